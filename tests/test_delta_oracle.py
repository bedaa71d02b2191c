"""The fp64 forms of the gated delta rule and of the group norm: closed cases and gradients against differences."""
import numpy as np
import pytest

import delta_oracle as do


def inputs(B=2, T=7, H=2, HV=4, K=5, V=3, seed=0):
    r = np.random.default_rng(seed)
    unit = lambda t: t / np.linalg.norm(t, axis=-1, keepdims=True)   # noqa: E731
    return (unit(r.normal(size=(B, T, H, K))), unit(r.normal(size=(B, T, H, K))), r.normal(size=(B, T, HV, V)),
            -r.uniform(size=(B, T, HV)), r.uniform(size=(B, T, HV)), r)


def test_full_strength_stores_the_value():
    """beta = 1 and a unit key: reading the key just written gives its value back."""
    q, k, v, g, _, _ = inputs(HV=2)
    o, _ = do.delta_fwd(k, k, v, g, np.ones_like(g), 1.0)
    np.testing.assert_allclose(o, v, atol=1e-12)


def test_orthogonal_keys_are_linear_attention():
    q, _, v, g, beta, _ = inputs(T=5, H=1, HV=1)
    k = np.broadcast_to(np.eye(5)[None, :, None, :], q.shape)
    o, _ = do.delta_fwd(q, k, v, 0 * g, beta, 0.5)
    scores = np.tril(np.einsum("bthk,bshk->bts", q, k))
    np.testing.assert_allclose(o[:, :, 0], 0.5 * scores @ (beta[..., None] * v)[:, :, 0], atol=1e-12)


def test_split_and_pack():
    q, k, v, g, beta, r = inputs(B=1, T=9)
    h0 = r.normal(size=(1, 4, 5, 3))
    o, ht = do.delta_fwd(q, k, v, g, beta, 0.4, h0)
    at = lambda t, s: t[:, s]   # noqa: E731
    first = [at(t, slice(0, 4)) for t in (q, k, v, g, beta)]
    second = [at(t, slice(4, None)) for t in (q, k, v, g, beta)]
    o1, h1 = do.delta_fwd(*first, 0.4, h0)
    o2, h2 = do.delta_fwd(*second, 0.4, h1)
    np.testing.assert_allclose(np.concatenate([o1, o2], 1), o, atol=1e-12)
    np.testing.assert_allclose(h2, ht, atol=1e-12)
    po, ph = do.delta_fwd(q, k, v, g, beta, 0.4, np.concatenate([h0, h1]), cu=[0, 4, 9])
    np.testing.assert_allclose(po, o, atol=1e-12)
    np.testing.assert_allclose(ph, np.concatenate([h1, ht]), atol=1e-12)


@pytest.mark.parametrize("cu", [None, [0, 3, 3, 8]])
def test_gradients_are_differences(cu):
    q, k, v, g, beta, r = inputs(B=1 if cu else 2, T=8)
    N = 3 if cu else 2
    h0, dht, dout = r.normal(size=(N, 4, 5, 3)), r.normal(size=(N, 4, 5, 3)), r.normal(size=v.shape)

    def loss(*x):
        o, ht = do.delta_fwd(*x[:5], 0.4, x[5], cu)
        return (o * dout).sum() + (ht * dht).sum()

    args = [q, k, v, g, beta, h0]
    grads = do.delta_bwd(q, k, v, g, beta, dout, 0.4, h0, dht, cu)
    for i, grad in enumerate(grads):
        way = r.normal(size=grad.shape)
        moved = lambda s: loss(*(a + s * way if j == i else a for j, a in enumerate(args)))   # noqa: E731
        assert abs((moved(1e-6) - moved(-1e-6)) / 2e-6 - (grad * way).sum()) < 1e-6 * np.abs(grad * way).sum()


@pytest.mark.parametrize("shape", [(3, 8), (2, 5, 8), (2, 2, 3, 8)])
@pytest.mark.parametrize("silu", [False, True])
def test_group_norm(shape, silu):
    r = np.random.default_rng(1)
    x, w, b, dy = r.normal(size=shape) + 1, r.normal(size=8), r.normal(size=8), r.normal(size=shape)
    (y, mean, rstd), _ = do.group_norm_fwd(x, 2, w, b, silu, 1e-5)
    flat = x.reshape(shape[0], -1, 8)
    assert np.allclose(mean[:, 1], flat[:, :, 4:].mean((1, 2))) and np.allclose(rstd[:, 0], 1 / np.sqrt(flat[:, :, :4].var((1, 2)) + 1e-5))
    grads, _ = do.group_norm_bwd(x, mean, rstd, dy, w, b, silu)
    loss = lambda x, w, b: (do.group_norm_fwd(x, 2, w, b, silu, 1e-5)[0][0] * dy).sum()   # noqa: E731
    for i, grad in enumerate(grads):
        way = r.normal(size=grad.shape)
        moved = lambda s: loss(*(a + s * way if j == i else a for j, a in enumerate((x, w, b))))   # noqa: E731
        assert abs((moved(1e-6) - moved(-1e-6)) / 2e-6 - (grad * way).sum()) < 1e-5 * np.abs(grad * way).sum() + 1e-8
