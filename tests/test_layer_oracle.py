"""The fp64 forms that the operators beside the chunkwise kernels are tested against, pinned by themselves: closed
forms, state-split invariance, and gradients against central differences."""
import numpy as np
import pytest

import layer_oracle as lo


def _scan_inputs(B, T, D, cu=None, seed=0):
    r = np.random.default_rng(seed)
    N = B if cu is None else len(cu) - 1
    return r.standard_normal((B, T, D)), -np.abs(r.standard_normal((B, T, D))) / 4, r.standard_normal((N, D)), r


def _difference(loss, args, i, step):
    """Central difference of the loss along ``step`` (of length 1e-5) in argument i."""
    up, down = ([a + sign * step if j == i else a for j, a in enumerate(args)] for sign in (1, -1))
    return (loss(*up) - loss(*down)) / 2e-5


def test_scan_closed_forms():
    x, g, h0, _ = _scan_inputs(2, 9, 3)
    np.testing.assert_allclose(lo.scan_fwd(x, 0 * g, h0)[0], np.cumsum(x, 1) + h0[:, None], rtol=1e-12)
    G = np.cumsum(g, 1)
    quad = np.einsum("btsd,bsd->btd", np.tril(np.ones((9, 9)))[None, :, :, None]
                     * np.exp(np.minimum(G[:, :, None] - G[:, None], 0)), x) + np.exp(G) * h0[:, None]
    h, ht, _, _ = lo.scan_fwd(x, g, h0)
    np.testing.assert_allclose(h, quad, rtol=1e-12)
    np.testing.assert_allclose(ht, h[:, -1], rtol=0)


def test_scan_split_and_pack():
    x, g, h0, _ = _scan_inputs(1, 11, 2, cu=[0, 4, 4, 11])
    h, ht, _, _ = lo.scan_fwd(x, g, h0, [0, 4, 4, 11])
    a, at, _, _ = lo.scan_fwd(x[:, :4], g[:, :4], h0[:1])
    b, bt, _, _ = lo.scan_fwd(x[:, 4:], g[:, 4:], h0[2:])
    np.testing.assert_array_equal(h, np.concatenate([a, b], 1))
    np.testing.assert_array_equal(ht, np.concatenate([at, h0[1:2], bt]))


@pytest.mark.parametrize("cu", [None, [0, 3, 3, 4, 10]])
def test_scan_gradients_against_differences(cu):
    x, g, h0, r = _scan_inputs(2 if cu is None else 1, 10, 2, cu, 1)
    dh, dht = r.standard_normal(x.shape), r.standard_normal(h0.shape)

    def loss(x, g, h0):
        h, ht, _, _ = lo.scan_fwd(x, g, h0, cu)
        return (h * dh).sum() + (ht * dht).sum()

    grads, _ = lo.scan_bwd(g, lo.scan_fwd(x, g, h0, cu)[0], dh, h0, dht, cu)
    args = [x, g, h0]
    for i, grad in enumerate(grads):
        for at in np.ndindex(args[i].shape):
            step = np.zeros_like(args[i])
            step[at] = 1e-5
            assert abs(_difference(loss, args, i, step) - grad[at]) < 1e-8


def test_gla_step_is_one_row_of_the_forward():
    import oracle
    from chunkwise_gated_linear_chunked_gb300 import build  # noqa: F401
    oracle.build()
    r = np.random.default_rng(3)
    q, k, g = (r.standard_normal((2, 1, 3, 8)).astype(np.float32) for _ in range(3))
    v, h0 = r.standard_normal((2, 1, 3, 4)).astype(np.float32), r.standard_normal((2, 3, 8, 4)).astype(np.float32)
    g = -np.abs(g)
    o, ht, _ = oracle.gla_fwd(q, k, v, g, 0.3, h0=h0)
    o1, new, _, _ = lo.gla_step(*(x[:, 0].astype(np.float64) for x in (q, k, v, g)), h0.astype(np.float64), 0.3)
    np.testing.assert_allclose(o1, o[:, 0], rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(new, ht, rtol=1e-12, atol=1e-13)


def test_norm_gradients_against_differences():
    r = np.random.default_rng(4)
    x, res, dy, ds = (r.standard_normal((3, 7)) for _ in range(4))
    w, eps = r.standard_normal(7), 1e-3

    def loss(x, res, w):
        y, s, _ = lo.norm_fwd(x, res, w, eps)
        return (y * dy).sum() + (s * ds).sum()

    y, s, rstd = lo.norm_fwd(x, res, w, eps)
    grad, dw, _, _ = lo.norm_bwd(s, rstd, w, dy, ds)
    args = [x, res, w]
    for i, gr in enumerate((grad, grad, dw)):
        for at in np.ndindex(args[i].shape):
            step = np.zeros_like(args[i])
            step[at] = 1e-5
            assert abs(_difference(loss, args, i, step) - gr[at]) < 1e-8


def test_quant_scales_partial_group():
    y = np.array([[1.0, -896.0, 4.0, 0.0, 0.0], [0, 0, 0, 0, 2.0]])
    scales, wide = lo.quant_scales(y, 2)
    np.testing.assert_allclose(scales, [[2, 4 / 448, 1e-30], [1e-30, 1e-30, 2 / 448]])
    np.testing.assert_allclose(wide[0], [2, 2, 4 / 448, 4 / 448, 1e-30])
    np.testing.assert_allclose(lo.quant_scales(y, 0)[0], [[2], [2 / 448]])
