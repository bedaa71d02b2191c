"""A gated delta layer as a model has it: keys and queries of unit length (norm_fwd with a weight of K^-0.5), the delta rule,
the group norm of its heads with SiLU; its gradients against the plain form's by autograd in fp64, and its tokens one by one
against the whole."""
import pytest
import torch

pytestmark = pytest.mark.gpu

H, HV, K, V = 2, 4, 64, 64


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture(scope="module")
def B():
    from chunkwise_gated_linear_chunked_gb300 import binding
    return binding


class Layer(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta, w, b):
        from chunkwise_gated_linear_chunked_gb300 import binding as B
        unit = torch.full((K,), K ** -0.5, device=q.device)
        qn, _, rq = B.norm_fwd(q, weight=unit, eps=0.0)
        kn, _, rk = B.norm_fwd(k, weight=unit, eps=0.0)
        o, _ = B.delta_fwd(qn, kn, v, g, beta)
        rows = o.reshape(-1, HV * V)
        y, mean, rstd = B.group_norm_fwd(rows, HV, weight=w, bias=b, activation="silu")
        ctx.save_for_backward(q, k, v, g, beta, w, b, qn, rq, kn, rk, rows, mean, rstd, unit)
        return y.reshape(v.shape)

    @staticmethod
    def backward(ctx, dy):
        from chunkwise_gated_linear_chunked_gb300 import binding as B
        q, k, v, g, beta, w, b, qn, rq, kn, rk, rows, mean, rstd, unit = ctx.saved_tensors
        drows, dw, db = B.group_norm_bwd(rows, mean, rstd, dy.reshape(rows.shape).contiguous(), weight=w, bias=b, activation="silu")
        dq, dk, dv, dg, dbeta, _ = B.delta_bwd(qn, kn, v, g, beta, drows.reshape(v.shape), want_dh0=False)
        return (B.norm_bwd(q, rq, dq, weight=unit, want_dw=False)[0], B.norm_bwd(k, rk, dk, weight=unit, want_dw=False)[0], dv, dg, dbeta,
                dw, db)


def plain(q, k, v, g, beta, w, b):
    q, k = (torch.nn.functional.normalize(t, dim=-1).repeat_interleave(HV // H, 2) for t in (q, k))
    S, rows = torch.zeros(q.shape[0], HV, K, V, dtype=q.dtype, device=q.device), []
    for t in range(q.shape[1]):
        S = g[:, t].exp()[..., None, None] * S
        row = beta[:, t, :, None] * (v[:, t] - torch.einsum("bhk,bhkv->bhv", k[:, t], S))
        S = S + k[:, t, ..., None] * row[..., None, :]
        rows.append(K ** -0.5 * torch.einsum("bhk,bhkv->bhv", q[:, t], S))
    o = torch.stack(rows, 1)
    o = (o - o.mean(-1, keepdim=True)) * (o.var(-1, unbiased=False, keepdim=True) + 1e-5).rsqrt()
    return torch.nn.functional.silu(o * w.reshape(HV, V) + b.reshape(HV, V))


def inputs(dtype, T):
    gen = torch.Generator(device="cuda").manual_seed(T)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=gen)   # noqa: E731
    q, k, v = (rand(2, T, n, 64).to(dtype) for n in (H, H, HV))
    return [q, k, v, -0.2 * rand(2, T, HV).abs(), rand(2, T, HV).sigmoid(), 1 + 0.1 * rand(HV * V), 0.1 * rand(HV * V)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_gradients(B, dtype):
    """fp32: operators within 1e-5 in four steps with order-one amplification.  bf16: the steps hand one another values
    rounded to 2^-8 (norm, delta rule, group norm, and back again: eight roundings at most), and the group norm divides by
    the spread of o, which the amplification of 4 below covers: heads' outputs have a spread near their size."""
    args = [t.requires_grad_(True) for t in inputs(dtype, 150)]
    wide = [t.detach().double().requires_grad_(True) for t in args]
    y, ref = Layer.apply(*args), plain(*wide)
    way = torch.randn(ref.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    rel = 1e-4 if dtype == torch.float32 else 4 * 8 * 2.0 ** -8
    assert (y.double() - ref).norm() <= rel * ref.norm()
    grads, refs = torch.autograd.grad(y, args, way.to(dtype)), torch.autograd.grad(ref, wide, way.to(dtype).double())
    for name, a, r in zip("q k v g beta w b".split(), grads, refs):
        assert torch.isfinite(a).all() and (a.double() - r).norm() <= rel * r.norm(), name


def test_tokens_one_by_one(B):
    args = inputs(torch.bfloat16, 70)
    whole = Layer.apply(*args)
    q, k, v, g, beta, w, b = args
    unit = torch.full((K,), K ** -0.5, device="cuda")
    pool = torch.zeros(2, HV, K, V, device="cuda")
    for t in range(70):
        qn, kn = (B.norm_fwd(x[:, t].contiguous(), weight=unit, eps=0.0)[0] for x in (q, k))
        o = B.delta_step(qn, kn, v[:, t].contiguous(), g[:, t].contiguous(), beta[:, t].contiguous(), pool)
        y, _, _ = B.group_norm_fwd(o.reshape(2, HV * V), HV, weight=w, bias=b, activation="silu")
        # o may round to neighbours in bf16 (2^-8 of its size), which the norm multiplies by its spread's reciprocal
        err = (y.reshape(2, HV, V).float() - whole[:, t].float()).norm() / whole[:, t].float().norm()
        assert err <= 2.0 ** -6
    assert B.layer_status() == B.GLA_OK
