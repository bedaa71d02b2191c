"""The gradients of gates of the gated delta rule over long sequences, token by token (fp32, and head sizes that the chunked
path does not take): sums of o.do - dv.v that cancel but for a few tokens' share, against the definition <S~, dS~> in fp64 on the
device."""
import pytest
import torch

import delta_oracle as do
from test_parity_delta import B, T32, TB, TH, _built, dev, make   # noqa: F401

pytestmark = pytest.mark.gpu

NAMES = ("q", "k", "v", "g", "beta")
BLOCK = 64   # rows after which a sum starts again from <S, dS>


def walk(body, state, ins, outs, back=False):
    """Calls body(rows of ins, rows of outs), which moves the state on, for every row in order, 91 or 128 rows a CUDA graph."""
    T = ins[0].shape[0]
    n = next(n for n in (128, 91, 1) if T % n == 0)
    these, those = ([t[:n].clone() for t in ts] for ts in (ins, outs))
    order = range(n - 1, -1, -1) if back else range(n)
    was = state.clone()
    body([t[0] for t in these], [t[0] for t in those])   # what the first call sets up cannot be captured
    state.copy_(was)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in order:
            body([t[i] for t in these], [t[i] for t in those])
    for lo in (range(T - n, -1, -n) if back else range(0, T, n)):
        for t, x in zip(these, ins):
            t.copy_(x[lo:lo + n])
        graph.replay()
        for t, x in zip(those, outs):
            x[lo:lo + n] = t


def definition(s, x, scale):
    """dg and dbeta of one dense sequence, and the sizes that rows' roundings are relative to: |o||do| + |dv||v| and |S||dS|
    (after a row) for dg, |x||Y| for dbeta; all [T, HV] in fp64 on the device."""
    per = s["v"].shape[2] // s["q"].shape[2]
    q, k = (s[n][0].cuda().double().repeat_interleave(per, 1) for n in ("q", "k"))
    v, beta, d = (t[0].cuda().double() for t in (s["v"], s["beta"], x["do"]))
    a = s["g"][0].cuda().double().exp()
    S, dS = (x[n][0].cuda().double() for n in ("h0", "dht"))
    old, rows, dx = v.new_empty(*k.shape, v.shape[-1]), torch.empty_like(v), torch.empty_like(v)
    dg, S_size, dS_size = (torch.empty_like(beta) for _ in range(3))

    def forward(ins, outs):
        k, v, a, beta = ins
        torch.mul(a[:, None, None], S, out=outs[0])
        outs[1].copy_(beta[:, None] * (v - (k[:, None] @ outs[0])[:, 0]))
        torch.baddbmm(outs[0], k[..., None], outs[1][:, None], out=S)
        outs[2].copy_(S.square().sum((1, 2)).sqrt())

    def backward(ins, outs):
        q, k, a, beta, d, old = ins
        outs[0].copy_(dS.square().sum((1, 2)).sqrt())
        dS.baddbmm_(q[..., None], scale * d[:, None])
        outs[1].copy_((k[:, None] @ dS)[:, 0])
        dS.baddbmm_(k[..., None], -beta[:, None, None] * outs[1][:, None])
        outs[2].copy_((dS * old).sum((1, 2)))
        dS.mul_(a[:, None, None])

    walk(forward, S, (k, v, a, beta), (old, rows, S_size))
    o = scale * (torch.einsum("thk,thkv->thv", q, old) + (q * k).sum(-1, keepdim=True) * rows)
    walk(backward, dS, (q, k, a, beta, d, old), (dS_size, dx, dg), back=True)
    size = lambda p, r: p.norm(dim=-1) * r.norm(dim=-1)   # noqa: E731
    y = rows / beta[..., None]
    return dg, (dx * y).sum(-1), size(o, d) + size(beta[..., None] * dx, v), S_size * dS_size, size(dx, y)


@pytest.mark.parametrize("T", [1001, 16384])
@pytest.mark.parametrize("dtype,heads", [(T32, (1, 3, 64, 64)), (T32, (1, 3, 37, 50)), (TB, (3, 3, 96, 80)), (TH, (1, 3, 64, 40))], ids=str)
def test_gate_gradients_of_long_sequences(B, dtype, heads, T):   # noqa: F811
    """Roundings are u / sqrt(3) in the mean square (u = 2^-24) and of random sign, and the partial sums of a product over D values
    sqrt(n / D) |a||b| / sqrt(D) long after n of them: such a product is off by less than u |a||b|.  A row's o.do is two of
    them, one after the other, dv.v, x and n one each; and a value of the state holds three roundings of its size for each token
    that it remembers, at most 64 for the gates here, which products average: (3 64 / 37)^0.5 = 2.3.  E = 4 u for all together.
    dg of a row is a sum over the rows behind it in its block, and <S, dS> at the block's end."""
    H, HV, K, V = heads
    s, x = make(dtype, T=T, H=H, HV=HV, K=K, V=V, seed=200 + T)
    s["g"] = s["g"] / 0.2 * torch.tensor([0.05, 1.6, 0.4])[torch.arange(HV) % 3]
    got = B.delta_bwd(*(dev(s[n]) for n in NAMES), dev(x["do"]), initial_state=dev(x["h0"]), dht=dev(x["dht"]))
    dg, db, rows, ends, both = definition(s, x, K ** -0.5)
    squares = torch.nn.functional.pad(rows.square(), (0, 0, 0, -T % BLOCK)).reshape(-1, BLOCK, HV)
    squares = squares.flip(1).cumsum(1).flip(1).reshape(-1, HV)[:T]
    last = torch.arange(T, device="cuda").div(BLOCK, rounding_mode="floor").mul(BLOCK).add(BLOCK - 1).clamp_max(T - 1)
    allowed = 4 * do.U * (squares + ends[last].square()).sqrt()
    for name, y, ref, tol in (("dg", got[3][0], dg, allowed), ("dbeta", got[4][0], db, 4 * do.U * both)):
        for part in (slice(None), slice(0, 256), slice(T - 256, T)):
            error, bound = (y.double() - ref)[part].norm(dim=0), tol[part].norm(dim=0)
            assert (error <= bound).all(), f"{name} of rows {part}: {error / bound} of what is allowed"


@pytest.mark.parametrize("dtype", [T32, TB, TH], ids=["f32", "bf16", "f16"])
def test_scratch_needs_no_zeroing(B, dtype):   # noqa: F811
    """A pack whose scratch is full of NaN."""
    s, x = make(dtype, lengths=[1, 0, 64, 65, 130, 3], H=2, HV=4, K=96, V=40, seed=210)
    args = [dev(s[n]) for n in NAMES] + [dev(x["do"])]
    kw = dict(initial_state=dev(x["h0"]), cu_seqlens=dev(x["cu"]))
    code = {T32: B.GLA_F32, TB: B.GLA_BF16, TH: B.GLA_F16}[dtype]
    need = B.lib().gla_delta_bwd_workspace_size(6, 1, 263, 2, 4, 96, 40, code, 1)
    scratch = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    for a, b in zip(B.delta_bwd(*args, workspace=scratch, **kw), B.delta_bwd(*args, **kw)):
        assert torch.equal(a, b)
