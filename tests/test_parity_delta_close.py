"""Gradients of gates and strengths of the gated delta rule head by head and row by row, each against what it is made of, and the
kernels that many heads and sequences run (64 columns a CTA)."""
import numpy as np
import pytest
import torch

import delta_oracle as do
from test_parity_delta import B, KIND, T32, TB, TH, _built, check_bwd, check_fwd, chunked, dev, f64, make   # noqa: F401

pytestmark = pytest.mark.gpu

NAMES = ("q", "k", "v", "g", "beta")


def check_gates(B, s, x, got):   # noqa: F811
    """Mean square bounds, over the rows of each sequence and head.  Token by token, E = 4 u: see the long sequences' test.  In
    chunks an operand is off by 2^-18 in the mean square: k S (1), its product with the inverse (3), the update (1) and the
    output's product (3) are 20^0.5 2^-18 together, once for each chunk that a state has passed, in forward and backward; they are
    of random sign over the V columns of a row's sum, which so are as much less than the lengths' product.  (An fp16 operand is
    nearer.)  dbeta = x.Y has two such factors; dg is a sum of o.do - dv.v over a group's rows behind (128; token by token 64), and
    <S, dS> at its end."""
    wide = [f64(s[n]) for n in NAMES]
    q, k, v, g, beta = wide
    K, V, HV = q.shape[-1], v.shape[-1], v.shape[2]
    keep, d, scale = {}, f64(x["do"]), K ** -0.5
    ref = do.delta_bwd(*wide, d, scale, f64(x["h0"]), f64(x["dht"]), x["cu"], keep)
    per, tiles = HV // q.shape[2], chunked(s["q"].dtype, K, V)
    fq, fb, fd, fv = np.repeat(q, per, 2).reshape(-1, HV, K), beta.reshape(-1, HV), d.reshape(-1, HV, V), v.reshape(-1, HV, V)
    dg, db, rg, rb = (t.reshape(-1, HV) for t in (f64(got[3]), f64(got[4]), ref[3], ref[4]))
    length = lambda t: np.linalg.norm(t, axis=-1)   # noqa: E731
    for n, (lo_, hi) in enumerate(do.sequences(*q.shape[:2], x["cu"])):
        if lo_ == hi:
            continue
        chunks = -(-(hi - lo_) // 64)
        E = 20 ** 0.5 * 2.0 ** -18 * (1 + chunks) ** 0.5 / V ** 0.5 + 4 * do.U if tiles else 4 * do.U
        at = range(lo_, hi)
        old, row, xs, behind = (np.stack([keep[r][i] for r in at]) for i in range(4))
        new = old + np.repeat(k, per, 2).reshape(-1, HV, K)[lo_:hi, ..., None] * row[..., None, :]
        o = scale * np.einsum("thk,thkv->thv", fq[lo_:hi], new)
        terms = length(o) * length(fd[lo_:hi]) + fb[lo_:hi] * length(xs) * length(fv[lo_:hi])
        ends = np.linalg.norm(new, axis=(2, 3)) * np.linalg.norm(behind, axis=(2, 3))
        group = 128 if tiles else 64
        size_g = np.zeros_like(terms)
        for a in range(0, hi - lo_, group):
            b = min(a + group, hi - lo_)
            size_g[a:b] = (np.cumsum(terms[a:b][::-1] ** 2, 0)[::-1] + ends[b - 1] ** 2) ** 0.5
        size_b = length(row) / fb[lo_:hi] * length(xs)
        for name, y, r, size in (("dg", dg, rg, size_g), ("dbeta", db, rb, 2 * size_b)):
            error, allowed = np.linalg.norm((y - r)[lo_:hi], axis=0), E * np.linalg.norm(size, axis=0)
            assert (error <= allowed).all(), f"{name} of sequence {n}: heads off by {error / allowed} of what is allowed"
            # a row alone: six times its own mean square
            bad = np.abs((y - r)[lo_:hi]) > 6 * E * size + 2.0 ** -149
            assert not bad.any(), f"{name} of sequence {n}: rows and heads {np.argwhere(bad)[:8].tolist()} off"


def fast_and_slow(s):
    """Heads in turn that forget within a few tokens, and that hardly do."""
    s["g"] = s["g"] / 0.2 * torch.tensor([0.2, 1.6, 0.02])[torch.arange(s["g"].shape[-1]) % 3]


CASES = [(T32, (1, 3, 64, 64)), (T32, (3, 3, 96, 80)), (T32, (1, 2, 37, 50)), (T32, (1, 2, 64, 256)), (TB, (1, 3, 128, 128)), (TB, (2, 4, 64, 16)),
         (TB, (1, 3, 128, 80)), (TB, (1, 2, 64, 240)), (TB, (1, 2, 96, 40)), (TH, (1, 3, 128, 64)), (TH, (1, 2, 64, 80)), (TH, (1, 2, 200, 33))]


@pytest.mark.parametrize("rows", [dict(Bn=2, T=257), dict(lengths=[1, 0, 64, 65, 130, 3, 193])], ids=str)
@pytest.mark.parametrize("dtype,heads", CASES, ids=lambda t: KIND.get(t, str(t)) if not isinstance(t, tuple) else str(t))
def test_gates_row_by_row(B, dtype, heads, rows):   # noqa: F811
    H, HV, K, V = heads
    s, x = make(dtype, H=H, HV=HV, K=K, V=V, seed=300 + K + V, **rows)
    fast_and_slow(s)
    got = B.delta_bwd(*(dev(s[n]) for n in NAMES), dev(x["do"]), initial_state=dev(x["h0"]), dht=dev(x["dht"]), cu_seqlens=dev(x["cu"]))
    check_gates(B, s, x, got)


@pytest.mark.parametrize("dtype", [TB, TH], ids=lambda t: KIND[t])
@pytest.mark.parametrize("V", [64, 80])
def test_more_heads_than_the_gpu_has_sms(B, dtype, V):   # noqa: F811
    """Keys of 128 where CTAs of 32 columns would be more than the SMs: CTAs of 64, the last of V = 80 with one group of four."""
    lengths = [130, 3, 64, 0, 65] * 2
    s, x = make(dtype, lengths=lengths, H=4, HV=8, K=128, V=V, seed=310 + V)
    assert len(lengths) * 8 * -(-V // 32) > torch.cuda.get_device_properties(0).multi_processor_count
    check_fwd(B, s, x, T32)
    check_fwd(B, s, x)
    check_gates(B, s, x, check_bwd(B, s, x))


def test_many_value_heads_of_a_key_head(B):   # noqa: F811
    """Gradients of one key head that 136 value heads share, of more than 2^31 values: the sum of those that 17 calls with eight
    heads each find, of which each is rounded to bf16 like the whole."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    T, HV, V = 1 << 17, 136, 128
    q, k = (torch.nn.functional.normalize(torch.randn(1, T, 1, 64, device="cuda", generator=gen), dim=-1).to(TB) for _ in range(2))
    v = torch.randn(1, T, HV, V, device="cuda", generator=gen, dtype=TB)
    g, beta = -0.1 * torch.rand(1, T, HV, device="cuda", generator=gen), torch.rand(1, T, HV, device="cuda", generator=gen)
    whole = B.delta_bwd(q, k, v, g, beta, v)[:2]
    sums, sizes = ([torch.zeros(q.shape, device="cuda") for _ in range(2)] for _ in range(2))
    for at in range(0, HV, 8):
        part = [t[:, :, at:at + 8].contiguous() for t in (v, g, beta)]
        for total, size, y in zip(sums, sizes, B.delta_bwd(q, k, *part, part[0])[:2]):
            total += y.float()
            size += y.float().abs()
    for name, y, total, size in zip(("dq", "dk"), whole, sums, sizes):
        # a rounding of each part and of the whole; the sums of 136 heads and of 17 parts in fp32
        allowed = 2.0 ** -8 * (total.abs() + size) * (1 + 2.0 ** -7) + 200 * do.U * size
        assert ((y.float() - total).abs() <= allowed).all(), name
