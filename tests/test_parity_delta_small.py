"""The gated delta rule on values far below one, in fp16 above all: its chunked path has operands of fp16, whose second term
ends at 2^-25 whatever the first one is.  Everything is linear in (v, h0) and, for the gradients, in (do, dht), so that
errors have to shrink with them: the bounds of ``delta_oracle`` as they stand, relative to what is compared."""
import numpy as np
import pytest
import torch

import delta_oracle as do
import test_parity_delta as parity
from test_parity_delta import B, T32, TB, TH, _built, check_bwd, check_fwd, dev, f64, make   # noqa: F401

pytestmark = pytest.mark.gpu

NAMES = ("q", "k", "v", "g", "beta")


def scaled(s, x, v=1.0, d=1.0):
    """The inputs with (v, h0) and (do, dht) multiplied by powers of two (a number, or one a column)."""
    s, x = dict(s), dict(x)
    s["v"], x["h0"] = (s["v"].float() * v).to(s["v"].dtype), x["h0"] * v
    x["do"], x["dht"] = (x["do"].float() * d).to(x["do"].dtype), x["dht"] * d
    return s, x


def bilinear(got, s, x, scale=None):
    """dbeta_i = x_i.Y_i, with x_i the gradient of the update row over beta and Y_i the row over beta: each is a row of values
    within the mean square bound of the chunked path, of its length, so that the product is within twice that of the two
    lengths; over a head's rows by their mean square."""
    keep, wide = {}, [f64(s[n]) for n in NAMES]
    scale = scale or wide[0].shape[-1] ** -0.5
    ref = do.delta_bwd(*wide, f64(x["do"]), scale, f64(x["h0"]), f64(x["dht"]), x["cu"], keep)
    rows, T = wide[3].shape[0] * wide[3].shape[1], wide[3].shape[1]
    beta = wide[4].reshape(rows, -1)
    size = np.stack([np.linalg.norm(keep[r][1], axis=-1) / beta[r] * np.linalg.norm(keep[r][2], axis=-1) for r in range(rows)])
    error = f64(got[4]).reshape(rows, -1) - ref[4].reshape(rows, -1)
    rel = 2 * do.bound("chunk", wide[0].shape[-1], wide[2].shape[-1], T, backward=True)
    off = np.linalg.norm(error, axis=0) / np.linalg.norm(size, axis=0)
    assert (off <= rel).all(), f"dbeta off by {off} of what it is made of, allowed {rel}"


def by_column(got, ref, rel, what):
    """Each column (the last axis) relative to its own largest value."""
    size = np.abs(ref).max(axis=tuple(range(ref.ndim - 1)), keepdims=True)
    off = (np.abs(f64(got) - ref) / size).reshape(-1, ref.shape[-1]).max(0)
    assert (off <= rel).all(), f"{what}: columns {np.argwhere(off > rel)[:, 0]} off by {off[off > rel]}, allowed {rel}"


@pytest.mark.parametrize("down", [0, 10, 13, 16, 20])
@pytest.mark.parametrize("heads", [(1, 2, 128, 128), (1, 1, 64, 80)], ids=str)
@pytest.mark.parametrize("dtype", [TH, TB], ids=["f16", "bf16"])
def test_small_values(B, dtype, heads, down):   # noqa: F811
    H, HV, K, V = heads
    s, x = scaled(*make(dtype, T=100, H=H, HV=HV, K=K, V=V, seed=80 + down), v=2.0 ** -down)
    check_fwd(B, s, x, T32)


@pytest.mark.parametrize("down", [0, 10, 13, 16, 20])
@pytest.mark.parametrize("heads", [(1, 2, 128, 128), (1, 1, 64, 80)], ids=str)
@pytest.mark.parametrize("dtype", [TH, TB], ids=["f16", "bf16"])
def test_small_gradients(B, dtype, heads, down):   # noqa: F811
    H, HV, K, V = heads
    s, x = scaled(*make(dtype, T=100, H=H, HV=HV, K=K, V=V, seed=90 + down), d=2.0 ** -down)
    bilinear(check_bwd(B, s, x), s, x)


@pytest.mark.parametrize("down", [(12, 12), (16, 4), (4, 16)], ids=str)
def test_small_values_and_gradients(B, down):   # noqa: F811
    s, x = scaled(*make(TH, lengths=[70, 1, 0, 130], H=2, HV=4, K=128, V=64, seed=100), v=2.0 ** -down[0], d=2.0 ** -down[1])
    check_fwd(B, s, x, T32)
    check_bwd(B, s, x)


@pytest.mark.parametrize("K", [64, 128])
def test_columns_of_many_sizes(B, K):   # noqa: F811
    """Columns of (v, h0), and of (do, dht), that are powers of two apart: none is the worse for a larger neighbour."""
    V = 96
    by = 2.0 ** -(torch.arange(V) * 7 % 19).float()
    s, x = scaled(*make(TH, T=140, K=K, V=V, seed=101), v=by, d=by)
    wide = [f64(s[n]) for n in NAMES]
    o, ht = B.delta_fwd(*(dev(s[n]) for n in NAMES), initial_state=dev(x["h0"]), out_dtype=T32)
    ro, rt = do.delta_fwd(*wide, K ** -0.5, f64(x["h0"]))
    rel = do.bound("chunk", K, V, 140)
    by_column(o, ro, rel, "o")
    by_column(ht, rt, rel, "ht")
    dh0 = B.delta_bwd(*(dev(s[n]) for n in NAMES), dev(x["do"]), initial_state=dev(x["h0"]), dht=dev(x["dht"]))[5]
    by_column(dh0, do.delta_bwd(*wide, f64(x["do"]), K ** -0.5, f64(x["h0"]), f64(x["dht"]))[5], 2 * rel, "dh0")
    check_bwd(B, s, x)


@pytest.mark.parametrize("scale", [2.0 ** -16, 1e-4, 100.0])
def test_scales(B, scale):   # noqa: F811
    s, x = make(TH, T=100, H=1, HV=2, K=64, V=64, seed=102)
    x["do"] = (x["do"].float() / max(scale, 1.0)).to(TH)
    check_fwd(B, s, x, T32, scale=scale)
    bilinear(check_bwd(B, s, x, scale=scale), s, x, scale)


def test_short_queries_and_weak_writes(B):   # noqa: F811
    """Queries far below unit length, and write strengths near zero."""
    s, x = make(TH, T=100, H=1, HV=2, K=128, V=64, seed=103)
    s["q"] = (s["q"].float() * 2.0 ** -10).to(TH)
    check_fwd(B, s, x, T32)
    check_bwd(B, s, x)
    s, x = make(TH, T=100, H=1, HV=2, K=128, V=64, h0=False, seed=104)
    s["beta"] = s["beta"] * 1e-4
    check_fwd(B, s, x, T32)
    check_bwd(B, s, x)


def test_products_beyond_the_range_of_their_factors(B):   # noqa: F811
    """Products of gradients with update rows that leave fp16's range (9.9e4), where no operand and no output does."""
    s, x = make(TH, T=64, K=64, V=64, h0=False, seed=105)
    s["v"], x["do"] = s["v"] * 16, x["do"] * 2048
    check_bwd(B, s, x)


@pytest.mark.parametrize("K", [64, 128])
def test_edges_in_fp16(B, K):   # noqa: F811
    """What the other types are tested with: cleared states and strengths of 0 to 2; and gates above zero."""
    parity.test_edges_of_gates_and_strengths(B, TH, K)
    parity.test_gates_above_zero(B, TH)


def test_rows_behind_and_repeats_in_fp16(B):   # noqa: F811
    """NaN behind the last sequence reaches no column's largest value; packs repeat bit for bit, in graphs and on streams."""
    parity.test_rows_behind_the_last_sequence(B, TH)
    parity.test_graph_and_other_stream(B, TH)
    s, x = make(TH, lengths=[3, 0, 64, 65, 1, 130, 200] * 12, H=2, HV=4, K=64, V=64, seed=10)
    args, kw = [dev(s[n]) for n in NAMES], dict(initial_state=dev(x["h0"]), cu_seqlens=dev(x["cu"]))
    one, two = B.delta_fwd(*args, **kw), B.delta_fwd(*args, **kw)
    assert all(torch.equal(a, b) for a, b in zip(one, two))
    one, two = (B.delta_bwd(*args, dev(x["do"]), dht=dev(x["dht"]), **kw) for _ in range(2))
    assert all(torch.equal(a, b) for a, b in zip(one, two))


def test_scratch_needs_no_zeroing_in_fp16(B):   # noqa: F811
    s, x = make(TH, lengths=[1, 0, 64, 65, 130, 3], H=2, HV=4, K=64, V=80, seed=106)
    args, kw = [dev(s[n]) for n in NAMES], dict(initial_state=dev(x["h0"]), cu_seqlens=dev(x["cu"]))
    sizes = (6, 1, 263, 2, 4, 64, 80)
    for call, need in ((B.delta_fwd, B.lib().gla_delta_fwd_workspace_size(*sizes, B.GLA_F16_OF16, 1)),
                       (lambda *a, **kw: B.delta_bwd(*a, dev(x["do"]), **kw), B.lib().gla_delta_bwd_workspace_size(*sizes, B.GLA_F16, 1))):
        scratch = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
        for a, b in zip(call(*args, workspace=scratch, **kw), call(*args, **kw)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [TH, TB], ids=["f16", "bf16"])
@pytest.mark.parametrize("K", [64, 128])
def test_a_large_row_among_ordinary_ones(B, K, dtype):   # noqa: F811
    """A value row, a query and an output's gradient a few thousand times the others': rows that it does not reach (those before
    it; for the gradients those behind) are as near as without it, relative to their own largest values."""
    s, x = make(dtype, T=60, K=K, V=64, seed=107)
    s["v"][0, 40], s["q"][0, 20], x["do"][0, 20] = s["v"][0, 40] * 4096, s["q"][0, 20] * 4096, x["do"][0, 20] * 2048
    wide = [f64(s[n]) for n in NAMES]
    o, _ = B.delta_fwd(*(dev(s[n]) for n in NAMES), initial_state=dev(x["h0"]), out_dtype=T32)
    ro, _ = do.delta_fwd(*wide, K ** -0.5, f64(x["h0"]))
    rows = [t for t in range(40) if t != 20]
    rel = do.bound("chunk", K, 64, 60)
    assert np.abs(f64(o) - ro)[0, rows].max() <= rel * np.abs(ro[0, rows]).max()
    got = B.delta_bwd(*(dev(s[n]) for n in NAMES), dev(x["do"]), initial_state=dev(x["h0"]), dht=dev(x["dht"]))
    ref = do.delta_bwd(*wide, f64(x["do"]), K ** -0.5, f64(x["h0"]), f64(x["dht"]))
    for name, i in (("dv", 2), ("dh0", 5)):
        y, r = (f64(got[i]), ref[i]) if name == "dh0" else (f64(got[i])[:, 21:40], ref[i][:, 21:40])
        own = 0 if name == "dh0" else (2.0 ** -11 if dtype == TH else 2.0 ** -8) * np.abs(r)
        assert (np.abs(y - r) <= 2 * rel * np.abs(r).max() + own).all(), name


def test_long_keys_and_weak_writes(B):   # noqa: F811
    """Keys of one entry of 100, as long as beta |k|^2 stays below 2: a chunk then adds to its state 6400 times its largest update
    row, from nothing, and no more than fits."""
    s, x = make(TH, T=130, K=64, V=64, h0=False, seed=108)
    s["k"][:] = 0
    s["k"][0, :, 0, 3] = 100
    s["beta"][:], s["v"] = 1e-5, s["v"].abs()
    check_fwd(B, s, x, T32)
    check_bwd(B, s, x)
