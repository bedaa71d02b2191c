"""GPU parity of the gated delta rule (forward, backward, one token) against the plain fp64 forms of ``delta_oracle``,
within its bounds plus the rounding of an output's type."""
import numpy as np
import pytest
import torch

import delta_oracle as do
import layer_oracle as lo

pytestmark = pytest.mark.gpu

T32, TB, TH = torch.float32, torch.bfloat16, torch.float16
KIND = {T32: "f32", TB: "bf16", TH: "f16"}


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture(scope="module")
def B():
    from chunkwise_gated_linear_chunked_gb300 import binding
    return binding


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def dev(t):
    return None if t is None else t.cuda()


def chunked(dtype, K, V):
    """Whether the tensor-core kernels take it."""
    return dtype != T32 and K in (64, 128) and V % 16 == 0


def make(dtype, Bn=1, T=64, H=1, HV=1, K=64, V=64, lengths=None, h0=True, seed=0, gate=0.2, tail=0):
    """Inputs of a call (on the host): a dict of tensors."""
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    cu = None
    if lengths is not None:
        ends = np.concatenate([[0], np.cumsum(lengths)])
        Bn, T, cu = 1, int(ends[-1]) + tail, torch.tensor(ends, dtype=torch.int32)
    N = Bn if cu is None else len(lengths)
    unit = lambda *s: (0.999 * torch.nn.functional.normalize(rand(*s), dim=-1)).to(dtype)   # noqa: E731
    s = dict(q=unit(Bn, T, H, K), k=unit(Bn, T, H, K), v=rand(Bn, T, HV, V).to(dtype),
             g=-gate * torch.rand(Bn, T, HV, generator=gen), beta=rand(Bn, T, HV).sigmoid())
    extra = dict(h0=0.5 * rand(N, HV, K, V) if h0 else None, cu=cu, do=rand(Bn, T, HV, V).to(dtype),
                 dht=0.5 * rand(N, HV, K, V) if h0 else None)
    return s, extra


def close(got, ref, size, rel, what, rounded=True):
    """|got - ref| <= rel size, plus the rounding to got's type; in rows that the reference knows."""
    known = ~np.isnan(ref)
    tol = rel * size + (lo.rounding(np.nan_to_num(ref), KIND[got.dtype]) if rounded else 0)
    bad = known & ~(np.abs(f64(got) - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, the first at {np.argwhere(bad)[0]}: {f64(got)[bad][0]} " \
                          f"for {ref[bad][0]}, allowed {np.broadcast_to(tol, ref.shape)[bad][0]}"


def check_fwd(B, s, x, out_dtype=None, scale=None):
    q, v = s["q"], s["v"]
    K, V, T = q.shape[-1], v.shape[-1], q.shape[1]
    o, ht = B.delta_fwd(*(dev(s[n]) for n in ("q", "k", "v", "g", "beta")), scale=scale, initial_state=dev(x["h0"]),
                        cu_seqlens=dev(x["cu"]), out_dtype=out_dtype)
    assert B.layer_status() == B.GLA_OK
    assert o.dtype == (out_dtype or q.dtype) and ht.dtype == T32
    ro, rt = do.delta_fwd(*(f64(s[n]) for n in ("q", "k", "v", "g", "beta")), scale or K ** -0.5, f64(x["h0"]), x["cu"])
    rel = do.bound("chunk" if chunked(q.dtype, K, V) else "scan", K, V, T)
    close(o, ro, do.largest(ro, (0, 1, 3)), rel, "o")
    close(ht, rt, do.largest(rt, (2, 3)), rel, "ht")
    return o, ht


def check_bwd(B, s, x, scale=None):
    q, v = s["q"], s["v"]
    K, V, T = q.shape[-1], v.shape[-1], q.shape[1]
    names = ("q", "k", "v", "g", "beta")
    got = B.delta_bwd(*(dev(s[n]) for n in names), dev(x["do"]), scale=scale, initial_state=dev(x["h0"]), dht=dev(x["dht"]),
                      cu_seqlens=dev(x["cu"]))
    assert B.layer_status() == B.GLA_OK
    keep, scale = {}, scale or K ** -0.5
    ref = do.delta_bwd(*(f64(s[n]) for n in names), f64(x["do"]), scale, f64(x["h0"]), f64(x["dht"]), x["cu"], keep)
    dq, dk, dv, dg, db, dh0 = ref
    rel = do.bound("chunk" if chunked(q.dtype, K, V) else "scan", K, V, T, backward=True)
    inside = slice(0, T if x["cu"] is None else int(x["cu"][-1]))
    per = v.shape[2] // q.shape[2]
    # a key head's gradients: sums over its value heads of products as large as the largest of dq, dk and dv here
    size_k = np.maximum(do.largest(dk, (0, 1, 3)), do.largest(dq, (0, 1, 3))) * per + \
        do.largest(dv.reshape(*dv.shape[:2], q.shape[2], -1), (0, 1, 3))
    size_v = do.largest(dv, (0, 1, 3)) + np.repeat(size_k, per, 2)
    size_dq = size_dk = size_k
    if chunked(q.dtype, K, V):   # operands of one 16-bit term: three roundings a term
        aq, ak = do.grad_sizes(f64(q), f64(s["k"]), f64(s["g"]), f64(s["beta"]), f64(x["do"]), scale, *q.shape[:2], x["cu"], keep)
        size_dq, size_dk = (size_k + 3 * lo.UNIT[KIND[q.dtype]] / rel * a[:, inside] for a in (aq, ak))
    # sums over a chunk of products of two rows: eight times (64 terms of random sign) the lengths' product
    long = lambda t: np.linalg.norm(t, axis=-1).max(initial=0.0)   # noqa: E731
    size_g = 8 * (long(dq) + long(dk) + long(dv) * (long(f64(v)[:, inside]) + 1)) + np.abs(f64(x["dht"]) if x["dht"] is not None else 0).max(initial=0.0)
    for name, y, r, size in (("dq", got[0], dq, size_dq), ("dk", got[1], dk, size_dk), ("dv", got[2], dv, size_v),
                             ("dg", got[3], dg, size_g), ("dbeta", got[4], db, size_g), ("dh0", got[5], dh0, do.largest(dh0, (2, 3)))):
        close(y[:, inside] if name != "dh0" else y, r[:, inside] if name != "dh0" else r, size, rel, name)
    return got


HEADS = [(1, 1, 64, 64), (2, 2, 128, 128), (1, 3, 128, 64), (2, 4, 64, 256), (1, 2, 128, 16), (1, 1, 64, 48), (3, 3, 96, 80), (1, 1, 7, 5),
         (1, 2, 128, 100), (1, 1, 256, 256), (1, 1, 1, 1), (1, 2, 64, 240), (1, 1, 128, 80)]
LENGTHS = [dict(Bn=1, T=1), dict(Bn=2, T=63), dict(Bn=1, T=64), dict(Bn=3, T=130), dict(lengths=[1, 0, 64, 65, 130, 3, 0])]


@pytest.mark.parametrize("types", [(T32, T32), (TB, TB), (TB, T32), (TH, TH), (TH, T32)], ids=lambda t: "-".join(KIND[x] for x in t))
@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("rows", LENGTHS, ids=str)
def test_forward(B, types, heads, rows):
    H, HV, K, V = heads
    s, x = make(types[0], H=H, HV=HV, K=K, V=V, seed=K + V, **rows)
    check_fwd(B, s, x, types[1])


@pytest.mark.parametrize("dtype", [T32, TB, TH], ids=lambda t: KIND[t])
@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("rows", LENGTHS, ids=str)
def test_backward(B, dtype, heads, rows):
    H, HV, K, V = heads
    s, x = make(dtype, H=H, HV=HV, K=K, V=V, seed=K + 2 * V, **rows)
    check_bwd(B, s, x)


@pytest.mark.parametrize("dtype", [T32, TB], ids=lambda t: KIND[t])
def test_no_states(B, dtype):
    """Without an initial state, a final one and their gradients."""
    s, x = make(dtype, Bn=2, T=150, H=2, HV=2, K=64, V=64, h0=False, seed=4)
    check_fwd(B, s, x, scale=0.7)
    check_bwd(B, s, x, scale=0.7)
    args = [dev(s[n]) for n in ("q", "k", "v", "g", "beta")]
    o, ht = B.delta_fwd(*args, output_final_state=False)
    assert ht is None and torch.equal(o, B.delta_fwd(*args)[0])
    got = B.delta_bwd(*args, dev(x["do"]), want_dh0=False)
    assert got[5] is None and all(torch.equal(a, b) for a, b in zip(got[:5], B.delta_bwd(*args, dev(x["do"]))[:5]))


@pytest.mark.parametrize("dtype", [T32, TB], ids=lambda t: KIND[t])
@pytest.mark.parametrize("K", [64, 128])
def test_edges_of_gates_and_strengths(B, dtype, K):
    """Gates of minus infinity (the state is cleared) and of zero, strengths of 0, 1 and 2, keys all the same, keys of zero."""
    s, x = make(dtype, Bn=1, T=200, H=1, HV=1, K=K, V=64, seed=5)
    s["g"][0, [0, 17, 18, 64, 100, 127, 199]] = -float("inf")
    s["g"][0, 30:50] = 0
    s["g"][0, 140] = -200.0
    s["beta"][0, 20:40], s["beta"][0, 60:70], s["beta"][0, 70:90] = 0, 1, 2
    s["k"][0, 90:120] = s["k"][0, 90]
    s["k"][0, 125] = 0
    check_fwd(B, s, x)
    check_bwd(B, s, x)


@pytest.mark.parametrize("dtype", [TB, TH], ids=lambda t: KIND[t])
@pytest.mark.parametrize("K", [64, 128])
@pytest.mark.parametrize("HV", [1, 8])
def test_gate_gradients_of_fast_decays(B, dtype, K, HV):
    """Gradients of gates after which little is left, behind a final state whose gradient is large: sums of products that
    cancel.  dg is <e^g S, dS>, and S, dS, the rows between them and the chunk's inverse are held in two 16-bit terms, each
    off by at most UNIT^2 of its size: 4 UNIT^2 of dg's norm.  (fp16's second term is a multiple of 2^-24: of values from
    2^-7 on, which make the norm, off by at most 2^-25, 2^-18 of them.)  And a row's o and dv are fp32 sums of 2 K / 16
    partial products of a tensor core, each cut to 24 bits: off by at most 2 K / 16 2^-23 of their size, of random signs over
    columns and rows, in sums of o dO and dv v that run over up to 128 rows."""
    s, x = make(dtype, T=400, H=1, HV=HV, K=K, V=128, gate=1.6, seed=71)
    x["dht"] = 2 * x["dht"]
    names = ("q", "k", "v", "g", "beta")
    dg = B.delta_bwd(*(dev(s[n]) for n in names), dev(x["do"]), initial_state=dev(x["h0"]), dht=dev(x["dht"]))[3]
    wide = [f64(s[n]) for n in names]
    o = do.delta_fwd(*wide, K ** -0.5, f64(x["h0"]))[0]
    _, _, dv, ref, _, _ = do.delta_bwd(*wide, f64(x["do"]), K ** -0.5, f64(x["h0"]), f64(x["dht"]))
    terms = ((o * f64(x["do"])) ** 2 + (dv * wide[2]) ** 2).sum(-1)
    sums = np.concatenate([np.cumsum(terms[:, a:a + 128][:, ::-1], 1) for a in range(0, 400, 128)], 1) ** 0.5
    bound = 4 * max(lo.UNIT[KIND[dtype]] ** 2, 2.0 ** -18) * np.linalg.norm(ref) + 2 * K / 16 * 2.0 ** -23 * np.linalg.norm(sums)
    error = np.linalg.norm(f64(dg) - ref)
    assert error <= bound


@pytest.mark.parametrize("dtype", [T32, TB], ids=lambda t: KIND[t])
def test_gates_above_zero(B, dtype):
    s, x = make(dtype, Bn=1, T=140, K=64, V=64, seed=6)
    s["g"] = 0.02 * torch.randn(s["g"].shape, generator=torch.Generator().manual_seed(1))
    s["beta"][:] = 0.9
    check_fwd(B, s, x)
    check_bwd(B, s, x)


@pytest.mark.parametrize("dtype", [T32, TB], ids=lambda t: KIND[t])
def test_rows_behind_the_last_sequence(B, dtype):
    """They are left as they were, and what lies in them reaches nothing."""
    s, x = make(dtype, lengths=[70, 5], tail=60, H=2, HV=2, K=64, V=64, seed=7)
    x["do"][0, 75:] = float("nan")
    for n in s:
        s[n][0, 75:] = float("nan")
    o, ht = check_fwd(B, s, x)
    got = check_bwd(B, s, x)
    for t in (ht, got[5]):
        assert torch.isfinite(t).all()
    out = torch.full_like(o, 7.0)
    lib, args = B.lib(), [dev(s[n]) for n in ("q", "k", "v", "g", "beta")]
    code = B.DELTA_CODE[dtype, dtype]
    need = lib.gla_delta_fwd_workspace_size(2, 1, 135, 2, 2, 64, 64, code, 1)
    ws, cu = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda"), dev(x["cu"])
    rc = lib.gla_delta_fwd(*(t.data_ptr() for t in args), out.data_ptr(), 0.125, None, None, cu.data_ptr(), 2, 1, 135, 2, 2, 64, 64,
                           code, lib.gla_scan_shared_workspace(), ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert rc == B.GLA_OK and (out[0, 75:] == 7).all() and (out[0, :75] != 7).any()


def test_bad_offsets_are_reported(B):
    for dtype in (T32, TB):
        s, x = make(dtype, lengths=[30, 40], K=64, V=64, seed=8)
        args = [dev(s[n]) for n in ("q", "k", "v", "g", "beta")]
        for cu in ([0, 80, 70], [0, 50, 30], [-3, 30, 70], [0, 30, 71]):
            cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
            B.delta_fwd(*args, cu_seqlens=cu)
            assert B.layer_status() == B.GLA_ERR_INVALID_ARG
            own = torch.zeros(256, dtype=torch.uint8, device="cuda")
            B.delta_bwd(*args, dev(x["do"]), cu_seqlens=cu, status=own)
            assert B.layer_status() == B.GLA_OK and B.get_status(own) == B.GLA_ERR_INVALID_ARG


@pytest.mark.parametrize("dtype", [T32, TB], ids=lambda t: KIND[t])
def test_state_in_place_and_in_pieces(B, dtype):
    """A sequence in two calls, the second on the state that the first left, updated in place."""
    s, x = make(dtype, Bn=2, T=192, H=1, HV=2, K=128, V=128, seed=9)
    whole, end = B.delta_fwd(*(dev(s[n]) for n in ("q", "k", "v", "g", "beta")), initial_state=dev(x["h0"]), out_dtype=T32)
    cut = lambda lo, hi: [dev(s[n][:, lo:hi].contiguous()) for n in ("q", "k", "v", "g", "beta")]   # noqa: E731
    first, state = B.delta_fwd(*cut(0, 128), initial_state=dev(x["h0"]), out_dtype=T32)
    lib, args, code = B.lib(), cut(128, 192), B.DELTA_CODE[dtype, T32]
    o = torch.empty(2, 64, 2, 128, device="cuda")
    ws = torch.empty(max(lib.gla_delta_fwd_workspace_size(2, 2, 64, 1, 2, 128, 128, code, 0), 256), dtype=torch.uint8, device="cuda")
    rc = lib.gla_delta_fwd(*(t.data_ptr() for t in args), o.data_ptr(), 128 ** -0.5, state.data_ptr(), state.data_ptr(), None, 2, 2, 64,
                           1, 2, 128, 128, code, lib.gla_scan_shared_workspace(), ws.data_ptr(), ws.numel(),
                           torch.cuda.current_stream().cuda_stream)
    assert rc == B.GLA_OK
    rel = 2 * do.bound("scan" if dtype == T32 else "chunk", 128, 128, 192)
    close(torch.cat([first, o], 1), f64(whole), do.largest(f64(whole), (0, 1, 3)), rel, "o")
    close(state, f64(end), do.largest(f64(end), (2, 3)), rel, "ht")


def test_many_sequences_repeat_bit_for_bit(B):
    lengths = [3, 0, 64, 65, 1, 130, 200] * 12
    for dtype in (T32, TB):
        s, x = make(dtype, lengths=lengths, H=2, HV=4, K=64, V=64, seed=10)
        args = [dev(s[n]) for n in ("q", "k", "v", "g", "beta")]
        kw = dict(initial_state=dev(x["h0"]), cu_seqlens=dev(x["cu"]))
        one, two = B.delta_fwd(*args, **kw), B.delta_fwd(*args, **kw)
        assert all(torch.equal(a, b) for a, b in zip(one, two))
        g1, g2 = (B.delta_bwd(*args, dev(x["do"]), dht=dev(x["dht"]), **kw) for _ in range(2))
        assert all(torch.equal(a, b) for a, b in zip(g1, g2))
        check_fwd(B, s, x)
        check_bwd(B, s, x)


@pytest.mark.parametrize("dtype", [T32, TB], ids=lambda t: KIND[t])
def test_graph_and_other_stream(B, dtype):
    s, x = make(dtype, Bn=2, T=100, H=2, HV=2, K=64, V=64, seed=11)
    args, g = [dev(s[n]) for n in ("q", "k", "v", "g", "beta")], dev(x["do"])
    want = (*B.delta_fwd(*args), *B.delta_bwd(*args, g))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = (*B.delta_fwd(*args, stream=side), *B.delta_bwd(*args, g, stream=side))
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = (*B.delta_fwd(*args), *B.delta_bwd(*args, g))
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


STEP_HEADS = [(1, 1, 64, 64), (2, 4, 128, 128), (2, 2, 128, 256), (3, 3, 96, 80), (1, 2, 7, 5), (1, 1, 256, 100), (2, 2, 200, 33)]


@pytest.mark.parametrize("types", [(T32, T32), (TB, TB), (TB, T32), (TH, TH), (TH, T32)], ids=lambda t: "-".join(KIND[x] for x in t))
@pytest.mark.parametrize("heads", STEP_HEADS, ids=str)
def test_step(B, types, heads):
    H, HV, K, V = heads
    s, x = make(types[0], Bn=5, T=1, H=H, HV=HV, K=K, V=V, seed=12)
    args = [dev(s[n][:, 0].contiguous()) for n in ("q", "k", "v", "g", "beta")]
    pool = torch.randn(8, HV, K, V, generator=torch.Generator().manual_seed(2)).cuda()
    slots = torch.tensor([6, -1, 0, 3, 7], dtype=torch.int32, device="cuda")
    was, live = pool.clone(), [0, 2, 3, 4]
    out = torch.full_like(pool, 9.0)
    o1 = B.delta_step(*args, pool, slots=slots, state_out=out, out_dtype=types[1])
    assert torch.equal(pool, was)
    o2 = B.delta_step(*args, pool, slots=slots, out_dtype=types[1])
    assert B.layer_status() == B.GLA_OK and torch.equal(o1, o2) and (o1[1] == 0).all()
    used = slots[live].long()
    rest = [i for i in range(8) if i not in used.tolist()]
    assert torch.equal(out[used], pool[used]) and (out[rest] == 9).all() and torch.equal(pool[rest], was[rest])
    ro, rt = do.delta_fwd(*(f64(s[n][live]) for n in ("q", "k", "v", "g", "beta")), K ** -0.5, f64(was[used]))
    # the output by way of q S~ + (q.k) n: a sum of K terms more
    rel = 2 * do.bound("scan", K, V, 1)
    size = do.largest(f64(was[used]), (2, 3))
    close(pool[used], rt, np.maximum(size, do.largest(rt, (2, 3))) * 2, rel, "state")
    close(o1[live], ro[:, 0], (K ** -0.5 * (K ** 0.5 * size[..., 0] + 4)), rel, "o")


def test_step_continues_a_prompt(B):
    """Prefill, then tokens one by one on the pool, inside a graph, as one forward over all."""
    s, x = make(TB, Bn=3, T=90, H=2, HV=4, K=128, V=128, seed=13)
    args = [dev(s[n]) for n in ("q", "k", "v", "g", "beta")]
    whole, end = B.delta_fwd(*args, out_dtype=T32)
    _, pool = B.delta_fwd(*(t[:, :80].contiguous() for t in args))
    token = [t[:, 80].contiguous() for t in args]
    B.delta_step(*token, pool.clone(), out_dtype=T32)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = B.delta_step(*token, pool, out_dtype=T32)
    rel = 2 * do.bound("chunk", 128, 128, 90)
    for t in range(80, 90):
        for dst, src in zip(token, args):
            dst.copy_(src[:, t])
        graph.replay()
        close(o, f64(whole[:, t]), do.largest(f64(whole), (1, 3))[:, 0], rel, f"token {t}")
    close(pool, f64(end), do.largest(f64(end), (2, 3)), rel, "state")


def test_bad_slots_are_reported(B):
    s, x = make(TB, Bn=2, T=1, K=64, V=64, seed=14)
    args = [dev(s[n][:, 0].contiguous()) for n in ("q", "k", "v", "g", "beta")]
    pool = torch.ones(3, 1, 64, 64, device="cuda")
    o = B.delta_step(*args, pool, slots=torch.tensor([3, -2], dtype=torch.int32, device="cuda"))
    assert B.layer_status() == B.GLA_ERR_INVALID_ARG and (o == 0).all() and (pool == 1).all()


def test_offsets_beyond_32_bits(B):
    """Values of more than 2^31 elements: the last head of the last rows as in a call with that head alone."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    T, HV, V = 1 << 17, 136, 128
    q, k = (torch.nn.functional.normalize(torch.randn(1, T, 1, 64, device="cuda", generator=gen), dim=-1).to(TB) for _ in range(2))
    v = torch.randn(1, T, HV, V, device="cuda", generator=gen, dtype=TB)
    g, beta = -0.1 * torch.rand(1, T, HV, device="cuda", generator=gen), torch.rand(1, T, HV, device="cuda", generator=gen)
    assert v.numel() > 1 << 31
    o, ht = B.delta_fwd(q, k, v, g, beta)
    last = [t[:, :, -1:].contiguous() for t in (v, g, beta)]
    one, end = B.delta_fwd(q, k, *last)
    assert torch.equal(o[:, :, -1:], one) and torch.equal(ht[:, -1:], end)
    del o
    got = B.delta_bwd(q, k, v, g, beta, v)
    one = B.delta_bwd(q, k, *last, last[0])
    for x, y in zip(got[2:5], one[2:5]):
        assert torch.equal(x[:, :, -1:], y)
    assert torch.equal(got[5][:, -1:], one[5])


def test_own_status_and_scratch(B):
    """A status word of the call's own that is too small, and scratch that is."""
    s, x = make(TB, Bn=1, T=70, K=64, V=64)
    args = [dev(s[n]) for n in ("q", "k", "v", "g", "beta")]
    with pytest.raises(B.GlaError):
        B.delta_fwd(*args, status=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(B.GlaError):
        B.delta_fwd(*args, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    need = B.lib().gla_delta_bwd_workspace_size(1, 1, 70, 1, 1, 64, 64, B.GLA_BF16, 0)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")   # NaN wherever it is read before it is written
    for a, b in zip(B.delta_bwd(*args, dev(x["do"]), workspace=ws), B.delta_bwd(*args, dev(x["do"]))):
        assert torch.equal(a, b)
    need = B.lib().gla_delta_fwd_workspace_size(1, 1, 70, 1, 1, 64, 64, B.GLA_BF16_OBF16, 0)
    for a, b in zip(B.delta_fwd(*args, workspace=torch.full((need,), 255, dtype=torch.uint8, device="cuda")), B.delta_fwd(*args)):
        assert torch.equal(a, b)


def test_fp16_range_is_reported(B):
    """A state that leaves fp16's range on the chunked path; token by token, and in bf16, it does not matter."""
    for dtype, K, want in ((TH, 64, "GLA_ERR_RANGE"), (TH, 96, "GLA_OK"), (TB, 64, "GLA_OK")):
        s, x = make(dtype, Bn=1, T=100, K=K, V=64, seed=15)
        args = [dev(s[n]) for n in ("q", "k", "v", "g", "beta")]
        o, ht = B.delta_fwd(*args, initial_state=1e5 * torch.ones(1, 1, K, 64, device="cuda"), out_dtype=T32)
        assert B.layer_status() == getattr(B, want)
        assert torch.isfinite(o).all() == (want == "GLA_OK")
        B.delta_bwd(*args, dev(x["do"]), dht=1e5 * torch.ones(1, 1, K, 64, device="cuda"))
        assert B.layer_status() == getattr(B, want)
        B.delta_bwd(*args, dev(x["do"]))
        assert B.layer_status() == B.GLA_OK


def test_nothing_to_do(B):
    z = lambda *s: torch.zeros(*s, device="cuda")   # noqa: E731
    o, ht = B.delta_fwd(z(0, 5, 2, 64), z(0, 5, 2, 64), z(0, 5, 2, 64), z(0, 5, 2), z(0, 5, 2))
    assert o.numel() == 0 and ht.numel() == 0
    for dtype in (T32, TB):
        q, h0 = z(2, 0, 2, 64).to(dtype), torch.randn(2, 2, 64, 64, device="cuda")
        o, ht = B.delta_fwd(q, q, q, z(2, 0, 2), z(2, 0, 2), initial_state=h0)
        assert o.shape == (2, 0, 2, 64) and torch.equal(ht, h0)
        assert (B.delta_fwd(q, q, q, z(2, 0, 2), z(2, 0, 2))[1] == 0).all()
        got = B.delta_bwd(q, q, q, z(2, 0, 2), z(2, 0, 2), q, dht=h0)
        assert torch.equal(got[5], h0) and got[0].numel() == 0
    assert B.delta_step(z(0, 2, 64), z(0, 2, 64), z(0, 2, 64), z(0, 2), z(0, 2), z(0, 2, 64, 64)).numel() == 0


def test_refusals(B):
    s, x = make(TB, Bn=2, T=10, H=2, HV=4, K=64, V=64)
    q, k, v, g, beta = (dev(s[n]) for n in ("q", "k", "v", "g", "beta"))
    do_, h0 = dev(x["do"]), dev(x["h0"])
    bad = [lambda: B.delta_fwd(q.cpu(), k, v, g, beta), lambda: B.delta_fwd(q, k[:, :5], v, g, beta),
           lambda: B.delta_fwd(q, k, v, g.bfloat16(), beta), lambda: B.delta_fwd(q, k, v, g, beta[..., :2].contiguous()),
           lambda: B.delta_fwd(q, k, v[:, :, :3].contiguous(), g[..., :3].contiguous(), beta[..., :3].contiguous()),
           lambda: B.delta_fwd(q, k, v.transpose(1, 2).contiguous().transpose(1, 2), g, beta),
           lambda: B.delta_fwd(q, k, v, g, beta, initial_state=h0[:1]), lambda: B.delta_fwd(q, k, v, g, beta, scale=-1.0),
           lambda: B.delta_fwd(q, k, v, g, beta, cu_seqlens=torch.tensor([0, 20], device="cuda")),
           lambda: B.delta_fwd(q, k, v, g, beta, cu_seqlens=torch.tensor([0, 20], dtype=torch.int32, device="cuda")),
           lambda: B.delta_fwd(q, k, v, g, beta, out_dtype=TH), lambda: B.delta_fwd(q[0], k[0], v[0], g[0], beta[0]),
           lambda: B.delta_bwd(q, k, v, g, beta, do_.float()), lambda: B.delta_bwd(q, k, v, g, beta, do_, dht=h0.bfloat16()),
           lambda: B.delta_step(q[:, 0].contiguous(), k[:, 0].contiguous(), v[:, 0].contiguous(), g[:, 0].contiguous(),
                                beta[:, 0].contiguous(), h0[:1])]
    for i, call in enumerate(bad):
        with pytest.raises(B.GlaError):
            call()
            pytest.fail(f"call {i} was not refused")
