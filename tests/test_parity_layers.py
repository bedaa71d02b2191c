"""GPU parity of the operators beside the chunkwise kernels (vector-state recurrence, one-token updates, residual
norm) against the plain fp64 forms in ``layer_oracle``, whose a-priori bounds are the tolerances: the fp32
evaluation's bound plus the rounding to the output's type."""
import numpy as np
import pytest
import torch

import layer_oracle as lo

pytestmark = pytest.mark.gpu

T32, TB, TH = torch.float32, torch.bfloat16, torch.float16
KIND = {T32: "f32", TB: "bf16", TH: "f16"}
SCAN_TYPES = [(T32, T32, T32), (TB, TB, T32), (TB, TB, TB), (TH, TH, T32), (TH, TH, TH), (TB, T32, T32), (TH, T32, T32)]


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


def within(x, ref, tol, what=""):
    """|x - ref| <= tol plus the rounding of x's type, elementwise."""
    got, tol = f64(x), tol + lo.rounding(ref, KIND[x.dtype])
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, the first at {np.argwhere(bad)[0]}: " \
                          f"{got[bad][0]} for {ref[bad][0]}, allowed {tol[bad][0]}"


def scan_inputs(types, Bn, T, D, lengths=None, h0=True, seed=0, gate=0.25):
    gen = torch.Generator().manual_seed(seed)
    cu = None
    if lengths is not None:
        Bn, T = 1, sum(lengths)
        cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32)
    N = Bn if cu is None else len(lengths)
    x = torch.randn(Bn, T, D, generator=gen).to(types[0])
    g = (-gate * torch.rand(Bn, T, D, generator=gen)).to(types[1])
    return x, g, torch.randn(N, D, generator=gen) if h0 else None, cu


SCAN_CASES = [   # B, T, D, lengths, initial state
    (1, 1, 1, None, True),
    (3, 1, 70, None, True),
    (2, 5, 64, None, False),
    (1, 127, 64, None, True),
    (2, 128, 65, None, True),
    (1, 129, 33, None, True),
    (2, 640, 200, None, True),
    (1, 1025, 129, None, False),
    (1, 4100, 96, None, True),
    (1, 9000, 8, None, True),
    (1, 0, 72, [1, 0, 2, 127, 128, 129, 300, 0], True),
    (1, 0, 40, [0, 0, 5], True),
    (1, 0, 64, [1000, 3, 2100], False),
]


@pytest.mark.parametrize("types", SCAN_TYPES, ids=lambda t: "-".join(KIND[x] for x in t))
@pytest.mark.parametrize("case", SCAN_CASES, ids=str)
def test_scan(B, case, types):
    Bn, T, D, lengths, with_h0 = case
    x, g, h0, cu = scan_inputs(types, Bn, T, D, lengths, with_h0, seed=D)
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    h, ht = B.scan_fwd(dev(x), dev(g), initial_state=dev(h0), cu_seqlens=dev(cu), out_dtype=types[2])
    ref, ref_t, tol, tol_t = lo.scan_fwd(f64(x), f64(g), f64(h0), cu)
    within(h, ref, tol, "h")
    within(ht, ref_t, tol_t, "ht")
    gen = torch.Generator().manual_seed(1)
    dh = torch.randn(h.shape, generator=gen).to(types[2])
    dht = torch.randn(ht.shape, generator=gen)
    dx, dg, dh0 = B.scan_bwd(dev(g), h, dev(dh), initial_state=dev(h0), dht=dev(dht), cu_seqlens=dev(cu),
                             dx_dtype=types[0])
    assert dx.dtype == types[0] and dg.dtype == types[1]
    refs, tols = lo.scan_bwd(f64(g), f64(h), f64(dh), f64(h0), f64(dht), cu)   # from the h that it was given
    for name, y, r, t in zip(("dx", "dg", "dh0"), (dx, dg, dh0), refs, tols):
        within(y, r, t, name)


@pytest.mark.parametrize("T,D", [(20000, 64), (5000, 1000)])
def test_scan_long_memory(B, T, D):
    """Gates of about -1e-4: the state remembers thousands of rows, over many time slices."""
    x, g, h0, _ = scan_inputs((T32, T32), 1, T, D, seed=2, gate=2e-4)
    h, ht = B.scan_fwd(x.cuda(), g.cuda(), initial_state=h0.cuda())
    ref, ref_t, tol, tol_t = lo.scan_fwd(f64(x), f64(g), f64(h0))
    within(h, ref, tol)
    within(ht, ref_t, tol_t)


def test_scan_many_short_sequences(B):
    lengths = [3, 0, 1, 7] * 300
    x, g, h0, cu = scan_inputs((TB, TB), 1, 0, 136, lengths, seed=3)
    h, ht = B.scan_fwd(x.cuda(), g.cuda(), initial_state=h0.cuda(), cu_seqlens=cu.cuda())
    ref, ref_t, tol, tol_t = lo.scan_fwd(f64(x), f64(g), f64(h0), cu)
    within(h, ref, tol)
    within(ht, ref_t, tol_t)


@pytest.mark.parametrize("types,D", [((TB, TB, TB), 128), ((T32, T32, T32), 77)], ids=["bf16", "f32"])
def test_scan_pack_of_many_lengths(B, types, D):
    """Enough sequences that short ones and long ones are walked by different kernels."""
    lengths = [3, 0, 64, 65, 1, 130, 700] * 160
    x, g, h0, cu = scan_inputs(types, 1, 0, D, lengths, seed=30)
    cu_d, h0_d, g_d = cu.cuda(), h0.cuda(), g.cuda()
    h, ht = B.scan_fwd(x.cuda(), g_d, initial_state=h0_d, cu_seqlens=cu_d)
    ref, ref_t, tol, tol_t = lo.scan_fwd(f64(x), f64(g), f64(h0), cu)
    within(h, ref, tol, "h")
    within(ht, ref_t, tol_t, "ht")
    dh = torch.randn(h.shape, generator=torch.Generator().manual_seed(31)).to(types[2]).cuda()
    grads = B.scan_bwd(g_d, h, dh, initial_state=h0_d, cu_seqlens=cu_d)
    refs, tols = lo.scan_bwd(f64(g), f64(h), f64(dh), f64(h0), None, cu)
    for name, y, r, t in zip(("dx", "dg", "dh0"), grads, refs, tols):
        within(y, r, t, name)


@pytest.mark.parametrize("types,Bn,T,D", [((TB, TB, TB), 24, 2100, 1000), ((TB, T32, T32), 10, 3000, 998)],
                         ids=["bf16", "f32-gate"])
def test_scan_more_tiles_than_run_at_once(B, types, Bn, T, D):
    """So many (sequence, channel tile) pairs that clusters come in waves."""
    x, g, h0, _ = scan_inputs(types, Bn, T, D, seed=32)
    g_d, h0_d = g.cuda(), h0.cuda()
    h, ht = B.scan_fwd(x.cuda(), g_d, initial_state=h0_d, out_dtype=types[2])
    ref, ref_t, tol, tol_t = lo.scan_fwd(f64(x), f64(g), f64(h0))
    within(h, ref, tol, "h")
    within(ht, ref_t, tol_t, "ht")
    dh = torch.randn(h.shape, generator=torch.Generator().manual_seed(33)).to(types[2])
    grads = B.scan_bwd(g_d, h, dh.cuda(), initial_state=h0_d, dx_dtype=types[0])
    refs, tols = lo.scan_bwd(f64(g), f64(h), f64(dh), f64(h0))
    for name, y, r, t in zip(("dx", "dg", "dh0"), grads, refs, tols):
        within(y, r, t, name)


def test_scan_many_batches_of_few_rows(B):
    for T in (1, 2, 9, 17):
        x, g, h0, _ = scan_inputs((TH, TH), 301, T, 72, seed=T)
        h, ht = B.scan_fwd(x.cuda(), g.cuda(), initial_state=h0.cuda(), out_dtype=TH)
        ref, ref_t, tol, tol_t = lo.scan_fwd(f64(x), f64(g), f64(h0))
        within(h, ref, tol)
        within(ht, ref_t, tol_t)


def test_scan_gradient_against_differences(B):
    """The fp32 gradients' inner product with a direction, against the fp64 loss's central difference along it."""
    x, g, h0, _ = scan_inputs((T32, T32), 2, 300, 10, seed=4)
    r = np.random.default_rng(5)
    dh, dht = r.standard_normal(x.shape).astype("f4"), r.standard_normal(h0.shape).astype("f4")
    h, _ = B.scan_fwd(x.cuda(), g.cuda(), initial_state=h0.cuda())
    grads = B.scan_bwd(g.cuda(), h, torch.tensor(dh).cuda(), initial_state=h0.cuda(), dht=torch.tensor(dht).cuda())
    _, tols = lo.scan_bwd(f64(g), f64(h), dh, f64(h0), dht)
    _, _, tol_h, _ = lo.scan_fwd(f64(x), f64(g), f64(h0))
    args = [f64(x), f64(g), f64(h0)]

    def loss(args):
        y, yt, _, _ = lo.scan_fwd(*args)
        return (y * dh).sum() + (yt * dht).sum()

    for i in range(3):
        v = r.standard_normal(args[i].shape)
        up, down = ([a + e * v if j == i else a for j, a in enumerate(args)] for e in (1e-6, -1e-6))
        slope = (loss(up) - loss(down)) / 2e-6
        got = (f64(grads[i]) * v).sum()
        allowed = ((tols[i] + lo.rounding(f64(grads[i]), "f32")) * np.abs(v)).sum()
        if i == 1:   # dg carries the error of the h that the forward wrote
            allowed += (np.abs(f64(grads[0]) * v) * np.abs(np.roll(tol_h + lo.rounding(f64(h), "f32"), 1, 1))).sum()
        # and the difference's own: third derivatives (in g) times 1e-12, cancellation of 1e-16 |loss| / 1e-6
        assert abs(slope - got) <= allowed + 1e-6 * (1 + abs(slope)) + 1e-9 * abs(loss(args))


def test_scan_strided_inputs_and_gradients(B):
    """x and g as column ranges of one projection; dx and dg as column ranges of one gradient."""
    for D, dtype in ((64, TB), (40, T32), (200, TH)):
        both = torch.randn(2, 150, 2 * D, generator=torch.Generator().manual_seed(6))
        both[..., D:] = -both[..., D:].abs() / 4
        both = both.to(dtype).cuda()
        x, g = both[..., :D], both[..., D:]
        h, ht = B.scan_fwd(x, g)
        h1, ht1 = B.scan_fwd(x.contiguous(), g.contiguous())
        assert torch.equal(h, h1) and torch.equal(ht, ht1)
        dh, grad = torch.randn_like(h), torch.full_like(both, 7)
        B.scan_bwd(g, h, dh, dx=grad[..., :D], dg=grad[..., D:])
        dx, dg, _ = B.scan_bwd(g.contiguous(), h, dh)
        assert torch.equal(grad, torch.cat([dx, dg], -1))
    # odd row spacing: 3 columns of padding between rows
    wide = torch.randn(1, 300, 80, device="cuda").to(TB)[..., :77]
    g = (-torch.rand(1, 300, 77, device="cuda")).to(TB)
    assert torch.equal(B.scan_fwd(wide, g)[0], B.scan_fwd(wide.contiguous(), g)[0])


def test_scan_resets_infinities_and_nan(B):
    """exp(-inf) and exp(lowest) are 0: the state restarts there.  A NaN or an infinity stays in its channel and in
    the rows after it, up to a reset (a NaN survives it: 0 times NaN)."""
    for dtype in (T32, TB):
        x, g, h0, _ = scan_inputs((dtype, dtype), 1, 700, 64, seed=7)
        x, g, h0 = x.cuda(), g.cuda(), h0.cuda()
        g[0, 300, :8] = -float("inf")
        g[0, 300, 8:16] = torch.finfo(dtype).min
        h, ht = B.scan_fwd(x, g, initial_state=h0)
        fresh, _ = B.scan_fwd(x[:, 300:].contiguous(), g[:, 300:].contiguous())
        assert torch.equal(h[0, 300, :16], x[0, 300, :16])
        ref, _, tol, _ = lo.scan_fwd(f64(x), f64(g), f64(h0))
        within(h, ref, tol)
        clean = h.clone()
        x[0, 500, 20] = float("nan")
        x[0, 600, 21] = float("inf")
        h, ht = B.scan_fwd(x, g, initial_state=h0)
        assert torch.isnan(h[0, 500:, 20]).all() and torch.isnan(ht[0, 20])
        assert torch.isinf(h[0, 600:, 21]).all() and torch.isinf(ht[0, 21])
        h[0, 500:, 20] = clean[0, 500:, 20]
        h[0, 600:, 21] = clean[0, 600:, 21]
        assert torch.equal(h, clean)


def test_scan_empty_calls(B):
    e = torch.empty(2, 0, 24, device="cuda", dtype=TB)
    h0 = torch.randn(2, 24, device="cuda")
    h, ht = B.scan_fwd(e, e, initial_state=h0)
    assert h.shape == (2, 0, 24) and torch.equal(ht, h0)
    assert torch.equal(B.scan_fwd(e, e)[1], torch.zeros(2, 24, device="cuda"))
    dx, dg, dh0 = B.scan_bwd(e, e, e, dht=h0)
    assert dx.shape == e.shape and torch.equal(dh0, h0)
    e = torch.empty(0, 5, 24, device="cuda")
    assert B.scan_fwd(e, e)[1].shape == (0, 24)


def test_scan_state_in_place_and_split(B):
    """ht over h0 in place, and a run cut in two by passing the state on."""
    x, g, h0, _ = scan_inputs((T32, T32), 2, 500, 96, seed=8)
    x, g, h0 = x.cuda(), g.cuda(), h0.cuda()
    ref, ref_t, tol, tol_t = lo.scan_fwd(f64(x), f64(g), f64(h0))
    state, ws = h0.clone(), torch.zeros(256, dtype=torch.uint8, device="cuda")
    h = torch.empty_like(x)
    for lo_, hi in ((0, 333), (333, 500)):
        xs, gs, hs = (t[:, lo_:hi].contiguous() for t in (x, g, h))
        rc = B.lib().gla_scan_fwd(xs.data_ptr(), gs.data_ptr(), hs.data_ptr(), state.data_ptr(), state.data_ptr(), None,
                                  2, 2, hi - lo_, 96, 96, 96, B.GLA_F32, ws.data_ptr(), 256,
                                  torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        h[:, lo_:hi] = hs
    within(h, ref, tol)
    within(state, ref_t, tol_t)


def test_scan_bad_offsets_are_reported(B):
    x = torch.zeros(1, 40, 64, device="cuda")
    for cu in ([0, 30, 20, 40], [0, 10, 39], [1, 40], [0, -5, 40], [0, 50, 40]):
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        B.scan_fwd(x, x, cu_seqlens=c, workspace=ws)
        assert B.get_status(ws) == B.GLA_ERR_INVALID_ARG and B.get_status(ws) == B.GLA_OK
        B.scan_bwd(x, x, x, cu_seqlens=c, workspace=ws)
        assert B.get_status(ws) == B.GLA_ERR_INVALID_ARG


def test_scan_rows_beyond_32_bit_offsets(B):
    """Rows 2^16 elements apart: the last ones lie beyond 2^31 elements."""
    T, ld, D = 34000, 1 << 16, 48
    buf = torch.empty(T * ld, dtype=TB, device="cuda")
    x, g = buf.as_strided((1, T, D), (T * ld, ld, 1)), buf.as_strided((1, T, D), (T * ld, ld, 1), 1024)
    x.copy_(torch.randn(1, T, D, device="cuda"))
    g.copy_(-torch.rand(1, T, D, device="cuda") / 4)
    h, ht = B.scan_fwd(x, g)
    h1, ht1 = B.scan_fwd(x.contiguous(), g.contiguous())
    assert torch.equal(h, h1) and torch.equal(ht, ht1)
    ref, _, tol, _ = lo.scan_fwd(f64(x), f64(g))
    within(h, ref, tol)


def test_scan_repeats_bit_for_bit(B):
    x, g, h0, cu = scan_inputs((TB, TB), 1, 0, 512, [3000, 17, 900], seed=9)
    args = dict(initial_state=h0.cuda(), cu_seqlens=cu.cuda())
    x, g = x.cuda(), g.cuda()
    first = B.scan_fwd(x, g, **args)
    dh = torch.randn_like(first[0])
    grads = B.scan_bwd(g, first[0], dh, **args)
    for _ in range(5):
        for a, b in zip(first + grads, B.scan_fwd(x, g, **args) + B.scan_bwd(g, first[0], dh, **args)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("types", SCAN_TYPES, ids=lambda t: "-".join(KIND[x] for x in t))
@pytest.mark.parametrize("Bn,D,S", [(1, 1, 1), (1, 1024, 3), (5, 77, 9), (64, 256, 64), (130, 40, 200)])
def test_scan_step(B, Bn, D, S, types):
    x, g, _, _ = scan_inputs(types, Bn, 1, D, seed=10)
    x, g = x[:, 0].cuda(), g[:, 0].cuda()
    state = torch.randn(S, D, generator=torch.Generator().manual_seed(11)).cuda()
    slots = torch.randperm(S, generator=torch.Generator().manual_seed(12))[:Bn].to(torch.int32)
    slots[Bn // 2] = -1 if Bn > 1 else slots[0]
    before = f64(state)
    h = B.scan_step(x, g, state, slots=slots.cuda(), out_dtype=types[2])
    ref, expected = np.zeros((Bn, D)), before.copy()
    for b, s in enumerate(slots.tolist()):
        if s >= 0:
            ref[b] = expected[s] = np.exp(f64(g)[b]) * before[s] + f64(x)[b]
    size = np.abs(f64(x)) + np.abs(before[slots.numpy()])
    within(h, ref, 4 * lo.U * size, "h")
    live = slots[slots >= 0].numpy()
    assert (np.delete(f64(state), live, 0) == np.delete(before, live, 0)).all()
    within(state[torch.from_numpy(live).long().cuda()], expected[live], 4 * lo.U * size[slots.numpy() >= 0], "state")
    # the forward's one row, and a state pool of its own to write
    out = torch.full_like(state, 5.0)
    start = torch.randn(Bn, D, device="cuda")
    pool = torch.zeros(S, D, device="cuda")
    pool[:Bn] = start
    same = B.scan_step(x, g, pool, slots=torch.arange(Bn, dtype=torch.int32, device="cuda"), state_out=out,
                       out_dtype=types[2])
    h1, ht1 = B.scan_fwd(x[:, None].contiguous(), g[:, None].contiguous(), initial_state=start, out_dtype=types[2])
    assert torch.equal(same, h1[:, 0]) and torch.equal(out[:Bn], ht1) and (out[Bn:] == 5).all()


STEP_CASES = [(1, 1, 64, 64, 1), (1, 8, 128, 128, 1), (3, 2, 128, 256, 7), (17, 5, 64, 128, 20), (40, 16, 128, 64, 41),
              (2, 3, 64, 256, 2)]


@pytest.mark.parametrize("types", SCAN_TYPES, ids=lambda t: "-".join(KIND[x] for x in t))
@pytest.mark.parametrize("case", STEP_CASES, ids=str)
def test_gla_step(B, case, types):
    Bn, H, K, V, S = case
    gen = torch.Generator().manual_seed(13)
    q, k, v = (torch.randn(Bn, H, d, generator=gen).to(types[0]) for d in (K, K, V))
    g = (-torch.rand(Bn, H, K, generator=gen)).to(types[1])
    state = torch.randn(S, H, K, V, generator=gen).cuda()
    slots = torch.randperm(S, generator=gen)[:Bn].to(torch.int32)
    before = f64(state)
    o, new, tol_o, tol_s = lo.gla_step(*(f64(t) for t in (q, k, v, g)), before[slots.numpy()], K ** -0.5)
    out = torch.full_like(state, 5.0)
    got = B.gla_step(q.cuda(), k.cuda(), v.cuda(), g.cuda(), state, slots=slots.cuda(), state_out=out,
                     out_dtype=types[2])
    within(got, o, tol_o, "o")
    within(out[slots.long().cuda()], new, tol_s, "state")
    others = np.delete(f64(out), slots.numpy(), 0)
    assert (others == 5).all() and (f64(state) == before).all()
    again = B.gla_step(q.cuda(), k.cuda(), v.cuda(), g.cuda(), state, slots=slots.cuda(), out_dtype=types[2])   # in place
    assert torch.equal(got, again) and torch.equal(state[slots.long().cuda()], out[slots.long().cuda()])


def test_gla_step_follows_the_forward(B):
    """A prompt through gla_fwd, then token by token: the outputs and states of one gla_fwd over all rows."""
    gen = torch.Generator().manual_seed(14)
    q, k, v = (torch.randn(2, 70, 4, 128, generator=gen).to(TB).cuda() for _ in range(3))
    g = (-torch.rand(2, 70, 4, 128, generator=gen) / 8).to(TB).cuda()
    o, ht = B.gla_fwd(q, k, v, g)
    cut = lambda t, a, b: t[:, a:b].contiguous()  # noqa: E731
    _, state = B.gla_fwd(*(cut(t, 0, 64) for t in (q, k, v, g)))
    for t in range(64, 70):
        step = B.gla_step(*(x[:, t].contiguous() for x in (q, k, v, g)), state)
        rel = (step - o[:, t]).norm() / o[:, t].norm()
        assert rel <= 5e-3   # the forward's own bound for bf16 inputs
    assert (state - ht).norm() / ht.norm() <= 5e-3


def test_steps_idle_and_bad_slots(B):
    """-1 marks an idle sequence; another slot outside the pool is reported; neither reads or writes a state."""
    gen = torch.Generator().manual_seed(15)
    for bad, code in ((-1, B.GLA_OK), (-2, B.GLA_ERR_INVALID_ARG), (3, B.GLA_ERR_INVALID_ARG),
                      (2 ** 31 - 1, B.GLA_ERR_INVALID_ARG)):
        slots = torch.tensor([2, bad], dtype=torch.int32).cuda()
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        state = torch.randn(3, 2, 64, 64, generator=gen).cuda()
        before = state.clone()
        q = torch.randn(2, 2, 64, generator=gen).cuda()
        o = B.gla_step(q, q, q, -q.abs(), state, slots=slots, workspace=ws)
        assert B.get_status(ws) == code
        assert (o[1] == 0).all() and torch.equal(state[:2], before[:2]) and not torch.equal(state[2], before[2])
        flat = torch.randn(3, 50, generator=gen).cuda()
        before = flat.clone()
        x = torch.randn(2, 50, generator=gen).cuda()
        h = B.scan_step(x, -x.abs(), flat, slots=slots, workspace=ws)
        assert B.get_status(ws) == code
        assert (h[1] == 0).all() and torch.equal(flat[:2], before[:2]) and not torch.equal(flat[2], before[2])


def test_gla_step_pool_beyond_32_bit_offsets(B):
    S = 131100   # 2^31 / (128 * 128) = 131072 states of one head
    pool = torch.empty(S, 1, 128, 128, device="cuda")
    gen = torch.Generator().manual_seed(16)
    q, k, v = (torch.randn(2, 1, 128, generator=gen).cuda() for _ in range(3))
    g = -torch.rand(2, 1, 128, generator=gen).cuda()
    slots = torch.tensor([S - 1, 0], dtype=torch.int32).cuda()
    start = torch.randn(2, 1, 128, 128, generator=gen).cuda()
    pool[slots.long()] = start
    o = B.gla_step(q, k, v, g, pool, slots=slots)
    assert torch.equal(o, B.gla_step(q, k, v, g, start)) and torch.equal(pool[slots.long()], start)


def norm_inputs(tx, tr, rows, D, seed=20, with_w=True):
    gen = torch.Generator().manual_seed(seed)
    x = (3 * torch.randn(rows, D, generator=gen)).to(tx)
    res = None if tr is None else torch.randn(rows, D, generator=gen).to(tr)
    return x, res, (1 + 0.2 * torch.randn(D, generator=gen)) if with_w else None


NORM_TYPES = [(T32, T32), (TB, TB), (TH, TH), (TB, T32), (TH, T32), (TB, None), (T32, None)]
NORM_SIZES = [(1, 1), (1, 2048), (5, 7), (33, 64), (130, 128), (3, 100), (9, 1000), (700, 96), (2, 1001), (65, 2048),
              (4, 4104), (3, 8192), (2, 16384), (2, 10007), (1, 16383)]


@pytest.mark.parametrize("types", NORM_TYPES, ids=lambda t: "-".join(KIND.get(x, "none") for x in t))
@pytest.mark.parametrize("rows,D", NORM_SIZES)
def test_norm_forward(B, rows, D, types):
    x, res, w = norm_inputs(*types, rows, D, with_w=rows != 33)
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    y, s, rstd = B.norm_fwd(dev(x), residual=dev(res), weight=dev(w), eps=1e-5)
    ry, rs, rr = lo.norm_fwd(f64(x), f64(res), f64(w), 1e-5)
    within(y, ry, 60 * lo.U * np.abs(ry), "y")
    within(rstd, rr, lo.RSTD_TOL * rr, "rstd")
    if res is not None:
        within(s, rs, lo.U * np.abs(rs), "s")
    for group in (0, 128):
        q, scales, s8, rstd8 = B.norm_quant_fwd(dev(x), residual=dev(res), weight=dev(w), eps=1e-5, group=group)
        assert torch.equal(rstd8, rstd) and torch.equal(s8, s)
        rscales, wide = lo.quant_scales(ry, group)
        within(scales, rscales, 64 * lo.U * rscales, "scales")
        v, got = ry / wide, q.float().cpu().double().numpy()
        step = np.maximum(np.abs(v) * 2.0 ** -4, 2.0 ** -10)   # half a step of e4m3
        assert (np.abs(got - v) <= step + 80 * lo.U * np.abs(v)).all()


@pytest.mark.parametrize("types", [t for t in NORM_TYPES if t[1] is not None],
                         ids=lambda t: "-".join(KIND.get(x, "none") for x in t))
@pytest.mark.parametrize("rows,D", NORM_SIZES)
def test_norm_backward(B, rows, D, types):
    tx, tr = types
    dy, s, w = norm_inputs(tx, tr, rows, D, seed=21)
    ds = None if rows == 5 else torch.randn(rows, D, generator=torch.Generator().manual_seed(22)).to(tr)
    rstd = (s.float().square().mean(-1) + 1e-5).rsqrt()
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    dx, dres, dw = B.norm_bwd(dev(s), dev(rstd), dev(dy), weight=dev(w), ds=dev(ds))
    grad, rdw, tol, tol_w = lo.norm_bwd(f64(s), f64(rstd), f64(w), f64(dy), f64(ds))
    within(dx, grad, tol, "dx")
    within(dres, grad, tol, "dres")
    within(dw, rdw, tol_w, "dw")
    assert dx.dtype == tx and dres.dtype == tr


@pytest.mark.parametrize("types", [(TB, TB), (TH, T32), (T32, T32)], ids=lambda t: "-".join(KIND[x] for x in t))
@pytest.mark.parametrize("rows,D", [(30001, 19), (9001, 130), (5001, 257), (3001, 517), (2001, 1001), (901, 2049), (701, 8001),
                                    (700, 8186)])
def test_norm_shifted_rows(B, rows, D, types):
    """Rows that start anywhere in a 16-byte unit, several turns of the grid, every output."""
    test_norm_forward(B, rows, D, types)
    test_norm_backward(B, rows, D, types)


@pytest.mark.parametrize("types", [(TB, TB), (TH, T32), (T32, T32)], ids=lambda t: "-".join(KIND[x] for x in t))
@pytest.mark.parametrize("rows,D", [(3001, 2048), (1301, 4096), (700, 4104), (457, 8192), (305, 8176)])
def test_norm_wide_rows_in_turns(B, rows, D, types):
    """Rows on whole units, several to a CTA one after the other, the last turn with fewer of them."""
    test_norm_forward(B, rows, D, types)
    test_norm_backward(B, rows, D, types)


@pytest.mark.parametrize("types", [(TB, TB), (TH, T32), (T32, T32)], ids=lambda t: "-".join(KIND[x] for x in t))
@pytest.mark.parametrize("rows,D", [(2, 3), (3, 1), (7, 2), (11, 3), (2, 5)])
def test_norm_rows_shorter_than_a_unit(B, rows, D, types):
    """Several rows in one 16-byte unit, the tensor's end inside it."""
    test_norm_forward(B, rows, D, types)
    test_norm_backward(B, rows, D, types)


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("tx", [TB, T32], ids=KIND.get)
@pytest.mark.parametrize("D", [3, 203, 1001])
def test_norm_shifted_rows_beside_nan(B, D, tx, group):
    """What a row reads of its neighbours' 16-byte units does not reach it: ordinary rows keep their bits."""
    x, res, w = (t.cuda() for t in norm_inputs(tx, tx, 9, D, seed=33))
    ok = torch.arange(9) % 2 == 0

    def run():
        y, s, rstd = B.norm_fwd(x, residual=res, weight=w)
        q, scales, _, _ = B.norm_quant_fwd(x, residual=res, weight=w, group=group)
        dx, _, _ = B.norm_bwd(s, rstd, x, weight=w, ds=res)
        return [t[ok] for t in (y, s, rstd, q.view(torch.uint8), scales, dx)]

    clean = run()
    x[~ok], res[~ok] = float("nan"), float("inf")
    for a, b in zip(clean, run()):
        assert torch.equal(a, b)


@pytest.mark.parametrize("rows,D", [(20011, 136), (3001, 1024)])
def test_norm_backward_many_rows(B, rows, D):
    dy, s, w = norm_inputs(TB, TB, rows, D, seed=23)
    rstd = (s.float().square().mean(-1) + 1e-5).rsqrt()
    dx, _, dw = B.norm_bwd(s.cuda(), rstd.cuda(), dy.cuda(), weight=w.cuda())
    grad, rdw, tol, tol_w = lo.norm_bwd(f64(s), f64(rstd), f64(w), f64(dy), None)
    within(dx, grad, tol, "dx")
    within(dw, rdw, tol_w, "dw")
    again = B.norm_bwd(s.cuda(), rstd.cuda(), dy.cuda(), weight=w.cuda())
    assert torch.equal(dw, again[2]) and torch.equal(dx, again[0])


def test_norm_gradient_against_differences(B):
    x, res, w = norm_inputs(T32, T32, 40, 90, seed=24)
    r = np.random.default_rng(25)
    dy, ds = (r.standard_normal(x.shape).astype("f4") for _ in range(2))
    _, s, rstd = B.norm_fwd(x.cuda(), residual=res.cuda(), weight=w.cuda(), eps=1e-5)
    dx, _, dw = B.norm_bwd(s, rstd, torch.tensor(dy).cuda(), weight=w.cuda(), ds=torch.tensor(ds).cuda())
    args = [f64(x), f64(res), f64(w)]

    def loss(args):
        y, t, _ = lo.norm_fwd(*args, 1e-5)
        return (y * dy).sum() + (t * ds).sum()

    _, _, tol, tol_w = lo.norm_bwd(f64(s), f64(rstd), f64(w), dy, ds)
    for i, (grad, t) in enumerate(((dx, tol), (dx, tol), (dw, tol_w))):
        v = r.standard_normal(args[i].shape)
        up, down = ([a + e * v if j == i else a for j, a in enumerate(args)] for e in (1e-5, -1e-5))
        slope, got = (loss(up) - loss(down)) / 2e-5, (f64(grad) * v).sum()
        # s and rstd carry roundings of u and RSTD_TOL, at which the gradient is evaluated
        allowed = ((t + (4 * lo.RSTD_TOL + 2 * lo.U) * (np.abs(f64(grad)) + 1)) * np.abs(v)).sum()
        assert abs(slope - got) <= allowed + 1e-6 * (1 + abs(slope))


def test_norm_special_rows(B):
    """Rows of zeros, infinities and NaN beside ordinary ones, which stay what they are."""
    x, res, w = norm_inputs(TB, T32, 6, 200, seed=26)
    x, res, w = x.cuda(), res.cuda(), w.cuda()
    clean = B.norm_fwd(x, residual=res, weight=w)
    clean8 = B.norm_quant_fwd(x, residual=res, weight=w, group=128)
    x[1], res[1] = 0, 0
    x[2, 5] = float("nan")
    x[3, 150] = float("inf")
    res[4, 7] = 3e38   # the square overflows: rstd is 0
    y, s, rstd = B.norm_fwd(x, residual=res, weight=w)
    q, scales, _, _ = B.norm_quant_fwd(x, residual=res, weight=w, group=128)
    for row in (0, 5):
        assert torch.equal(y[row], clean[0][row]) and torch.equal(q[row].float(), clean8[0][row].float())
    assert (y[1] == 0).all() and (q[1].float() == 0).all() and (scales[1] == torch.tensor(1e-30, device="cuda")).all()
    assert torch.isnan(y[2]).all() and torch.isnan(q[2].float()).all() and torch.isnan(scales[2]).all()
    assert rstd[3] == 0 and torch.isnan(y[3, 150]) and (y[3, :150] == 0).all()
    assert torch.isnan(scales[3, 1]) and torch.isnan(q[3, 128:].float()).all() and (q[3, :128].float() == 0).all()
    assert rstd[4] == 0 and (y[4] == 0).all()


def test_norm_in_place_and_leading_shape(B):
    x, res, w = norm_inputs(TB, TB, 12, 96, seed=27)
    x, res, w = x.cuda().view(3, 4, 96), res.cuda().view(3, 4, 96), w.cuda()
    y, s, rstd = B.norm_fwd(x, residual=res, weight=w)
    assert y.shape == (3, 4, 96) and rstd.shape == (3, 4)
    y2 = torch.empty_like(y)
    rc = B.lib().gla_norm_fwd(x.data_ptr(), res.data_ptr(), w.data_ptr(), y2.data_ptr(), res.data_ptr(), None, 12, 96, 1e-6,
                              B.GLA_BF16, torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and torch.equal(y2, y) and torch.equal(res, s)
    dy, ds = torch.randn_like(y), torch.randn_like(y)
    dx, _, dw = B.norm_bwd(s, rstd, dy, weight=w, ds=ds)
    ws = torch.empty(int(B.lib().gla_norm_bwd_workspace_size(12, 96)), dtype=torch.uint8, device="cuda")
    rc = B.lib().gla_norm_bwd(s.data_ptr(), rstd.data_ptr(), w.data_ptr(), dy.data_ptr(), ds.data_ptr(), None,
                              ds.data_ptr(), None, 12, 96, B.GLA_BF16, ws.data_ptr(), ws.numel(),
                              torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and torch.equal(ds, dx)   # the gradient of the residual over ds in place
    empty = torch.empty(0, 96, device="cuda", dtype=TB)
    assert B.norm_fwd(empty, residual=empty, weight=w)[0].shape == (0, 96)
    dx, _, dw = B.norm_bwd(empty, torch.empty(0, device="cuda"), empty, weight=w)
    assert (dw == 0).all()


def test_norm_rows_beyond_32_bit_offsets(B):
    rows, D = 270000, 8192   # 2.2e9 elements
    x = torch.zeros(rows, D, dtype=TB, device="cuda")
    x[-2:] = torch.randn(2, D, device="cuda")
    w = torch.randn(D, device="cuda")
    y, _, rstd = B.norm_fwd(x, weight=w)
    y1, _, rstd1 = B.norm_fwd(x[-2:].contiguous(), weight=w)
    assert torch.equal(y[-2:], y1) and torch.equal(rstd[-2:], rstd1) and (y[:1000] == 0).all()
    dx, _, dw = B.norm_bwd(x, rstd, y, weight=w)
    dx1, _, dw1 = B.norm_bwd(x[-2:].contiguous(), rstd1, y1, weight=w)
    assert torch.equal(dx[-2:], dx1)
    np.testing.assert_allclose(f64(dw), f64(dw1), rtol=1e-6)   # the other rows add zeros


def test_calls_on_another_stream(B):
    """Outputs and workspaces belong to the stream that the call runs on."""
    x, g, h0, _ = scan_inputs((TB, TB), 2, 900, 256, seed=28)
    x, g, h0 = x.cuda(), g.cuda(), h0.cuda()
    w = torch.ones(256, device="cuda")
    ref = B.scan_fwd(x, g, initial_state=h0)
    ref_n = B.norm_bwd(x, torch.ones(2, 900, device="cuda"), g, weight=w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        a = B.scan_fwd(x, g, initial_state=h0, stream=side)
        b = B.norm_bwd(x, torch.ones(2, 900, device="cuda"), g, weight=w, stream=side)
        B.scan_fwd(x, g, initial_state=h0)
        side.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(a, ref)) and all(torch.equal(p, q) for p, q in zip(b, ref_n))


def test_calls_in_a_graph(B):
    """One token through norm, recurrence and GLA update, captured once and replayed on new inputs."""
    D, H = 256, 2
    x, w = torch.randn(4, D, device="cuda").to(TB), torch.ones(D, device="cuda")
    state, pool = torch.zeros(4, D, device="cuda"), torch.zeros(4, H, 128, 128, device="cuda")

    def token():
        y, _, _ = B.norm_fwd(x, weight=w)
        h = B.scan_step(y, -y.abs(), state)
        qkv = h.view(4, H, 128)
        return B.gla_step(qkv, qkv, qkv, -qkv.abs(), pool)

    token()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = token()
    for seed in range(3):
        x.copy_(torch.randn(4, D, generator=torch.Generator().manual_seed(seed)).to(TB))
        kept, kept_pool = state.clone(), pool.clone()
        graph.replay()
        got, after, after_pool = o.clone(), state.clone(), pool.clone()
        state.copy_(kept)
        pool.copy_(kept_pool)
        assert torch.equal(token(), got) and torch.equal(state, after) and torch.equal(pool, after_pool)


def test_binding_refusals(B):
    x = torch.randn(2, 8, 64, device="cuda")
    code = lambda e: e.value.code  # noqa: E731
    for call in (lambda: B.scan_fwd(x[0], x[0]),                                       # not [B, T, D]
                 lambda: B.scan_fwd(x, x[:, :4]),
                 lambda: B.scan_fwd(x.transpose(1, 2).contiguous().transpose(1, 2), x),  # channels not adjacent
                 lambda: B.scan_fwd(x, x, initial_state=torch.zeros(3, 64, device="cuda")),
                 lambda: B.scan_fwd(x, x, cu_seqlens=torch.zeros(2, device="cuda", dtype=torch.int64)),
                 lambda: B.scan_fwd(x.cpu(), x.cpu()),
                 lambda: B.scan_bwd(x, x, x[:, :4]),
                 lambda: B.scan_step(x[0], x[0], torch.zeros(3, 64, device="cuda")),
                 lambda: B.scan_step(x[0], x[0], torch.zeros(8, 64, device="cuda"), slots=torch.zeros(4, device="cuda")),
                 lambda: B.gla_step(x, x, x, x, torch.zeros(2, 8, 64, 32, device="cuda")),
                 lambda: B.norm_fwd(x, residual=x[:1]),
                 lambda: B.norm_fwd(x.transpose(0, 1)),
                 lambda: B.norm_fwd(x, weight=torch.ones(63, device="cuda")),
                 lambda: B.norm_bwd(x, torch.ones(2, device="cuda"), x)):
        with pytest.raises(B.GlaError) as e:
            call()
        assert code(e) == B.GLA_ERR_INVALID_ARG
    for call in (lambda: B.scan_fwd(x.double(), x.double()), lambda: B.scan_fwd(x, x.bfloat16()),
                 lambda: B.gla_step(x, x, x, x, torch.zeros(2, 8, 64, 64, device="cuda"), out_dtype=TB),
                 lambda: B.norm_fwd(x.double()), lambda: B.norm_fwd(x.bfloat16(), residual=x.half()),
                 lambda: B.norm_quant_fwd(x, group=64)):
        with pytest.raises(B.GlaError) as e:
            call()
        assert code(e) == B.GLA_ERR_UNSUPPORTED
    with pytest.raises(B.GlaError) as e:   # a column range that starts off the 16-byte grid
        B.scan_fwd(torch.randn(2, 8, 130, device="cuda")[..., 1:65], x)
    assert code(e) == B.GLA_ERR_ALIGNMENT


def test_kernel_names(B):
    x, w = torch.randn(2, 40, 64, device="cuda"), torch.ones(64, device="cuda")
    timer = B.KernelTimer()
    cu = torch.arange(0, 2001, 2, dtype=torch.int32, device="cuda")   # enough sequences for both kernels
    pack = torch.randn(1, 2000, 128, device="cuda")
    for call, names in ((lambda: B.scan_fwd(pack, -pack.abs(), cu_seqlens=cu), ["scan_fwd_rows", "scan_fwd"]),
                        (lambda: B.scan_bwd(pack, pack, pack, cu_seqlens=cu), ["scan_bwd_rows", "scan_bwd"]),
                        (lambda: B.scan_fwd(x[:, :9].contiguous(), x[:, :9].contiguous()), ["scan_fwd_rows"]),
                        (lambda: B.scan_fwd(x, -x.abs()), ["scan_fwd"]), (lambda: B.scan_bwd(x, x, x), ["scan_bwd"]),
                        (lambda: B.scan_step(x[0], x[0], x[0].clone()), ["scan_step"]),
                        (lambda: B.gla_step(x, x, x, x, torch.zeros(2, 40, 64, 64, device="cuda")), ["gla_step"]),
                        (lambda: B.norm_fwd(x, weight=w), ["norm_fwd"]),
                        (lambda: B.norm_quant_fwd(x, weight=w), ["norm_quant_fwd"]),
                        (lambda: B.norm_bwd(x, x[..., 0].contiguous(), x, weight=w), ["norm_bwd", "norm_dw"])):
        with timer:
            call()
        torch.cuda.synchronize()
        assert [n for n, _ in timer.results()] == names


def test_short_and_checked_calls_agree(B):
    """The usual calls go the short way (a workspace argument sends the same call the checked one), to the same results."""
    x, g, h0, cu = (t.cuda() for t in scan_inputs((TB, TB), 1, 0, 96, [30, 0, 200], seed=40))
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    B.scan_fwd(x, g)   # the status workspace exists from here on
    h, ht = B.scan_fwd(x, g, h0, cu_seqlens=cu)
    pool, slots = torch.randn(5, 96, device="cuda"), torch.tensor([4, 1], dtype=torch.int32).cuda()
    q = torch.randn(2, 3, 64, device="cuda").to(TH)
    states = torch.randn(2, 3, 64, 64, device="cuda")
    w, res = torch.randn(96, device="cuda"), torch.randn(1, 230, 96, device="cuda")
    rows, x2 = x[0, :2].contiguous(), -x[0, 2:4].abs().contiguous()
    short = [B._calls.scan_fwd(x, g, h0, True, cu, None), B._calls.scan_fwd(x, g, None, False, None, T32),
             B._calls.scan_bwd(g, h, x, h0, ht, cu, None, True), B._calls.scan_bwd(g, h, x, None, None, None, TB, False),
             B._calls.scan_step(rows, x2, pool.clone(), slots, None, T32),
             B._calls.gla_step(q, q, q, -q.abs(), states.clone(), None, None, None, TH),
             B._calls.gla_step(q, q, q, -q.abs(), states.clone(), 0.25, None, None, None),
             B._calls.norm_fwd(x, res, w, 1e-6), B._calls.norm_fwd(x, None, None, 1e-6),
             B._calls.norm_quant_fwd(x, res, w, 1e-6, 0), B._calls.norm_quant_fwd(x, None, w, 1e-6, 128),
             B._calls.norm_bwd(res, res[..., 0].contiguous(), x, w, res, True, ws),
             B._calls.norm_bwd(x, res[..., 0].contiguous(), x, w, None, False, ws)]
    checked = [B._scan_fwd_checked(x, g, h0, True, cu, None, None, ws, stream=None),
               B._scan_fwd_checked(x, g, None, False, None, T32, None, ws, stream=None),
               B._scan_bwd_checked(g, h, x, h0, ht, cu, None, True, None, None, ws, stream=None),
               B._scan_bwd_checked(g, h, x, None, None, None, TB, False, None, None, ws, stream=None),
               B._scan_step_checked(rows, x2, pool.clone(), slots, None, T32, ws, stream=None),
               B._gla_step_checked(q, q, q, -q.abs(), states.clone(), None, None, None, TH, ws, stream=None),
               B._gla_step_checked(q, q, q, -q.abs(), states.clone(), 0.25, None, None, None, ws, stream=None),
               B._norm_fwd_checked(x, res, w, 1e-6, stream=None), B._norm_fwd_checked(x, None, None, 1e-6, stream=None),
               B._norm_quant_fwd_checked(x, res, w, 1e-6, 0, stream=None),
               B._norm_quant_fwd_checked(x, None, w, 1e-6, 128, stream=None),
               B._norm_bwd_checked(res, res[..., 0].contiguous(), x, w, res, True, ws, stream=None),
               B._norm_bwd_checked(x, res[..., 0].contiguous(), x, w, None, False, ws, stream=None)]
    for a, b in zip(short, checked):
        a, b = (v if isinstance(v, tuple) else (v,) for v in (a, b))
        assert len(a) == len(b)
        for p, r in zip(a, b):
            assert (p is None) == (r is None)
            if p is not None:
                assert p.dtype == r.dtype and p.shape == r.shape and torch.equal(p.float(), r.float())
    out = B.norm_bwd(x, res[..., 0].contiguous(), x, weight=w)
    assert out[0] is out[1]
    for unusual in ((x.cpu(), g, None, True, None, None), (x[..., ::2], g, None, True, None, None),
                    (x, g.float(), None, True, None, TB), (x, g[:, :5], None, True, None, None),
                    (x, g, h0[:1], True, cu, None), (x, g, h0.half(), True, cu, None), (1, g, None, True, None, None),
                    (x, g, None, True, cu.long(), None), (x[0], g[0], None, True, None, None)):
        assert B._calls.scan_fwd(*unusual) is None
    assert B._calls.gla_step(q, q, q, q, states[:1], None, None, None, None) is None
    assert B._calls.gla_step(q, q, q, q, states, -1.0, None, None, None) is None
    assert B._calls.norm_fwd(x, res.half(), w, 1e-6) is None
    assert B._calls.norm_quant_fwd(x, None, w, 1e-6, 64) is None
