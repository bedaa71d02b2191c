"""The vector-state recurrence with gates above zero.  Sums of gates over a stretch of rows may leave the range of an
fp32 exponential while every state, and every row's share of it, stays inside: the answer is then finite, whatever
the length, the layout and the number of CTAs that a sequence is cut over."""
import numpy as np
import pytest
import torch

import layer_oracle as lo

pytestmark = pytest.mark.gpu

T32, TB, TH = torch.float32, torch.bfloat16, torch.float16
KIND = {T32: "f32", TB: "bf16", TH: "f16"}
TYPES = [(T32, T32, T32), (TB, TB, T32), (TB, TB, TB), (TH, TH, T32), (TB, T32, T32)]   # x, gate, output
# sequences, rows, channels: threads alone; one tile; clusters (rows on whole units, in pairs, anywhere); many sequences
SIZES = [(2, 16, 64), (1, 128, 64), (1, 700, 64), (2, 900, 66), (1, 700, 33), (1, 5000, 64), (400, 300, 64)]


@pytest.fixture(scope="module")
def B():
    import __graft_entry__
    __graft_entry__.build()
    from chunkwise_gated_linear_chunked_gb300 import binding
    return binding


def f64(t):
    return t.detach().cpu().double().numpy()


def gates(kind, T, D, gen):
    """Log-decays [T, D] that rise and fall in turn: their running sums stay within about 130 of where they start, and
    span more than the 88 of an fp32 exponential (slow: 84)."""
    size = 0.9 + 0.2 * torch.rand(T, D, generator=gen)
    turn = 8 if kind == "steep" else 60
    up = (torch.arange(T) // turn) % 4   # +60, +60, -60, -60, ... or the other way round
    sign = torch.where(up < 2, 1.0, -1.0)[:, None]
    return {"rise": size * sign, "fall": -size * sign, "slow": 0.7 * size * sign, "steep": 6 * size * sign}[kind]


def walk(g, start, add, reverse=False):
    """fp64 states s_t = exp(g_t) (s_{t-1} + before) + after of one sequence and their bounds.  ``add`` [T, D] enters
    after the decay (the forward's x) or before it (reverse: the backward's dh, rows last to first; the values returned
    are then those before the decay, with the final state).  Of a row's decay: exp within (4 + |g|) u, product and sum
    2 u; where rows are composed by the sum of their gates, 16 of them at most, u of that sum's parts in each row."""
    T, D = g.shape
    out, tol = np.zeros((T, D)), np.zeros((T, D))
    parts = 16 * np.abs(g).max()
    s, H, W = start.copy(), np.abs(start), np.zeros(D)
    for t in (range(T - 1, -1, -1) if reverse else range(T)):
        a, per = np.exp(g[t]), 6 + np.abs(g[t]) + parts
        if reverse:
            s, H = s + add[t], H + np.abs(add[t])
            out[t], tol[t] = s, lo.U * (W + 100 * H)
            s, H, W = a * s, a * H, a * (W + per * H)
        else:
            s, H, W = a * s + add[t], a * H + np.abs(add[t]), a * (W + per * H)
            out[t], tol[t] = s, lo.U * (W + 100 * H)
    return out, tol, s, lo.U * (W + 100 * H)


def within(x, ref, tol, what):
    got, tol = f64(x), tol + lo.rounding(ref, KIND[x.dtype])
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, the first at {np.argwhere(bad)[0]}: " \
                          f"{got[bad][0]} for {ref[bad][0]}, allowed {tol[bad][0]}"


def in_range(ref):
    """The channels whose fp64 states stay well inside fp32's range, at least two thirds of them."""
    on = np.abs(ref).max(0) < 1e37
    assert on.mean() > 0.66
    return np.flatnonzero(on)


@pytest.mark.parametrize("types", TYPES, ids=lambda t: "-".join(KIND[x] for x in t))
@pytest.mark.parametrize("kind,start", [("rise", 1e-24), ("fall", 1e24), ("slow", 1e-20), ("steep", 1e-24)])
@pytest.mark.parametrize("N,T,D", SIZES)
def test_rise_and_fall(B, N, T, D, kind, start, types):
    """States from a start far from one, that come back to it: forward and backward against fp64.  Every second
    channel starts at zero and stays there until its inputs begin.  Channels whose running sum drifts so far that their
    fp64 states leave fp32's range have no answer; most have one."""
    gen = torch.Generator().manual_seed(T + D)
    g = gates(kind, T, D, gen).to(types[1])
    small = min(start, 1 / start)   # of what is added on the way, wherever the gates' running sum is
    x = (small * torch.randn(T, D, generator=gen)).to(types[0])
    x[:min(T, 400) // 2, ::2] = 0
    h0 = start * torch.randn(D, generator=gen)
    h0[::2] = 0
    many = lambda t: t[None].repeat(N, *[1] * t.dim()).cuda()  # noqa: E731
    h, ht = B.scan_fwd(many(x), many(g), initial_state=many(h0), out_dtype=types[2])
    ref, tol, end, tol_end = walk(f64(g), f64(h0), f64(x))
    on = in_range(ref)
    h, ht = h[..., on], ht[..., on]
    within(h[0], ref[:, on], tol[:, on], "h")
    within(ht[0], end[on], tol_end[on], "ht")
    assert torch.equal(h, h[:1].expand_as(h)) and torch.equal(ht, ht[:1].expand_as(ht))
    if types[0] == TH:
        return   # dx has x's type, whose range ends at 65504
    # backward: the same gates walked from the end; h of order one, as it is given
    rev = g.flip(0)
    hs = torch.randn(T, D, generator=gen).to(types[2])
    dh = (small * torch.randn(T, D, generator=gen)).to(types[2])
    dh[T - min(T, 400) // 2:, ::2] = 0
    dht = start * torch.randn(D, generator=gen)
    dht[::2] = 0
    dx, dg, dh0 = B.scan_bwd(many(rev), many(hs), many(dh), dht=many(dht), dx_dtype=types[0])
    lam, tol, mu, tol_mu = walk(f64(rev), f64(dht), f64(dh), reverse=True)
    on = in_range(lam)
    within(dx[0][:, on], lam[:, on], tol[:, on], "dx")
    within(dh0[0][on], mu[on], tol_mu[on], "dh0")
    prev = np.concatenate([np.zeros((1, D)), f64(hs)[:-1]])
    a = np.exp(f64(rev))
    own = (8 + np.abs(f64(rev))) * lo.U * np.abs(a * lam)   # the row's own decay and two products
    within(dg[0][:, on], (a * lam * prev)[:, on], ((a * tol + own) * np.abs(prev))[:, on], "dg")
    dx, dg = dx[..., on], dg[..., on]
    assert torch.equal(dx, dx[:1].expand_as(dx)) and torch.equal(dg, dg[:1].expand_as(dg))


@pytest.mark.parametrize("N,T,D", SIZES)
def test_zeros_stay_zeros(B, N, T, D):
    """A zero state under growth: zeros, and gradients of zeros likewise."""
    g, z = torch.ones(N, T, D, device="cuda"), torch.zeros(N, T, D, device="cuda")
    h, ht = B.scan_fwd(z, g)
    assert (h == 0).all() and (ht == 0).all()
    dx, dg, dh0 = B.scan_bwd(g, z, z)
    assert (dx == 0).all() and (dg == 0).all() and (dh0 == 0).all()


def test_masked_tail_of_a_gradient(B):
    """No gradient in the last rows and none of the final state, which is what a masked loss leaves."""
    g, h = torch.full((1, 1000, 64), 0.5, device="cuda"), torch.randn(1, 1000, 64, device="cuda")
    dh = torch.zeros(1, 1000, 64, device="cuda")
    dh[:, 99] = 1e-10
    dx, dg, dh0 = B.scan_bwd(g, h, dh)
    assert (dx[:, 100:] == 0).all() and (dg[:, 100:] == 0).all()
    lam, tol, mu, tol_mu = walk(f64(g[0]), np.zeros(64), f64(dh[0]), reverse=True)
    within(dx[0], lam, tol, "dx")
    within(dh0[0], mu, tol_mu, "dh0")


@pytest.mark.parametrize("N,T,D", [(1, 400, 64), (1, 2000, 66), (1, 400, 33), (400, 400, 64)])
def test_an_overflow_stays(B, N, T, D):
    """A state that passes the largest fp32 value is infinite from there on, also when the gates fall again."""
    g = torch.ones(N, T, D, device="cuda")
    g[:, 200:] = -0.25
    h0 = torch.ones(N, D, device="cuda")
    h0[:, 1::2] = -1
    h0[:, ::4] = 0
    h, ht = B.scan_fwd(torch.zeros_like(g), g, initial_state=h0)
    assert torch.equal(h[:, 100:], (h0 * float("inf")).nan_to_num(0, float("inf"), -float("inf"))[:, None].expand(N, T - 100, D))
    assert torch.equal(ht, h[:, -1])


def test_steep_decays(B):
    """Gates below -87.3, whose decays are subnormal: within 2^-126 of the state, beside the relative bound."""
    g = torch.linspace(-104, -80, 64 * 3).repeat_interleave(2).view(3, 2, 64)   # sequences, rows, channels
    x, h0 = torch.zeros(3, 2, 64), torch.full((3, 64), 1e38)
    x[:, 1] = 1
    h, _ = B.scan_fwd(x.cuda(), g.cuda(), initial_state=h0.cuda())
    state = f64(h0)
    for t in range(2):
        gt, xt = f64(g[:, t]), f64(x[:, t])
        ref = np.exp(gt) * state + xt
        tol = np.abs(state) * (np.exp(gt) * (2.0 ** -22 + np.abs(gt) * 2.0 ** -24) + 2.0 ** -126) + 2 * lo.U * np.abs(ref)
        within(h[:, t], ref, tol, f"row {t}")
        state = f64(h[:, t])
