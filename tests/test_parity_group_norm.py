"""GPU parity of the group norm (forward, backward) against the plain fp64 forms of ``delta_oracle``, within their bounds
plus the rounding of an output's type."""
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


def within(got, ref, tol, what):
    tol = tol + lo.rounding(ref, KIND[got.dtype])
    bad = ~(np.abs(f64(got) - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, the first at {np.argwhere(bad)[0]}: {f64(got)[bad][0]} " \
                          f"for {ref[bad][0]}, allowed {tol[bad][0]}"


def check(B, x, G, w, b, act, seed=0, eps=1e-5):
    d = lambda t: None if t is None else t.cuda()   # noqa: E731
    y, mean, rstd = B.group_norm_fwd(d(x), G, weight=d(w), bias=d(b), activation=act, eps=eps)
    refs, tols = do.group_norm_fwd(f64(x), G, f64(w), f64(b), act == "silu", eps)
    for name, got, ref, tol in zip(("y", "mean", "rstd"), (y, mean, rstd), refs, tols):
        within(got, ref, tol, name)
    dy = torch.randn(x.shape, generator=torch.Generator().manual_seed(seed)).to(x.dtype)
    got = B.group_norm_bwd(d(x), mean, rstd, d(dy), weight=d(w), bias=d(b), activation=act)
    refs, tols = do.group_norm_bwd(f64(x), f64(mean), f64(rstd), f64(dy), f64(w), f64(b), act == "silu")
    assert (got[1] is None) == (w is None) and (got[2] is None) == (b is None)
    for name, y, ref, tol in zip(("dx", "dw", "db"), got, refs, tols):
        if y is not None:
            within(y, ref, tol, name)
    return got


SHAPES = [   # shape, groups
    ((1, 8), 1), ((5, 64), 4), ((3, 39), 3), ((130, 2048), 16), ((7, 1000), 8), ((9, 520), 40), ((2, 4096), 1), ((3, 4095), 1),
    ((4, 300), 300), ((40, 1536), 2), ((3, 8200), 2), ((2, 9000), 1),
    ((2, 5, 16), 2), ((3, 7, 5, 24), 4), ((2, 1001, 520), 40), ((1, 300, 13), 13), ((1, 257, 13), 1), ((2, 64, 2056), 8), ((2, 33, 4100), 4),
    ((1, 1, 8), 2), ((2, 3, 3000), 3), ((17, 9, 128), 1), ((1, 1024, 64), 32),
]


@pytest.mark.parametrize("dtype", [T32, TB, TH], ids=lambda t: KIND[t])
@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("shape,G", SHAPES, ids=str)
def test_group_norm(B, dtype, act, shape, G):
    gen = torch.Generator().manual_seed(shape[-1])
    C = shape[-1]
    x = (torch.randn(shape, generator=gen) * (1 + 0.3 * torch.rand(C, generator=gen)) + torch.randn(C, generator=gen)).to(dtype)
    check(B, x, G, 1 + 0.2 * torch.randn(C, generator=gen), 0.3 * torch.randn(C, generator=gen), act)


@pytest.mark.parametrize("shape,G", [((20, 256), 4), ((2, 50, 96), 6)], ids=str)
def test_without_weights(B, shape, G):
    x = torch.randn(shape, generator=torch.Generator().manual_seed(1))
    w, b = torch.full((shape[-1],), 1.5), torch.full((shape[-1],), -0.25)
    for args in ((None, None), (w, None), (None, b)):
        check(B, x, G, *args, "silu")
    d = [t.cuda() for t in B.group_norm_fwd(x.cuda(), G)]
    assert B.group_norm_bwd(x.cuda(), d[1], d[2], x.cuda(), weight=w.cuda(), bias=b.cuda(), want_dw=False)[1:] == (None, None)


@pytest.mark.parametrize("shape,G", [((6, 512), 4), ((2, 700, 64), 8)], ids=str)
def test_mean_far_from_zero(B, shape, G):
    """A mean of 1000 beside a spread of 1: the variance comes from differences, not from squares' differences."""
    gen = torch.Generator().manual_seed(2)
    check(B, torch.randn(shape, generator=gen) + 1000, G, None, None, None)


@pytest.mark.parametrize("shape,G", [((6, 64), 4), ((2, 90, 64), 8)], ids=str)
def test_constants_and_outliers(B, shape, G):
    x = torch.full(shape, 3.0)
    y, mean, rstd = B.group_norm_fwd(x.cuda(), G, eps=1e-4)
    assert (y == 0).all() and (mean == 3).all() and (rstd - 100).abs().max() < 1e-3
    x = torch.randn(shape, generator=torch.Generator().manual_seed(3))
    x.view(shape[0], -1)[:, 0] = 1e4     # the first value of a group, about which sums are taken
    check(B, x, G, None, None, "silu")


@pytest.mark.parametrize("shape,G", [((4, 64), 4), ((2, 90, 64), 8)], ids=str)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nan_stays_in_its_group(B, shape, G, bad):
    x = torch.randn(shape, generator=torch.Generator().manual_seed(4)).cuda()
    want, _, _ = B.group_norm_fwd(x, G)
    x.view(shape[0], -1, G, 64 // G)[1, -1, 2, 3] = bad
    y, mean, rstd = B.group_norm_fwd(x, G)
    hit = torch.zeros_like(x, dtype=torch.bool)
    hit.view(shape[0], -1, G, 64 // G)[1, :, 2] = True
    assert torch.isnan(y[hit]).all() and torch.equal(y[~hit], want[~hit])
    assert torch.isnan(rstd[1, 2]) and torch.isfinite(rstd).sum() == rstd.numel() - 1


def test_repeats_graph_and_other_stream(B):
    for shape, G in (((500, 1024), 8), ((3, 1200, 96), 6)):
        x = torch.randn(shape, generator=torch.Generator().manual_seed(5)).to(TB).cuda()
        w, b = (torch.randn(shape[-1], generator=torch.Generator().manual_seed(i)).cuda() for i in (6, 7))
        call = lambda **kw: B.group_norm_fwd(x, G, weight=w, bias=b, activation="silu", **kw)   # noqa: E731
        want = call()
        back = lambda **kw: B.group_norm_bwd(x, want[1], want[2], x, weight=w, bias=b, activation="silu", **kw)   # noqa: E731
        want_back = back()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = (*call(stream=side), *back(stream=side))
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(p, r) for p, r in zip(got, (*want, *want_back)))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = (*call(), *back())
        for _ in range(2):
            for t in got:
                t.zero_()
            graph.replay()
            assert all(torch.equal(p, r) for p, r in zip(got, (*want, *want_back)))


@pytest.mark.parametrize("shape,G", [((1 << 21, 1040), 8), ((2, 1 << 20, 1040), 8)], ids=str)
def test_offsets_beyond_32_bits(B, shape, G):
    x = torch.randn(shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(8), dtype=TB)
    assert x.numel() > 1 << 31
    w = torch.randn(shape[-1], device="cuda")
    y, mean, rstd = B.group_norm_fwd(x, G, weight=w, bias=w, activation="silu")
    one = B.group_norm_fwd(x[-1:].contiguous(), G, weight=w, bias=w, activation="silu")
    # one sample alone is cut into other slices: statistics within their bound of one another
    assert (mean[-1:] - one[1]).abs().max() <= 2 * do.SUM and ((rstd[-1:] - one[2]) / one[2]).abs().max() <= 4 * do.SUM
    assert (y[-1:].float() - one[0].float()).abs().max() <= 2 ** -7 * one[0].abs().max()   # neighbours in bf16
    del y
    dx, dw, db = B.group_norm_bwd(x, mean, rstd, x, weight=w, bias=w, activation="silu")
    alone = B.group_norm_bwd(x[-1:].contiguous(), mean[-1:].contiguous(), rstd[-1:].contiguous(), x[-1:].contiguous(), weight=w, bias=w,
                             activation="silu")[0]
    assert (dx[-1:].float() - alone.float()).abs().max() <= 2 ** -7 * alone.abs().max()


def test_nothing_to_do(B):
    x, w = torch.zeros(0, 7, 64, device="cuda"), torch.ones(64, device="cuda")
    y, mean, rstd = B.group_norm_fwd(x, 4, weight=w)
    assert y.shape == x.shape and mean.shape == (0, 4)
    dx, dw, db = B.group_norm_bwd(x, mean, rstd, x, weight=w, bias=w)
    assert dx.shape == x.shape and (dw == 0).all() and (db == 0).all()


def test_refusals(B):
    x, w = torch.zeros(4, 6, 64, device="cuda"), torch.ones(64, device="cuda")
    mean = torch.zeros(4, 8, device="cuda")
    bad = [lambda: B.group_norm_fwd(x.cpu(), 4), lambda: B.group_norm_fwd(x, 5), lambda: B.group_norm_fwd(x, 0),
           lambda: B.group_norm_fwd(x[..., 0, 0], 1), lambda: B.group_norm_fwd(x.transpose(0, 1), 4), lambda: B.group_norm_fwd(x.double(), 4),
           lambda: B.group_norm_fwd(x, 4, weight=w.half()), lambda: B.group_norm_fwd(x, 4, bias=w[:32]), lambda: B.group_norm_fwd(x, 4, activation="gelu"),
           lambda: B.group_norm_fwd(x, 4, eps=-1.0), lambda: B.group_norm_fwd(x[:, :0], 4),
           lambda: B.group_norm_bwd(x, mean[:3], mean, x), lambda: B.group_norm_bwd(x, mean, mean, x.bfloat16()),
           lambda: B.group_norm_bwd(x, mean, mean[:, :4], x), lambda: B.group_norm_bwd(x, mean[0], mean[0], x)]
    for i, call in enumerate(bad):
        with pytest.raises(B.GlaError):
            call()
            pytest.fail(f"call {i} was not refused")
