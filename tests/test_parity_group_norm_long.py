"""The group norm where a thread has many rows: statistics beside outliers, and sums of weight gradients, against fp64 on the
device."""
import pytest
import torch

import delta_oracle as do
from test_parity_group_norm import B, T32, TB, TH, _built   # noqa: F401

pytestmark = pytest.mark.gpu


def statistics(x, G):
    """mean, rstd (eps 1e-5) and the mean magnitude of each group, in fp64, sample by sample."""
    out = []
    for t in x:
        p = t.double().reshape(-1, G, x.shape[-1] // G)
        mean = p.mean((0, 2))
        out.append((mean, ((p - mean[:, None]).square().mean((0, 2)) + 1e-5).rsqrt(), p.abs().mean((0, 2))))
    return [torch.stack(t) for t in zip(*out)]


@pytest.mark.parametrize("dtype", [T32, TB], ids=["f32", "bf16"])
@pytest.mark.parametrize("value", [1e4, -300.0])
def test_outliers_before_many_rows(B, dtype, value):   # noqa: F811
    """An outlier as the first value that a thread has, of some thousand: its squares are sums over blocks of at most 32 rows about
    a value near the block's, which lose at most 32 units to the cancellation, and the blocks' join is a sum of what they are: the
    bound on sums as it stands."""
    N, S, C, G = 304, 65536, 16, 1
    x = torch.randn(N, S, C, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(dtype)
    x[:, 0] = value
    x[::2, 1] = 3 * value
    _, mean, rstd = B.group_norm_fwd(x, G)
    m, r, size = statistics(x, G)
    assert ((mean - m).abs() <= do.SUM * size).all()
    off = ((rstd - r) / r).abs()
    assert (off <= do.SUM + (do.SUM * size * r) ** 2).all(), f"{off.max()} off"


def test_means_far_from_zero_over_many_rows(B):   # noqa: F811
    x = torch.randn(304, 65536, 16, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)) + 1000
    _, mean, rstd = B.group_norm_fwd(x, 4)
    m, r, size = statistics(x, 4)
    assert ((mean - m).abs() <= 16 * do.U * size).all()   # of 1000 itself, not of a sum of them
    assert ((rstd - r) / r).abs().max() <= do.SUM


@pytest.mark.parametrize("shape,G", [((1 << 21, 1040), 8), ((2, 1 << 20, 1040), 8)], ids=str)
def test_sums_over_two_million_rows(B, shape, G):   # noqa: F811
    """mean, rstd, dw and db of more than 2^31 values.  A thread adds as many values one after the other as its lanes have
    groups (three CTAs an SM of eight groups of 130 channels; a slice's rows where there are positions), then come at most 512
    partial sums of 32 threads, and their join: so many roundings of the sums' magnitudes."""
    gen = torch.Generator(device="cuda").manual_seed(8)
    C, sms = shape[-1], torch.cuda.get_device_properties(0).multi_processor_count
    x = torch.randn(shape, device="cuda", generator=gen, dtype=TB)
    dy = torch.randn(shape, device="cuda", generator=gen, dtype=TB)
    w = torch.rand(C, device="cuda", generator=gen) + 0.5
    _, mean, rstd = B.group_norm_fwd(x, G, weight=w, bias=w)
    _, dw, db = B.group_norm_bwd(x, mean, rstd, dy, weight=w, bias=w)
    tokens = len(shape) == 2
    count = (shape[0] * G // (3 * sms * 8) if tokens else shape[1] // (sms * 2 // shape[0])) + 1 + 512 + 40
    sums = torch.zeros(4, C, device="cuda", dtype=torch.float64)
    for n in range(0, shape[0], 1 << 15 if tokens else 1):
        part, grad = x[n:n + (1 << 15)], dy[n:n + (1 << 15)]
        if tokens:
            m, r, size = (t.squeeze(1) for t in _moments(part.reshape(-1, 1, G, C // G)))
            assert ((mean[n:n + (1 << 15)] - m).abs() <= do.SUM * size).all()
            assert ((rstd[n:n + (1 << 15)] / r - 1).abs() <= do.SUM).all()
            blocks = [(part, grad, mean[n:n + (1 << 15)], rstd[n:n + (1 << 15)])]
        else:
            part, grad = x[n], dy[n]
            total, square = torch.zeros(2, G, device="cuda", dtype=torch.float64)
            for lo in range(0, shape[1], 1 << 15):
                p = part[lo:lo + (1 << 15)].double().reshape(-1, G, C // G)
                total += p.sum((0, 2))
                square += p.square().sum((0, 2))   # the mean is near zero: nothing cancels
            m = total / (shape[1] * (C // G))
            r = (square / (shape[1] * (C // G)) - m * m + 1e-5).rsqrt()
            assert ((mean[n] - m).abs() <= do.SUM).all() and ((rstd[n] / r - 1).abs() <= do.SUM).all()
            blocks = [(part[lo:lo + (1 << 15)], grad[lo:lo + (1 << 15)], mean[n:n + 1], rstd[n:n + 1]) for lo in range(0, shape[1], 1 << 15)]
        for p, d, m, r in blocks:
            d = d.double()
            m, r = (t.double().repeat_interleave(C // G, 1) for t in (m, r))
            xh = (p.double() - m) * r
            sums += torch.stack([(d * xh).sum(0), d.sum(0), (d * xh).abs().sum(0), d.abs().sum(0)])
    # xh itself: the difference, and the product with rstd
    assert ((dw - sums[0]).abs() <= (count + 8) * do.U * sums[2] + 4 * do.U * sums[3]).all()
    assert ((db - sums[1]).abs() <= count * do.U * sums[3]).all()


def _moments(p):
    """mean, rstd and the mean magnitude of [N, S, G, W] by sample and group, [N, 1, G] in fp64."""
    p = p.double()
    mean = p.mean((1, 3), keepdim=True)
    return tuple(t.squeeze(3) for t in (mean, ((p - mean).square().mean((1, 3), keepdim=True) + 1e-5).rsqrt(), p.abs().mean((1, 3), keepdim=True)))
