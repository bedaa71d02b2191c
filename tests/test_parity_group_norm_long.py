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
