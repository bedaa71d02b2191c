"""The norm's backward on wide rows, several to a CTA: by registers and by shared memory, on either side of the rule that
chooses, against the plain fp64 form."""
import pytest
import torch

from test_parity_layers import KIND, T32, TB, TH, test_norm_backward as check_backward

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    import __graft_entry__
    __graft_entry__.build()
    from chunkwise_gated_linear_chunked_gb300 import binding
    return binding


@pytest.mark.parametrize("types", [(TB, TB), (TH, TH), (TB, T32), (T32, T32)], ids=lambda t: "-".join(KIND[x] for x in t))
@pytest.mark.parametrize("rows,D", [(901, 3600), (901, 4096), (701, 4500), (501, 7000), (501, 8000), (501, 8184)])
def test_backward(B, rows, D, types):
    check_backward(B, rows, D, types)
    # the same bits again, and a single turn's rows alone give the same gradients
    gen = torch.Generator(device="cuda").manual_seed(D)
    s, ds = (torch.randn(rows, D, device="cuda", generator=gen).to(types[1]) for _ in range(2))
    dy, w = torch.randn(rows, D, device="cuda", generator=gen).to(types[0]), torch.rand(D, device="cuda", generator=gen)
    rstd = (s.float().square().mean(-1) + 1e-5).rsqrt()
    dx, dres, dw = B.norm_bwd(s, rstd, dy, weight=w, ds=ds)
    again = B.norm_bwd(s, rstd, dy, weight=w, ds=ds)
    assert torch.equal(dx, again[0]) and torch.equal(dres, again[1]) and torch.equal(dw, again[2])
    few = B.norm_bwd(s[:8], rstd[:8], dy[:8], weight=w, ds=ds[:8])
    assert torch.equal(dx[:8], few[0]) and torch.equal(dres[:8], few[1])
