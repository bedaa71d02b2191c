"""README's gated delta layer, run as it stands there."""
import pathlib
import re

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16], ids=["f32", "bf16", "f16"])
def test_recipe_with_keys_of_zero(dtype):
    """Rows of padding have keys (and queries and values) of zero: they come out as numbers, and store nothing."""
    import __graft_entry__
    __graft_entry__.build()
    from chunkwise_gated_linear_chunked_gb300 import binding
    text = (pathlib.Path(__file__).parent.parent / "README.md").read_text()
    code, = (c for c in re.findall(r"```python\n(.*?)```", text, re.S) if "delta_bwd" in c)
    B, T, H, HV, K, V = 1, 70, 2, 4, 64, 64
    gen = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=gen)   # noqa: E731
    q, k, v = (rand(B, T, n, 64).to(dtype) for n in (H, H, HV))
    for t in (q, k, v):
        t[:, 60:] = 0
    g, beta = -rand(B, T, HV).abs(), rand(B, T, HV).sigmoid()
    space = dict(torch=torch, binding=binding, B=B, T=T, H=H, HV=HV, K=K, V=V, q=q, k=k, v=v, g=g, beta=beta, h0=0.1 * rand(B, HV, K, V),
                 cu=torch.tensor([0, T], dtype=torch.int32, device="cuda"), w=rand(HV * V), b=rand(HV * V), dy=rand(B * T, HV * V).to(dtype),
                 pool=torch.zeros(2, HV, K, V, device="cuda"), slots=torch.tensor([1], dtype=torch.int32, device="cuda"))
    # one token, of zeros too
    space.update(q1=q[:, -1].contiguous(), k1=k[:, -1].contiguous(), v1=v[:, -1].contiguous(), g1=g[:, -1].contiguous(), beta1=beta[:, -1].contiguous())
    exec(code, space)
    assert binding.layer_status() == binding.GLA_OK
    for name in ("k", "rstd", "o", "ht", "y", "do", "dq", "dk", "dv", "dg", "dbeta", "dh0", "pool"):
        assert torch.isfinite(space[name]).all(), name
    assert (space["k"][:, 60:] == 0).all()
    length = space["k"][:, :60].float().norm(dim=-1)
    assert (length - 1).abs().max() <= 2 ** -7   # half a step of bf16 a value, and the norm's
    # and back through the norm of the keys
    dk = binding.norm_bwd(k, space["rstd"], space["dk"], weight=space["unit"], want_dw=False)[0]
    assert torch.isfinite(dk).all()
