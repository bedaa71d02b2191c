"""The binding's short way (the _calls module) and its checked way give the same results, for the gated delta rule and the
group norm."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def calls(B):
    gen = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=gen)   # noqa: E731
    out = []
    for dtype in (torch.float32, torch.bfloat16):
        q, k, v = (0.1 * rand(1, 150, n, 64) for n in (2, 2, 4))
        q, k, v, g, beta = q.to(dtype), k.to(dtype), v.to(dtype), -rand(1, 150, 4).abs(), rand(1, 150, 4).sigmoid()
        cu, h0 = torch.tensor([0, 70, 70, 150], dtype=torch.int32, device="cuda"), rand(3, 4, 64, 64)
        for kw in (dict(), dict(cu_seqlens=cu, initial_state=h0, scale=0.3)):
            out += B.delta_fwd(q, k, v, g, beta, **kw)
            out += B.delta_bwd(q, k, v, g, beta, v, **kw)
        out.append(B.delta_fwd(q, k, v, g, beta, output_final_state=False, out_dtype=torch.float32)[0])
        out += B.delta_bwd(q, k, v, g, beta, v, want_dh0=False)[:5]
        pool, slots = rand(160, 4, 64, 64), torch.randperm(160, device="cuda", generator=gen)[:150].to(torch.int32)
        out += [B.delta_step(q[0], k[0], v[0], g[0], beta[0], pool, slots=slots, out_dtype=torch.float32), pool]
        for x, groups in ((v.reshape(150, 256), 4), (v, 16)):
            y, mean, rstd = B.group_norm_fwd(x, groups, activation="silu")
            w, b = rand(x.shape[-1]), rand(x.shape[-1])
            out += [y, mean, rstd, *B.group_norm_fwd(x, groups, weight=w, bias=b, eps=1e-3)]
            out += B.group_norm_bwd(x, mean, rstd, x, weight=w, bias=b, activation="silu")
            out.append(B.group_norm_bwd(x, mean, rstd, x, weight=w, want_dw=False)[0])
    return out


def test_both_ways_agree(monkeypatch):
    from chunkwise_gated_linear_chunked_gb300 import binding as B
    assert not isinstance(B._calls, B._NoCalls)
    taken = []
    real = B._calls

    class Counted:
        def __getattr__(self, name):
            def call(*args):
                got = getattr(real, name)(*args)
                taken.append((name, got is not None))
                return got
            return call

    monkeypatch.setattr(B, "_calls", Counted())
    short = calls(B)
    assert len(taken) == 30 and all(t for _, t in taken), [n for n, t in taken if not t]   # the short way took every call
    monkeypatch.setattr(B, "_calls", B._NoCalls())
    checked = calls(B)
    assert len(short) == len(checked) and all(torch.equal(a, b) for a, b in zip(short, checked))
