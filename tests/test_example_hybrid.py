"""The hybrid model of examples/: it learns, its gradients are those of its plain torch form, and decoding token by
token continues a prompt as one forward over all tokens does."""
import importlib.util
import os

import pytest
import torch
import torch.nn.functional as F

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lm():
    import __graft_entry__
    __graft_entry__.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_lm.py")
    spec = importlib.util.spec_from_file_location("hybrid_lm", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def plain_forward(lm, m, tokens):
    """The model in torch operations, in fp64, one row after the other."""
    p = {k: v.detach().double().requires_grad_(True) for k, v in m.p.items()}
    stream = p["embed"][tokens]
    x = torch.zeros_like(stream)

    def norm(x, stream, w):
        s = x + stream
        return s * (s.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w, s

    for i in range(lm.LAYERS):
        y, stream = norm(x, stream, p[f"norm{i}"])
        z = y @ p[f"in{i}"].T
        rows = []
        if m.is_gla(i):
            q, k, v, gate = (t.reshape(*t.shape[:-1], lm.HEADS, lm.HEAD_DIM) for t in z.chunk(4, -1))
            a = (F.logsigmoid(gate) / 16).exp()
            S = torch.zeros(tokens.shape[0], lm.HEADS, lm.HEAD_DIM, lm.HEAD_DIM, dtype=torch.float64, device=z.device)
            for t in range(tokens.shape[1]):
                S = a[:, t, ..., None] * S + k[:, t, ..., None] * v[:, t, ..., None, :]
                rows.append(lm.HEAD_DIM ** -0.5 * (q[:, t, ..., None] * S).sum(-2))
        else:
            u, gate = z.chunk(2, -1)
            a = (F.logsigmoid(gate) / 4).exp()
            h = torch.zeros_like(u[:, 0])
            for t in range(tokens.shape[1]):
                h = a[:, t] * h + u[:, t]
                rows.append(h)
        x = torch.stack(rows, 1).reshape(stream.shape) @ p[f"out{i}"].T
    return norm(x, stream, p["norm_out"])[0] @ p["logits"].T, p


def test_fp32_gradients_match_the_plain_form(lm):
    """fp32 operators of relative error 1e-5 at most, in four layers with order-one amplification: 1e-3 overall."""
    torch.backends.cuda.matmul.allow_tf32 = False
    m = lm.Model(torch.float32)
    tokens = lm.batch(2, 70, 0)
    ref, p = plain_forward(lm, m, tokens[:, :-1])
    F.cross_entropy(ref.reshape(-1, lm.VOCAB), tokens[:, 1:].reshape(-1)).backward()
    for w in m.p.values():
        w.requires_grad_(True)
    logits = m.forward(tokens[:, :-1])
    F.cross_entropy(logits.reshape(-1, lm.VOCAB), tokens[:, 1:].reshape(-1)).backward()
    assert (logits - ref).norm() <= 1e-4 * ref.norm()
    for name, w in m.p.items():
        assert (w.grad - p[name].grad).norm() <= 1e-3 * p[name].grad.norm(), name


def test_it_learns(lm):
    losses = lm.train(lm.Model(), 60)
    assert losses[-1] < 0.7 * losses[0]


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 1e-4), (torch.bfloat16, 5e-2)], ids=["fp32", "bf16"])
def test_decoding_continues_the_forward(lm, dtype, tol):
    """fp32: as above.  bf16: 2^-8 of each rounding, some dozen of them on the way, and 8-bit activations 2^-4."""
    m = lm.Model(dtype, seed=3)
    tokens = lm.batch(5, 89, 2)[:, :90]
    full = m.forward(tokens)
    slots = torch.tensor([6, 0, 3, 7, 2], dtype=torch.int32).cuda()
    server, small = lm.Server(m, 8), lm.Server(m, 8, eight_bit=True)
    last = server.prefill(tokens[:, :80], slots)
    small.prefill(tokens[:, :80], slots)
    assert (last - full[:, 79]).norm() <= tol * full[:, 79].norm()
    for t in range(80, 90):
        got = server.step(tokens[:, t], slots)
        assert (got - full[:, t]).norm() <= tol * full[:, t].norm()
        eight = small.step(tokens[:, t], slots)
        assert (eight - full[:, t]).norm() <= 0.2 * full[:, t].norm()


def test_generation(lm):
    m = lm.Model(seed=4)
    slots = torch.arange(3, dtype=torch.int32).cuda()
    prompt = lm.batch(3, 40, 5)[:, :40]
    out = lm.generate(lm.Server(m, 3), prompt, slots, 12)
    # the graph's tokens are those of the same loop without a graph
    server = lm.Server(m, 3)
    tokens = server.prefill(prompt, slots).argmax(-1)
    for i in range(12):
        assert torch.equal(out[:, i], tokens)
        tokens = server.step(tokens, slots).argmax(-1)
