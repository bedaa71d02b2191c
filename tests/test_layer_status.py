"""What kernels report when the caller keeps no workspace can be read: bad offsets and bad slots of every call, by the
short way and the checked one, on other streams, and of a captured call that is the process's first."""
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def B():
    import __graft_entry__
    __graft_entry__.build()
    from chunkwise_gated_linear_chunked_gb300 import binding
    return binding


def calls(B):
    x = torch.zeros(1, 40, 64, device="cuda")
    bad_cu = torch.tensor([0, 30, 20, 40], dtype=torch.int32, device="cuda")
    rows, pool = torch.zeros(2, 64, device="cuda"), torch.zeros(3, 64, device="cuda")
    q, states = torch.zeros(2, 2, 64, device="cuda"), torch.zeros(3, 2, 64, 64, device="cuda")
    bad = torch.tensor([1, 3], dtype=torch.int32, device="cuda")
    return [lambda s: B.scan_fwd(x, x, cu_seqlens=bad_cu, stream=s),
            lambda s: B.scan_bwd(x, x, x, cu_seqlens=bad_cu, stream=s),
            lambda s: B.scan_step(rows, rows, pool, slots=bad, stream=s),
            lambda s: B.gla_step(q, q, q, q, states, slots=bad, stream=s)]


@pytest.mark.gpu
@pytest.mark.parametrize("which", range(4))
def test_default_calls_report(B, which):
    call, side = calls(B)[which], torch.cuda.Stream()
    torch.cuda.synchronize()
    B.layer_status()   # whatever came before
    assert B.layer_status() == B.GLA_OK
    for stream in (None, side, None):   # the usual call goes the short way, one with a stream the checked one
        call(stream)
        assert B.layer_status(stream=stream) == B.GLA_ERR_INVALID_ARG
        assert B.layer_status(stream=stream) == B.GLA_OK
    with torch.cuda.stream(side):
        call(None)
        assert B.layer_status(device=0) == B.GLA_ERR_INVALID_ARG
    assert B.layer_status() == B.GLA_OK


@pytest.mark.gpu
def test_own_workspace_is_apart(B):
    x, ws = torch.zeros(1, 40, 64, device="cuda"), torch.zeros(256, dtype=torch.uint8, device="cuda")
    B.layer_status()
    B.scan_fwd(x, x, cu_seqlens=torch.tensor([1, 40], dtype=torch.int32, device="cuda"), workspace=ws)
    assert B.layer_status() == B.GLA_OK and B.get_status(ws) == B.GLA_ERR_INVALID_ARG


FIRST = """
import torch
from chunkwise_gated_linear_chunked_gb300 import binding as B
x, state = torch.ones(2, 64, device="cuda"), torch.zeros(3, 64, device="cuda")
slots = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    h = B.scan_step(x, x, state, slots=slots) if {short} else B._scan_step_checked(x, x, state, slots, None, None, None, stream=None)
graph.replay()
assert B.layer_status() == B.GLA_OK
slots.copy_(torch.tensor([0, 7], dtype=torch.int32))
for _ in range(2):
    graph.replay()
    assert B.layer_status() == B.GLA_ERR_INVALID_ARG and B.layer_status() == B.GLA_OK
slots.copy_(torch.tensor([0, 2], dtype=torch.int32))
graph.replay()
assert B.layer_status() == B.GLA_OK and bool((state[0] > 1).all())
print("fine")
"""


@pytest.mark.gpu
@pytest.mark.parametrize("short", [True, False])
def test_first_call_in_a_capture(B, short):
    got = subprocess.run([sys.executable, "-c", FIRST.format(short=short)], cwd=ROOT, capture_output=True, text=True,
                         timeout=300)
    assert got.returncode == 0 and got.stdout.strip() == "fine", got.stdout + got.stderr
