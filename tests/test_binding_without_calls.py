"""The binding's short cut (the _calls module) is optional: without it, or with one that does not load, every function
is there and takes the checked way to the same kernels."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SETUP = """
import torch
from chunkwise_gated_linear_chunked_gb300 import build
build.calls_lib = lambda: {path!r}
from chunkwise_gated_linear_chunked_gb300 import binding as B
"""
REFUSALS = """
x = torch.zeros(2, 8, 64)
for call in (lambda: B.scan_fwd(x, x), lambda: B.scan_bwd(x, x, x), lambda: B.scan_step(x[0], x[0], x[0]),
             lambda: B.gla_step(x, x, x, x, x), lambda: B.norm_fwd(x), lambda: B.norm_quant_fwd(x),
             lambda: B.norm_bwd(x, x[..., 0], x)):
    try:
        call()
    except B.GlaError as e:
        assert e.code == B.GLA_ERR_INVALID_ARG
    else:
        raise SystemExit("not refused")
assert B.gla_fwd and B.workspace_size(2, 100, 2, 64, 64, 2) > 0
print("fine")
"""
RESULTS = """
gen = torch.Generator(device="cuda").manual_seed(0)
x, g = (torch.randn(2, 300, 64, device="cuda", generator=gen) for _ in range(2))
g = -g.abs()
h, ht = B.scan_fwd(x, g)
grads = B.scan_bwd(g, h, x, dht=ht)
y, s, rstd = B.norm_fwd(x, residual=g)
q, scales, _, _ = B.norm_quant_fwd(x, residual=g, group=128)
dx, _, dw = B.norm_bwd(s, rstd, x, weight=torch.ones(64, device="cuda"))
state = ht.clone()
h1 = B.scan_step(x[:, 0].contiguous(), g[:, 0].contiguous(), state)
pool = torch.ones(2, 300, 64, 64, device="cuda")
o = B.gla_step(x, x, x, g, pool)
assert B.layer_status() == B.GLA_OK
print([float(t.double().sum()) for t in (h, ht, *grads, y, s, rstd, q.float(), scales, dx, dw, state, h1, pool, o)])
"""


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunkwise_gated_linear_chunked_gb300 import build
    build.build()


def run(code):
    got = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert got.returncode == 0, got.stdout + got.stderr
    return got.stdout.strip().splitlines()[-1]


@pytest.mark.parametrize("there", [False, True], ids=["missing", "broken"])
def test_import_without_the_module(tmp_path, there):
    path = tmp_path / "_calls.so"
    if there:
        path.write_bytes(b"not a module")
    assert run(SETUP.format(path=str(path)) + REFUSALS) == "fine"


def test_refusals_with_the_module():
    from chunkwise_gated_linear_chunked_gb300 import build
    assert run(SETUP.format(path=build.calls_lib()) + REFUSALS) == "fine"


@pytest.mark.parametrize("compiler", ["no-such-compiler", "false"])
def test_build_without_a_host_compiler(monkeypatch, tmp_path, compiler):
    """What cannot be compiled is left out with a warning, an earlier module with it; libgla.so stands."""
    from chunkwise_gated_linear_chunked_gb300 import build
    earlier = tmp_path / "_calls.so"
    earlier.write_bytes(b"of an earlier state")
    monkeypatch.setenv("CXX", compiler)
    monkeypatch.setattr(build, "calls_lib", lambda: str(earlier))
    monkeypatch.setattr(build, "calls_stale", lambda: True)
    with pytest.warns(RuntimeWarning, match="_calls"):
        assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not earlier.exists()


@pytest.mark.gpu
def test_same_results_without_the_module(tmp_path):
    from chunkwise_gated_linear_chunked_gb300 import build
    assert os.path.exists(build.calls_lib())
    assert run(SETUP.format(path=str(tmp_path / "none.so")) + RESULTS) == \
        run(SETUP.format(path=build.calls_lib()) + RESULTS)
