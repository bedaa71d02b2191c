"""Refusals of the operators beside the chunkwise kernels: every bad argument is answered before any CUDA work.
Pointers are fake addresses that the library only inspects (alignment, overlap) and never dereferences."""
import ctypes

import pytest

A = 1 << 24   # fake aligned device addresses far apart


@pytest.fixture(scope="module")
def gla():
    from chunkwise_gated_linear_chunked_gb300 import build
    build.build()
    from chunkwise_gated_linear_chunked_gb300 import binding
    return binding


def scan(gla, x=A, g=2 * A, h=3 * A, h0=None, ht=None, cu=None, N=2, B=2, T=100, D=64, ldx=None, ldg=None, dtype=1,
         ws=64 * A, wsb=256):
    return gla.lib().gla_scan_fwd(x, g, h, h0, ht, cu, N, B, T, D, D if ldx is None else ldx,
                                  D if ldg is None else ldg, dtype, ws, wsb, None)


def scan_bwd(gla, g=A, h=2 * A, dh=3 * A, h0=None, dht=None, dx=4 * A, dg=5 * A, dh0=None, cu=None, N=2, B=2, T=100,
             D=64, ldg=None, lddx=None, lddg=None, dtype=2, ws=64 * A, wsb=256):
    ld = [D if v is None else v for v in (ldg, lddx, lddg)]
    return gla.lib().gla_scan_bwd(g, h, dh, h0, dht, dx, dg, dh0, cu, N, B, T, D, *ld, dtype, ws, wsb, None)


def scan_step(gla, x=A, g=2 * A, h=3 * A, h0=4 * A, ht=4 * A, slots=None, B=2, S=2, D=64, ldx=None, ldg=None, dtype=1,
              ws=64 * A, wsb=256):
    return gla.lib().gla_scan_step(x, g, h, h0, ht, slots, B, S, D, D if ldx is None else ldx,
                                   D if ldg is None else ldg, dtype, ws, wsb, None)


def step(gla, q=A, k=2 * A, v=3 * A, g=4 * A, o=5 * A, scale=0.1, h0=6 * A, ht=6 * A, slots=None, B=2, S=2, H=2,
         K=64, V=64, dtype=1, ws=64 * A, wsb=256):
    return gla.lib().gla_step(q, k, v, g, o, ctypes.c_float(scale), h0, ht, slots, B, S, H, K, V, dtype, ws, wsb, None)


def norm(gla, x=A, res=2 * A, w=3 * A, y=4 * A, s=5 * A, rstd=6 * A, rows=10, D=64, eps=1e-6, dtype=1):
    return gla.lib().gla_norm_fwd(x, res, w, y, s, rstd, rows, D, ctypes.c_float(eps), dtype, None)


def quant(gla, x=A, res=2 * A, w=3 * A, q=4 * A, scales=7 * A, s=5 * A, rstd=6 * A, rows=10, D=64, eps=1e-6, group=0,
          dtype=1):
    return gla.lib().gla_norm_quant_fwd(x, res, w, q, scales, s, rstd, rows, D, ctypes.c_float(eps), group, dtype, None)


def norm_bwd(gla, s=A, rstd=2 * A, w=3 * A, dy=4 * A, ds=5 * A, dx=6 * A, dres=None, dw=7 * A, rows=10, D=64, dtype=1,
             ws=64 * A, wsb=1 << 40):
    return gla.lib().gla_norm_bwd(s, rstd, w, dy, ds, dx, dres, dw, rows, D, dtype, ws, wsb, None)


def test_scan_refusals(gla):
    assert scan(gla, dtype=7) == gla.GLA_ERR_UNSUPPORTED
    assert scan(gla, dtype=1 | gla.GLA_HEAD_FIRST) == gla.GLA_ERR_UNSUPPORTED
    assert scan(gla, N=3) == gla.GLA_ERR_INVALID_ARG
    assert scan(gla, cu=40 * A) == gla.GLA_ERR_INVALID_ARG               # a pack has B == 1
    assert scan(gla, D=0) == gla.GLA_ERR_INVALID_ARG
    assert scan(gla, T=-1) == gla.GLA_ERR_INVALID_ARG
    assert scan(gla, ldx=63) == gla.GLA_ERR_INVALID_ARG
    assert scan(gla, N=70000, B=70000, T=70000) == gla.GLA_ERR_UNSUPPORTED
    assert scan(gla, x=None) == gla.GLA_ERR_INVALID_ARG
    assert scan(gla, g=2 * A + 2) == gla.GLA_ERR_ALIGNMENT
    assert scan(gla, h0=9 * A + 4) == gla.GLA_ERR_ALIGNMENT
    assert scan(gla, ws=None) == gla.GLA_ERR_WORKSPACE
    assert scan(gla, wsb=255) == gla.GLA_ERR_WORKSPACE
    assert scan(gla, ws=64 * A + 16) == gla.GLA_ERR_ALIGNMENT
    assert scan(gla, h=A + 1024) == gla.GLA_ERR_INVALID_ARG               # h overlaps x
    assert scan(gla, h0=9 * A, ht=9 * A + 64) == gla.GLA_ERR_INVALID_ARG  # partial overlap of the states
    assert scan(gla, ht=64 * A) == gla.GLA_ERR_INVALID_ARG
    assert gla.lib().gla_scan_workspace_size() == 256
    assert scan(gla, N=0, B=0, x=None, g=None, h=None) == gla.GLA_OK      # nothing to do


def test_scan_bwd_refusals(gla):
    assert scan_bwd(gla, dtype=-1) == gla.GLA_ERR_UNSUPPORTED
    assert scan_bwd(gla, lddx=8) == gla.GLA_ERR_INVALID_ARG
    assert scan_bwd(gla, dx=None) == gla.GLA_ERR_INVALID_ARG
    assert scan_bwd(gla, dh=3 * A + 8) == gla.GLA_ERR_ALIGNMENT
    assert scan_bwd(gla, dx=A) == gla.GLA_ERR_INVALID_ARG
    assert scan_bwd(gla, dg=4 * A + 128) == gla.GLA_ERR_INVALID_ARG       # same rows of 64, not column ranges
    assert scan_bwd(gla, dg=4 * A + 112, lddx=128, lddg=128) == gla.GLA_ERR_INVALID_ARG   # ranges that share bytes
    assert scan_bwd(gla, dg=4 * A + 128, lddx=128, lddg=192) == gla.GLA_ERR_INVALID_ARG
    assert scan_bwd(gla, dh0=64 * A) == gla.GLA_ERR_INVALID_ARG
    # dx and dg as the halves of one [rows, 2 D] gradient pass the check (and stop at the missing workspace)
    assert scan_bwd(gla, N=0, B=0, dg=4 * A + 128, lddx=128, lddg=128) == gla.GLA_OK


def test_step_refusals(gla):
    assert scan_step(gla, S=3) == gla.GLA_ERR_INVALID_ARG                 # no slots: one state per sequence
    assert scan_step(gla, h0=None) == gla.GLA_ERR_INVALID_ARG
    assert scan_step(gla, ldg=8) == gla.GLA_ERR_INVALID_ARG
    assert scan_step(gla, slots=9 * A + 4) == gla.GLA_ERR_ALIGNMENT
    assert scan_step(gla, h0=4 * A, ht=4 * A + 256) == gla.GLA_ERR_INVALID_ARG
    assert scan_step(gla, h=4 * A) == gla.GLA_ERR_INVALID_ARG
    assert scan_step(gla, wsb=8) == gla.GLA_ERR_WORKSPACE
    assert scan_step(gla, dtype=9) == gla.GLA_ERR_UNSUPPORTED
    assert step(gla, K=96) == gla.GLA_ERR_UNSUPPORTED
    assert step(gla, V=32) == gla.GLA_ERR_UNSUPPORTED
    assert step(gla, dtype=8) == gla.GLA_ERR_UNSUPPORTED
    assert step(gla, scale=0.0) == gla.GLA_ERR_INVALID_ARG
    assert step(gla, scale=float("nan")) == gla.GLA_ERR_INVALID_ARG
    assert step(gla, S=5) == gla.GLA_ERR_INVALID_ARG
    assert step(gla, o=None) == gla.GLA_ERR_INVALID_ARG
    assert step(gla, v=3 * A + 4) == gla.GLA_ERR_ALIGNMENT
    assert step(gla, o=6 * A + 64) == gla.GLA_ERR_INVALID_ARG             # o overlaps the states
    assert step(gla, ws=None) == gla.GLA_ERR_WORKSPACE
    assert step(gla, B=0, S=0) == gla.GLA_OK


def test_norm_refusals(gla):
    for f in (norm, quant):
        assert f(gla, dtype=2) == gla.GLA_ERR_UNSUPPORTED
        assert f(gla, dtype=4 | gla.GLA_RES_F32) == gla.GLA_ERR_UNSUPPORTED
        assert f(gla, D=0) == gla.GLA_ERR_INVALID_ARG
        assert f(gla, D=16385) == gla.GLA_ERR_UNSUPPORTED
        assert f(gla, rows=-1) == gla.GLA_ERR_INVALID_ARG
        assert f(gla, eps=-1.0) == gla.GLA_ERR_INVALID_ARG
        assert f(gla, eps=float("inf")) == gla.GLA_ERR_INVALID_ARG
        assert f(gla, x=None) == gla.GLA_ERR_INVALID_ARG
        assert f(gla, w=3 * A + 4) == gla.GLA_ERR_ALIGNMENT
        assert f(gla, s=A) == gla.GLA_ERR_INVALID_ARG                     # s overlaps x
        assert f(gla, s=2 * A + 16) == gla.GLA_ERR_INVALID_ARG            # s partly over res
        assert f(gla, rows=0) == gla.GLA_OK
    assert norm(gla, y=2 * A) == gla.GLA_ERR_INVALID_ARG
    assert quant(gla, group=64) == gla.GLA_ERR_UNSUPPORTED
    assert quant(gla, group=-1) == gla.GLA_ERR_INVALID_ARG
    assert quant(gla, scales=None) == gla.GLA_ERR_INVALID_ARG
    assert quant(gla, scales=4 * A) == gla.GLA_ERR_INVALID_ARG


def test_norm_bwd_refusals(gla):
    assert norm_bwd(gla, dtype=3 + 4) == gla.GLA_ERR_UNSUPPORTED
    assert norm_bwd(gla, D=20000) == gla.GLA_ERR_UNSUPPORTED
    assert norm_bwd(gla, dx=None) == gla.GLA_ERR_INVALID_ARG
    assert norm_bwd(gla, rstd=None) == gla.GLA_ERR_INVALID_ARG
    assert norm_bwd(gla, dw=7 * A + 8) == gla.GLA_ERR_ALIGNMENT
    assert norm_bwd(gla, ws=None) == gla.GLA_ERR_WORKSPACE
    assert norm_bwd(gla, wsb=100) == gla.GLA_ERR_WORKSPACE
    assert norm_bwd(gla, dx=A) == gla.GLA_ERR_INVALID_ARG                 # dx over s
    assert norm_bwd(gla, dx=4 * A, dres=4 * A) == gla.GLA_ERR_INVALID_ARG  # both over dy
    assert norm_bwd(gla, dw=64 * A) == gla.GLA_ERR_INVALID_ARG
    assert gla.lib().gla_norm_bwd_workspace_size(100, 0) == 0
    assert gla.lib().gla_norm_bwd_workspace_size(100, 20000) == 0
    assert gla.lib().gla_norm_bwd_workspace_size(100, 64) >= 256


def test_earlier_entry_points_refuse_the_layers_types(gla):
    """fp16 outputs (GLA_F16_OF16) belong to the recurrence and the one-token updates only."""
    lib, ws = gla.lib(), 64 * A
    assert lib.gla_fwd(A, 2 * A, 3 * A, 4 * A, 5 * A, 0.1, None, None, None, 2, 2, 100, 2, 64, 64, 64, gla.GLA_F16_OF16, ws,
                       1 << 40, None) == gla.GLA_ERR_UNSUPPORTED
    assert gla.workspace_size(2, 100, 2, 64, 64, 2, 64, gla.GLA_F16_OF16) == 0
    assert gla.bwd_workspace_size(2, 100, 2, 64, 64, 2, 64, gla.GLA_F16_OF16) == 0
    assert lib.gla_wy_fwd(A, 2 * A, 3 * A, 4 * A, None, 5 * A, 6 * A, None, 2, 2, 100, 2, 2, 64, 64, 64, gla.GLA_F16_OF16, ws,
                          1 << 40, None) == gla.GLA_ERR_UNSUPPORTED
    assert lib.gla_chunk_local_cumsum(A, 2 * A, None, 1, 1, 10, 1, 64, 64, gla.GLA_F16_OF16, None) == gla.GLA_ERR_UNSUPPORTED
