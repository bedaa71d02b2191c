"""Refusals of the gated delta rule and the group norm: every bad argument is answered before any CUDA work.  Pointers are
fake addresses that the library only inspects (alignment, overlap) and never dereferences."""
import ctypes

import pytest

A = 1 << 24   # fake aligned device addresses far apart


@pytest.fixture(scope="module")
def gla():
    from chunkwise_gated_linear_chunked_gb300 import build
    build.build()
    from chunkwise_gated_linear_chunked_gb300 import binding
    return binding


def fwd(gla, q=A, k=2 * A, v=3 * A, g=4 * A, beta=5 * A, o=6 * A, scale=0.1, h0=None, ht=None, cu=None, N=2, B=2, T=100, H=1, HV=2,
        K=64, V=64, dtype=2, status=60 * A, ws=64 * A, wsb=1 << 22):
    return gla.lib().gla_delta_fwd(q, k, v, g, beta, o, ctypes.c_float(scale), h0, ht, cu, N, B, T, H, HV, K, V, dtype, status, ws, wsb, None)


def bwd(gla, q=A, k=2 * A, v=3 * A, g=4 * A, beta=5 * A, do=6 * A, scale=0.1, h0=None, dht=None, dq=7 * A, dk=8 * A, dv=9 * A, dg=10 * A,
        dbeta=11 * A, dh0=None, cu=None, N=2, B=2, T=100, H=1, HV=2, K=64, V=64, dtype=1, status=60 * A, ws=64 * A, wsb=1 << 30):
    return gla.lib().gla_delta_bwd(q, k, v, g, beta, do, ctypes.c_float(scale), h0, dht, dq, dk, dv, dg, dbeta, dh0, cu, N, B, T, H, HV, K, V,
                                   dtype, status, ws, wsb, None)


def step(gla, q=A, k=2 * A, v=3 * A, g=4 * A, beta=5 * A, o=6 * A, scale=0.1, h0=7 * A, ht=7 * A, slots=None, B=2, S=2, H=1, HV=2, K=64, V=64,
         dtype=2, status=60 * A):
    return gla.lib().gla_delta_step(q, k, v, g, beta, o, ctypes.c_float(scale), h0, ht, slots, B, S, H, HV, K, V, dtype, status, None)


def norm(gla, x=A, w=2 * A, b=3 * A, y=4 * A, mean=5 * A, rstd=6 * A, N=4, S=10, C=64, G=4, eps=1e-5, act=1, dtype=1, ws=64 * A, wsb=1 << 22):
    return gla.lib().gla_group_norm_fwd(x, w, b, y, mean, rstd, N, S, C, G, ctypes.c_float(eps), act, dtype, ws, wsb, None)


def norm_bwd(gla, x=A, mean=2 * A, rstd=3 * A, w=4 * A, b=5 * A, dy=6 * A, dx=7 * A, dw=8 * A, db=9 * A, N=4, S=10, C=64, G=4, act=1, dtype=1,
             ws=64 * A, wsb=1 << 22):
    return gla.lib().gla_group_norm_bwd(x, mean, rstd, w, b, dy, dx, dw, db, N, S, C, G, act, dtype, ws, wsb, None)


@pytest.mark.parametrize("call", [fwd, bwd], ids=["fwd", "bwd"])
def test_delta_refusals(gla, call):
    bad = gla.GLA_ERR_INVALID_ARG
    for dtype in (4, 5, 7, -1, 1 | gla.GLA_HEAD_FIRST):
        assert call(gla, dtype=dtype) == gla.GLA_ERR_UNSUPPORTED
    for kw in (dict(K=257), dict(V=257), dict(B=70000, N=70000, T=70000), dict(T=1 << 30, HV=8), dict(N=1 << 30, B=1 << 30, T=1)):
        assert call(gla, **kw) == gla.GLA_ERR_UNSUPPORTED
    for kw in (dict(N=3), dict(cu=40 * A), dict(K=0), dict(V=0), dict(H=0), dict(HV=0), dict(H=2, HV=3), dict(T=-1), dict(scale=0.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(q=None), dict(k=None), dict(v=None), dict(g=None), dict(beta=None)):
        assert call(gla, **kw) == bad
    for kw in (dict(q=A + 8), dict(g=4 * A + 4), dict(h0=20 * A + 4), dict(status=60 * A + 16)):
        assert call(gla, **kw) == gla.GLA_ERR_ALIGNMENT
    assert call(gla, status=None) == gla.GLA_ERR_WORKSPACE
    assert call(gla, N=0, B=0) == gla.GLA_OK


def test_delta_fwd_overlaps(gla):
    bad = gla.GLA_ERR_INVALID_ARG
    for kw in (dict(o=A), dict(o=4 * A), dict(ht=A), dict(o=60 * A), dict(h0=20 * A, ht=20 * A + 256), dict(ht=6 * A)):
        assert fwd(gla, **kw) == bad
    assert fwd(gla, o=None) == bad
    need = gla.lib().gla_delta_fwd_workspace_size
    assert need(2, 2, 100, 1, 2, 257, 64, 2, 0) == 0 and need(2, 2, 100, 1, 2, 64, 64, 0, 0) == 0


def test_delta_bwd_overlaps(gla):
    bad = gla.GLA_ERR_INVALID_ARG
    for kw in (dict(dq=A), dict(dk=7 * A), dict(dv=6 * A), dict(dg=5 * A), dict(dbeta=10 * A), dict(dh0=7 * A), dict(dht=20 * A, dh0=20 * A),
               dict(dq=64 * A), dict(dq=None), dict(dbeta=None), dict(do=None)):
        assert bwd(gla, **kw) == bad
    for dtype in (gla.GLA_BF16_OBF16, gla.GLA_F16_OF16):
        assert bwd(gla, dtype=dtype) == gla.GLA_ERR_UNSUPPORTED
    assert bwd(gla, ws=None) == gla.GLA_ERR_WORKSPACE and bwd(gla, wsb=1000) == gla.GLA_ERR_WORKSPACE
    assert bwd(gla, ws=64 * A + 16) == gla.GLA_ERR_ALIGNMENT
    need = gla.lib().gla_delta_bwd_workspace_size
    assert need(2, 2, 100, 1, 2, 64, 64, gla.GLA_BF16_OBF16, 0) == 0 and need(2, 2, 100, 1, 3, 64, 64, 1, 0) > 0
    assert need(2, 2, 100, 2, 3, 64, 64, 1, 0) == 0


def test_step_refusals(gla):
    bad = gla.GLA_ERR_INVALID_ARG
    for kw in (dict(S=3), dict(H=2, HV=3), dict(K=0), dict(scale=-1.0), dict(o=None), dict(h0=None), dict(o=7 * A), dict(h0=7 * A, ht=7 * A + 512),
               dict(B=-1)):
        assert step(gla, **kw) == bad
    for kw in (dict(dtype=4), dict(K=300), dict(V=300), dict(B=1 << 28, S=1 << 28)):
        assert step(gla, **kw) == gla.GLA_ERR_UNSUPPORTED
    assert step(gla, v=3 * A + 4) == gla.GLA_ERR_ALIGNMENT and step(gla, slots=9 * A + 4) == gla.GLA_ERR_ALIGNMENT
    assert step(gla, status=None) == gla.GLA_ERR_WORKSPACE
    assert step(gla, B=0, S=0) == gla.GLA_OK


@pytest.mark.parametrize("call", [norm, norm_bwd], ids=["fwd", "bwd"])
def test_group_norm_refusals(gla, call):
    bad = gla.GLA_ERR_INVALID_ARG
    for dtype in (2, 4, -1, 1 | gla.GLA_RES_F32):
        assert call(gla, dtype=dtype) == gla.GLA_ERR_UNSUPPORTED
    for kw in (dict(G=5), dict(G=0), dict(C=0), dict(S=0), dict(N=-1), dict(act=2), dict(act=-1), dict(x=None), dict(mean=None)):
        assert call(gla, **kw) == bad
    assert call(gla, N=1 << 40, S=1 << 40) == gla.GLA_ERR_UNSUPPORTED
    assert call(gla, w=30 * A + 4) == gla.GLA_ERR_ALIGNMENT
    assert call(gla, ws=None) == gla.GLA_ERR_WORKSPACE and call(gla, wsb=16) == gla.GLA_ERR_WORKSPACE
    assert call(gla, ws=64 * A + 32) == gla.GLA_ERR_ALIGNMENT


def test_group_norm_overlaps(gla):
    bad = gla.GLA_ERR_INVALID_ARG
    for kw in (dict(y=A), dict(y=2 * A), dict(mean=4 * A), dict(rstd=5 * A), dict(y=64 * A), dict(eps=-1.0), dict(eps=float("inf")), dict(y=None)):
        assert norm(gla, **kw) == bad
    for kw in (dict(dx=A), dict(dx=6 * A), dict(dw=7 * A), dict(db=8 * A), dict(dw=4 * A), dict(dx=64 * A), dict(dx=None), dict(dy=None)):
        assert norm_bwd(gla, **kw) == bad
    assert norm(gla, N=0) == gla.GLA_OK and norm_bwd(gla, N=0, dw=None, db=None) == gla.GLA_OK
    need = gla.lib().gla_group_norm_workspace_size
    assert need(4, 10, 64, 5, 1, 1) == 0 and need(4, 1, 64, 4, 1, 0) == 0 and need(4, 1, 64, 4, 1, 1) > 0 and need(4, 10, 64, 4, 1, 0) > 0
