"""Host-side argument checks of the activation checkpoints, the step's gradients from them and the norm
step (no GPU: validation runs before any launch, the addresses are never dereferenced)."""
import ctypes

import pytest

A = 1 << 32


@pytest.fixture(scope="module")
def M():
    from stream_residual_fusion_gb300 import build
    build.build()
    import stream_residual_fusion_gb300.mhc as m
    return m


def _addr(i, off=0):
    return ctypes.c_void_p(A + i * (1 << 28) + off)


@pytest.mark.parametrize("call", ["mhc_checkpoint_save", "mhc_checkpoint_load"])
def test_checkpoint_validation(M, call):
    f = getattr(M.lib, call)
    p = [_addr(i) for i in range(3)]
    assert f(*p, -1, 64, None) == M.MHC_ERR_SHAPE
    assert f(*p, 4, 0, None) == M.MHC_ERR_SHAPE
    assert f(*p, 4, 60, None) == M.MHC_ERR_SHAPE
    assert f(*p, (1 << 38) + 1, 64, None) == M.MHC_ERR_SHAPE
    assert f(None, None, None, 0, 64, None) == M.MHC_OK
    for i in range(3):
        q = list(p)
        q[i] = None
        assert f(*q, 4, 64, None) == M.MHC_ERR_NULL
        q[i] = _addr(i, 8)
        assert f(*q, 4, 64, None) == M.MHC_ERR_ALIGN
    assert f(p[0], p[1], p[0], 4, 64, None) == M.MHC_ERR_ALIAS


def test_checkpoint_sizes(M):
    s = M.lib.mhc_checkpoint_scale_bytes
    assert s(10, 32) == 10 and s(10, 40) == 20 and s(7, 5120) == 7 * 160
    assert s(0, 32) == 0 and s(4, 20) == 0 and s(-1, 32) == 0


def _bwd(M, N=256, n=4, d=5120, iters=20, flags=0, ptrs=None, ws=None, ws_bytes=1 << 40):
    p = [_addr(i) for i in range(26)] if ptrs is None else ptrs
    ws = _addr(30) if ws is None else ws
    return M.lib.mhc_fused_step_backward_ckpt(*p, N, n, d, iters, 1e-6, 1e-6, flags, ws, ws_bytes, None)


def test_step_backward_ckpt_validation(M):
    for kw in (dict(n=1), dict(N=-1), dict(iters=0), dict(iters=4097), dict(d=5120 + 32), dict(flags=0x2)):
        assert _bwd(M, **kw) == M.MHC_ERR_SHAPE, kw
    for i in range(26):
        p = [_addr(k) for k in range(26)]
        p[i] = None
        assert _bwd(M, ptrs=p) == M.MHC_ERR_NULL, i
        p[i] = _addr(i, 4)
        assert _bwd(M, ptrs=p) == M.MHC_ERR_ALIGN, i
    assert _bwd(M, ws=ctypes.c_void_p(0)) == M.MHC_ERR_WORKSPACE
    p = [_addr(k) for k in range(26)]
    p[17] = p[1]                                   # gX over X's scales
    assert _bwd(M, ptrs=p) == M.MHC_ERR_ALIAS
    p = [_addr(k) for k in range(26)]
    p[18] = _addr(0, 256 * 4 * 5120 - 16)          # gF over the end of X's codes
    assert _bwd(M, ptrs=p) == M.MHC_ERR_ALIAS
    assert _bwd(M, ws=_addr(2)) == M.MHC_ERR_ALIAS
    assert M.lib.mhc_backward_ckpt_workspace_bytes(256, 4, 5120 + 32) == 0
    assert M.lib.mhc_backward_ckpt_workspace_bytes(256, 1, 5120) == 0


# X, F, gate, pre, post, comb, gain_post, gain_pre, X_out, y
def _norm(M, N=16, n=4, d=512, flags=0, **change):
    p = [_addr(i) for i in range(10)]
    for i, v in change.items():
        p[int(i[1:])] = v
    return M.lib.mhc_norm_step(*p, N, n, d, 1.0, 1e-6, flags, None)


def test_norm_step_validation(M):
    for kw in (dict(n=2), dict(N=-1), dict(d=0), dict(d=100), dict(d=32776), dict(flags=0x2), dict(flags=0x8)):
        assert _norm(M, **kw) == M.MHC_ERR_SHAPE, kw
    assert _norm(M, N=0) == M.MHC_OK
    for i in (0, 1, 3, 4, 5, 7, 8, 9):             # the gate and the post gain may be missing
        assert _norm(M, **{f"p{i}": None}) == M.MHC_ERR_NULL, i
    for i in range(10):
        assert _norm(M, **{f"p{i}": _addr(i, 4)}) == M.MHC_ERR_ALIGN, i
    # one stream: all three weights, or none of them unless they are shared ones
    assert _norm(M, n=1, p3=None) == M.MHC_ERR_NULL
    none = dict(p3=None, p4=None, p5=None)
    assert _norm(M, **none) == M.MHC_ERR_NULL
    assert _norm(M, n=1, flags=M.WEIGHTS_SHARED, **none) == M.MHC_ERR_NULL
    assert _norm(M, flags=M.GATE_SIGMOID, p2=None) == M.MHC_ERR_NULL
    assert _norm(M, p9=_addr(8, 64)) == M.MHC_ERR_ALIAS
    assert _norm(M, p8=_addr(0, 64)) == M.MHC_ERR_ALIAS       # X_out == X only exactly
    assert _norm(M, p9=_addr(2)) == M.MHC_ERR_ALIAS           # y over the gate
    # shared weights are one row of 64 bytes: an output inside it overlaps, the one row alone
    assert _norm(M, flags=M.WEIGHTS_SHARED, p9=_addr(5, 48)) == M.MHC_ERR_ALIAS


# (X, F, gate, pre, post, comb, gain_post, gain_pre, gXp, gy,
#  gX, gF, ggate, gpre, gpost, gcomb, ggain_post, ggain_pre)
def _norm_bwd(M, ckpt, N=16, n=4, d=512, flags=0, ws=None, ws_bytes=1 << 40, **change):
    p = [_addr(i) for i in range(18)]
    for i, v in change.items():
        p[int(i[1:])] = v
    ws = _addr(30) if ws is None else ws
    tail = (N, n, d, 1.0, 1e-6, flags, ws, ws_bytes, None)
    if ckpt:
        return M.lib.mhc_norm_step_backward_ckpt(p[0], _addr(20), p[1], _addr(21), *p[2:], *tail)
    return M.lib.mhc_norm_step_backward(*p, *tail)


@pytest.mark.parametrize("ckpt", [False, True])
def test_norm_step_backward_validation(M, ckpt):
    for kw in (dict(n=2), dict(N=-1), dict(d=100), dict(d=32776), dict(flags=0x2)):
        assert _norm_bwd(M, ckpt, **kw) == M.MHC_ERR_SHAPE, kw
    for i in (0, 1, 3, 7, 8, 9, 10, 11, 12, 13, 14, 15, 16, 17):
        assert _norm_bwd(M, ckpt, **{f"p{i}": None}) == M.MHC_ERR_NULL, i
    for i in range(18):
        assert _norm_bwd(M, ckpt, **{f"p{i}": _addr(i, 4)}) == M.MHC_ERR_ALIGN, i
    assert _norm_bwd(M, ckpt, ws=ctypes.c_void_p(0)) == M.MHC_ERR_WORKSPACE
    assert _norm_bwd(M, ckpt, ws=_addr(30, 8)) == M.MHC_ERR_ALIGN
    for out, on in ((10, 0), (10, 8), (11, 1), (11, 9), (12, 2), (13, 3), (16, 6), (17, 7), (17, 16)):
        assert _norm_bwd(M, ckpt, **{f"p{out}": _addr(on)}) == M.MHC_ERR_ALIAS, (out, on)
    assert _norm_bwd(M, ckpt, ws=_addr(9)) == M.MHC_ERR_ALIAS
    assert _norm_bwd(M, ckpt, n=1, p3=None, p4=None) == M.MHC_ERR_NULL
    assert M.lib.mhc_norm_step_backward_workspace_bytes(0, 4, 512) == 0
    assert M.lib.mhc_norm_step_backward_workspace_bytes(4, 2, 512) == 0
    assert M.lib.mhc_norm_step_backward_workspace_bytes(4, 4, 511) == 0
