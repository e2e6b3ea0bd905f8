"""What the norm, gradient-norm and MXFP4 calls refuse, before anything is launched (no GPU:
addresses are never dereferenced)."""

import ctypes
import os

import pytest
import torch

import delayed_scaling_gemm_amd as dsg

needs_lib = pytest.mark.skipif(not os.path.exists(dsg.LIB_PATH), reason="libfp8ds.so not built")
P = 0x10000
NAN = float("nan")


@needs_lib
def test_exports():
    lib = ctypes.CDLL(dsg.LIB_PATH)
    for n in ("fp8ds_rmsnorm", "fp8ds_rmsnorm_rowwise", "fp8ds_rmsnorm_mx", "fp8ds_rmsnorm_bwd",
              "fp8ds_rmsnorm_bwd_workspace", "fp8ds_grad_norm", "fp8ds_grad_norm_workspace",
              "fp8ds_grad_clip", "fp8ds_adamw_clip", "fp8ds_cast_mxfp4", "fp8ds_dequant_mxfp4",
              "fp8ds_gemm_mxfp4"):
        assert hasattr(lib, n), n


@needs_lib
def test_rmsnorm_refusals():
    L = dsg.lib()

    def head(x=P, xt=1, ldx=64, res=P, ldr=64, ht=1, gamma=P, gt=1, rows=4, cols=64, eps=1e-5, h=P,
             ldh=64, y=P, yt=1, ldy=64, rstd=P, fmt=0):
        return x, xt, ldx, res, ldr, ht, gamma, gt, rows, cols, eps, h, ldh, y, yt, ldy, rstd, fmt

    def plain(scale=P, q=P, ldq=64, used=None, am=None, sat=None, **kw):
        return L.fp8ds_rmsnorm(*head(**kw), scale, q, ldq, used, am, sat, None)

    def row(q=P, scale=P, margin=0, **kw):
        return L.fp8ds_rmsnorm_rowwise(*head(**kw), margin, q, 64, scale, None, None, None)

    def mx(q=P, ldq=64, s=P, lds=2, **kw):
        return L.fp8ds_rmsnorm_mx(*head(**kw), q, ldq, s, lds, None)

    for call in (plain, row, mx):
        assert call(xt=4) == -3 and call(ht=2) == -3 and call(gt=-1) == -3 and call(yt=9) == -3
        assert call(xt=0, ht=1) == -6                        # fp32 into a BF16 stream
        assert call(rows=-1) == -2 and call(cols=-64) == -2 and call(rows=1 << 31) == -2
        assert call(ldx=63) == -2 and call(ldr=63) == -2 and call(ldh=32) == -2 and call(ldy=0) == -2
        assert call(eps=NAN) == -7 and call(eps=-1.0) == -7 and call(eps=float("inf")) == -7
        assert call(x=None) == -1 and call(gamma=None) == -1 and call(q=None) == -1
        assert call(x=P + 1) == -4 and call(h=P + 1) == -4 and call(rstd=P + 2) == -4
        assert call(gamma=P + 1) == -4
    assert plain(scale=None) == -1 and plain(scale=None, q=None, am=P) == -1
    assert plain(fmt=2) == -3 and row(fmt=2) == -3 and mx(fmt=3) == -3
    assert plain(ldq=60) == -2 and row(margin=127) == -2 and row(scale=None) == -1
    assert mx(cols=48, ldq=64) == -2 and mx(s=None) == -1 and mx(lds=1) == -2 and mx(ldq=32) == -2
    assert mx(fmt=2, ldq=31) == -2
    for bad in (dict(x=P + 2), dict(ldx=65), dict(gamma=P + 4), dict(q=P + 4), dict(ldq=68),
                dict(h=P + 8), dict(y=P + 4)):
        assert mx(**bad) == -4, bad
    # nothing to do: nothing is launched
    assert plain(rows=0) == 0 and row(rows=0) == 0 and mx(cols=0, ldq=0) == 0


@needs_lib
def test_rmsnorm_bwd_refusals():
    L = dsg.lib()
    need = L.fp8ds_rmsnorm_bwd_workspace(4, 64)
    assert need == 64 * 4 and L.fp8ds_rmsnorm_bwd_workspace(0, 64) == 0
    assert L.fp8ds_rmsnorm_bwd_workspace(-1, 64) == -2
    # partial sums are bounded whatever the rows
    assert L.fp8ds_rmsnorm_bwd_workspace(1 << 22, 4096) <= 1024 * 4096 * 4

    def call(dy=P, dt=1, lddy=64, h=P, ht=1, ldh=64, rstd=P, gamma=P, gt=1, dres=P, lddr=64, rows=4,
             cols=64, dx=P, lddx=64, dg=P, ws=P, n=need, fmt=0, scale=P, q=P, ldq=64, used=None,
             am=None, sat=None):
        return L.fp8ds_rmsnorm_bwd(dy, dt, lddy, h, ht, ldh, rstd, gamma, gt, dres, lddr, rows, cols,
                                   dx, lddx, dg, ws, n, fmt, scale, q, ldq, used, am, sat, None)

    assert call(dt=2) == -3 and call(ht=5) == -3 and call(gt=2) == -3 and call(fmt=2) == -3
    assert call(dt=0, ht=1) == -6
    for bad in (dict(dy=None), dict(h=None), dict(rstd=None), dict(gamma=None), dict(dx=None),
                dict(dg=None), dict(ws=None), dict(q=None), dict(scale=None),
                dict(scale=None, q=None, am=P)):
        assert call(**bad) == -1, bad
    for bad in (dict(rows=-1), dict(lddy=63), dict(lddr=1), dict(lddx=0), dict(ldq=63),
                dict(n=need - 1)):
        assert call(**bad) == -2, bad
    for bad in (dict(dy=P + 1), dict(dx=P + 1), dict(ws=P + 8), dict(dg=P + 2), dict(rstd=P + 1)):
        assert call(**bad) == -4, bad


@needs_lib
def test_grad_norm_and_clip_refusals():
    L = dsg.lib()

    def arrays(ptrs=(P, P), types=(1, 0), counts=(10, 20)):
        n = len(ptrs)
        return n, (ctypes.c_void_p * n)(*ptrs), (ctypes.c_int * n)(*types), (ctypes.c_int64 * n)(*counts)

    def norm(arr=None, gs=1.0, mx=1.0, norm=P, coef=P, ws=P, nb=None):
        return L.fp8ds_grad_norm(*(arr or arrays()), gs, mx, norm, coef, ws,
                                 L.fp8ds_grad_norm_workspace() if nb is None else nb, None)

    def clip(arr=None, out=(P + 64, P + 128), out_types=(1, 1), coef=P):
        n, p, t, c = arr or arrays()
        o = None if out is None else (ctypes.c_void_p * len(out))(*out)
        return L.fp8ds_grad_clip(n, p, t, c, o, None if out_types is None else (ctypes.c_int * 2)(*out_types),
                                 coef, None)

    for call in (norm, clip):
        assert call(arrays(types=(1, 2))) == -3 and call(arrays(counts=(1, -1))) == -2
        assert call(arrays(ptrs=(P, None))) == -1 and call(arrays(ptrs=(P + 1, P))) == -4
        assert call(arrays(counts=(1 << 40, 1 << 40))) == -2
        assert call((5000,) + arrays()[1:]) == -2 and call((-1,) + arrays()[1:]) == -2
        assert call((2, None) + arrays()[2:]) == -1
    assert norm(norm=None) == -1 and norm(norm=P + 1) == -4 and norm(gs=0.0) == -7
    assert norm(gs=NAN) == -7 and norm(mx=0.0) == -7 and norm(mx=NAN) == -7
    big = arrays(counts=(65536, 1))
    assert norm(big, ws=None) == -1 and norm(big, nb=8) == -2 and norm(big, ws=P + 8) == -4
    assert clip(coef=None) == -1 and clip(out=(P + 64, None)) == -1 and clip(out_types=(1, 7)) == -3
    assert clip(arrays(types=(0, 0)), out=(P, P + 256), out_types=(1, 0)) == -6  # in place, other type
    assert clip(out=(P + 64, P + 2), out_types=(1, 0)) == -4 and clip(out_types=None) == -1
    assert L.fp8ds_grad_clip(0, None, None, None, None, None, P, None) == 0
    assert clip(arrays(ptrs=(None, None), counts=(0, 0)), out=None) == 0
    hp = (1e-3, 0.9, 0.999, 1e-8, 0.0, 1.0)
    assert L.fp8ds_adamw_clip(P, P, 1, P, P, 4, 4, *hp, None, 1, None, 0, None, None, None, None, None,
                              None, None) == -1
    assert L.fp8ds_adamw_clip(P, P, 1, P, P, 4, 4, *hp[:5], 0.0, P, 1, None, 0, None, None, None, None,
                              None, None, None) == -7


@needs_lib
def test_mxfp4_refusals():
    L = dsg.lib()

    def cast(x=P, xt=1, rows=64, cols=64, q=P, s=P, qt=P, st=P):
        return L.fp8ds_cast_mxfp4(x, xt, rows, cols, q, s, qt, st, None)

    assert cast(xt=3) == -3 and cast(rows=-1) == -2 and cast(cols=48) == -2 and cast(rows=40) == -2
    assert cast(x=None) == -1 and cast(q=None) == -1 and cast(s=None) == -1 and cast(st=None) == -1
    assert cast(qt=None) == -1 and cast(x=P + 8) == -4 and cast(q=P + 4) == -4 and cast(qt=P + 8) == -4
    assert cast(rows=0) == 0 and cast(rows=65536 * 128, cols=32) == -2
    d = lambda q=P, s=P, rows=4, cols=64, y=P, yt=1: L.fp8ds_dequant_mxfp4(q, s, rows, cols, y, yt, None)  # noqa: E731
    assert d(yt=2) == -3 and d(cols=33) == -2 and d(q=None) == -1 and d(s=None) == -1
    assert d(y=P + 8) == -4 and d(q=P + 8) == -4 and d(rows=0) == 0

    def gemm(M=64, N=64, K=128, a=P, fa=2, lda=128, sa=P, ldsa=4, b=P, ldb=128, sb=P, ldsb=4, c=P, ct=1,
             ldc=64, am=None):
        return L.fp8ds_gemm_mxfp4(M, N, K, a, fa, lda, sa, ldsa, b, ldb, sb, ldsb, c, ct, ldc, am, None)

    assert gemm(fa=3) == -3 and gemm(ct=2) == -3
    for bad in (dict(M=-1), dict(K=100), dict(lda=96), dict(ldb=64), dict(ldc=63), dict(ldsa=3),
                dict(ldsb=0), dict(M=65535 * 64 + 1), dict(lda=1 << 50)):
        assert gemm(**bad) == -2, bad
    for bad in (dict(a=None), dict(b=None), dict(sa=None), dict(sb=None), dict(c=None)):
        assert gemm(**bad) == -1, bad
    for bad in (dict(a=P + 8), dict(b=P + 4), dict(lda=144), dict(ldb=136), dict(c=P + 1),
                dict(fa=0, lda=136), dict(am=P + 2)):
        assert gemm(**bad) == -4, bad
    assert gemm(M=0) == 0 and gemm(N=0) == 0


def test_binding_refuses_host_and_odd_tensors():
    x, g = torch.zeros(4, 64), torch.ones(64)
    q = torch.zeros(4, 64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        dsg.fp8ds_rmsnorm(x, g, 1e-5, y=x)
    with pytest.raises(ValueError, match="2-D"):
        dsg.fp8ds_rmsnorm_rowwise(x[0], g, 1e-5, dsg.E4M3, 0, q, g)
    with pytest.raises(ValueError, match="CUDA"):
        dsg.fp8ds_rmsnorm_bwd(x, x, g, g, x, g, None)
    with pytest.raises(ValueError, match="CUDA"):
        dsg.fp8ds_grad_norm([x], 1.0, g)
    with pytest.raises(ValueError, match="CUDA"):
        dsg.fp8ds_grad_clip([x], g)
    with pytest.raises(ValueError, match="CUDA"):
        dsg.fp8ds_cast_mxfp4(x, q, q)
    with pytest.raises(ValueError, match="CUDA"):
        dsg.fp8ds_dequant_mxfp4(q, q, x)
    with pytest.raises(ValueError, match="CUDA"):
        dsg.fp8ds_gemm_mxfp4(4, 4, 64, q, dsg.E2M1, 64, q, 2, q, 64, q, 2, x, 4)
