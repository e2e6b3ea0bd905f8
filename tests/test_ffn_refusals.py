"""What the gated products, the norms around a residual addition and Muon refuse, before anything is
launched (no GPU: addresses are never dereferenced)."""

import ctypes
import os

import pytest
import torch

import delayed_scaling_gemm_amd as dsg

pytestmark = pytest.mark.skipif(not os.path.exists(dsg.LIB_PATH), reason="libfp8ds.so not built")
P = 0x10000
NAN, INF = float("nan"), float("inf")


def test_exports():
    lib = ctypes.CDLL(dsg.LIB_PATH)
    for n in ("fp8ds_gated_gemm", "fp8ds_gated_gemm_bwd", "fp8ds_rmsnorm_sandwich",
              "fp8ds_rmsnorm_sandwich_rowwise", "fp8ds_rmsnorm_sandwich_mx", "fp8ds_rmsnorm_sandwich_bwd",
              "fp8ds_rmsnorm_sandwich_bwd_workspace", "fp8ds_muon_workspace", "fp8ds_muon_direction",
              "fp8ds_muon_apply"):
        assert hasattr(lib, n), n


@pytest.mark.parametrize("bwd", [False, True])
def test_gated_refusals(bwd):
    fn = dsg.lib().fp8ds_gated_gemm_bwd if bwd else dsg.lib().fp8ds_gated_gemm

    def call(M=4, F=32, K=64, A=P, fa=0, lda=64, sa=P, B=P, fb=0, ldb=64, sb=P, act=0, gu=P, ldgu=64, y=P,
             yt=1, ldy=64, fmt=0, scale=P, q=P, ldq=64, used=None, am=None, sat=None, mma=0):
        return fn(M, F, K, A, fa, lda, sa, B, fb, ldb, sb, act, gu, ldgu, y, yt, ldy, fmt, scale, q, ldq, used,
                  am, sat, mma, None)

    assert call(fa=2) == -3 and call(fb=7) == -3 and call(fmt=2) == -3 and call(act=2) == -3
    assert call(act=-1) == -3 and call(yt=2) == -3 and call(mma=2) == -3
    assert call(fb=1) == -6
    if not bwd:
        assert call(fa=1) == -6
    for bad in (dict(M=-1), dict(F=-1), dict(K=-1), dict(M=1 << 31), dict(F=1 << 30), dict(K=1 << 31),
                dict(M=1 << 30, F=1 << 20), dict(lda=63), dict(ldb=63), dict(ldgu=63), dict(ldy=31),
                dict(ldq=31), dict(ldgu=1 << 60)):
        assert call(**bad) == -2, bad
    if bwd:
        assert call(ldy=63) == -2 and call(ldq=63) == -2
    for bad in (dict(scale=None), dict(q=None), dict(scale=None, q=None, used=P), dict(sa=None),
                dict(scale=None, q=None, sat=P), dict(sb=None), dict(A=None), dict(B=None),
                dict(y=None, scale=None, q=None, **({} if bwd else dict(gu=None)))):
        assert call(**bad) == -1, bad
    if bwd:
        assert call(gu=None) == -1
    for bad in (dict(A=P + 8), dict(B=P + 1), dict(lda=72), dict(ldb=72), dict(gu=P + 1), dict(y=P + 1),
                dict(y=P + 2, yt=0), dict(sa=P + 2), dict(scale=P + 1), dict(am=P + 2), dict(sat=P + 4),
                dict(used=P + 1)):
        assert call(**bad) == -4, bad
    # nothing to do: nothing is launched
    assert call(M=0) == 0 and call(F=0, ldy=0, ldq=0) == 0 and call(M=0, q=None) == 0
    assert call(M=0, scale=None) == -1


def test_sandwich_refusals():
    L = dsg.lib()

    def head(x=P, xt=1, ldx=64, pg=P, pt=1, e1=1e-6, gate=P, gate_t=0, t=None, alpha=1.0, res=P, ldr=64,
             ht=1, gamma=P, gt=1, rows=4, cols=64, eps=1e-5, h=P, ldh=64, y=P, yt=1, ldy=64, r1=P, r2=P,
             fmt=0):
        return (x, xt, ldx, pg, pt, e1, gate, gate_t, t, alpha, res, ldr, ht, gamma, gt, rows, cols, eps, h,
                ldh, y, yt, ldy, r1, r2, fmt)

    def plain(scale=P, q=P, ldq=64, used=None, am=None, sat=None, **kw):
        return L.fp8ds_rmsnorm_sandwich(*head(**kw), scale, q, ldq, used, am, sat, None)

    def row(q=P, scale=P, margin=0, **kw):
        return L.fp8ds_rmsnorm_sandwich_rowwise(*head(**kw), margin, q, 64, scale, None, None, None)

    def mx(q=P, ldq=64, s=P, lds=2, **kw):
        return L.fp8ds_rmsnorm_sandwich_mx(*head(**kw), q, ldq, s, lds, None)

    for call in (plain, row, mx):
        assert call(xt=4) == -3 and call(ht=2) == -3 and call(gt=-1) == -3 and call(yt=9) == -3
        assert call(pt=3) == -3 and call(gate_t=5) == -3
        assert call(xt=0, ht=1) == -6
        assert call(rows=-1) == -2 and call(cols=-64) == -2 and call(rows=1 << 31) == -2
        assert call(ldx=63) == -2 and call(ldr=63) == -2 and call(ldh=32) == -2 and call(ldy=0) == -2
        for e in (NAN, -1.0, INF):
            assert call(eps=e) == -7 and call(e1=e) == -7
        assert call(alpha=NAN) == -7 and call(alpha=INF) == -7
        for n in ("x", "gamma", "q", "pg", "res", "h"):
            assert call(**{n: None}) == -1, n
        for bad in (dict(x=P + 1), dict(h=P + 1), dict(res=P + 1), dict(r1=P + 2), dict(r2=P + 2),
                    dict(gamma=P + 1), dict(pg=P + 1), dict(gate=P + 2), dict(t=P + 1)):
            assert call(**bad) == -4, bad
    assert plain(scale=None) == -1 and plain(scale=None, q=None, am=P) == -1
    assert plain(fmt=2) == -3 and row(fmt=2) == -3 and mx(fmt=3) == -3
    assert plain(ldq=60) == -2 and row(margin=127) == -2 and row(scale=None) == -1
    assert mx(cols=48) == -2 and mx(s=None) == -1 and mx(lds=1) == -2 and mx(ldq=32) == -2
    for bad in (dict(x=P + 2), dict(ldx=65), dict(gamma=P + 4), dict(pg=P + 8), dict(gate=P + 4),
                dict(q=P + 4), dict(ldq=68), dict(h=P + 8), dict(y=P + 4), dict(res=P + 2)):
        assert mx(**bad) == -4, bad
    assert plain(rows=0) == 0 and row(rows=0) == 0 and mx(cols=0, ldq=0) == 0


def test_sandwich_bwd_refusals():
    L = dsg.lib()
    need = L.fp8ds_rmsnorm_sandwich_bwd_workspace(4, 64)
    assert need == 2 * 64 * 4 and L.fp8ds_rmsnorm_sandwich_bwd_workspace(0, 64) == 0
    assert L.fp8ds_rmsnorm_sandwich_bwd_workspace(-1, 64) == -2
    assert L.fp8ds_rmsnorm_sandwich_bwd_workspace(1 << 22, 4096) <= 2 * 1024 * 4096 * 4

    def call(dy=P, xt=1, lddy=64, h=P, ht=1, ldh=64, r2=P, gamma=P, gt=1, x=P, ldx=64, r1=P, pg=P, pt=1,
             gate=P, gate_t=0, t=P, alpha=1.0, dres=P, lddr=64, rows=4, cols=64, dh=P, lddh=64, dx=P,
             lddx=64, dg=P, dpg=P, dgate=P, dt=P, ws=P, n=need, fmt=0, scale=P, q=P, ldq=64, used=None,
             am=None, sat=None):
        return L.fp8ds_rmsnorm_sandwich_bwd(dy, xt, lddy, h, ht, ldh, r2, gamma, gt, x, ldx, r1, pg, pt, gate,
                                            gate_t, t, alpha, dres, lddr, rows, cols, dh, lddh, dx, lddx, dg,
                                            dpg, dgate, dt, ws, n, fmt, scale, q, ldq, used, am, sat, None)

    for n in ("xt", "ht", "gt", "pt", "gate_t"):
        assert call(**{n: 2}) == -3, n
    assert call(fmt=2) == -3 and call(xt=0, ht=1) == -6 and call(alpha=NAN) == -7
    for n in ("lddy", "ldh", "ldx", "lddr", "lddh", "lddx", "ldq"):
        assert call(**{n: 63}) == -2, n
    assert call(rows=-1) == -2 and call(cols=1 << 31) == -2 and call(n=need - 1) == -2
    for n in ("dy", "h", "r2", "gamma", "x", "r1", "pg", "dh", "dg", "dpg", "ws", "q", "scale"):
        assert call(**{n: None}) == -1, n
    assert call(gate=None) == -1 and call(t=None) == -1  # their gradients are asked for
    for bad in (dict(dy=P + 1), dict(h=P + 1), dict(x=P + 1), dict(dres=P + 1), dict(dh=P + 1),
                dict(dx=P + 1), dict(gamma=P + 1), dict(pg=P + 1), dict(gate=P + 1), dict(dg=P + 2),
                dict(dpg=P + 2), dict(dgate=P + 1), dict(dt=P + 2), dict(r1=P + 1), dict(r2=P + 1),
                dict(t=P + 2), dict(ws=P + 8)):
        assert call(**bad) == -4, bad
    assert call(cols=0, scale=None, q=None) == 0


def test_muon_refusals():
    L = dsg.lib()
    need = L.fp8ds_muon_workspace(100, 200)
    assert need > 0 and L.fp8ds_muon_workspace(0, 5) == 0 and L.fp8ds_muon_workspace(-1, 5) == -2
    assert L.fp8ds_muon_workspace((1 << 19) + 1, 5) == -2 and L.fp8ds_muon_workspace(1 << 18, 1 << 18) == -2
    assert L.fp8ds_muon_workspace(100, 200) == L.fp8ds_muon_workspace(200, 100)
    bad_coefs = (ctypes.c_float * 15)(*([1.0] * 14 + [NAN]))

    def call(g=P, gt=1, ldg=200, m=P, rows=100, cols=200, mu=0.95, nest=1, gs=1.0, coef=None, am=None,
             steps=5, coefs=None, eps=1e-7, o=P, ot=1, ldo=200, ws=P, n=need):
        return L.fp8ds_muon_direction(g, gt, ldg, m, rows, cols, mu, nest, gs, coef, am, steps, coefs, eps,
                                      o, ot, ldo, ws, n, None)

    assert call(gt=2) == -3 and call(ot=-1) == -3
    assert call(rows=-1) == -2 and call(cols=1 << 20) == -2 and call(n=need - 1) == -2
    assert call(ldg=199) == -2 and call(ldo=199) == -2
    for bad in (dict(mu=1.0), dict(mu=-0.1), dict(mu=NAN), dict(gs=0.0), dict(gs=INF), dict(eps=0.0),
                dict(eps=NAN), dict(steps=0), dict(steps=17),
                dict(coefs=ctypes.cast(bad_coefs, ctypes.c_void_p))):
        assert call(**bad) == -7, bad
    assert call(g=None) == -1 and call(o=None) == -1 and call(ws=None) == -1
    for bad in (dict(g=P + 1), dict(m=P + 4), dict(o=P + 2, ot=0), dict(ws=P + 8), dict(coef=P + 2), dict(am=P + 1)):
        assert call(**bad) == -4, bad
    assert call(rows=0, g=None, o=None, ws=None) == 0

    def apply(w=P, o=P, ot=1, rows=100, cols=200, lr=0.1, wd=0.0, adj=1.0, am0=None, fmt=0, scale=P, q=P,
              qt=None, used=None, am=None, sat=None):
        return L.fp8ds_muon_apply(w, o, ot, rows, cols, lr, wd, adj, am0, fmt, scale, q, qt, used, am, sat, None)

    assert apply(ot=3) == -3 and apply(fmt=2) == -3
    assert apply(rows=-1) == -2 and apply(rows=1 << 20, cols=1 << 20) == -2
    assert apply(rows=65535 * 128 + 1, cols=1, qt=P) == -2
    assert apply(lr=NAN) == -7 and apply(wd=INF) == -7 and apply(adj=NAN) == -7
    assert apply(w=None) == -1 and apply(o=None) == -1 and apply(q=None) == -1
    assert apply(scale=None) == -1 and apply(scale=None, q=None, am=P) == -1
    for bad in (dict(w=P + 4), dict(o=P + 2), dict(q=P + 1), dict(qt=P + 8), dict(scale=P + 1),
                dict(used=P + 2), dict(am=P + 1), dict(sat=P + 4), dict(am0=P + 2)):
        assert apply(**bad) == -4, bad
    assert apply(rows=0, w=None, o=None) == 0


def test_binding_refusals():
    """The Python side's own checks, made before any call (CPU tensors are never passed on)."""
    u8, f32 = torch.uint8, torch.float32
    x, w, s = torch.zeros(4, 32, dtype=u8), torch.zeros(6, 32, dtype=u8), torch.ones(1)
    y = torch.zeros(4, 3)
    with pytest.raises(ValueError, match="contracted"):
        dsg.fp8ds_gated_gemm(x, dsg.E4M3, s, torch.zeros(6, 16, dtype=u8), dsg.E4M3, s, 0, y=y)
    with pytest.raises(ValueError, match="rows, expected the gate"):
        dsg.fp8ds_gated_gemm(x, dsg.E4M3, s, torch.zeros(5, 32, dtype=u8), dsg.E4M3, s, 0, y=y)
    with pytest.raises(ValueError, match="CUDA"):
        dsg.fp8ds_gated_gemm(x, dsg.E4M3, s, w, dsg.E4M3, s, 0, y=y)
    v = torch.ones(32)
    with pytest.raises(ValueError, match="2-D"):
        dsg.fp8ds_rmsnorm_sandwich(v, v, 1e-6, v, v, 1e-6, v)
    with pytest.raises(ValueError, match="2-D"):
        dsg.fp8ds_muon_direction(v, v, x)
    with pytest.raises(ValueError, match="one shape"):
        dsg.fp8ds_muon_direction(y, torch.zeros(3, 4), x)
    with pytest.raises(ValueError, match="numbers for"):
        dsg.fp8ds_muon_direction(y, y, x, coefs=[(1.0, 2.0, 3.0)])
    with pytest.raises(ValueError, match="one shape"):
        dsg.fp8ds_muon_apply(y, torch.zeros(3, 4, dtype=f32), 0.1)
