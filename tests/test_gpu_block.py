"""The residual stack (delayed_scaling_gemm_amd/block.py) on the GPU.

With an FP32 residual stream every fused step has a composition of separate calls with
the same roundings (norm to FP32, then its cast; gradients clipped into FP32, then AdamW;
weights updated, then cast), so the two have to agree bit for bit.  Gradients are also
held against autograd in fp64 without any quantisation: X and W are rounded by at most
2^-4, dY by 2^-3, relative to each value (E4M3, E5M2 in their normal range), so a dW of
two blocks is a sum of terms off by at most (1 + 2^-4)^3 (1 + 2^-3)^2 - 1 = 0.52 with
signs at random: its direction is asked to keep a cosine of 0.95 (rms errors of 1/sqrt(3)
of those, added in squares, give 1 - 0.18^2 / 2 = 0.98)."""

import pytest

torch = pytest.importorskip("torch")

import delayed_scaling_gemm_amd as dsg  # noqa: E402
from delayed_scaling_gemm_amd.block import NormLinearStack  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
HP = dict(beta1=0.9, beta2=0.999, eps=1e-8)


def u8(*shape):
    return torch.empty(shape, dtype=U8, device=DEV)


def inputs(T, C, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, C, generator=g).to(BF).to(DEV)
    dy = (torch.randn(T, C, generator=g) / T).to(BF).to(DEV)
    return x, dy


class Plain:
    """The same stack from separate calls, one per step of the formulas."""

    def __init__(self, s):
        self.s, self.L, self.C = s, s.layers, s.width
        self.w = [w.clone() for w in s.w]
        self.gamma = [g.clone() for g in s.gamma]
        self.mom = [(torch.zeros_like(p), torch.zeros_like(p)) for p in self.w + self.gamma]
        self.history, self.cursor = torch.zeros_like(s.history), torch.zeros_like(s.cursor)
        self.scale = torch.ones_like(s.scale)
        self.step = 0

    def cast(self, x, fmt, i, q, q_t=None):
        dsg.fp8ds_cast_acc(x, fmt, self.scale[i:i + 1], q, q_t, self.used[i:i + 1],
                           self.amax[i:i + 1])

    def run(self, x, dy):
        L, C, T = self.L, self.C, x.shape[0]
        self.used, self.amax = torch.zeros_like(self.scale), torch.zeros_like(self.scale)
        one = lambda i: self.used[i:i + 1]  # noqa: E731
        h, hs, rs, xqs, wqs = x.float(), [], [], [], []
        for i in range(L):
            y32, r = torch.empty(T, C, device=DEV), torch.empty(T, device=DEV)
            dsg.fp8ds_rmsnorm(h, self.gamma[i], self.s.eps, y=y32, rstd=r)
            xq, wq, wqt = u8(T, C), u8(C, C), u8(C, C)
            self.cast(y32, dsg.E4M3, i, xq)
            self.cast(self.w[i], dsg.E4M3, L + i, wq, wqt)
            out = torch.empty(T, C, dtype=BF, device=DEV)
            dsg.fp8ds_gemm(dsg.OP_N, dsg.OP_T, T, C, C, xq, dsg.E4M3, C, one(i), wqt, dsg.E4M3, C,
                           one(L + i), out, C)
            hs.append(h), rs.append(r), xqs.append(xq), wqs.append(wq)
            h = h + out.float()
        y, r = torch.empty(T, C, dtype=BF, device=DEV), torch.empty(T, device=DEV)
        dsg.fp8ds_rmsnorm(h, self.gamma[L], self.s.eps, y=y, rstd=r)
        hs.append(h), rs.append(r)
        ws = u8(dsg.fp8ds_rmsnorm_bwd_workspace(T, C))
        dres, dws, dgs, g = None, [None] * L, [None] * (L + 1), dy
        for i in range(L, -1, -1):
            dh, dgs[i] = torch.empty(T, C, device=DEV), torch.empty(C, device=DEV)
            dsg.fp8ds_rmsnorm_bwd(g, hs[i], rs[i], self.gamma[i], dh, dgs[i], ws, dres)
            dres = dh
            if i == 0:
                break
            j, dq = i - 1, u8(T, C)
            self.cast(dh, dsg.E5M2, 2 * L + j, dq)
            g, dws[j] = torch.empty(T, C, dtype=BF, device=DEV), torch.empty(C, C, dtype=BF, device=DEV)
            dsg.fp8ds_gemm(dsg.OP_N, dsg.OP_T, T, C, C, dq, dsg.E5M2, C, one(2 * L + j), wqs[j],
                           dsg.E4M3, C, one(L + j), g, C)
            dsg.fp8ds_gemm(dsg.OP_T, dsg.OP_N, C, C, T, xqs[j], dsg.E4M3, C, one(j), dq, dsg.E5M2, C,
                           one(2 * L + j), dws[j], C)
        dsg.fp8ds_scale_update(self.history, self.cursor, self.amax, self.s.fmts, dsg.ALGO_MAX, 0,
                               self.scale)
        self.step += 1
        return y, dh, dws + dgs

    def optimize(self, grads, lr, max_norm, decay):
        norm, coef = torch.zeros(1, device=DEV), torch.zeros(1, device=DEV)
        dsg.fp8ds_grad_norm(grads, max_norm, norm, coef, u8(dsg.fp8ds_grad_norm_workspace()))
        out = [torch.empty(g.shape, device=DEV) for g in grads]
        dsg.fp8ds_grad_clip(grads, coef, out)
        for i, p in enumerate(self.w + self.gamma):
            dsg.fp8ds_adamw(p, out[i], *self.mom[i], lr, **HP,
                            weight_decay=decay if i < self.L else 0.0, step=self.step)
        return norm, coef


@pytest.mark.parametrize("T,C,layers", [(1, 32, 1), (17, 160, 2), (96, 64, 3), (300, 256, 2)])
def test_steps_equal_the_separate_calls(T, C, layers):
    torch.manual_seed(T + C)
    s = NormLinearStack(layers, C, stream_dtype=F32)
    p = Plain(s)
    for step in range(3):
        x, dy = inputs(T, C, 10 * T + step)
        y, dx = s.forward(x), s.backward(dy)
        py, pdx, pg = p.run(x, dy)
        assert torch.equal(y, py) and torch.equal(dx, pdx)
        for a, b in zip(s.grads(), pg):
            assert torch.equal(a, b)
        assert torch.equal(s.scale, p.scale) and torch.equal(s.history, p.history)
        s.optimizer_step(1e-2, 1e-3, weight_decay=0.1, **HP)
        norm, coef = p.optimize(pg, 1e-2, 1e-3, 0.1)
        assert torch.equal(s.norm, norm) and torch.equal(s.coef, coef)
        for a, b in zip(s.w + s.gamma, p.w + p.gamma):
            assert torch.equal(a, b)


@pytest.mark.parametrize("stream", [BF, F32])
def test_gradients_against_autograd(stream):
    T, C, L = 256, 128, 2
    torch.manual_seed(1)
    s = NormLinearStack(L, C, stream_dtype=stream)
    x, dy = inputs(T, C, 2)
    for _ in range(2):  # the second step casts with the scales of the first one's amaxes
        s.forward(x), s.backward(dy)
    got = [g.double().cpu() for g in s.grads()]
    leaf = lambda t: t.double().cpu().requires_grad_()  # noqa: E731
    w, gamma = [leaf(t) for t in s.w], [leaf(t) for t in s.gamma]
    norm = lambda h, g: h / torch.sqrt((h * h).mean(-1, keepdim=True) + s.eps) * g  # noqa: E731
    h = x.double().cpu()
    for i in range(L):
        h = h + norm(h, gamma[i]) @ w[i]
    norm(h, gamma[L]).backward(dy.double().cpu())
    for a, b in zip(got, [t.grad for t in w + gamma]):
        assert (a * b).sum() / (a.norm() * b.norm()) > 0.95
        assert abs(a.norm() / b.norm() - 1) < 0.2


def test_training_lowers_the_loss():
    T, C = 256, 64
    torch.manual_seed(3)
    s = NormLinearStack(2, C)
    x, t = inputs(T, C, 4)[0], inputs(T, C, 5)[0].float()
    losses = []
    for _ in range(40):
        y = s.forward(x).float()
        losses.append(((y - t) ** 2).sum().item() / T)
        s.backward((2 * (y - t) / T).to(BF))
        s.optimizer_step(1e-2, 1.0)
        assert float(s.norm) > 0 and 0 < float(s.coef) <= 1
    assert losses[-1] < losses[0]


def test_a_bad_gradient_skips_the_whole_step():
    T, C = 64, 64
    s = NormLinearStack(2, C)
    x, dy = inputs(T, C, 6)
    s.forward(x), s.backward(dy), s.optimizer_step(1e-2, 1.0)
    before = [p.clone() for p in s.w + s.gamma]
    dy[3, 5] = float("inf")
    s.forward(x), s.backward(dy), s.optimizer_step(1e-2, 1.0)
    assert not torch.isfinite(s.norm).item()
    for a, b in zip(s.w + s.gamma, before):
        assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", [dsg.E2M1, dsg.E4M3, dsg.E5M2])
@pytest.mark.parametrize("T", [1, 5, 130])
def test_decode_equals_the_separate_calls(T, fmt):
    C, L = 160, 2
    torch.manual_seed(7)
    s = NormLinearStack(L, C, stream_dtype=F32)
    s.quantize()
    x = inputs(T, C, 8)[0]
    y = s.decode(x, fmt)
    h = x.float()
    for i in range(L):
        y32 = torch.empty(T, C, device=DEV)
        dsg.fp8ds_rmsnorm(h, s.gamma[i], s.eps, y=y32)
        q, qs = u8(T, C // 2 if fmt == dsg.E2M1 else C), u8(T, C // 32)
        if fmt == dsg.E2M1:
            dsg.fp8ds_cast_mxfp4(y32, q, qs)
        else:
            dsg.fp8ds_cast_mx(y32, fmt, q, qs)
        wt, wts = u8(C, C // 2), u8(C, C // 32)
        dsg.fp8ds_cast_mxfp4(s.w[i].t().contiguous(), wt, wts)
        out = torch.empty(T, C, dtype=BF, device=DEV)
        dsg.fp8ds_gemm_mxfp4(T, C, C, q, fmt, C, qs, C // 32, wt, C, wts, C // 32, out, C)
        h = h + out.float()
    ref = torch.empty(T, C, dtype=BF, device=DEV)
    dsg.fp8ds_rmsnorm(h, s.gamma[L], s.eps, y=ref)
    assert torch.equal(y, ref)
    assert torch.equal(x, inputs(T, C, 8)[0])  # the caller's x is left alone


def test_decode_in_bf16_stream_and_after_training():
    T, C = 9, 64
    s = NormLinearStack(2, C)
    x, dy = inputs(T, C, 9)
    s.quantize()
    before = s.decode(x).clone()
    s.forward(x), s.backward(dy), s.optimizer_step(1e-1, 1.0)
    assert bool(s.decode(x, dsg.E4M3).isfinite().all())
    s.quantize()
    assert not torch.equal(s.decode(x), before)
