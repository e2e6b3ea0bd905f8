"""The stack of gated feed-forward blocks (delayed_scaling_gemm_amd/ffn.py) on the GPU.

With an FP32 residual stream each fused step has a composition of separate calls with the same
roundings (the gated product to FP32, then its cast; norms to FP32, then theirs; weights updated, then
cast), so the two have to agree bit for bit.  Gradients are also held against autograd in fp64 without
any quantisation: the products' operands are rounded by at most 2^-4 (E4M3) and 2^-3 (E5M2) relative to
each value, of either sign, so over the up to nine rounded operands on a gradient's way through two
blocks the relative error's root mean square is below sqrt(5 2^-8 + 4 2^-6) / sqrt(3) = 0.17, and the
cosine above 1 - 0.17^2 / 2 = 0.985 for values all of one binade's worst: 0.95 is asked."""

import math

import pytest

torch = pytest.importorskip("torch")

import delayed_scaling_gemm_amd as dsg  # noqa: E402
from delayed_scaling_gemm_amd.ffn import A, DGU, DY, W, WD, X, GatedFeedForwardStack  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


def u8(*shape):
    return torch.empty(shape, dtype=U8, device=DEV)


def f32(*shape):
    return torch.empty(shape, device=DEV)


def inputs(T, C, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, C, generator=g).to(BF).to(DEV)
    dy = (torch.randn(T, C, generator=g) / T).to(BF).to(DEV)
    return x, dy


class Plain:
    """The same stack from separate calls, one per step of the formulas."""

    def __init__(self, s):
        self.s, self.L, self.C, self.F = s, s.layers, s.width, s.inner
        copy = lambda ts: [t.clone() for t in ts]  # noqa: E731
        self.w, self.wd, self.gamma = copy(s.w), copy(s.wd), copy(s.gamma)
        self.pg, self.gate = copy(s.post_gamma), copy(s.gate)
        self.mom = [[torch.zeros(self.C, self.F, device=DEV) for _ in range(2)] for _ in s.w]
        self.momd = [torch.zeros_like(t) for t in s.wd]
        self.moments = [(torch.zeros_like(p), torch.zeros_like(p)) for p in self.vectors()]
        self.history, self.cursor = torch.zeros_like(s.history), torch.zeros_like(s.cursor)
        self.scale, self.step = torch.ones_like(s.scale), 0

    def vectors(self):
        return self.gamma + self.pg + self.gate

    def at(self, which, i):
        n = which * self.L + i
        return self.used[n:n + 1]

    def cast(self, x, fmt, which, i, q, q_t=None):
        n = which * self.L + i
        dsg.fp8ds_cast_acc(x, fmt, self.scale[n:n + 1], q, q_t, self.used[n:n + 1], self.amax[n:n + 1])

    def run(self, x, dy):
        L, C, F, T, s = self.L, self.C, self.F, x.shape[0], self.s
        self.used, self.amax = torch.zeros_like(self.scale), torch.zeros_like(self.scale)
        h, y32, r = x.float(), f32(T, C), f32(T)
        dsg.fp8ds_rmsnorm(h, self.gamma[0], s.eps, y=y32, rstd=r)
        hs, rs, kept = [h], [r], []
        for i in range(L):
            xq, wq, wqt, dq, dqt = u8(T, C), u8(C, 2 * F), u8(2 * F, C), u8(F, C), u8(C, F)
            self.cast(y32, dsg.E4M3, X, i, xq)
            self.cast(self.w[i], dsg.E4M3, W, i, wq, wqt)
            self.cast(self.wd[i], dsg.E4M3, WD, i, dq, dqt)
            gu, a = torch.empty(T, 2 * F, dtype=BF, device=DEV), f32(T, F)
            dsg.fp8ds_gated_gemm(xq, dsg.E4M3, self.at(X, i), wqt, dsg.E4M3, self.at(W, i), s.act, gu=gu, y=a)
            aq, out = u8(T, F), torch.empty(T, C, dtype=BF, device=DEV)
            self.cast(a, dsg.E4M3, A, i, aq)
            dsg.fp8ds_gemm(dsg.OP_N, dsg.OP_T, T, C, F, aq, dsg.E4M3, F, self.at(A, i), dqt, dsg.E4M3, F,
                           self.at(WD, i), out, C)
            h, r1, r2, y32 = f32(T, C), f32(T), f32(T), f32(T, C)
            dsg.fp8ds_rmsnorm_sandwich(out, self.pg[i], s.post_eps, hs[-1], self.gamma[i + 1], s.eps, h,
                                       alpha=s.alpha, gate=self.gate[i], y=y32, post_rstd=r1, rstd=r2)
            hs.append(h), rs.append(r2), kept.append((xq, wq, dq, gu, aq, out, r1))
        y = y32.to(BF)
        g, dres, grads = dy, None, {}
        for i in range(L - 1, -1, -1):
            xq, wq, dq, gu, aq, out, r1 = kept[i]
            dh, dx = f32(T, C), f32(T, C)
            dg, dpg, dgate = f32(C), f32(C), f32(C)
            ws = u8(dsg.fp8ds_rmsnorm_sandwich_bwd_workspace(T, C))
            # (types of dy, x and dx are one: in FP32 they hold the same values)
            dsg.fp8ds_rmsnorm_sandwich_bwd(g.float(), hs[i + 1], rs[i + 1], self.gamma[i + 1], out.float(),
                                           r1, self.pg[i], dh, dg, dpg, ws, alpha=s.alpha,
                                           gate=self.gate[i], dgate=dgate, dres=dres, dx=dx)
            yq, gq, dgu = u8(T, C), u8(T, 2 * F), f32(T, 2 * F)
            self.cast(dx, dsg.E5M2, DY, i, yq)
            dsg.fp8ds_gated_gemm_bwd(yq, dsg.E5M2, self.at(DY, i), dq, dsg.E4M3, self.at(WD, i), s.act, gu,
                                     dgu=dgu)
            self.cast(dgu, dsg.E5M2, DGU, i, gq)
            dwd, dw = torch.empty(F, C, dtype=BF, device=DEV), torch.empty(C, 2 * F, dtype=BF, device=DEV)
            dsg.fp8ds_gemm(dsg.OP_T, dsg.OP_N, F, C, T, aq, dsg.E4M3, F, self.at(A, i), yq, dsg.E5M2, C,
                           self.at(DY, i), dwd, C)
            dsg.fp8ds_gemm(dsg.OP_T, dsg.OP_N, C, 2 * F, T, xq, dsg.E4M3, C, self.at(X, i), gq, dsg.E5M2,
                           2 * F, self.at(DGU, i), dw, 2 * F)
            g = torch.empty(T, C, dtype=BF, device=DEV)
            dsg.fp8ds_gemm(dsg.OP_N, dsg.OP_T, T, C, 2 * F, gq, dsg.E5M2, 2 * F, self.at(DGU, i), wq,
                           dsg.E4M3, 2 * F, self.at(W, i), g, C)
            grads[i], dres = (dw, dwd, dg, dpg, dgate), dh
        dh, dg0 = f32(T, C), f32(C)
        dsg.fp8ds_rmsnorm_bwd(g, hs[0], rs[0], self.gamma[0], dh, dg0,
                              u8(max(16, dsg.fp8ds_rmsnorm_bwd_workspace(T, C))), dres)
        dsg.fp8ds_scale_update(self.history, self.cursor, self.amax, s.fmts, s.algo, 0, self.scale)
        self.step += 1
        by = lambda k: [grads[i][k] for i in range(L)]  # noqa: E731
        return y, dh, by(0) + by(1) + [dg0] + by(2) + by(3) + by(4)

    def optimize(self, grads, lr, max_norm, decay):
        L, F, C = self.L, self.F, self.C
        norm, coef = torch.zeros(1, device=DEV), torch.zeros(1, device=DEV)
        dsg.fp8ds_grad_norm(grads, max_norm, norm, coef, u8(dsg.fp8ds_grad_norm_workspace()))
        adjust = 0.2 * math.sqrt(max(C, F))
        for i in range(L):
            o = []
            for k in range(2):
                g = grads[i][:, k * F:(k + 1) * F].contiguous()
                o.append(torch.empty(C, F, dtype=BF, device=DEV))
                dsg.fp8ds_muon_direction(g, o[k], u8(dsg.fp8ds_muon_workspace(C, F)),
                                         momentum=self.mom[i][k], grad_coef=coef)
            dsg.fp8ds_muon_apply(self.w[i], torch.cat(o, 1), lr, decay, adjust)
            od = torch.empty(F, C, dtype=BF, device=DEV)
            dsg.fp8ds_muon_direction(grads[L + i], od, u8(dsg.fp8ds_muon_workspace(F, C)),
                                     momentum=self.momd[i], grad_coef=coef)
            dsg.fp8ds_muon_apply(self.wd[i], od, lr, decay, adjust)
        for p, g, (m, v) in zip(self.vectors(), grads[2 * L:], self.moments):
            dsg.fp8ds_adamw(p, g, m, v, lr, 0.9, 0.999, 1e-8, 0.0, self.step, grad_coef=coef)


@pytest.mark.parametrize("T,C,F,layers,act", [(1, 32, 48, 1, 0), (17, 160, 96, 2, 1), (96, 64, 256, 3, 0),
                                              (300, 256, 272, 2, 0)])
def test_steps_equal_the_separate_calls(T, C, F, layers, act):
    torch.manual_seed(T + C)
    s = GatedFeedForwardStack(layers, C, F, act=act, alpha=0.5, stream_dtype=F32)
    for p in s.gate + s.post_gamma:
        p.add_(0.1 * torch.randn_like(p))
    p = Plain(s)
    for step in range(3):
        x, dy = inputs(T, C, 10 * T + step)
        y, dx = s.forward(x), s.backward(dy)
        py, pdx, pg = p.run(x, dy)
        assert torch.equal(y, py) and torch.equal(dx, pdx)
        for a, b in zip(s.grads(), pg):
            assert torch.equal(a, b)
        assert torch.equal(s.scale, p.scale) and torch.equal(s.history, p.history)
        s.optimizer_step(1e-2, 1e-3, weight_decay=0.1)
        p.optimize(pg, 1e-2, 1e-3, 0.1)
        for a, b in zip(s.w + s.wd + s.vectors(), p.w + p.wd + p.vectors()):
            assert torch.equal(a, b)


@pytest.mark.parametrize("stream", [BF, F32])
@pytest.mark.parametrize("act", [0, 1])
def test_gradients_against_autograd(stream, act):
    T, C, F, L = 256, 128, 192, 2
    torch.manual_seed(1)
    s = GatedFeedForwardStack(L, C, F, act=act, alpha=0.7, stream_dtype=stream)
    for w in s.w + s.wd:
        w.mul_(4)  # gates that are not near 0
    x, dy = inputs(T, C, 2)
    for _ in range(2):  # the second step casts with the scales of the first one's amaxes
        s.forward(x), s.backward(dy)
    got = [g.double().cpu() for g in s.grads()]
    leaf = lambda t: t.double().cpu().requires_grad_()  # noqa: E731
    w, wd, gamma = [leaf(t) for t in s.w], [leaf(t) for t in s.wd], [leaf(t) for t in s.gamma]
    pg, gate = [leaf(t) for t in s.post_gamma], [leaf(t) for t in s.gate]
    norm = lambda h, g, e: h / torch.sqrt((h * h).mean(-1, keepdim=True) + e) * g  # noqa: E731
    fn = torch.nn.functional
    h = x.double().cpu()
    for i in range(L):
        gu = norm(h, gamma[i], s.eps) @ w[i]
        g = fn.silu(gu[:, :F]) if act == 0 else fn.gelu(gu[:, :F], approximate="tanh")
        h = h + s.alpha * gate[i] * norm((g * gu[:, F:]) @ wd[i], pg[i], s.post_eps)
    norm(h, gamma[L], s.eps).backward(dy.double().cpu())
    for a, b in zip(got, [t.grad for t in w + wd + gamma + pg + gate]):
        assert (a * b).sum() / (a.norm() * b.norm()) > 0.95
        assert abs(a.norm() / b.norm() - 1) < 0.2


def test_a_bad_gradient_skips_the_whole_step():
    T, C = 64, 64
    s = GatedFeedForwardStack(2, C, 96)
    x, dy = inputs(T, C, 6)
    s.forward(x), s.backward(dy), s.optimizer_step(1e-2, 1.0)
    keep = lambda: s.w + s.wd + s.vectors() + s.momentum + s.momentum_d  # noqa: E731
    before = [p.clone() for p in keep()]
    dy[3, 5] = float("inf")
    s.forward(x), s.backward(dy), s.optimizer_step(1e-2, 1.0)
    assert not torch.isfinite(s.norm).item()
    for a, b in zip(keep(), before):
        assert torch.equal(a, b)
    y = s.forward(x)
    assert torch.isfinite(y).all()


@pytest.mark.parametrize("T", [1, 5, 16, 40])
def test_decode_is_the_forward_pass(T):
    """The same weights and scales: the same bits; captured too, whatever ran before."""
    C, F = 160, 176
    torch.manual_seed(7)
    s = GatedFeedForwardStack(2, C, F, alpha=0.5)
    x, dy = inputs(64, C, 8)
    for _ in range(3):
        s.forward(x), s.backward(dy), s.optimizer_step(1e-2, 1.0)
    xs = [inputs(T, C, 20 + i)[0] for i in range(3)]
    want = [s.forward(v).clone() for v in xs]  # (the first one with the optimizer's FP8 weights)
    # forward() casts the weights anew from the second call on, with the same scales
    for v, y in zip(xs, want):
        assert torch.equal(s.decode(v), y)
    v = xs[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = s.decode(v)
    for i in (1, 2, 0):
        v.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])
        s.decode(inputs(T + 3, C, 99)[0])  # other buffers than the graph's


def test_decode_after_quantize():
    T, C, F = 9, 64, 96
    s = GatedFeedForwardStack(2, C, F)
    s.quantize()
    x = inputs(T, C, 9)[0]
    a = s.decode(x).clone()
    assert torch.isfinite(a).all()
    s.w[0].mul_(-1)  # the other sign of gate and up: another output, after the codes are made anew
    assert torch.equal(s.decode(x), a)
    s.quantize()
    assert not torch.equal(s.decode(x), a)


def test_side_stream_steps_equal_the_default_stream_steps():
    T, C, F = 48, 64, 80
    runs = []
    for side in (False, True):
        torch.manual_seed(11)
        s = GatedFeedForwardStack(2, C, F)
        stream = torch.cuda.Stream() if side else None
        x, dy = inputs(T, C, 12)
        torch.cuda.synchronize()
        for _ in range(3):
            y = s.forward(x, stream=stream)
            s.backward(dy, stream=stream), s.optimizer_step(1e-2, 1.0, stream=stream)
        torch.cuda.synchronize()
        runs.append([y] + s.w + s.wd + s.vectors())
    assert all(torch.equal(a, b) for a, b in zip(*runs))
