"""A residual stack of gated feed-forward blocks with a norm on either side of each, trained and served,
composed from the C-ABI calls.

  h_0 = x
  a_l = act(n_l Wg_l) * (n_l Wu_l),  n_l = RMSNorm(h_l; gamma_l)
  h_(l+1) = h_l + alpha gate_l RMSNorm(a_l Wd_l; post_gamma_l),   y = RMSNorm(h_L; gamma_L)

Training (:meth:`GatedFeedForwardStack.forward`, :meth:`~GatedFeedForwardStack.backward`,
:meth:`~GatedFeedForwardStack.optimizer_step`), delayed scaling in the HYBRID recipe:

  fwd:  fp8ds_gated_gemm multiplies by gate and up, activates and writes the down projection's E4M3
        operand; fp8ds_rmsnorm_sandwich normalises its output, gates and adds it, normalises the
        stream and writes the next block's operand.  Neither operand has a 16-bit copy.
  bwd:  fp8ds_rmsnorm_sandwich_bwd gives the stream's gradient and the down projection's E5M2 dY;
        fp8ds_gated_gemm_bwd takes that through the down projection and the activation to the
        E5M2 dY of gate and up together, whose dX and dW are one product each.
  opt:  fp8ds_grad_norm over all gradients; Muon for the matrices, gate and up each for itself
        (fp8ds_muon_direction, fp8ds_muon_apply, which writes the next forward's FP8 weights), AdamW
        for gammas and gates.  A norm that is not finite skips the whole step.

Serving (:meth:`~GatedFeedForwardStack.decode`): the same FP8 weights and the scales that training left
(or :meth:`~GatedFeedForwardStack.quantize` makes), any number of tokens, nothing kept.

Weights are stored [in, out], gate and up side by side as [width, 2 inner].  Everything stays on one
stream, without a host synchronisation.  A decode can be captured into a graph; the training calls
alternate amax sets and count steps on the host, so a graph of one would repeat that step's.
"""

from __future__ import annotations

import math

import torch

from . import (ACT_SILU, ALGO_MAX, E4M3, E5M2, MMA_EXACT, OP_N, OP_T, fp8ds_adamw, fp8ds_cast_acc,
               fp8ds_cast_current, fp8ds_gated_gemm, fp8ds_gated_gemm_bwd, fp8ds_gemm, fp8ds_grad_norm,
               fp8ds_grad_norm_workspace, fp8ds_muon_apply, fp8ds_muon_direction, fp8ds_muon_workspace,
               fp8ds_rmsnorm, fp8ds_rmsnorm_bwd, fp8ds_rmsnorm_bwd_workspace, fp8ds_rmsnorm_sandwich,
               fp8ds_rmsnorm_sandwich_bwd, fp8ds_rmsnorm_sandwich_bwd_workspace,
               fp8ds_scale_update_clear)
from .buffers import Buffers

# tensors of a block with a scaling history: both inputs, both weights, both output gradients
X, A, W, WD, DGU, DY = range(6)
_FMT = (E4M3, E4M3, E4M3, E4M3, E5M2, E5M2)


class GatedFeedForwardStack(Buffers):
    """``layers`` blocks of width ``width`` and inner width ``inner`` (multiples of 16).  ``alpha`` is
    the residual scale, ``stream_dtype`` the type of the residual stream h."""

    def __init__(self, layers: int, width: int, inner: int, act: int = ACT_SILU, alpha: float = 1.0,
                 eps: float = 1e-5, post_eps: float = 1e-6, hist_len: int = 16, algo: int = ALGO_MAX,
                 margin: int = 0, stream_dtype=torch.bfloat16, device="cuda", mma: int = MMA_EXACT):
        if layers < 1 or width < 16 or width % 16 or inner < 16 or inner % 16:
            raise ValueError(f"layers {layers} must be positive, width {width} and inner {inner} "
                             "multiples of 16")
        if stream_dtype not in (torch.bfloat16, torch.float32):
            raise TypeError("the residual stream is bf16 or fp32")
        self.layers, self.width, self.inner, self.act = layers, width, inner, act
        self.alpha, self.eps, self.post_eps = alpha, eps, post_eps
        self.algo, self.margin, self.mma = algo, margin, mma
        self.stream_dtype = stream_dtype
        super().__init__(device)
        f32 = dict(dtype=torch.float32, device=self.device)
        # fp32 masters: [gate | up] and down of each block, a gamma per norm, a gate per block
        self.w = [torch.empty(width, 2 * inner, **f32).normal_(std=0.02) for _ in range(layers)]
        self.wd = [torch.empty(inner, width, **f32).normal_(std=0.02) for _ in range(layers)]
        self.gamma = [torch.ones(width, **f32) for _ in range(layers + 1)]
        self.post_gamma = [torch.ones(width, **f32) for _ in range(layers)]
        self.gate = [torch.ones(width, **f32) for _ in range(layers)]
        # Muon's momenta: gate's and up's are matrices of their own, one after the other
        self.momentum = [torch.zeros(2, width, inner, **f32) for _ in range(layers)]
        self.momentum_d = [torch.zeros(inner, width, **f32) for _ in range(layers)]
        self.moments = [(torch.zeros_like(p), torch.zeros_like(p)) for p in self.vectors()]
        n = 6 * layers
        self.fmts = [f for f in _FMT for _ in range(layers)]
        self.history = torch.zeros(n, hist_len, **f32)
        self.cursor = torch.zeros(n, dtype=torch.int32, device=self.device)
        self.scale = torch.ones(n, **f32)
        self.scale_used = torch.zeros(n, **f32)
        # amax of all histories, two sets used in turn: the scale update that ends a step zeroes the
        # next step's
        self._amax = torch.zeros(2, n, **f32)
        self.norm = torch.zeros(1, **f32)
        self.coef = torch.ones(1, **f32)
        self.steps = 0
        self._prepared = False  # optimizer_step wrote this step's FP8 weights
        self._pending = False   # a forward has not met its backward yet
        self._fresh = False     # a backward's gradients have not been applied yet

    def vectors(self):
        """Gammas, post-gammas and gates, in the order of their gradients in :meth:`grads`."""
        return self.gamma + self.post_gamma + self.gate

    def _state(self, which, layer):
        """(scale, scale_used, amax of this step) of a tensor of a block."""
        i = which * self.layers + layer
        return self.scale[i:i + 1], self.scale_used[i:i + 1], self._amax[self.steps & 1, i:i + 1]

    def _codes(self, i):
        """Buffers of block i's FP8 weights: [in, out] and transposed, of both matrices."""
        C, F, u8 = self.width, self.inner, torch.uint8
        return (self._buf(f"wq{i}", (C, 2 * F), u8), self._buf(f"wqt{i}", (2 * F, C), u8),
                self._buf(f"dq{i}", (F, C), u8), self._buf(f"dqt{i}", (C, F), u8))

    def _check(self, x, what="x"):
        if x.dim() != 2 or x.shape[1] != self.width:
            raise ValueError(f"{what} is {tuple(x.shape)}, the stack [tokens, {self.width}]")

    def forward(self, x, stream=None):
        """``x`` [tokens, width] BF16 (or of the stream's type) -> y [tokens, width] BF16."""
        self._check(x)
        T, C, F, u8, bf = x.shape[0], self.width, self.inner, torch.uint8, torch.bfloat16
        self._use(stream)
        rstd = self._buf("rstd", (self.layers + 1, T), torch.float32)
        post = self._buf("post_rstd", (self.layers, T), torch.float32)
        h = self._buf("h0", (T, C), self.stream_dtype)
        xq = self._buf("xq0", (T, C), u8)
        s, su, am = self._state(X, 0)
        fp8ds_rmsnorm(x, self.gamma[0], self.eps, None, h, None, rstd[0], E4M3, s, xq, su, am, stream=stream)
        y = self._buf("y", (T, C), bf)
        for i in range(self.layers):
            wq, wqt, dq, dqt = self._codes(i)
            if not self._prepared:
                for p, q, qt, which in ((self.w[i], wq, wqt, W), (self.wd[i], dq, dqt, WD)):
                    s, su, am = self._state(which, i)
                    fp8ds_cast_acc(p, E4M3, s, q, qt, su, am, stream=stream)
            gu, aq = self._buf(f"gu{i}", (T, 2 * F), bf), self._buf(f"aq{i}", (T, F), u8)
            s, su, am = self._state(A, i)
            fp8ds_gated_gemm(xq, E4M3, self._state(X, i)[1], wqt, E4M3, self._state(W, i)[1], self.act,
                             gu=gu, scale=s, q=aq, scale_used=su, amax=am, stream=stream, mma=self.mma)
            out = self._buf(f"out{i}", (T, C), bf)
            fp8ds_gemm(OP_N, OP_T, T, C, F, aq, E4M3, F, su, dqt, E4M3, F, self._state(WD, i)[1], out, C,
                       None, stream, mma=self.mma)
            nxt, cast = self._buf(f"h{i + 1}", (T, C), self.stream_dtype), {}
            if i + 1 < self.layers:
                s, su, am = self._state(X, i + 1)
                xq = self._buf(f"xq{i + 1}", (T, C), u8)
                cast = dict(fmt=E4M3, scale=s, q=xq, scale_used=su, amax=am)
            else:
                cast = dict(y=y)
            fp8ds_rmsnorm_sandwich(out, self.post_gamma[i], self.post_eps, h, self.gamma[i + 1], self.eps,
                                   nxt, alpha=self.alpha, gate=self.gate[i], post_rstd=post[i],
                                   rstd=rstd[i + 1], stream=stream, **cast)
            h = nxt
        self._prepared, self._pending = False, True
        return y

    def backward(self, dy, stream=None):
        """``dy`` [tokens, width] BF16 -> the gradient of x, of the stream's type; the parameters' are
        in :meth:`grads`.  Ends the step: the scales move on."""
        T, C, F, u8, f32 = dy.shape[0], self.width, self.inner, torch.uint8, torch.float32
        bf = torch.bfloat16
        rstd = self._bufs.get("rstd")
        if not self._pending or tuple(dy.shape) != (rstd.shape[1], C):
            raise RuntimeError("backward() needs a forward() of this shape before it")
        self._use(stream)
        post = self._bufs["post_rstd"]
        ws = self._buf("ws", (max(16, fp8ds_rmsnorm_sandwich_bwd_workspace(T, C),
                                  fp8ds_rmsnorm_bwd_workspace(T, C)),), u8)
        yq, gq = self._buf("dyq", (T, C), u8), self._buf("dguq", (T, 2 * F), u8)
        dh = self._buf("dh", (T, C), self.stream_dtype)  # in place: the stream's gradient
        dres = None
        for i in range(self.layers - 1, -1, -1):
            s, syu, am = self._state(DY, i)
            vec = [self._buf(f"{n}{i + k}", (C,), f32) for n, k in (("dg", 1), ("dpg", 0), ("dgate", 0))]
            fp8ds_rmsnorm_sandwich_bwd(dy, self._bufs[f"h{i + 1}"], rstd[i + 1], self.gamma[i + 1],
                                       self._bufs[f"out{i}"], post[i], self.post_gamma[i], dh, vec[0],
                                       vec[1], ws, alpha=self.alpha, gate=self.gate[i], dgate=vec[2],
                                       dres=dres, fmt=E5M2, scale=s, q=yq, scale_used=syu, amax=am,
                                       stream=stream)
            dres = dh
            s, sgu, am = self._state(DGU, i)
            fp8ds_gated_gemm_bwd(yq, E5M2, syu, self._bufs[f"dq{i}"], E4M3, self._state(WD, i)[1], self.act,
                                 self._bufs[f"gu{i}"], fmt=E5M2, scale=s, q=gq, scale_used=sgu, amax=am,
                                 stream=stream, mma=MMA_EXACT)
            dwd = self._buf(f"dwd{i}", (F, C), bf)
            fp8ds_gemm(OP_T, OP_N, F, C, T, self._bufs[f"aq{i}"], E4M3, F, self._state(A, i)[1], yq, E5M2,
                       C, syu, dwd, C, None, stream)
            fp8ds_gemm(OP_T, OP_N, C, 2 * F, T, self._bufs[f"xq{i}"], E4M3, C, self._state(X, i)[1], gq,
                       E5M2, 2 * F, sgu, self._buf(f"dw{i}", (C, 2 * F), bf), 2 * F, None, stream)
            dy = self._buf("dx", (T, C), bf)
            fp8ds_gemm(OP_N, OP_T, T, C, 2 * F, gq, E5M2, 2 * F, sgu, self._bufs[f"wq{i}"], E4M3, 2 * F,
                       self._state(W, i)[1], dy, C, None, stream)
        fp8ds_rmsnorm_bwd(dy, self._bufs["h0"], rstd[0], self.gamma[0], dh, self._buf("dg0", (C,), f32),
                          ws, dres, stream=stream)
        now = self.steps & 1
        fp8ds_scale_update_clear(self.history, self.cursor, self._amax[now], self.fmts, self.algo,
                                 self.margin, self.scale, self._amax[now ^ 1], stream=stream)
        self.steps += 1
        self._pending, self._fresh = False, True
        return dh

    def grads(self):
        """The last backward's gradients: every block's [gate | up] (BF16 [width, 2 inner]), every down
        projection's (BF16 [inner, width]), then those of :meth:`vectors` (FP32)."""
        L, b = range(self.layers), self._bufs
        return ([b[f"dw{i}"] for i in L] + [b[f"dwd{i}"] for i in L]
                + [b[f"dg{i}"] for i in range(self.layers + 1)] + [b[f"dpg{i}"] for i in L]
                + [b[f"dgate{i}"] for i in L])

    def optimizer_step(self, lr, max_norm, vector_lr=None, mu=0.95, nesterov=True, ns_steps=5,
                       weight_decay=0.0, beta1=0.9, beta2=0.999, eps=1e-8, grad_scale=1.0, stream=None):
        """Muon for the matrices (updates of root mean square 0.2 ``lr``), AdamW with ``vector_lr``
        (``lr`` if None) for the vectors, on gradients clipped to the global norm ``max_norm``, and the
        FP8 weights of the next forward.  A norm that is not finite skips the step.

        Once for a :meth:`backward`, before the next :meth:`forward`: it writes the FP8 weights that a
        pending backward would read."""
        if self._pending or not self._fresh:
            raise RuntimeError("optimizer_step() comes once after each backward(), before the next "
                               "forward()")
        self._use(stream)
        C, F, L, u8, bf = self.width, self.inner, self.layers, torch.uint8, torch.bfloat16
        g = self.grads()
        ws = self._buf("norm_ws", (fp8ds_grad_norm_workspace(),), u8)
        fp8ds_grad_norm(g, max_norm, self.norm, self.coef, ws, grad_scale, stream)
        mws = self._buf("muon_ws", (fp8ds_muon_workspace(C, F),), u8)
        muon = dict(mu=mu, nesterov=nesterov, steps=ns_steps, grad_scale=grad_scale, grad_coef=self.coef,
                    grad_amax=self.norm, stream=stream)
        adjust = 0.2 * math.sqrt(max(C, F))
        both, down = self._buf("o", (C, 2 * F), bf), self._buf("od", (F, C), bf)
        for i in range(L):
            wq, wqt, dq, dqt = self._codes(i)
            for k in range(2):  # gate and up are matrices of their own, side by side
                part = slice(k * F, (k + 1) * F)
                fp8ds_muon_direction(g[i][:, part], both[:, part], mws, momentum=self.momentum[i][k], **muon)
            fp8ds_muon_direction(g[L + i], down, mws, momentum=self.momentum_d[i], **muon)
            for p, o, q, qt, which in ((self.w[i], both, wq, wqt, W), (self.wd[i], down, dq, dqt, WD)):
                s, su, am = self._state(which, i)
                fp8ds_muon_apply(p, o, lr, weight_decay, adjust, E4M3, s, q, qt, su, am,
                                 grad_amax=self.norm, stream=stream)
        for p, gp, (m, v) in zip(self.vectors(), g[2 * L:], self.moments):
            fp8ds_adamw(p, gp, m, v, lr if vector_lr is None else vector_lr, beta1, beta2, eps, 0.0,
                        self.steps, grad_scale=grad_scale, grad_amax=self.norm, grad_coef=self.coef,
                        stream=stream)
        self._prepared, self._fresh = True, False

    def quantize(self, stream=None):
        """FP8 weights with current scales for :meth:`decode`, where training has not left any that
        fit the weights (after they were loaded, say).  The activations' scales are the state's:
        train, or set ``scale``."""
        if self._pending:
            raise RuntimeError("quantize() would overwrite the weights that a pending backward() reads")
        self._use(stream)
        for i in range(self.layers):
            wq, wqt, dq, dqt = self._codes(i)
            for p, q, qt, which in ((self.w[i], wq, wqt, W), (self.wd[i], dq, dqt, WD)):
                n = which * self.layers + i
                fp8ds_cast_current(p, E4M3, self.margin, q, self.scale_used[n:n + 1],
                                   self._buf("amax", (1,), torch.float32), qt, stream=stream)
        # (an optimizer step's scales are lost with its codes: the next forward casts anew)
        self._prepared = False

    def decode(self, x, stream=None):
        """:meth:`forward` with the FP8 weights that are there (of an :meth:`optimizer_step` or a
        :meth:`quantize`) and the present scales; any number of tokens, nothing kept for a backward
        pass and no amax taken."""
        self._check(x)
        if "wqt0" not in self._bufs:
            raise RuntimeError("decode() needs the FP8 weights of a training step or of quantize()")
        T, C, F, u8, bf = x.shape[0], self.width, self.inner, torch.uint8, torch.bfloat16
        self._use(stream)
        h, xq = self._buf("sh", (T, C), self.stream_dtype), self._buf("sxq", (T, C), u8)
        aq, out, y = self._buf("saq", (T, F), u8), self._buf("sout", (T, C), bf), self._buf("sy", (T, C), bf)
        fp8ds_rmsnorm(x, self.gamma[0], self.eps, None, h, None, None, E4M3, self._state(X, 0)[0], xq,
                      stream=stream)
        for i in range(self.layers):
            _, wqt, _, dqt = self._codes(i)
            sa = self._state(A, i)[0]
            fp8ds_gated_gemm(xq, E4M3, self._state(X, i)[0], wqt, E4M3, self._state(W, i)[1], self.act,
                             scale=sa, q=aq, stream=stream, mma=self.mma)
            fp8ds_gemm(OP_N, OP_T, T, C, F, aq, E4M3, F, sa, dqt, E4M3, F, self._state(WD, i)[1], out, C,
                       None, stream, mma=self.mma)
            last = i + 1 == self.layers
            cast = dict(y=y) if last else dict(fmt=E4M3, scale=self._state(X, i + 1)[0], q=xq)
            fp8ds_rmsnorm_sandwich(out, self.post_gamma[i], self.post_eps, h, self.gamma[i + 1], self.eps, h,
                                   alpha=self.alpha, gate=self.gate[i], stream=stream, **cast)
        return y
