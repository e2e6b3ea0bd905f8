"""A residual stack of RMSNorm and FP8 Linear blocks, trained and served, composed from the
C-ABI calls.

  h_0 = x,   h_(l+1) = h_l + Linear_l(RMSNorm_l(h_l)),   y = RMSNorm_L(h_L)

Training (:meth:`NormLinearStack.forward`, :meth:`~NormLinearStack.backward`,
:meth:`~NormLinearStack.optimizer_step`), delayed scaling in the HYBRID recipe:

  fwd:  fp8ds_rmsnorm adds the last Linear's output to the stream, normalises and writes the
        next Linear's E4M3 operand in one pass: X has no 16-bit copy.
  bwd:  dX of a Linear goes through fp8ds_rmsnorm_bwd, which adds the stream's gradient and
        writes both the new one and, in E5M2, the dY operand of the Linear below.
  opt:  fp8ds_grad_norm over every dW and dgamma; fp8ds_adamw scales by its coefficient on the
        device, skips the whole step where the norm is not finite, and writes the next
        forward's FP8 weights.
  One scale update for the histories of all X, W and dY ends the step.

Serving (:meth:`~NormLinearStack.quantize`, :meth:`~NormLinearStack.decode`): the weights in
MXFP4, fp8ds_rmsnorm_mx writes the activations in blocks of 32 (E2M1, E4M3 or E5M2) and
fp8ds_gemm_mxfp4 multiplies them.  No calibration, any number of tokens.

Weights are stored [in, out].  Everything stays on one stream, without a host
synchronisation.  A decode can be captured into a graph; the training calls alternate amax sets
and count steps on the host, so a graph of one would repeat that step's.
"""

from __future__ import annotations

import torch

from . import (ALGO_MAX, E2M1, E4M3, E5M2, MMA_EXACT, MMA_FP8, OP_N, OP_T, fp8ds_adamw,
               fp8ds_cast_acc, fp8ds_cast_mxfp4, fp8ds_gemm, fp8ds_gemm_mxfp4, fp8ds_grad_norm,
               fp8ds_grad_norm_workspace, fp8ds_rmsnorm, fp8ds_rmsnorm_bwd,
               fp8ds_rmsnorm_bwd_workspace, fp8ds_rmsnorm_mx, fp8ds_scale_update_clear)
from .buffers import Buffers
from .linear import DY, FP8_FWD_MIN_K, W, X


class NormLinearStack(Buffers):
    """``layers`` blocks of width ``width`` (a multiple of 32).  ``stream_dtype`` is the type of
    the residual stream h: BF16, or FP32 where its additions should not round."""

    def __init__(self, layers: int, width: int, eps: float = 1e-5, hist_len: int = 16,
                 algo: int = ALGO_MAX, margin: int = 0, stream_dtype=torch.bfloat16,
                 device="cuda", mma_bwd: int = MMA_EXACT, mma_decode: int = MMA_EXACT):
        if layers < 1 or width < 32 or width % 32:
            raise ValueError(f"layers {layers} must be positive, width {width} a multiple of 32")
        if stream_dtype not in (torch.bfloat16, torch.float32):
            raise TypeError("the residual stream is bf16 or fp32")
        self.layers, self.width, self.eps = layers, width, eps
        self.algo, self.margin = algo, margin
        # datapaths of the backward products, and of decode()'s with MXFP8 activations
        self.mma_bwd, self.mma_decode = mma_bwd, mma_decode
        self.stream_dtype = stream_dtype
        super().__init__(device)
        f32 = dict(dtype=torch.float32, device=self.device)
        # fp32 masters and their moments; a gamma per norm, the last one's too
        self.w = [torch.empty(width, width, **f32).normal_(std=0.02) for _ in range(layers)]
        self.gamma = [torch.ones(width, **f32) for _ in range(layers + 1)]
        self.moments = [(torch.zeros_like(p), torch.zeros_like(p)) for p in self.w + self.gamma]
        # scaling state: all X, then all W, then all dY
        n = 3 * layers
        self.fmts = [E4M3] * (2 * layers) + [E5M2] * layers
        self.history = torch.zeros(n, hist_len, **f32)
        self.cursor = torch.zeros(n, dtype=torch.int32, device=self.device)
        self.scale = torch.ones(n, **f32)
        self.scale_used = torch.zeros(n, **f32)
        # amax of all histories, two sets used in turn: the scale update that ends a step
        # zeroes the next step's
        self._amax = torch.zeros(2, n, **f32)
        self.norm = torch.zeros(1, **f32)
        self.coef = torch.ones(1, **f32)
        self.steps = 0
        self._prepared = False  # optimizer_step wrote this step's FP8 weights
        self._pending = False   # a forward has not met its backward yet
        self._fresh = False     # a backward's gradients have not been applied yet

    def _state(self, which, layer):
        """(scale, scale_used, amax of this step) of X, W or dY of a layer."""
        i = which * self.layers + layer
        return (self.scale[i:i + 1], self.scale_used[i:i + 1],
                self._amax[self.steps & 1, i:i + 1])

    def _h(self, i, tokens):
        return self._buf(f"h{i}", (tokens, self.width), self.stream_dtype)

    def forward(self, x, stream=None):
        """``x`` [tokens, width] BF16 (or of the stream's type) -> y [tokens, width] BF16."""
        T, C, u8, bf = x.shape[0], self.width, torch.uint8, torch.bfloat16
        if x.dim() != 2 or x.shape[1] != C:
            raise ValueError(f"x is {tuple(x.shape)}, the stack [tokens, {C}]")
        self._use(stream)
        rstd = self._buf("rstd", (self.layers + 1, T), torch.float32)
        mma = MMA_FP8 if C >= FP8_FWD_MIN_K else MMA_EXACT
        residual = None
        for i in range(self.layers):
            s, su, am = self._state(X, i)
            xq = self._buf(f"xq{i}", (T, C), u8)
            h = self._h(i, T)
            fp8ds_rmsnorm(x, self.gamma[i], self.eps, residual, h, None, rstd[i], E4M3, s, xq, su,
                          am, stream=stream)
            s, su, am = self._state(W, i)
            wq = self._buf(f"wq{i}", (C, C), u8)
            wqt = self._buf(f"wqt{i}", (C, C), u8)
            if not self._prepared:
                fp8ds_cast_acc(self.w[i], E4M3, s, wq, wqt, su, am, stream=stream)
            x = self._buf("x", (T, C), bf)  # free again: the norm has put the last one into h
            fp8ds_gemm(OP_N, OP_T, T, C, C, xq, E4M3, C, self._state(X, i)[1], wqt, E4M3, C, su, x,
                       C, None, stream, mma=mma)
            residual = h
        y = self._buf("y", (T, C), bf)
        fp8ds_rmsnorm(x, self.gamma[-1], self.eps, residual, self._h(self.layers, T), y,
                      rstd[-1], stream=stream)
        self._prepared, self._pending = False, True
        return y

    def backward(self, dy, stream=None):
        """``dy`` [tokens, width] (BF16) -> the gradient of x, of the stream's type; the weights'
        are in :meth:`grads`.  Ends the step: the scales move on."""
        T, C, u8, f32 = dy.shape[0], self.width, torch.uint8, torch.float32
        rstd = self._bufs.get("rstd")
        if not self._pending or tuple(dy.shape) != (rstd.shape[1], C):
            raise RuntimeError("backward() needs a forward() of this shape before it")
        self._use(stream)
        ws = self._buf("ws", (max(16, fp8ds_rmsnorm_bwd_workspace(T, C)),), u8)
        dq = self._buf("dq", (T, C), u8)
        dres = None
        for i in range(self.layers, -1, -1):
            h = self._h(i, T)
            dh = self._buf("dh", (T, C), self.stream_dtype)  # in place: the stream's gradient
            cast = {}
            if i > 0:  # the operand of the Linear whose output h_i took in
                s, su, am = self._state(DY, i - 1)
                cast = dict(fmt=E5M2, scale=s, q=dq, scale_used=su, amax=am)
            fp8ds_rmsnorm_bwd(dy, h, rstd[i], self.gamma[i], dh, self._buf(f"dg{i}", (C,), f32), ws,
                              dres, stream=stream, **cast)
            if i == 0:
                break
            j = i - 1
            dy = self._buf("dx", (T, C), torch.bfloat16)
            fp8ds_gemm(OP_N, OP_T, T, C, C, dq, E5M2, C, su, self._bufs[f"wq{j}"], E4M3, C,
                       self._state(W, j)[1], dy, C, None, stream, mma=self.mma_bwd)
            dw = self._buf(f"dw{j}", (C, C), torch.bfloat16)
            fp8ds_gemm(OP_T, OP_N, C, C, T, self._bufs[f"xq{j}"], E4M3, C,
                       self._state(X, j)[1], dq, E5M2, C, su, dw, C, None, stream,
                       mma=self.mma_bwd)
            dres = dh
        now = self.steps & 1
        fp8ds_scale_update_clear(self.history, self.cursor, self._amax[now], self.fmts, self.algo,
                                 self.margin, self.scale, self._amax[now ^ 1], stream=stream)
        self.steps += 1
        self._pending, self._fresh = False, True
        return dh

    def grads(self):
        """The last backward's gradients: every dW (BF16 [in, out]), then every dgamma (FP32)."""
        return ([self._bufs[f"dw{i}"] for i in range(self.layers)]
                + [self._bufs[f"dg{i}"] for i in range(self.layers + 1)])

    def optimizer_step(self, lr, max_norm, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0,
                       grad_scale=1.0, stream=None):
        """AdamW with the gradients clipped to the global norm ``max_norm`` (gammas without
        decay), and the FP8 weights of the next forward.  ``norm`` and ``coef`` hold the norm
        (times ``grad_scale``) and the factor; a norm that is not finite skips the step.

        Once for a :meth:`backward`, before the next :meth:`forward`: it writes the FP8 weights
        that a pending backward would read."""
        if self._pending or not self._fresh:
            raise RuntimeError("optimizer_step() comes once after each backward(), before the next "
                               "forward()")
        self._use(stream)
        C, u8, g = self.width, torch.uint8, self.grads()
        ws = self._buf("norm_ws", (fp8ds_grad_norm_workspace(),), u8)
        fp8ds_grad_norm(g, max_norm, self.norm, self.coef, ws, grad_scale, stream)
        for i, p in enumerate(self.w + self.gamma):
            m, v = self.moments[i]
            cast, decay = {}, 0.0
            if i < self.layers:
                s, su, am = self._state(W, i)
                cast = dict(fmt=E4M3, scale=s, q=self._buf(f"wq{i}", (C, C), u8),
                            q_t=self._buf(f"wqt{i}", (C, C), u8), scale_used=su, amax=am)
                decay = weight_decay
            fp8ds_adamw(p, g[i], m, v, lr, beta1, beta2, eps, decay, self.steps,
                        grad_scale=grad_scale, grad_amax=self.norm, stream=stream,
                        grad_coef=self.coef, **cast)
        self._prepared, self._fresh = True, False

    def quantize(self, stream=None):
        """Write the weights' MXFP4 codes for :meth:`decode`."""
        self._use(stream)
        C, u8 = self.width, torch.uint8
        for i, w in enumerate(self.w):
            # the product reads W^T blocked along in: the cast's transposed copy
            fp8ds_cast_mxfp4(w, self._buf("m4", (C, C // 2), u8),
                             self._buf("m4s", (C, C // 32), u8),
                             self._buf(f"m4t{i}", (C, C // 2), u8),
                             self._buf(f"m4st{i}", (C, C // 32), u8), stream)

    def decode(self, x, fmt=E4M3, stream=None):
        """:meth:`forward` with the weights of the last :meth:`quantize` and the activations in
        MX blocks of ``fmt``; any number of tokens, nothing kept for a backward pass."""
        if "m4t0" not in self._bufs:
            raise RuntimeError("decode() needs the weights of a preceding quantize()")
        T, C, u8, bf = x.shape[0], self.width, torch.uint8, torch.bfloat16
        if x.dim() != 2 or x.shape[1] != C:
            raise ValueError(f"x is {tuple(x.shape)}, the stack [tokens, {C}]")
        self._use(stream)
        q = self._buf("sq", (T, C // 2 if fmt == E2M1 else C), u8)
        qs = self._buf("sqs", (T, C // 32), u8)
        h, residual = self._buf("sh", (T, C), self.stream_dtype), None
        for i in range(self.layers):
            fp8ds_rmsnorm_mx(x, self.gamma[i], self.eps, fmt, q, qs, residual, h, stream=stream)
            x = self._buf("sx", (T, C), bf)
            fp8ds_gemm_mxfp4(T, C, C, q, fmt, C, qs, C // 32, self._bufs[f"m4t{i}"],
                             C, self._bufs[f"m4st{i}"], C // 32, x, C, None, stream,
                             self.mma_decode)
            residual = h  # in place from here on
        y = self._buf("sy", (T, C), bf)
        fp8ds_rmsnorm(x, self.gamma[-1], self.eps, residual, None, y, stream=stream)
        return y
