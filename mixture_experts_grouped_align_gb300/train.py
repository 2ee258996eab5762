"""One training step of a bf16 MoE layer: routed experts, a dense shared expert beside them, and
the router's auxiliary losses.

Forward, for x [T, K]:
    logits = x Wr^T (fp32);  ids, w = top-k routing (moe_align)
    gu = x W1[e]^T per pair;  h = w * silu(g) u, gu kept as an MXFP8 checkpoint;  o = h W2[e]^T
    gs = x Ws1^T + bs1;       hs = silu(g) u,   gs kept as an MXFP8 checkpoint
    y = hs Ws2^T + bs2 + sum_j o_tj
Backward, from dy [T, K]: the activations' gradients come from the checkpoints, which also give
the activations again for the weight gradients; the routing weights' gradients join the
balance and z losses' in d_logits.

Marshalling only: products, activations, losses and sums run in the library's kernels; torch moves
data, namely the transposed copies of w1 and w2 and the rounding of d_logits to bf16.  The products take
bf16 operands, so dx and the router's gradient see the logits' gradient within 2^-9 of itself, as
every gradient that passes from one product to the next here; ``d_logits`` itself is fp32.  A
caller who wants more of the router's gradient has it there.

``TrainLayer`` refers to the caller's weights, which may change in place between steps (not between
a forward and its backward), and holds what lives from a forward to its backward: the routing, and
the pre-activations as MXFP8 checkpoints (33/64 of their bf16 bytes).  Everything else is scratch,
which layers can share.
"""
from __future__ import annotations

import math

import torch

from . import (Ctx, MoeError, moe_act_backward, moe_act_checkpoint, moe_align, moe_align_capacity, moe_dense_bias_grad,
               moe_dense_gemm, moe_grouped_gemm, moe_pair_sum, moe_router_loss, moe_router_loss_workspace_size,
               moe_wgrad, moe_wgrad_workspace_size)

BLOCK_M = 128


def _check(t, what, dtype, device, shape=None, numel=0):
    """MoeError unless ``t`` is a dense, 16-byte aligned tensor of ``dtype`` on ``device``, of exactly
    ``shape`` or of at least ``numel`` elements: the kernels read and write whole rows from its
    address on."""
    if not isinstance(t, torch.Tensor):
        raise MoeError(-1, f"{what}: need a torch tensor, got {type(t).__name__}")
    size_ok = t.numel() >= numel if shape is None else tuple(t.shape) == tuple(shape)
    if t.dtype != dtype or not size_ok or not t.is_contiguous() or t.data_ptr() % 16 or t.device != device:
        need = f"shape {tuple(shape)}" if shape is not None else f"at least {numel} elements"
        raise MoeError(-1, f"{what}: need a contiguous, 16-byte aligned {dtype} tensor of {need} on {device}, got {t.dtype} "
                           f"{tuple(t.shape)}, strides {t.stride()}, on {t.device}")


def _apart(a, b, what):
    """MoeError if the two dense tensors share memory."""
    if a.data_ptr() < b.data_ptr() + b.numel() * b.element_size() and b.data_ptr() < a.data_ptr() + a.numel() * a.element_size():
        raise MoeError(-1, f"{what} must not overlap")


class Scratch:
    """Device buffers of which nothing is needed between two passes of a layer: pre-activations and
    their gradients (one buffer), activations, pair rows, transposed weights, workspaces.  Layers
    whose passes follow one another in one stream can share one; it grows as layers are made (so make them
    before a pass is captured into a graph)."""

    def __init__(self, device):
        self.device, self.version, self._buffers = torch.device(device), 0, {}

    def reserve(self, name, nbytes):
        have = self._buffers.get(name)
        if have is None or have.numel() < nbytes:
            self._buffers[name] = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
            self.version += 1

    def view(self, name, dtype, *shape):
        n = dtype.itemsize
        for s in shape:
            n *= s
        return self._buffers[name][:n].view(dtype).view(shape)

    def nbytes(self):
        return sum(b.numel() for b in self._buffers.values())


class TrainLayer:
    """wr [E, K], w1 [E, 2I, K], w2 [E, K, I], ws1 [2Is, K], ws2 [K, Is], bs1 [2Is], bs2 [K]: bf16
    device tensors; K, I and Is multiples of 64, 1 <= k <= 32, k <= E <= 1024.  Batches of up to
    ``max_rows`` tokens.

    Every operand is checked before anything is launched (MoeError): type, shape, density,
    alignment and device, and that what a pass writes lies apart from what it still reads.

    ``scratch``: a ``Scratch`` to share with other layers (``other.scratch``); its own by default."""

    def __init__(self, wr, w1, w2, ws1, bs1, ws2, bs2, k, max_rows, balance_coef=0.01, z_coef=0.001, scratch=None):
        for what, t, dims in (("wr", wr, 2), ("w2", w2, 3), ("ws2", ws2, 2)):  # those that the sizes come from
            if not isinstance(t, torch.Tensor) or t.dim() != dims:
                raise MoeError(-1, f"{what}: need a torch tensor of {dims} dimensions")
        self.wr, self.w1, self.w2, self.ws1, self.bs1, self.ws2, self.bs2 = wr, w1, w2, ws1, bs1, ws2, bs2
        self.E, self.K, self.k = wr.shape[0], wr.shape[1], k
        self.I, self.Is = w2.shape[2], ws2.shape[1]
        if any(n % 64 for n in (self.K, self.I, self.Is)):
            raise ValueError("K, I and Is must be multiples of 64 (moe_wgrad)")
        if not (1 <= k <= 32 and k <= self.E <= 1024):
            raise ValueError("need 1 <= k <= 32 and k <= E <= 1024 (moe_router_loss)")
        self._check_weights()
        self.coef = (balance_coef, z_coef)
        dev, bf = wr.device, torch.bfloat16
        T, P, E, K, I, Is = max_rows, max_rows * k, self.E, self.K, self.I, self.Is
        self.max_rows, self.x = T, None
        new = lambda *shape, dtype=bf: torch.empty(shape, dtype=dtype, device=dev)  # noqa: E731
        i32, u8, f32 = torch.int32, torch.uint8, torch.float32
        self.logits, self.ids, self.w = new(T, E, dtype=f32), new(T, k, dtype=i32), new(T, k, dtype=f32)
        self.cap, blocks = moe_align_capacity(P, E, BLOCK_M)
        self.sorted, self.expert_ids, self.ntpp = new(self.cap, dtype=i32), new(blocks, dtype=i32), new(4, dtype=i32)
        self.codes, self.scales = new(P, 2 * I, dtype=u8), new(P, 2 * I // 32, dtype=u8)
        self.codes_s, self.scales_s = new(T, 2 * Is, dtype=u8), new(T, 2 * Is // 32, dtype=u8)
        # every token once, for the dense layers' weight gradients (one expert)
        self.cap1, blocks1 = moe_align_capacity(T, 1, BLOCK_M)
        self.sorted1, self.expert_ids1, self.ntpp1 = new(self.cap1, dtype=i32), new(blocks1, dtype=i32), new(4, dtype=i32)
        self.zeros = torch.zeros((T, 1), dtype=i32, device=dev)
        self.d_logits = new(T, E, dtype=f32)
        # the router's gradient products take E in multiples of 64: columns of zeros in d_logits and
        # rows of zeros in a copy of wr
        self.Ep = (E + 63) // 64 * 64
        self.grad_wr = new(self.Ep, K, dtype=f32)
        self.counts, self.prob_mean, self.loss = new(E, dtype=i32), new(E, dtype=f32), new(3, dtype=f32)
        self.status = torch.zeros(4, dtype=i32, device=dev)
        self.grads = {"wr": self.grad_wr[:E], "w1": new(E, 2 * I, K, dtype=f32), "w2t": new(E, I, K, dtype=f32),
                      "ws1": new(2 * Is, K, dtype=f32), "ws2": new(K, Is, dtype=f32), "bs1": new(2 * Is, dtype=f32),
                      "bs2": new(K, dtype=f32)}
        need = max(moe_router_loss_workspace_size(E), 256,
                   *(moe_wgrad_workspace_size(e, n, kin, BLOCK_M, c) for e, n, kin, c in
                     [(E, 2 * I, K, self.cap), (E, I, K, self.cap), (1, 2 * Is, K, self.cap1), (1, K, Is, self.cap1)]))
        self.scratch = Scratch(dev) if scratch is None else scratch
        if self.scratch.device != dev:
            raise MoeError(-1, f"scratch: need one on {dev}, got {self.scratch.device}")
        # name: (type, shape, what it is reserved as)
        self._views, self._bound = {
            "workspace": (u8, (need,), "workspace"),
            # the experts' input gradients contract over their outputs: a transposed copy of w2, then of
            # w1, made by every backward from the weights as they are then
            "wt": (bf, (E * 2 * I * K,), "wt"),
            "gu": (bf, (P, 2 * I), "gu"), "dgu": (bf, (P, 2 * I), "gu"),  # gu is done with when its checkpoint is written
            "h": (bf, (P, I), "h"), "dh": (bf, (P, I), "dh"), "dw": (f32, (T, k), "dw"),
            "o": (bf, (P, K), "pairs"), "dx_pairs": (bf, (P, K), "pairs"),
            "gs": (bf, (T, 2 * Is), "gs"), "dgs": (bf, (T, 2 * Is), "gs"),
            "hs": (bf, (T, Is), "hs"), "dhs": (bf, (T, Is), "dhs"),
            "routed": (bf, (T, K), "rows"), "dx_router": (bf, (T, K), "rows"),
            "d_logits16": (bf, (T, self.Ep), "d_logits16"), "wr_rows": (bf, (self.Ep if self.Ep != E else 0, K), "wr_rows"),
        }, None
        for dtype, shape, buffer in self._views.values():
            self.scratch.reserve(buffer, dtype.itemsize * math.prod(shape))

    def _bind(self):
        """Attributes for the scratch, again where another layer has made it grow."""
        if self._bound != self.scratch.version:
            for name, (dtype, shape, buffer) in self._views.items():
                setattr(self, name, self.scratch.view(buffer, dtype, *shape))
            self._bound = self.scratch.version

    def _check_weights(self):
        E, K, I, Is, dev = self.E, self.K, self.I, self.Is, self.wr.device
        for what, shape in (("wr", (E, K)), ("w1", (E, 2 * I, K)), ("w2", (E, K, I)), ("ws1", (2 * Is, K)), ("bs1", (2 * Is,)),
                            ("ws2", (K, Is)), ("bs2", (K,))):
            _check(getattr(self, what), what, torch.bfloat16, dev, shape)
        if dev.type != "cuda":
            raise MoeError(-1, f"wr: need weights on a CUDA device, got {dev}")

    def _ctx(self):
        self._bind()
        return Ctx(workspace=self.workspace, dev_status=self.status)

    def forward(self, x, y):
        """x [T, K] bf16 -> y [T, K] bf16.  x is needed again by ``backward``."""
        dev, bf = self.wr.device, torch.bfloat16
        self._check_weights()
        _check(x, "x", bf, dev, (x.shape[0] if isinstance(x, torch.Tensor) and x.dim() else 0, self.K))
        if x.shape[0] > self.max_rows:
            raise MoeError(-3, f"x: {x.shape[0]} rows, the layer was made for up to {self.max_rows}")
        _check(y, "y", bf, dev, numel=x.numel())
        _apart(x, y, "x and y")
        T, k, E, K, I, Is, c = x.shape[0], self.k, self.E, self.K, self.I, self.Is, self._ctx()
        self.T, self.x = T, x
        if T == 0:
            return y
        moe_dense_gemm(x, self.wr, "nk", None, None, 1.0, T, E, K, "none", self.logits, c)
        cap, _ = moe_align_capacity(T * k, E, BLOCK_M)
        moe_align(self.logits, self.ids, self.w, T, k, E, BLOCK_M, self.sorted, cap, self.expert_ids, self.ntpp, None, c)
        args = (T, k, self.sorted, self.expert_ids, self.ntpp, BLOCK_M, cap)
        moe_grouped_gemm("bf16", E, 2 * I, K, x, None, 0, self.w1, None, None, *args, self.gu, c)
        moe_act_checkpoint(self.gu, self.w, T * k, I, "swiglu", self.h, self.codes, self.scales, c)
        moe_grouped_gemm("bf16", E, K, I, self.h, None, 1, self.w2, None, None, *args, self.o, c)
        moe_pair_sum(self.o, None, T, k, K, self.routed, c)
        moe_dense_gemm(x, self.ws1, "nk", self.bs1, None, 1.0, T, 2 * Is, K, "none", self.gs, c)
        moe_act_checkpoint(self.gs, None, T, Is, "swiglu", self.hs, self.codes_s, self.scales_s, c)
        moe_dense_gemm(self.hs, self.ws2, "nk", self.bs2, self.routed, 1.0, T, K, Is, "none", y, c)
        return y

    def backward(self, dy, dx, token_mask=None):
        """dy [T, K] bf16, the gradient of y -> dx [T, K] bf16, the weights' gradients in
        ``grads`` (fp32; "w2t" is [E, I, K]), the losses in ``loss`` (total, balance, z) and the
        experts' counts in ``counts``.

        token_mask [T] bytes: 0 for padding rows.  They count for nothing in the losses, and their
        routing weights are constants: d_logits is zero there, whatever dy is.  So dy has to be zero
        in padding rows, as it is where nothing reads y's; otherwise the terms that run through
        those tokens' routing weights are missing from dx and the router's gradient, while the
        experts' gradients have the tokens' terms."""
        if self.x is None:
            raise MoeError(-1, "backward needs a forward before it")
        x, dev, bf = self.x, self.wr.device, torch.bfloat16
        self._check_weights()
        for t, what in ((dy, "dy"), (dx, "dx")):
            _check(t, what, bf, dev, numel=x.numel())
        for t, what in ((dy, "dy and dx"), (x, "x and dx")):
            _apart(t, dx, what)
        if token_mask is not None:
            _check(token_mask, "token_mask", torch.uint8, dev, numel=x.shape[0])
        T, k, E, K, I, Is, c, g = self.T, self.k, self.E, self.K, self.I, self.Is, self._ctx(), self.grads
        if T == 0:
            for t in (*g.values(), self.loss, self.counts, self.prob_mean):
                t.zero_()
            return dx
        cap, _ = moe_align_capacity(T * k, E, BLOCK_M)
        args = (T, k, self.sorted, self.expert_ids, self.ntpp, BLOCK_M, cap)
        # routed experts: dh, then the activation from its checkpoint (h is w h again)
        w2t = self.wt[:E * I * K].view(E, I, K).copy_(self.w2.transpose(1, 2))
        moe_grouped_gemm("bf16", E, I, K, dy, None, 0, w2t, None, None, *args, self.dh, c)
        moe_act_backward(self.codes, self.scales, self.dh, self.w, T * k, I, "swiglu", self.dgu, self.h, self.dw, c)
        moe_wgrad(self.h, dy, 0, T, k, E, I, K, *args[2:], g["w2t"], 0, c)
        moe_wgrad(self.dgu, x, 0, T, k, E, 2 * I, K, *args[2:], g["w1"], 0, c)
        w1t = self.wt.view(E, K, 2 * I).copy_(self.w1.transpose(1, 2))
        moe_grouped_gemm("bf16", E, K, 2 * I, self.dgu, None, 1, w1t, None, None, *args, self.dx_pairs, c)
        # router: the routing weights' gradient joins the auxiliary losses'
        moe_router_loss(self.logits, self.ids, self.w, self.dw, token_mask, T, k, E, *self.coef, self.counts,
                        self.prob_mean, self.loss, self.d_logits, c)
        self.d_logits16[:T, :E].copy_(self.d_logits[:T])
        wr = self.wr
        if self.Ep != E:
            self.d_logits16[:T, E:].zero_()
            wr = self.wr_rows
            wr[:E].copy_(self.wr)
            wr[E:].zero_()
        moe_dense_gemm(self.d_logits16, wr, "kn", None, None, 1.0, T, K, self.Ep, "none", self.dx_router, c)
        moe_pair_sum(self.dx_pairs, self.dx_router, T, k, K, dx, c)
        # shared expert
        cap1, _ = moe_align_capacity(T, 1, BLOCK_M)
        moe_align(None, self.zeros, None, T, 1, 1, BLOCK_M, self.sorted1, cap1, self.expert_ids1, self.ntpp1, None, c)
        one = (self.sorted1, self.expert_ids1, self.ntpp1, BLOCK_M, cap1)
        moe_dense_gemm(dy, self.ws2, "kn", None, None, 1.0, T, Is, K, "none", self.dhs, c)
        moe_act_backward(self.codes_s, self.scales_s, self.dhs, None, T, Is, "swiglu", self.dgs, self.hs, None, c)
        moe_wgrad(dy, self.hs, 0, T, 1, 1, K, Is, *one, g["ws2"], 0, c)
        moe_wgrad(self.dgs, x, 0, T, 1, 1, 2 * Is, K, *one, g["ws1"], 0, c)
        moe_dense_bias_grad(dy, T, K, g["bs2"], c)
        moe_dense_bias_grad(self.dgs, T, 2 * Is, g["bs1"], c)
        moe_wgrad(self.d_logits16, x, 0, T, 1, 1, self.Ep, K, *one, self.grad_wr, 0, c)
        moe_dense_gemm(self.dgs, self.ws1, "kn", None, dx, 1.0, T, K, 2 * Is, "none", dx, c)
        return dx
