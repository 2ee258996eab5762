"""Convenience wrapper: one MoE layer resident on a CUDA device.

Holds the weights, the alignment buffers and the workspace, and runs one step of the
path -- bucket padding (W4A16 MXFP4 only), routing + alignment, the forward -- through
the C ABI.  Marshalling only: every step runs in the library's kernels.

``prewarm`` captures one CUDA graph of routing + alignment + forward per token bucket (the
bucket values up to the layer's row capacity: 97 of them for 20000 rows), so that a serving
loop never captures or sets up kernels on the hot path; ``step_bucketed`` pads a batch to
its bucket and replays that bucket's graph ("Bound Triton MoE JIT specializations via
token-dim bucketing and warmup", TensorRT-LLM PR 15311, Description: bucketing bounds the
set of specializations and a prewarm builds all of them up front).

``ServeBlock`` is the layer in a residual stream: the norm before it in the operands' own format, the
router, and a dense shared expert with the low-rank adapters of the requests in a batch.
"""
from __future__ import annotations

import torch

from . import (Ctx, MoeError, moe_act_checkpoint, moe_adapter_gemm, moe_adapter_gemm_workspace_size, moe_align,
               moe_align_capacity, moe_bucket, moe_bucket_pad, moe_dense_gemm, moe_forward, moe_forward_workspace_size,
               moe_residual_norm)
from .train import _check

BLOCK_M = 128


class DeviceLayer:
    """Weights (torch uint8 / bf16 device tensors in the C ABI layouts) + buffers for up
    to ``max_rows`` token rows."""

    def __init__(self, quant, E, K, I, k, w1, w1_scale, b1, w2, w2_scale, b2, max_rows,
                 device="cuda", block_m=BLOCK_M, pad=True, activation="swiglu"):
        self.quant, self.E, self.K, self.I, self.k = quant, E, K, I, k
        self.activation = activation
        self.w1, self.w1_scale, self.b1 = w1, w1_scale, b1
        self.w2, self.w2_scale, self.b2 = w2, w2_scale, b2
        self.block_m = block_m
        self.pad = pad and quant == "mxfp4"
        rows = moe_bucket(max_rows) if self.pad and max_rows > 0 else max_rows
        self.max_rows = rows
        self.device = device
        P = rows * k
        self.cap, self.cap_blocks = moe_align_capacity(P, E, block_m)
        dev = device
        self.topk_ids = torch.empty((rows, k), dtype=torch.int32, device=dev)
        self.topk_w = torch.empty((rows, k), dtype=torch.float32, device=dev)
        self.sorted = torch.empty(self.cap, dtype=torch.int32, device=dev)
        self.expert_ids = torch.empty(max(self.cap_blocks, 1), dtype=torch.int32, device=dev)
        self.ntpp = torch.zeros(4, dtype=torch.int32, device=dev)
        self.expert_offsets = torch.empty(E + 1 + (-(E + 1)) % 4, dtype=torch.int32, device=dev)
        self.x_pad = torch.zeros((rows, K), dtype=torch.bfloat16, device=dev)
        self.logits_pad = torch.zeros((rows, E), dtype=torch.float32, device=dev)
        self.ws_bytes = moe_forward_workspace_size(rows, k, K, I, self.cap)
        self.workspace = torch.empty(max(self.ws_bytes, 256), dtype=torch.uint8, device=dev)
        self.status = torch.zeros(4, dtype=torch.int32, device=dev)
        self._ctx_cache = {}
        self.graphs = {}  # bucket rows -> torch.cuda.CUDAGraph (prewarm)
        self._graph_stream = None
        self._y_graph = None

    def ctx(self, stream=None, events=None):
        key = (stream, None if events is None else tuple(id(e) for e in events))
        c = self._ctx_cache.get(key)
        if c is None:
            c = Ctx(stream=stream, workspace=self.workspace, dev_status=self.status, events=events)
            if len(self._ctx_cache) > 64:
                self._ctx_cache.clear()
            self._ctx_cache[key] = c
        return c

    def rows_for(self, T):
        return moe_bucket(T) if (self.pad and T > 0) else T

    def step(self, x, logits, T, y, stream=None, events=None, x_scale=None):
        """x [T, K] bf16 (MXFP8: E4M3 codes with x_scale [T, K/32] E8M0), logits [T, E] fp32
        on the device -> y [T, K] bf16.  ``events`` (4 torch.cuda.Event) are recorded around
        the forward's kernels."""
        ctx = self.ctx(stream)
        if self.pad:
            _, T_rows = moe_bucket_pad(T, self.quant, x, self.x_pad, self.K * 2, logits,
                                       self.logits_pad, self.E, ctx)
            xs, ls = self.x_pad, self.logits_pad
        else:
            T_rows, xs, ls = T, x, logits
        cap, _ = moe_align_capacity(T_rows * self.k, self.E, self.block_m)
        moe_align(ls, self.topk_ids, self.topk_w, T_rows, self.k, self.E, self.block_m,
                  self.sorted, cap, self.expert_ids, self.ntpp, self.expert_offsets, ctx)
        moe_forward(self.quant, self.E, self.K, self.I, self.w1, self.w1_scale, self.b1, self.w2,
                    self.w2_scale, self.b2, xs, x_scale, T_rows, T, self.k, self.topk_w, self.sorted,
                    self.expert_ids, self.ntpp, self.expert_offsets, self.block_m, cap, y,
                    self.ctx(stream, events) if events else ctx, activation=self.activation)
        return T_rows

    # ------------------------------------------------------------------ bucket graphs
    def buckets(self, max_tokens=None):
        """The bucket values up to ``max_tokens`` (default: the row capacity), ascending."""
        hi = self.max_rows if max_tokens is None else min(max_tokens, self.max_rows)
        out, b = [], 1
        while b <= hi:
            out.append(b)
            b = moe_bucket(b + 1)
        return out

    def _bucket_body(self, b, stream):
        """Routing + alignment + forward of ``b`` padded rows from x_pad / logits_pad into
        the graph output buffer (every row of the bucket is computed; callers slice)."""
        ctx = self.ctx(stream)
        cap, _ = moe_align_capacity(b * self.k, self.E, self.block_m)
        moe_align(self.logits_pad, self.topk_ids, self.topk_w, b, self.k, self.E, self.block_m,
                  self.sorted, cap, self.expert_ids, self.ntpp, self.expert_offsets, ctx)
        moe_forward(self.quant, self.E, self.K, self.I, self.w1, self.w1_scale, self.b1, self.w2,
                    self.w2_scale, self.b2, self.x_pad, None, b, b, self.k, self.topk_w, self.sorted,
                    self.expert_ids, self.ntpp, self.expert_offsets, self.block_m, cap, self._y_graph, ctx,
                    activation=self.activation)

    def prewarm(self, max_tokens=None):
        """Captures the graph of every bucket up to ``max_tokens``; returns the bucket list."""
        if not self.pad:
            raise ValueError("bucket graphs need a padded (W4A16 MXFP4) layer")
        if self._graph_stream is None:
            self._graph_stream = torch.cuda.Stream(device=self.device)
            self._y_graph = torch.empty((self.max_rows, self.K), dtype=torch.bfloat16, device=self.device)
        s = self._graph_stream
        s.wait_stream(torch.cuda.current_stream())
        todo = [b for b in self.buckets(max_tokens) if b not in self.graphs]
        with torch.cuda.stream(s):
            for b in todo:  # one eager run of each shape first: launch setup stays out of capture
                self._bucket_body(b, s)
        s.synchronize()
        for b in todo:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                self._bucket_body(b, s)
            self.graphs[b] = g
        torch.cuda.synchronize()
        return self.buckets(max_tokens)

    def step_bucketed(self, x, logits, T):
        """Pads x [T, K] / logits [T, E] to bucket(T) rows and replays that bucket's graph;
        returns y [T, K] (a view of the graph's output buffer, valid until the next call)."""
        b = moe_bucket(T)
        g = self.graphs.get(b)
        if g is None:
            raise KeyError(f"no graph for bucket {b}: call prewarm() first")
        s = self._graph_stream
        s.wait_stream(torch.cuda.current_stream())
        moe_bucket_pad(T, self.quant, x, self.x_pad, self.K * 2, logits, self.logits_pad, self.E,
                       self.ctx(s))
        with torch.cuda.stream(s):
            g.replay()
        torch.cuda.current_stream().wait_stream(s)
        return self._y_graph[:T]


class ServeBlock:
    """A DeviceLayer behind its norm, in a residual stream, with its router and a shared expert:

        s = residual + branch;  n = rmsnorm(s) * norm_w      (an MXFP8 layer reads n in MXFP8)
        y = experts(n, router n) + swiglu(n ws1^T + bs1) ws2^T + bs2

    norm_w [K], wr [E, K], ws1 [2Is, K], bs1 [2Is], ws2 [K, Is], bs2 [K]: bf16; ``shared`` = (ws1, bs1, ws2,
    bs2) or None.  ``adapters``: a pair (for ws1 and for ws2; either may be None) of (a [L, r, in], b [L, out, r]
    bf16, scale [L] fp32 or None): low-rank adapters, of which each request of a batch names one.  Is is a
    multiple of 8, with adapters for ws1 of 32.  The stream is bf16, or fp32 (``stream_f32``).  Up to
    ``max_requests`` requests a batch.

    Weights are checked when the block is made, and a step's operands before anything is launched (MoeError):
    type, size, density, alignment and device, and that what is written lies apart from what is still read."""

    def __init__(self, layer, norm_w, wr, shared=None, adapters=(None, None), eps=1e-5, stream_f32=False, max_requests=512):
        bf, dev = torch.bfloat16, norm_w.device
        self.layer, self.norm_w, self.wr, self.shared, self.adapters, self.eps = layer, norm_w, wr, shared, adapters, eps
        T, K, E = layer.max_rows, layer.K, layer.E
        if tuple(norm_w.shape) != (K,) or tuple(wr.shape) != (E, K):
            raise MoeError(-1, f"need norm_w [{K}] and wr [{E}, {K}], got {tuple(norm_w.shape)} and {tuple(wr.shape)}")
        for what, t in (("norm_w", norm_w), ("wr", wr)):
            _check(t, what, bf, layer.status.device, t.shape)
        if any(adapters) and shared is None:
            raise MoeError(-1, "adapters need a shared expert")
        new = lambda *s, dtype=bf: torch.empty(s, dtype=dtype, device=dev)  # noqa: E731
        self.stream, self.normed = new(T, K, dtype=torch.float32 if stream_f32 else bf), new(T, K)
        self._own = [(t, t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in (self.stream, self.normed)]
        self.logits = new(T, E, dtype=torch.float32)
        mx = layer.quant == "mxfp8"
        self.codes = new(T, K, dtype=torch.uint8) if mx else None
        self.scales = new(T, K // 32, dtype=torch.uint8) if mx else None
        self.max_requests, ranks = max_requests, [0]
        if shared is not None:
            ws1, bs1, ws2, bs2 = shared
            Is = self.Is = ws2.shape[1]
            if tuple(ws1.shape) != (2 * Is, K) or ws2.shape[0] != K:
                raise MoeError(-1, f"need ws1 [{2 * Is}, {K}] and ws2 [{K}, {Is}], got {tuple(ws1.shape)} and {tuple(ws2.shape)}")
            for what, t, n in (("ws1", ws1, 2 * Is * K), ("bs1", bs1, 2 * Is), ("ws2", ws2, K * Is), ("bs2", bs2, K)):
                _check(t, what, bf, dev, numel=n)
            for pair, (n_in, n_out) in zip(adapters, ((K, 2 * Is), (Is, K))):
                if pair is None:
                    continue
                a, b = pair[:2]
                if a.dim() != 3 or a.shape[2] != n_in or tuple(b.shape) != (a.shape[0], n_out, a.shape[1]):
                    raise MoeError(-1, f"adapters: need a [L, r, {n_in}] and b [L, {n_out}, r], got {tuple(a.shape)} and {tuple(b.shape)}")
                _check(a, "adapters' a", bf, dev, a.shape)
                _check(b, "adapters' b", bf, dev, b.shape)
                if len(pair) > 2 and pair[2] is not None:
                    _check(pair[2], "adapters' scale", torch.float32, dev, numel=a.shape[0])
                ranks.append(a.shape[1])
            if adapters[0] is not None and Is % 32:  # refused by moe_act_checkpoint, at the first batch with an adapter
                raise MoeError(-2, f"adapters for ws1 need a shared width that is a multiple of 32, got {Is}")
            self.hs = new(T, Is)
            if adapters[0] is not None:  # added before the activation, so the pre-activations are kept
                self.gs = new(T, 2 * Is)
                self.held = new(T, 2 * Is, dtype=torch.uint8), new(T, 2 * Is // 32, dtype=torch.uint8)
        # the adapters' workspace is no smaller for more requests up to 1024 (beyond, other kernels run), and
        # largest at whole 256s of rows, or at all; requests may be more than rows
        need = max([256] + [moe_adapter_gemm_workspace_size(t, min(1024, max_requests), max(ranks))
                            for t in {T, *range(256, T, 256)} if max(ranks)])
        self.workspace = new(need, dtype=torch.uint8)
        self.status = torch.zeros(4, dtype=torch.int32, device=dev)

    def _adapt(self, which, x, T, n_out, n_in, row_offsets, adapter, out, ctx):
        a, b, scale = (*self.adapters[which], None)[:3]
        moe_adapter_gemm(x, a, b, scale, row_offsets, adapter, out, T, n_out, n_in, a.shape[1], a.shape[0], adapter.shape[0], out,
                         ctx)

    def _check_step(self, branch, residual, T, y, row_offsets, adapter):
        dev, n, bf = self.norm_w.device, T * self.layer.K, torch.bfloat16
        # rows, and whether they may begin where the block's stream or its norm does: the stream may be written over
        # the residual and the norm over the branch
        rows = [(y, "y", bf, None)]
        if branch is not None:
            rows.append((branch, "branch", bf, self.normed))
        if residual is not None:
            rows.append((residual, "residual", self.stream.dtype, self.stream))
        for t, what, dtype, same in rows:
            _check(t, what, dtype, dev, numel=n)
            at, size = t.data_ptr(), n * dtype.itemsize
            for own, start, end in self._own:
                if at < end and start < at + size and not (own is same and at == start):
                    raise MoeError(-1, f"{what} and the block's rows must not overlap")
        if adapter is not None:
            _check(adapter, "adapter", torch.int32, dev, (adapter.shape[0],))
            _check(row_offsets, "row_offsets", torch.int32, dev, numel=adapter.shape[0] + 1)

    def step(self, branch, residual, T, y, row_offsets=None, adapter=None):
        """branch [T, K] bf16 or None, residual [T, K] in the stream's type -> y [T, K] bf16 and the stream
        [T, K] (the block's own, until its next step).  With adapters: row_offsets [R + 1] and adapter [R] int32 on
        the device (-1: none), rows of no request having none."""
        K, E, L = self.layer.K, self.layer.E, self.layer
        if T > L.max_rows:
            raise MoeError(-3, f"{T} rows, the layer was made for up to {L.max_rows}")
        adapt = adapter is not None and adapter.shape[0] > 0
        if adapt and adapter.shape[0] > self.max_requests:
            raise MoeError(-3, f"{adapter.shape[0]} requests, the block was made for up to {self.max_requests}")
        if T > 0:
            self._check_step(branch, residual, T, y, row_offsets, adapter if adapt and any(self.adapters) else None)
        ctx = Ctx(workspace=self.workspace, dev_status=self.status)
        moe_residual_norm(branch, residual, None, self.norm_w, T, K, self.eps, 0.0, None, 0, self.stream, self.normed, self.codes,
                          self.scales, ctx)
        if T == 0:
            return y, self.stream[:0]
        moe_dense_gemm(self.normed, self.wr, "nk", None, None, 1.0, T, E, K, "none", self.logits, ctx)
        L.step(self.normed if self.codes is None else self.codes, self.logits, T, y, stream=torch.cuda.current_stream(),
               x_scale=self.scales)
        if self.shared is not None:
            ws1, bs1, ws2, bs2 = self.shared
            if adapt and self.adapters[0] is not None:
                moe_dense_gemm(self.normed, ws1, "nk", bs1, None, 1.0, T, 2 * self.Is, K, "none", self.gs, ctx)
                self._adapt(0, self.normed, T, 2 * self.Is, K, row_offsets, adapter, self.gs, ctx)
                moe_act_checkpoint(self.gs, None, T, self.Is, "swiglu", self.hs, *self.held, ctx)
            else:
                moe_dense_gemm(self.normed, ws1, "nk", bs1, None, 1.0, T, self.Is, K, "swiglu", self.hs, ctx)
            moe_dense_gemm(self.hs, ws2, "nk", bs2, y, 1.0, T, K, self.Is, "none", y, ctx)
            if adapt and self.adapters[1] is not None:
                self._adapt(1, self.hs, T, K, self.Is, row_offsets, adapter, y, ctx)
        return y, self.stream[:T]
