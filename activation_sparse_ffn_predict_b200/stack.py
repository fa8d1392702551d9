"""A decode step over a stack of FFN layers: predictor then sparse FFN per layer.

One step takes the B tokens' FFN inputs for every layer (``x[l]``), runs the
predictor and the sparse FFN (one asf_predict_sparse_ffn call) for
l = 0..L-1 in order on one stream, and leaves y[l], idx[l], count[l] on the
device.  The launch sequence is captured
once into a CUDA graph; kernels inside it overlap through programmatic
dependent launch (each waits for its predecessor before reading its inputs).
"""
from __future__ import annotations

from typing import List, Optional, Sequence, Union

import torch

from .api import (FFN, Predictor, Workspace, asf_dense_ffn, asf_predict, asf_predict_sparse_ffn, asf_read_error,
                  asf_sparse_ffn, asf_workspace_bytes)
from .attention import KVCache, asf_kv_append, asf_tree_attention
from .w4 import W4FFN, W4Matrix, asf_w4_matmul, asf_w4_sparse_ffn


class AttentionStage:
    """The attention in front of a stack's FFN layers, for the stack's B tokens.

    Layer l appends k[l], v[l] [B, heads, head_dim] to caches[l], runs the
    tokens' tree attention with q[l] [B, q_heads, head_dim], and leaves the
    layer's FFN input in the stack's x[l]: the attention output itself (then
    q_heads * head_dim is the hidden size), or its product with the 4-bit
    projection out[l] [hidden, q_heads * head_dim].  The caller fills q, k, v
    and, for all layers alike, table [R, max_pages], lens [R], begin [R + 1]
    and anc [B]."""

    def __init__(self, caches: Sequence[KVCache], q_heads: int, requests: int, max_pages: int, batch: int,
                 out: Optional[Sequence[W4Matrix]] = None):
        c0, n = caches[0], len(caches)
        if any((c.heads, c.head_dim, c.page, c.device) != (c0.heads, c0.head_dim, c0.page, c0.device) for c in caches):
            raise ValueError("the layers' caches must have one head layout, page size and device")
        if out is not None and (len(out) != n
                                or any((m.k, m.rows) != (q_heads * c0.head_dim, out[0].rows) for m in out)):
            raise ValueError("one projection of q_heads * head_dim columns per layer, all of one hidden size")
        self.caches, self.out, self.R, self.max_pages = list(caches), out, int(requests), int(max_pages)
        half = lambda *s: torch.zeros(*s, dtype=torch.float16, device=c0.device)  # noqa: E731
        ints = lambda *s: torch.zeros(*s, dtype=torch.int32, device=c0.device)  # noqa: E731
        self.q = half(n, batch, q_heads, c0.head_dim)
        self.k, self.v = half(n, batch, c0.heads, c0.head_dim), half(n, batch, c0.heads, c0.head_dim)
        self.o = half(batch, q_heads, c0.head_dim)
        self.table, self.lens, self.begin, self.anc = ints(requests, max_pages), ints(requests), ints(requests + 1), ints(batch)
        self.ws = Workspace.for_attention(c0, q_heads, requests, batch)
        self.ws_out = _widest_w4(out, batch) if out is not None else None
        self.width = out[0].rows if out is not None else q_heads * c0.head_dim

    def launches(self) -> int:
        """Kernels per layer: append, attention, the merge of split keys unless the table is too
        short for a split, and the projection."""
        c = self.caches[0]
        sms = torch.cuda.get_device_properties(c.device).multi_processor_count
        split = _attention_splits(self.max_pages * c.page, c.heads, c.head_dim, self.q.shape[2] // c.heads, self.R,
                                  self.q.shape[1], sms)
        return 2 + int(split) + int(self.out is not None)

    def enqueue(self, l: int, x: torch.Tensor, stream=None) -> None:
        o = self.o if self.out is not None else x.view(self.o.shape)
        asf_kv_append(self.caches[l], self.table, self.lens, self.begin, self.k[l], self.v[l], self.ws, stream)
        asf_tree_attention(self.caches[l], self.table, self.lens, self.begin, self.q[l], self.anc, o, self.ws,
                           stream=stream)
        if self.out is not None:
            asf_w4_matmul(self.out[l], o.view(x.shape[0], -1), x, self.ws_out, stream=stream)


class LayerStack:
    def __init__(self, preds: Sequence[Optional[Predictor]], ffns: Sequence[Union[FFN, W4FFN]], batch: int,
                 tau: float = 0.5, mode: str = "predict", device=None, combined: bool = True,
                 attention: Optional[AttentionStage] = None):
        """mode: "predict" (predictor + sparse FFN), "sparse" (sparse FFN over
        caller-filled idx/count), or "dense" (all neurons).  combined: in
        predict mode, one asf_predict_sparse_ffn call per layer instead of
        asf_predict followed by asf_sparse_ffn (same results).  FFNs of 4-bit
        rows (all layers or none) take the predicted list from asf_predict.
        attention: what computes x[l] before each layer; without it the caller
        fills x.  Layers share the hidden size; neurons, predictor widths, groups
        and activations may differ (idx is as wide as the widest layer)."""
        if mode not in ("predict", "sparse", "dense"):
            raise ValueError("mode must be predict, sparse or dense")
        self.preds = list(preds)
        self.ffns = list(ffns)
        self.L = len(self.ffns)
        self.B = int(batch)
        self.tau = float(tau)
        self.mode = mode
        self.combined = bool(combined)
        f0 = self.ffns[0]
        dev = device if device is not None else f0.tensors[1].device
        self.w4 = isinstance(f0, W4FFN)
        if any(isinstance(f, W4FFN) != self.w4 for f in self.ffns):
            raise ValueError("4-bit FFNs: all layers or none")
        if self.w4:
            self.combined = False
        predict = mode == "predict"
        p0 = self.preds[0] if (self.preds and predict) else None
        self.d, self.n = f0.d, max(f.n for f in self.ffns)
        if any(f.d != self.d for f in self.ffns):
            raise ValueError("the layers must have one hidden size")
        if predict and (len(self.preds) < self.L or any(
                p is None or p.d != self.d or p.n > f.n or p.dtype != p0.dtype for p, f in zip(self.preds, self.ffns))):
            raise ValueError("a predictor per layer, of its hidden size, no more neurons and one dtype")
        self.dtype = (p0.dtype if p0 is not None else torch.float16) if self.w4 else f0.dtype
        self.attention = attention
        if attention is not None and (attention.width != self.d or attention.q.shape[:2] != (self.L, self.B)
                                      or self.dtype != torch.float16):
            raise ValueError("the attention stage must have the stack's layers and batch and give its fp16 input")
        self.x = torch.zeros(self.L, self.B, self.d, dtype=self.dtype, device=dev)
        self.y = torch.zeros(self.L, self.B, self.d, dtype=torch.float32, device=dev)
        self.idx = torch.zeros(self.L, self.n, dtype=torch.int32, device=dev)
        self.count = torch.zeros(self.L, dtype=torch.int32, device=dev)
        # one workspace for all layers, as large as the layer that needs most asks for
        pairs = [(p if predict else None, None if self.w4 else f)
                 for p, f in zip(self.preds if predict else self.ffns, self.ffns)]
        self.ws = Workspace(*max(pairs, key=lambda pf: asf_workspace_bytes(*pf, self.B)), self.B, device=dev) \
            if predict or not self.w4 else None
        self.ws_w4 = _widest_w4(self.ffns, self.B) if self.w4 else None
        self.graph: Optional[torch.cuda.CUDAGraph] = None

    def launches_per_step(self) -> int:
        """Kernels this library launches per step, following its dispatch.
        Predictor: the layer-1 kernel, the layer-2 ring kernel once per group
        of up to 8 tokens (all groups OR into one union mask), and the
        compaction kernel -- except in the combined call when the one-kernel
        sparse FFN (batches up to 4 whose per-lane accumulators fit) ranks the
        mask itself.  FFN: the one-kernel FFN and its reduction when it holds
        the batch; otherwise, for 5-32 tokens with fp16 weights, the
        tensor-core gate/up kernel once per 16 tokens, the tensor-core down
        projection and the reduction of its splits; else gate/up and down on
        the CUDA cores; gate/up and down for 4-bit rows.  The attention stage
        adds its own."""
        attention = getattr(self, "attention", None)
        before = attention.launches() if attention is not None else 0
        if getattr(self, "w4", False):
            return self.L * (before + 2 + (2 + -(-self.B // 8) if self.mode == "predict" else 0))
        fused = _fused_sparse_ffn(self.d, self.dtype, self.B)
        if fused:
            ffn = 2
        elif self.dtype == torch.float16 and self.B > 4:
            ffn = -(-self.B // 16) + 2
        else:
            ffn = 2
        if self.mode != "predict":
            return self.L * (before + ffn)
        pred = 1 + -(-self.B // 8)
        compact = 0 if (self.combined and fused) else 1
        return self.L * (before + pred + compact + ffn)

    def enqueue(self, stream=None) -> None:
        for l in range(self.L):
            x, y = self.x[l], self.y[l]
            if self.attention is not None:
                self.attention.enqueue(l, x, stream)
            if self.w4:
                cnt = self.count[l:l + 1]
                if self.mode == "predict":
                    asf_predict(self.preds[l], x, self.tau, self.idx[l], cnt, self.ws, stream)
                dense = self.mode == "dense"
                asf_w4_sparse_ffn(self.ffns[l], x, None if dense else self.idx[l], None if dense else cnt, y, self.ws_w4,
                                  stream)
                continue
            if self.mode == "dense":
                asf_dense_ffn(self.ffns[l], x, y, self.ws, stream)
                continue
            cnt = self.count[l:l + 1]
            if self.mode == "predict" and self.combined:
                asf_predict_sparse_ffn(self.preds[l], self.ffns[l], x, self.tau, self.idx[l], cnt, y, self.ws,
                                       stream)
                continue
            if self.mode == "predict":
                asf_predict(self.preds[l], x, self.tau, self.idx[l], cnt, self.ws, stream)
            asf_sparse_ffn(self.ffns[l], x, self.idx[l], cnt, y, self.ws, stream)

    def read_error(self, stream=None) -> int:
        """asf_read_error over all of the stack's workspaces: the first error, or 0."""
        stage = self.attention
        spaces = [self.ws, self.ws_w4] + ([stage.ws, stage.ws_out] if stage is not None else [])
        return next((e for e in [asf_read_error(w, stream) for w in spaces if w is not None] if e), 0)

    def capture(self, warmup: int = 2) -> None:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(warmup):
                self.enqueue()
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph(keep_graph=True)     # keeps the node list readable
        with torch.cuda.graph(g):
            self.enqueue()
        g.instantiate()
        torch.cuda.synchronize()
        self.graph = g

    def kernel_nodes(self) -> Optional[int]:
        """Kernel launches recorded in the captured graph (None if the CUDA
        runtime bindings cannot read it): the measured counterpart of
        launches_per_step()."""
        if self.graph is None:
            return None
        try:
            from cuda.bindings import runtime as rt
            graph = rt.cudaGraph_t(init_value=self.graph.raw_cuda_graph())
            err, _, num = rt.cudaGraphGetNodes(graph, 0)
            if err != rt.cudaError_t.cudaSuccess:
                return None
            err, nodes, num = rt.cudaGraphGetNodes(graph, num)
            if err != rt.cudaError_t.cudaSuccess:
                return None
            kernels = 0
            for nd in nodes[:num]:
                err, kind = rt.cudaGraphNodeGetType(nd)
                if err == rt.cudaError_t.cudaSuccess and kind == rt.cudaGraphNodeType.cudaGraphNodeTypeKernel:
                    kernels += 1
            return kernels
        except Exception:
            return None

    def step(self) -> None:
        if self.graph is None:
            self.enqueue()
        else:
            self.graph.replay()

    def release(self) -> None:
        self.graph = None


def _widest_w4(ops: Sequence[Union[W4FFN, W4Matrix]], batch: int) -> Workspace:
    """A workspace that is enough for each of the operators in turn."""
    return Workspace.for_w4(max(ops, key=lambda op: op.workspace_bytes(batch)), batch)


def _attention_splits(keys: int, heads: int, head_dim: int, grp: int, R: int, T: int, sms: int) -> bool:
    """Whether asf_tree_attention may split a request's keys (and then launches the merge) for a table
    of that many keys: from 512 keys on, or 1024 or 2048 where few units have a cluster of 4 or 8 CTAs each."""
    rows = -(-T // R) * grp
    wm = 1 if rows <= 16 else 2 if rows <= 32 else 8
    units = heads * (T * grp // (16 * wm) + R)
    room = sms * (3 if head_dim <= 64 else 2)
    if wm <= 2 and 256 < keys <= 2048 and units * 8 <= sms:
        return False
    if wm <= 2 and 64 < keys <= 1024 and units * 4 <= room:
        return False
    return keys > 512


def _fused_sparse_ffn(d: int, dtype, B: int) -> bool:
    """Whether the library runs the one-kernel sparse FFN for this shape: up to
    4 tokens, and at most 64 fp32 accumulators per lane (d / (8 warps x 32
    lanes x elements per 16 bytes), rounded up to 1, 2, 4 or 6 chunks, times
    elements per chunk times the token group)."""
    if B > 4:
        return False
    v = 8 if dtype == torch.float16 else 4
    q = -(-(d // v) // 256)
    q = next((c for c in (1, 2, 4, 6) if q <= c), None)
    nb = next(c for c in (1, 2, 4) if B <= c)
    return q is not None and q * v * nb <= 64


def build_layers(weights: List, device, hot_rows: Optional[Sequence[int]] = None,
                 l2_next: bool = False) -> tuple:
    """Predictor and FFN descriptors for a list of ``synthetic.LayerWeights`` on ``device``.

    hot_rows[l] (optional) is the number of leading rows of layer l that the
    offline profile found active for most tokens (the prefetch hint).  With
    l2_next, layer l's sparse FFN prefetches the predictor weights of layer
    l+1 (of layer 0 after the last layer: the next token's first layer) into
    L2; off by default, since the benchmark stack measured faster without it."""
    preds, ffns = [], []
    for l, w in enumerate(weights):
        preds.append(Predictor(w.W1, w.b1, w.W2, w.b2))
        ffns.append(FFN(w.act, w.Wg, w.Wu, w.WdT, w.bias, hot_rows=(hot_rows[l] if hot_rows else 0)))
    if l2_next:
        link_l2_next(preds, ffns)
    return preds, ffns


def link_l2_next(preds: Sequence[Predictor], ffns: Sequence[FFN]) -> None:
    """Point each layer's L2 hint at the next layer's predictor weights (cyclic)."""
    L = len(ffns)
    for l in range(L):
        nxt = preds[(l + 1) % L]
        ffns[l].set_l2_next(nxt.tensors[0], nxt.tensors[2])
