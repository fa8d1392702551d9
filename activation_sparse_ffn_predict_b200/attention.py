"""Tree attention over a paged key/value cache, and eviction from it: tensor-level
binding of asf_kv_append, asf_tree_attention, asf_tree_attention_scored and
asf_kv_evict (include/asffn.h, "Tree attention" and "Eviction")."""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _lib as L
from .api import Workspace, _invoke, _ptr

_I32, _F16, _F32 = torch.int32, torch.float16, torch.float32


class KVCache:
    """A layer's keys and values, fp16 [pages, page, heads, head_dim] each; strides are
    multiples of 8 elements and at least head_dim, the last dimension is contiguous."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        for name, x in (("k", k), ("v", v)):
            if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dtype != torch.float16 or x.dim() != 4:
                raise ValueError(f"{name} must be a float16 CUDA tensor [pages, page, heads, head_dim]")
            if x.numel() == 0 or x.stride(3) != 1:
                raise ValueError(f"{name} must not be empty, and its last dimension contiguous")
        if k.shape != v.shape or k.stride() != v.stride() or k.device != v.device:
            raise ValueError("k and v must have one shape, layout and device")
        self.k, self.v, self.device, self.index = k, v, k.device, k.device.index
        self.pages, self.page, self.heads, self.head_dim = (int(n) for n in k.shape)
        self.desc = L.asf_kv_cache(self.pages, self.page, self.heads, self.head_dim, k.data_ptr(), v.data_ptr(),
                                   # the stride of a dimension of one is never used, and torch's can be anything
                                   *(int(k.stride(i)) if k.shape[i] > 1 else self.head_dim for i in range(3)))
        self._ref = ctypes.byref(self.desc)

    def workspace_bytes(self, q_heads: int, requests: int, tokens: int, scored_pages: Optional[int] = None) -> int:
        if scored_pages is not None:
            return int(L.load().asf_attention_scored_workspace_bytes(self._ref, int(q_heads), int(requests), int(tokens),
                                                                     int(scored_pages)))
        return int(L.load().asf_attention_workspace_bytes(self._ref, int(q_heads), int(requests), int(tokens)))


def _requests(cache: KVCache, table, lens, begin):
    on, of, n, b = cache.index, table.shape, lens.shape, begin.shape    # each shape read once: a tenth of a microsecond
    if len(of) != 2 or len(n) != 1 or n[0] != of[0]:
        raise ValueError("table must be [R, max_pages] and lens [R]")
    R, max_pages = of
    if len(b) != 1 or b[0] != R + 1:
        raise ValueError("begin must be [R + 1]")
    return _ptr(table, "table", on, _I32), max_pages, R, _ptr(lens, "lens", on, _I32), _ptr(begin, "begin", on, _I32)


def asf_kv_append(cache: KVCache, table: torch.Tensor, lens: torch.Tensor, begin: torch.Tensor, k: torch.Tensor,
                  v: torch.Tensor, ws: Workspace, stream=None) -> None:
    """Write the tokens' k and v [T, heads, head_dim] at positions lens[r] + i of their requests.

    k and v may be rows of the cache only where the call does not write: copy them where it may."""
    of = k.shape
    if len(of) != 3 or of[1] != cache.heads or of[2] != cache.head_dim or v.shape != of:
        raise ValueError("k and v must be [T, heads, head_dim]")
    dev = cache.device
    req = _requests(cache, table, lens, begin)
    kp, vp = _ptr(k, "k", dev.index, _F16), _ptr(v, "v", dev.index, _F16)
    _invoke("asf_kv_append", dev, stream, cache._ref, *req, of[0], kp, vp, ws.on(dev), ws.nbytes)


def _attend(cache: KVCache, table, lens, begin, q, anc, o, ws, scale):
    of = q.shape
    if len(of) != 3 or of[2] != cache.head_dim or o.shape != of:
        raise ValueError("q and o must be [T, q_heads, head_dim]")
    n = anc.shape
    if len(n) != 1 or n[0] != of[0]:
        raise ValueError("anc must be [T]")
    on = cache.index
    req = _requests(cache, table, lens, begin)
    qp, op = _ptr(q, "q", on, _F16), _ptr(o, "o", on, _F16)
    ap = _ptr(anc, "anc", on, _I32)
    return (cache._ref, *req, of[0], of[1], qp, ap, cache.head_dim ** -0.5 if scale is None else scale, op)


def asf_tree_attention(cache: KVCache, table: torch.Tensor, lens: torch.Tensor, begin: torch.Tensor, q: torch.Tensor,
                       anc: torch.Tensor, o: torch.Tensor, ws: Workspace, scale: Optional[float] = None,
                       stream=None) -> None:
    """o [T, q_heads, head_dim] = attention of the call's tokens over their requests' keys.

    table int32 [R, max_pages], lens int32 [R], begin int32 [R + 1]; anc int32 [T]: which of the call's
    tokens each token sees, beside every key before lens.  scale: head_dim ** -0.5 unless given."""
    args = _attend(cache, table, lens, begin, q, anc, o, ws, scale)
    _invoke("asf_tree_attention", cache.device, stream, *args, ws.on(cache.device), ws.nbytes)


def asf_tree_attention_scored(cache: KVCache, table: torch.Tensor, lens: torch.Tensor, begin: torch.Tensor,
                              q: torch.Tensor, anc: torch.Tensor, o: torch.Tensor, scores: torch.Tensor, ws: Workspace,
                              scale: Optional[float] = None, stream=None) -> None:
    """asf_tree_attention that adds to scores fp32 [R, heads, S] the weight that each cached key received.

    Every token of the call counts: those of a verified tree go through it by themselves, drafts through
    asf_tree_attention.  S covers the positions seen; the call's own tokens' positions are set instead.  ws:
    Workspace.for_attention(..., scored_pages=the table's width)."""
    args = _attend(cache, table, lens, begin, q, anc, o, ws, scale)
    of = scores.shape
    if len(of) != 3 or of[0] != lens.shape[0] or of[1] != cache.heads:
        raise ValueError("scores must be [R, heads, S]")
    sp = _ptr(scores, "scores", cache.index, _F32)
    _invoke("asf_tree_attention_scored", cache.device, stream, *args, sp, of[2], ws.on(cache.device), ws.nbytes)


def asf_kv_evict(cache: KVCache, table: torch.Tensor, lens: torch.Tensor, scores: torch.Tensor, keep: int,
                 table_out: torch.Tensor, lens_out: torch.Tensor, scores_out: torch.Tensor, kept: torch.Tensor,
                 ws: Workspace, first: int = 0, recent: int = 0, stream=None) -> None:
    """Each request's kv heads keep `keep` keys each, on the pages of table_out [R, max_pages]: the first `first`,
    the last `recent` and those with the largest scores fp32 [R, heads, S], in their order.

    lens_out int32 [R], kept int32 [R, heads, keep] (the old positions) and scores_out fp32 [R, heads,
    >= keep] are written as far as keys are kept."""
    on, of, n, old, new = cache.index, scores.shape, lens.shape, table.shape, table_out.shape
    R = n[0] if len(n) == 1 else -1
    if len(old) != 2 or len(new) != 2 or old[0] != R or new[0] != R:
        raise ValueError("table and table_out must be [R, max_pages], lens [R]")
    if len(of) != 3 or of[0] != R or of[1] != cache.heads:
        raise ValueError("scores must be [R, heads, S]")
    to, sel = scores_out.shape, kept.shape
    if lens_out.shape != n or len(sel) != 3 or sel[0] != R or sel[1] != cache.heads or sel[2] != keep:
        raise ValueError("lens_out must be [R] and kept [R, heads, keep]")
    if len(to) != 3 or to[0] != R or to[1] != cache.heads:
        raise ValueError("scores_out must be [R, heads, S_out]")
    _invoke("asf_kv_evict", cache.device, stream, cache._ref, _ptr(table, "table", on, _I32), old[1], R,
            _ptr(lens, "lens", on, _I32), _ptr(scores, "scores", on, _F32), of[2], int(keep), int(first), int(recent),
            _ptr(table_out, "table_out", on, _I32), new[1], _ptr(lens_out, "lens_out", on, _I32),
            _ptr(scores_out, "scores_out", on, _F32), to[2], _ptr(kept, "kept", on, _I32), ws.on(cache.device), ws.nbytes)
