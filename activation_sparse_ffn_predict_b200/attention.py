"""Tree attention over a paged key/value cache: tensor-level binding of
asf_kv_append and asf_tree_attention (include/asffn.h, "Tree attention")."""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _lib as L
from .api import Workspace, _arg, _invoke


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
        self.k, self.v, self.device = k, v, k.device
        self.pages, self.page, self.heads, self.head_dim = (int(n) for n in k.shape)
        self.desc = L.asf_kv_cache(self.pages, self.page, self.heads, self.head_dim, k.data_ptr(), v.data_ptr(),
                                   # the stride of a dimension of one is never used, and torch's can be anything
                                   *(int(k.stride(i)) if k.shape[i] > 1 else self.head_dim for i in range(3)))
        self._ref = ctypes.byref(self.desc)

    def workspace_bytes(self, q_heads: int, requests: int, tokens: int) -> int:
        return int(L.load().asf_attention_workspace_bytes(self._ref, int(q_heads), int(requests), int(tokens)))


def _requests(cache: KVCache, table, lens, begin):
    dev, of = cache.device, table.shape
    if len(of) != 2 or lens.shape != of[:1]:
        raise ValueError("table must be [R, max_pages] and lens [R]")
    R, max_pages = of
    if begin.shape != (R + 1,):
        raise ValueError("begin must be [R + 1]")
    return (_arg(table, "table", dev, torch.int32), max_pages, R, _arg(lens, "lens", dev, torch.int32),
            _arg(begin, "begin", dev, torch.int32))


def asf_kv_append(cache: KVCache, table: torch.Tensor, lens: torch.Tensor, begin: torch.Tensor, k: torch.Tensor,
                  v: torch.Tensor, ws: Workspace, stream=None) -> None:
    """Write the tokens' k and v [T, heads, head_dim] at positions lens[r] + i of their requests.

    k and v may be rows of the cache only where the call does not write: copy them where it may."""
    of = k.shape
    if len(of) != 3 or of[1] != cache.heads or of[2] != cache.head_dim or v.shape != of:
        raise ValueError("k and v must be [T, heads, head_dim]")
    dev = cache.device
    req = _requests(cache, table, lens, begin)
    kp, vp = _arg(k, "k", dev, torch.float16), _arg(v, "v", dev, torch.float16)
    _invoke("asf_kv_append", dev, stream, cache._ref, *req, of[0], kp, vp, ws.on(dev), ws.nbytes)


def asf_tree_attention(cache: KVCache, table: torch.Tensor, lens: torch.Tensor, begin: torch.Tensor, q: torch.Tensor,
                       anc: torch.Tensor, o: torch.Tensor, ws: Workspace, scale: Optional[float] = None,
                       stream=None) -> None:
    """o [T, q_heads, head_dim] = attention of the call's tokens over their requests' keys.

    table int32 [R, max_pages], lens int32 [R], begin int32 [R + 1]; anc int32 [T]: which of the call's
    tokens each token sees, beside every key before lens.  scale: head_dim ** -0.5 unless given."""
    of = q.shape
    if len(of) != 3 or of[2] != cache.head_dim or o.shape != of:
        raise ValueError("q and o must be [T, q_heads, head_dim]")
    if anc.shape != of[:1]:
        raise ValueError("anc must be [T]")
    dev = cache.device
    req = _requests(cache, table, lens, begin)
    qp, op = _arg(q, "q", dev, torch.float16), _arg(o, "o", dev, torch.float16)
    ap = _arg(anc, "anc", dev, torch.int32)
    if scale is None:
        scale = cache.head_dim ** -0.5
    _invoke("asf_tree_attention", dev, stream, cache._ref, *req, of[0], of[1], qp, ap, scale, op, ws.on(dev),
            ws.nbytes)
