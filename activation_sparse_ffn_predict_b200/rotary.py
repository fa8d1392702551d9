"""Rotary positions: tensor-level binding of the asf_rotary_* calls
(include/asffn.h, "Rotary positions")."""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from . import _lib as L
from .api import _DT, Workspace, _invoke, _ptr, check
from .attention import _F16, _I32, KVCache, _requests

_LAYOUT = {"half": L.ASF_ROTARY_HALF, "pairs": L.ASF_ROTARY_PAIRS}
_SCALING = {"none": L.ASF_ROTARY_PLAIN, "linear": L.ASF_ROTARY_LINEAR, "ntk": L.ASF_ROTARY_NTK, "yarn": L.ASF_ROTARY_YARN}


class Rotary:
    """How heads of head_dim columns turn: the first rot_dim of them (all by default), paired
    by "half" (columns j and j + rot_dim / 2) or as neighbouring "pairs".

    The frequencies are those of `base` under `scaling` ("none", "linear", "ntk" or "yarn", for contexts
    `factor` times the `original` one), or the given ones in radians per position, with `scale` for
    their cosines and sines."""

    def __init__(self, head_dim: int, rot_dim: Optional[int] = None, base: float = 10000.0, layout: str = "half",
                 scaling: str = "none", factor: float = 1.0, original: int = 4096,
                 frequencies: Optional[Sequence[float]] = None, scale: Optional[float] = None, device="cuda"):
        if layout not in _LAYOUT or scaling not in _SCALING:
            raise ValueError("layout must be 'half' or 'pairs', scaling 'none', 'linear', 'ntk' or 'yarn'")
        rot_dim = int(head_dim) if rot_dim is None else int(rot_dim)
        if rot_dim < 2 or rot_dim % 2 or rot_dim > head_dim or head_dim > L.ASF_MAX_ROTARY_DIM:
            raise ValueError("rot_dim must be even and at most head_dim, head_dim at most %d" % L.ASF_MAX_ROTARY_DIM)
        n = rot_dim // 2
        freq, mul, turns = (ctypes.c_double * n)(), ctypes.c_float(1.0), (ctypes.c_uint64 * n)()
        if frequencies is None:
            check(L.load().asf_rotary_frequencies(rot_dim, float(base), _SCALING[scaling], float(factor), float(original),
                                                  freq, ctypes.byref(mul)), "asf_rotary_frequencies")
        else:
            if len(frequencies) != n:
                raise ValueError("one frequency per pair")
            freq[:] = [float(f) for f in frequencies]
        check(L.load().asf_rotary_turns(freq, n, turns), "asf_rotary_turns")
        self.head_dim, self.rot_dim, self.layout = int(head_dim), rot_dim, layout
        self.frequencies, self.scale = list(freq), float(mul.value if scale is None else scale)
        signed = [t - (1 << 64) if t >> 63 else t for t in turns]
        self.turns = torch.tensor(signed, dtype=torch.int64, device=device)
        self.device, self.index = self.turns.device, self.turns.device.index
        if self.device.type != "cuda":
            raise ValueError("device must be a CUDA device")
        self.desc = L.asf_rotary(self.head_dim, rot_dim, _LAYOUT[layout], self.scale, self.turns.data_ptr())
        self._ref = ctypes.byref(self.desc)


def _rows(t: torch.Tensor, name: str, index: int, dtype, of):
    """Address of a tensor of the shape `of`, [T, heads, head_dim] with its last dimension contiguous, on CUDA
    device `index`, and its token and head strides (never read for a dimension of one)."""
    if not isinstance(t, torch.Tensor) or t.get_device() != index:
        raise ValueError(f"{name} must be a tensor on cuda:{index}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must have dtype {dtype}, got {t.dtype}")
    token, head, one = t.stride()
    T, heads, D = of
    if one != 1 and D != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return t.data_ptr(), token if T > 1 else heads * D, head if heads > 1 else D


def asf_rotary_apply(rot: Rotary, x: torch.Tensor, pos: torch.Tensor, y: torch.Tensor, stream=None) -> None:
    """y [T, heads, head_dim] = x turned by its tokens' positions pos int32 [T]; y may be x.

    fp16 or fp32; token and head strides are free (slices of a joint projection)."""
    of = x.shape
    if len(of) != 3 or of[2] != rot.head_dim or y.shape != of:
        raise ValueError("x and y must be [T, heads, head_dim]")
    dt = x.dtype
    code = _DT.get(dt)
    if code is None:
        raise ValueError("x must be float16 or float32")
    n = pos.shape
    if len(n) != 1 or n[0] != of[0]:
        raise ValueError("pos must be [T]")
    on = rot.index
    xp, xt, xh = _rows(x, "x", on, dt, of)
    yp, yt, yh = _rows(y, "y", on, dt, of)
    _invoke("asf_rotary_apply", rot.device, stream, rot._ref, xp, code, of[0], of[1], xt, xh,
            _ptr(pos, "pos", on, _I32), yp, yt, yh)


def asf_rotary_append(rot: Rotary, cache: KVCache, table: torch.Tensor, lens: torch.Tensor, begin: torch.Tensor,
                      pos: torch.Tensor, q: torch.Tensor, q_out: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                      ws: Workspace, stream=None) -> None:
    """asf_kv_append of k turned by pos int32 [T], and of v as it is; q_out [T, q_heads, head_dim] = q turned.

    q, k and v may be slices of one joint projection (heads contiguous, tokens apart)."""
    of, kv = q.shape, k.shape
    if len(of) != 3 or of[2] != cache.head_dim or q_out.shape != of:
        raise ValueError("q and q_out must be [T, q_heads, head_dim]")
    if len(kv) != 3 or kv[0] != of[0] or kv[1] != cache.heads or kv[2] != cache.head_dim or v.shape != kv:
        raise ValueError("k and v must be [T, heads, head_dim]")
    n = pos.shape
    if len(n) != 1 or n[0] != of[0]:
        raise ValueError("pos must be [T]")
    dev, on, D = cache.device, cache.index, cache.head_dim
    if rot.index != on:
        raise ValueError(f"the rotary table must be on {dev}")
    req = _requests(cache, table, lens, begin)
    qp, qs, qh = _rows(q, "q", on, _F16, of)
    kp, ks, kh = _rows(k, "k", on, _F16, kv)
    vp, vs, vh = _rows(v, "v", on, _F16, kv)
    if qh != D or kh != D or vh != D:
        raise ValueError("the heads of q, k and v must be contiguous")
    _invoke("asf_rotary_append", dev, stream, rot._ref, cache._ref, *req, of[0], _ptr(pos, "pos", on, _I32), of[1],
            qp, qs, _ptr(q_out, "q_out", on, _F16), kp, ks, vp, vs, ws.on(dev), ws.nbytes)
