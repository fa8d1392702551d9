"""4-bit weights with group scales: tensor-level binding of the asf_w4_* calls
(include/asffn.h, "4-bit weights"; the layout of a row is described there)."""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _lib as L
from .api import _ACT, _DT, Workspace, _arg, _invoke, _ptr


def asf_w4_row_bytes(k: int, group: int) -> int:
    """Bytes of one 4-bit row of k weights."""
    n = int(L.load().asf_w4_row_bytes(int(k), int(group)))
    if n == 0:
        raise ValueError("k must be a positive multiple of 8 up to %d and group 32, 64 or 128" % L.ASF_W4_MAX_K)
    return n


def _bytes_of(data: torch.Tensor, name: str) -> int:
    if not isinstance(data, torch.Tensor) or not data.is_cuda or data.dtype != torch.uint8:
        raise ValueError(f"{name} must be a uint8 CUDA tensor")
    if not data.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return data.data_ptr()


class W4Matrix:
    """4-bit rows [m, k]: data is uint8 [m, >= asf_w4_row_bytes(k, group)]."""

    def __init__(self, data: torch.Tensor, k: int, group: int = 128):
        ptr = _bytes_of(data, "data")
        if data.dim() != 2 or data.shape[0] < 1 or data.shape[1] < asf_w4_row_bytes(k, group) or data.shape[1] % 16:
            raise ValueError("data must be [m, row bytes], row bytes a multiple of 16 that holds a row")
        self.data, self.device = data, data.device
        self.rows, self.k, self.group = int(data.shape[0]), int(k), int(group)
        self.desc = L.asf_w4_matrix(self.rows, self.k, self.group, ptr, int(data.shape[1]))
        self._ref = ctypes.byref(self.desc)

    @classmethod
    def quantize(cls, W: torch.Tensor, group: int = 128, stream=None) -> "W4Matrix":
        """A 4-bit copy of W [m, k] (fp16 or fp32)."""
        if W.dim() != 2:
            raise ValueError("W must be [m, k]")
        mat = cls(torch.empty(W.shape[0], asf_w4_row_bytes(W.shape[1], group), dtype=torch.uint8, device=W.device),
                  W.shape[1], group)
        asf_w4_quantize(W, mat, stream)
        return mat

    def workspace_bytes(self, max_batch: int, lora: Optional["LoraSet"] = None) -> int:
        if lora is not None:
            return int(L.load().asf_w4_lora_workspace_bytes(self._ref, lora._ref, int(max_batch)))
        return int(L.load().asf_w4_workspace_bytes(self._ref, None, int(max_batch)))


class LoraSet:
    """Low-rank adapters of one projection: A [n, rank, k] and B [n, m, rank], fp16 or fp32, scale fp32 [n] (1 without);
    rank a multiple of 8 up to 256: adapters of smaller ranks are padded with zeros."""

    def __init__(self, A: torch.Tensor, B: torch.Tensor, scale: Optional[torch.Tensor] = None):
        if not isinstance(A, torch.Tensor) or not A.is_cuda or A.dtype not in _DT or A.dim() != 3:
            raise ValueError("A must be a float16 or float32 CUDA tensor [n, rank, k]")
        n, rank, k = A.shape
        if B.dim() != 3 or B.shape[0] != n or B.shape[2] != rank or A.numel() == 0 or B.numel() == 0:
            raise ValueError("B must be [n, m, rank]")
        if scale is not None and scale.shape != (n,):
            raise ValueError("scale must be [n]")
        self.A, self.B, self.scale, self.device = A, B, scale, A.device
        self.adapters, self.rank, self.k, self.rows, self.dtype = int(n), int(rank), int(k), int(B.shape[1]), A.dtype
        self.desc = L.asf_lora(self.adapters, self.rank, self.k, self.rows, _DT[A.dtype], _arg(A, "A", A.device),
                               _arg(B, "B", A.device, A.dtype),
                               _arg(scale, "scale", A.device, torch.float32) if scale is not None else None)
        self._ref = ctypes.byref(self.desc)


class W4FFN:
    """One FFN layer of 4-bit rows: data is uint8 [n, m, asf_w4_row_bytes(d, group)] with
    m = 3 (gate | up | down, "reglu") or 2 (up | down, "relu"); bias fp32 [n]."""

    def __init__(self, act: str, data: torch.Tensor, bias: torch.Tensor, d: int, group: int = 128):
        if act not in _ACT:
            raise ValueError("act must be 'reglu' or 'relu'")
        ptr = _bytes_of(data, "data")
        mats = 3 if act == "reglu" else 2
        if data.dim() != 3 or data.shape[0] < 1 or data.shape[1] != mats or data.shape[2] != asf_w4_row_bytes(d, group):
            raise ValueError("data must be [n, %d, asf_w4_row_bytes(d, group)]" % mats)
        if bias.shape != (data.shape[0],):
            raise ValueError("bias must be [n]")
        self.act, self.d, self.n, self.group = act, int(d), int(data.shape[0]), int(group)
        self.device = data.device
        self.data, self.bias = data, bias
        self.tensors = (data, bias)
        self.desc = L.asf_w4_ffn(self.d, self.n, self.group, _ACT[act], ptr, mats * int(data.shape[2]),
                                 _arg(bias, "bias", self.device, torch.float32))
        self._ref = ctypes.byref(self.desc)

    @classmethod
    def quantize(cls, act: str, Wg: Optional[torch.Tensor], Wu: torch.Tensor, WdT: torch.Tensor, bias: torch.Tensor,
                 group: int = 128, stream=None) -> "W4FFN":
        """A 4-bit copy of a layer's rows (each [n, d], fp16 or fp32)."""
        if act not in _ACT:
            raise ValueError("act must be 'reglu' or 'relu'")
        mats = [Wg, Wu, WdT] if act == "reglu" else [Wu, WdT]
        if any(W is None or W.dim() != 2 or W.shape != Wu.shape for W in mats):
            raise ValueError("the layer's matrices must all be [n, d]")
        n, d = Wu.shape
        rb = asf_w4_row_bytes(d, group)
        data = torch.empty(n, len(mats), rb, dtype=torch.uint8, device=Wu.device)
        for i, W in enumerate(mats):
            _quantize(W, L.asf_w4_matrix(n, d, int(group), data.data_ptr() + i * rb, len(mats) * rb), data.device, stream)
        return cls(act, data, bias, d, group)

    def workspace_bytes(self, max_batch: int) -> int:
        return int(L.load().asf_w4_workspace_bytes(None, self._ref, int(max_batch)))


def _quantize(src: torch.Tensor, desc, device, stream) -> None:
    if src.dtype not in _DT:
        raise ValueError("weights must be float16 or float32")
    sp = _arg(src, "src", device)
    _invoke("asf_w4_quantize", device, stream, sp, _DT[src.dtype], ctypes.byref(desc))


def asf_w4_quantize(src: torch.Tensor, mat: W4Matrix, stream=None) -> None:
    """mat's rows = src [m, k] (fp16 or fp32) in 4 bits."""
    if src.shape != (mat.rows, mat.k):
        raise ValueError("src must be [rows, k] of the matrix")
    _quantize(src, mat.desc, mat.device, stream)


def asf_w4_dequantize(mat: W4Matrix, dst: torch.Tensor, stream=None) -> None:
    """dst [m, k] (fp16 or fp32) = the weights that mat's rows stand for."""
    if dst.shape != (mat.rows, mat.k) or dst.dtype not in _DT:
        raise ValueError("dst must be [rows, k], float16 or float32")
    dp = _arg(dst, "dst", mat.device)
    _invoke("asf_w4_dequantize", mat.device, stream, mat._ref, dp, _DT[dst.dtype])


def _product(mat: W4Matrix, x, y, bias, relu):
    xd, yd, of, to = x.dtype, y.dtype, x.shape, y.shape
    xt, yt = _DT.get(xd), _DT.get(yd)
    if xt is None or len(of) != 2 or of[1] != mat.k:
        raise ValueError("x must be [B, k], float16 or float32")
    B = of[0]
    if yt is None or len(to) != 2 or to[0] != B or to[1] != mat.rows:
        raise ValueError("y must be [B, rows], float16 or float32")
    on, bp = mat.device.index, None
    if bias is not None:
        if bias.shape != (mat.rows,):
            raise ValueError("bias must be [rows]")
        bp = _ptr(bias, "bias", on, torch.float32)
    return _ptr(x, "x", on, xd), xt, B, bp, int(bool(relu)), _ptr(y, "y", on, yd), yt


def asf_w4_matmul(mat: W4Matrix, x: torch.Tensor, y: torch.Tensor, ws: Workspace,
                  bias: Optional[torch.Tensor] = None, relu: bool = False, stream=None) -> None:
    """y [B, m] = x [B, k] times the 4-bit rows (+ bias [m], then ReLU); x and y fp16 or fp32."""
    _invoke("asf_w4_matmul", mat.device, stream, mat._ref, *_product(mat, x, y, bias, relu), ws.on(mat.device), ws.nbytes)


def asf_w4_matmul_lora(mat: W4Matrix, lora: LoraSet, which: torch.Tensor, x: torch.Tensor, y: torch.Tensor, ws: Workspace,
                       bias: Optional[torch.Tensor] = None, relu: bool = False, stream=None) -> None:
    """asf_w4_matmul with each token's own adapter beside it: which int32 [B], negative for none; x in the
    adapters' dtype.  ws: Workspace.for_w4(mat, B, lora=lora)."""
    args, n = _product(mat, x, y, bias, relu), which.shape
    if len(n) != 1 or n[0] != args[2]:
        raise ValueError("which must be [B]")
    if lora.device.index != mat.device.index or x.dtype is not lora.dtype:
        raise ValueError(f"the adapters must be on {mat.device} and in x's dtype")
    _invoke("asf_w4_matmul_lora", mat.device, stream, mat._ref, lora._ref, _ptr(which, "which", mat.device.index, torch.int32),
            *args, ws.on(mat.device), ws.nbytes)


def asf_w4_sparse_ffn(ffn: W4FFN, x: torch.Tensor, idx: Optional[torch.Tensor], count: Optional[torch.Tensor],
                      y: torch.Tensor, ws: Workspace, stream=None) -> None:
    """asf_sparse_ffn over 4-bit rows (x fp16 or fp32, y fp32); idx and count both None: all neurons."""
    xt, of = _DT.get(x.dtype), x.shape
    if xt is None or len(of) != 2 or of[1] != ffn.d:
        raise ValueError("x must be [B, d], float16 or float32")
    if y.shape != of:
        raise ValueError("y must be [B, d]")
    dev = ffn.device
    ip = cp = None
    if (idx is None) != (count is None):
        raise ValueError("idx and count come together")
    if idx is not None:
        if idx.numel() < ffn.n or count.numel() < 1:
            raise ValueError("idx must hold n entries and count one")
        ip, cp = _arg(idx, "idx", dev, torch.int32), _arg(count, "count", dev, torch.int32)
    xp, yp = _arg(x, "x", dev), _arg(y, "y", dev, torch.float32)
    _invoke("asf_w4_sparse_ffn", dev, stream, ffn._ref, xp, xt, of[0], ip, cp, yp, ws.on(dev), ws.nbytes)
