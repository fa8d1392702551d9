"""4-bit rows with group scales in numpy: the format byte by byte, and the
float64 products over it (include/asffn.h, "4-bit weights")."""
from __future__ import annotations

import numpy as np


def padded(k: int) -> int:
    return -(-k // 128) * 128


def row_bytes(k: int, group: int) -> int:
    scales = -(-padded(k) // 512) * (512 // group) * 2
    return padded(k) // 2 + -(-scales // 16) * 16


def w4_codes(W, group: int):
    """(codes 0..15 [m, kp], scales fp16 [m, kp/group]) by the definition, in binary32."""
    W = np.asarray(W, dtype=np.float32)
    m, k = W.shape
    w = np.zeros((m, padded(k)), np.float32)
    w[:, :k] = W
    w = w.reshape(m, -1, group)
    with np.errstate(all="ignore"):
        top = np.max(np.where(np.isnan(w), np.float32(np.inf), np.abs(w)), axis=2)
        s = (top / np.float32(7)).astype(np.float16)
        bad = ~np.isfinite(s)
        sf = s.astype(np.float32)[..., None]
        c = np.where((sf > 0) & ~bad[..., None], np.rint(w / sf), np.float32(0))
    c = np.clip(np.nan_to_num(c), -8, 7).astype(np.int64) + 8
    s[bad] = np.nan
    return c.reshape(m, -1), s


def w4_pack(W, group: int) -> np.ndarray:
    """uint8 [m, row_bytes]: every byte of the rows."""
    c, s = w4_codes(W, group)
    m, kp = c.shape
    out = np.zeros((m, row_bytes(np.asarray(W).shape[1], group)), np.uint8)
    for i in range(kp):
        j, t, e = i % 128 // 32, i % 32 // 8, i % 8
        bit = 16 * (e % 2) + 4 * (e // 2)
        out[:, i // 128 * 64 + (4 * t + j) * 4 + bit // 8] |= (c[:, i] << (bit % 8)).astype(np.uint8)
    out[:, kp // 2:kp // 2 + 2 * s.shape[1]] = s.view(np.uint8).reshape(m, -1)
    return out


def w4_unpack(rows, k: int, group: int) -> np.ndarray:
    """float64 [..., k] of uint8 rows [..., row_bytes]."""
    rows = np.asarray(rows)
    i = np.arange(k)
    j, t, e = i % 128 // 32, i % 32 // 8, i % 8
    bit = 16 * (e % 2) + 4 * (e // 2)
    c = (rows[..., i // 128 * 64 + (4 * t + j) * 4 + bit // 8] >> (bit % 8).astype(np.uint8)) & 15
    kp = padded(k)
    s = np.ascontiguousarray(rows[..., kp // 2:kp // 2 + 2 * (kp // group)]).view(np.float16).astype(np.float64)
    return (c.astype(np.float64) - 8) * s[..., i // group]


def w4_ffn(act: str, data, bias, d: int, group: int, x, idx) -> np.ndarray:
    """Sparse FFN over the listed neurons; data uint8 [n, mats, row_bytes]."""
    idx = np.asarray(idx, dtype=np.int64)
    x = np.asarray(x, np.float64)
    if idx.size == 0:
        return np.zeros((x.shape[0], d))
    w = w4_unpack(np.asarray(data)[idx], d, group)
    a = np.maximum(x @ w[:, 0].T + np.asarray(bias, np.float64)[idx], 0)
    if act == "reglu":
        a = a * (x @ w[:, 1].T)
    return a @ w[:, -1]
