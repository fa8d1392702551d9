"""4-bit rows without a GPU: the format's description against itself, and the
arguments that the calls refuse before any launch."""
import ctypes

import numpy as np
import pytest

from activation_sparse_ffn_predict_b200 import _lib as L
from activation_sparse_ffn_predict_b200 import build as B
from oracle import w4 as O

FAKE = 1 << 20          # aligned, never dereferenced: every case fails validation first


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("k", [8, 128, 136, 512, 1000, 4096])
def test_row_bytes_and_round_trip(lib, k, group):
    assert lib.asf_w4_row_bytes(k, group) == O.row_bytes(k, group)
    rng = np.random.default_rng(k + group)
    W = rng.standard_normal((3, k)).astype(np.float32)
    W[1, :] = 0
    rows = O.w4_pack(W, group)
    back = O.w4_unpack(rows, k, group)
    c, s = O.w4_codes(W, group)
    scale = np.repeat(s.astype(np.float64), group, axis=1)[:, :k]
    assert np.array_equal(back, (c[:, :k] - 8) * scale)
    # half a step of rounding, and what the fp16 scale's rounding (2^-11 of up to 7 steps) adds at the clamp
    assert np.all(np.abs(back - W) <= scale * (0.5 + 7 * 2.0 ** -11 + 1e-6))
    assert np.all(back[1] == 0)


@pytest.mark.parametrize("k,group", [(0, 32), (-8, 32), (12, 32), (64, 16), (64, 256), (L.ASF_W4_MAX_K + 8, 32)])
def test_row_bytes_refuses(lib, k, group):
    assert lib.asf_w4_row_bytes(k, group) == 0


def test_struct_layout_matches_header():
    assert ctypes.sizeof(L.asf_w4_matrix) == 32 and L.asf_w4_matrix.data.offset == 16
    assert ctypes.sizeof(L.asf_w4_ffn) == 40 and L.asf_w4_ffn.bias.offset == 32


def _mat(rows=64, k=256, group=128, data=FAKE, stride=None):
    return L.asf_w4_matrix(rows, k, group, data, O.row_bytes(k, group) if stride is None else stride)


BAD_MATS = [
    (dict(data=0), L.ASF_ERR_INVALID_ARG), (dict(rows=0), L.ASF_ERR_INVALID_ARG),
    (dict(k=0, stride=16), L.ASF_ERR_INVALID_ARG), (dict(k=252, stride=144), L.ASF_ERR_MISALIGNED),
    (dict(group=16, stride=256), L.ASF_ERR_UNSUPPORTED), (dict(data=FAKE + 8), L.ASF_ERR_MISALIGNED),
    (dict(stride=152), L.ASF_ERR_MISALIGNED), (dict(stride=128), L.ASF_ERR_INVALID_ARG),
    (dict(k=L.ASF_W4_MAX_K + 8, stride=1 << 20), L.ASF_ERR_UNSUPPORTED)]


@pytest.mark.parametrize("kw,status", BAD_MATS)
def test_matrix_descriptors_refused(lib, kw, status):
    m = ctypes.byref(_mat(**kw))
    assert lib.asf_w4_quantize(FAKE, L.ASF_F16, m, None) == status
    assert lib.asf_w4_dequantize(m, FAKE, L.ASF_F16, None) == status
    assert lib.asf_w4_matmul(m, FAKE, L.ASF_F16, 1, None, 0, FAKE, L.ASF_F32, FAKE, 1 << 40, None) == status
    assert lib.asf_w4_workspace_bytes(m, None, 1) == 0


def test_matmul_refuses(lib):
    m = _mat()
    need = lib.asf_w4_workspace_bytes(ctypes.byref(m), None, 4)
    assert need > 4096

    def call(x=FAKE, dt=L.ASF_F16, B=4, bias=None, relu=0, y=FAKE, ydt=L.ASF_F32, ws=FAKE, wsb=need - 1):
        return lib.asf_w4_matmul(ctypes.byref(m), x, dt, B, bias, relu, y, ydt, ws, wsb, None)

    assert call() == L.ASF_ERR_WORKSPACE
    assert call(ws=0, wsb=need) == L.ASF_ERR_WORKSPACE
    assert call(ws=FAKE + 16, wsb=need) == L.ASF_ERR_WORKSPACE
    assert call(x=0) == call(y=0) == call(B=0) == call(B=33) == call(relu=2) == L.ASF_ERR_INVALID_ARG
    assert call(dt=7) == call(ydt=3) == L.ASF_ERR_UNSUPPORTED
    assert call(x=FAKE + 8) == call(y=FAKE + 2) == call(bias=FAKE + 2) == L.ASF_ERR_MISALIGNED
    assert lib.asf_w4_matmul(None, FAKE, 1, 1, None, 0, FAKE, L.ASF_F32, FAKE, 1 << 40, None) == L.ASF_ERR_INVALID_ARG
    assert lib.asf_w4_quantize(0, L.ASF_F16, ctypes.byref(m), None) == L.ASF_ERR_INVALID_ARG
    assert lib.asf_w4_quantize(FAKE + 2, L.ASF_F16, ctypes.byref(m), None) == L.ASF_ERR_MISALIGNED
    assert lib.asf_w4_quantize(FAKE, 9, ctypes.byref(m), None) == L.ASF_ERR_UNSUPPORTED
    assert lib.asf_w4_dequantize(ctypes.byref(m), 0, L.ASF_F16, None) == L.ASF_ERR_INVALID_ARG
    assert lib.asf_w4_dequantize(ctypes.byref(m), FAKE, 9, None) == L.ASF_ERR_UNSUPPORTED


def _ffn(d=256, n=100, group=64, act=L.ASF_ACT_REGLU, data=FAKE, stride=None, bias=FAKE):
    mats = 3 if act == L.ASF_ACT_REGLU else 2
    return L.asf_w4_ffn(d, n, group, act, data, mats * O.row_bytes(d, group) if stride is None else stride, bias)


def test_sparse_ffn_refuses(lib):
    f = _ffn()
    need = lib.asf_w4_workspace_bytes(None, ctypes.byref(f), 32)

    def call(f=f, x=FAKE, dt=L.ASF_F32, B=32, idx=FAKE, cnt=FAKE, y=FAKE, ws=FAKE, wsb=need - 1):
        return lib.asf_w4_sparse_ffn(ctypes.byref(f), x, dt, B, idx, cnt, y, ws, wsb, None)

    assert call() == call(idx=None, cnt=None) == L.ASF_ERR_WORKSPACE
    assert call(idx=None) == call(cnt=None) == call(x=0) == call(y=0) == call(B=0) == call(B=33) == L.ASF_ERR_INVALID_ARG
    assert call(dt=5) == L.ASF_ERR_UNSUPPORTED
    assert call(x=FAKE + 4) == call(idx=FAKE + 1) == call(cnt=FAKE + 2) == L.ASF_ERR_MISALIGNED
    assert call(f=_ffn(act=5)) == call(f=_ffn(group=48, stride=1 << 12)) == L.ASF_ERR_UNSUPPORTED
    assert call(f=_ffn(bias=0)) == call(f=_ffn(data=0)) == call(f=_ffn(n=0)) == L.ASF_ERR_INVALID_ARG
    assert call(f=_ffn(stride=2 * O.row_bytes(256, 64))) == L.ASF_ERR_INVALID_ARG
    assert call(f=_ffn(d=252, stride=1 << 12)) == call(f=_ffn(bias=FAKE + 1)) == L.ASF_ERR_MISALIGNED


def test_workspace_grows_with_the_batch(lib):
    f, m = _ffn(d=4096, n=11008), _mat(rows=1000, k=8192)
    got = [lib.asf_w4_workspace_bytes(ctypes.byref(m), ctypes.byref(f), b) for b in range(1, 33)]
    assert got == sorted(got)
    assert lib.asf_w4_workspace_bytes(None, None, 1) == 0
    assert lib.asf_w4_workspace_bytes(ctypes.byref(m), None, 0) == lib.asf_w4_workspace_bytes(ctypes.byref(m), None, 33) == 0


def test_overlap_and_too_many_rows_are_refused(lib):
    m = ctypes.byref(_mat())
    ws = lib.asf_w4_workspace_bytes(m, None, 1)
    for y in (FAKE, FAKE + 2 * 256 - 4):
        assert lib.asf_w4_matmul(m, FAKE, L.ASF_F16, 1, None, 0, y, L.ASF_F32, FAKE, ws, None) == L.ASF_ERR_INVALID_ARG
    assert lib.asf_w4_workspace_bytes(ctypes.byref(_mat(rows=L.ASF_W4_MAX_ROWS + 1)), None, 1) == 0
    assert lib.asf_w4_matmul(m, FAKE, L.ASF_F16, 1, None, 0, FAKE + 1, L.ASF_F16, FAKE, ws, None) == L.ASF_ERR_MISALIGNED


def test_quantize_and_dequantize_refuse_shared_memory(lib):
    m = _mat()                                              # 64 rows of 256, at FAKE
    end = 64 * O.row_bytes(256, 128)
    for dt, size in ((L.ASF_F16, 2), (L.ASF_F32, 4)):
        for at in (FAKE, FAKE + end - 16, FAKE - 64 * 256 * size + 16):
            assert lib.asf_w4_quantize(at, dt, ctypes.byref(m), None) == L.ASF_ERR_INVALID_ARG
            assert lib.asf_w4_dequantize(ctypes.byref(m), at, dt, None) == L.ASF_ERR_INVALID_ARG
    rows = _mat(stride=512)                                 # 4-bit rows inside the rows that they come from
    assert lib.asf_w4_quantize(FAKE, L.ASF_F16, ctypes.byref(rows), None) == L.ASF_ERR_INVALID_ARG
