"""Arguments of the 4-bit product with adapters that are refused before any launch (no GPU)."""
import ctypes

import pytest

from activation_sparse_ffn_predict_b200 import _lib as L
from activation_sparse_ffn_predict_b200 import build as B

FAKE = 1 << 20          # aligned, never dereferenced: every case fails validation first


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


def _mat(m=64, k=256, group=128, data=FAKE, stride=None):
    return L.asf_w4_matrix(m, k, group, data, stride if stride is not None else 144)


def _lora(n=3, r=16, k=256, m=64, dt=1, a=FAKE, b=FAKE, s=FAKE):
    return L.asf_lora(n, r, k, m, dt, a, b, s)


def test_struct_layout_matches_header():
    assert ctypes.sizeof(L.asf_lora) == 48 and L.asf_lora.A.offset == 24


def test_workspace(lib):
    mat, lora = ctypes.byref(_mat()), ctypes.byref(_lora())
    sizes = [lib.asf_w4_lora_workspace_bytes(mat, lora, b) for b in range(1, 33)]
    assert sizes == sorted(sizes) and sizes[0] > lib.asf_w4_workspace_bytes(mat, None, 1)
    for b in (0, 33):
        assert lib.asf_w4_lora_workspace_bytes(mat, lora, b) == 0
    for bad in (_lora(k=264), _lora(m=63), _lora(r=12), _lora(r=0), _lora(n=0), _lora(a=0), _lora(b=0), _lora(dt=2),
                _lora(r=L.ASF_MAX_LORA_RANK + 8)):
        assert lib.asf_w4_lora_workspace_bytes(mat, ctypes.byref(bad), 4) == 0
    assert lib.asf_w4_lora_workspace_bytes(ctypes.byref(_mat(group=48)), lora, 4) == 0
    assert lib.asf_w4_lora_workspace_bytes(None, lora, 4) == lib.asf_w4_lora_workspace_bytes(mat, None, 4) == 0


def test_arguments_refused(lib):
    need = lib.asf_w4_lora_workspace_bytes(ctypes.byref(_mat()), ctypes.byref(_lora()), 4)

    def mul(mat=None, lora=None, which=FAKE, x=2 * FAKE, dt=1, n=4, bias=FAKE, relu=0, y=4 * FAKE, yt=0, ws=8 * FAKE, wsb=need - 1):
        return lib.asf_w4_matmul_lora(ctypes.byref(mat or _mat()), ctypes.byref(lora or _lora()), which, x, dt, n, bias, relu, y, yt,
                                      ws, wsb, None)

    assert mul() == mul(ws=0, wsb=1 << 40) == mul(ws=8 * FAKE + 64, wsb=1 << 40) == L.ASF_ERR_WORKSPACE
    for kw in (dict(which=0), dict(x=0), dict(y=0), dict(n=0), dict(n=33), dict(relu=2), dict(lora=_lora(k=264)), dict(lora=_lora(m=65)),
               dict(lora=_lora(n=0)), dict(lora=_lora(r=0)), dict(lora=_lora(a=0)), dict(lora=_lora(b=0)), dict(lora=_lora(n=-1)),
               dict(y=2 * FAKE + 16, wsb=1 << 40), dict(mat=_mat(data=0), wsb=1 << 40), dict(mat=_mat(stride=128), wsb=1 << 40)):
        assert mul(**kw) == L.ASF_ERR_INVALID_ARG, kw
    for kw in (dict(dt=0), dict(yt=2), dict(lora=_lora(dt=2)), dict(lora=_lora(r=L.ASF_MAX_LORA_RANK + 8)),
               dict(mat=_mat(group=48), wsb=1 << 40)):
        assert mul(**kw) == L.ASF_ERR_UNSUPPORTED, kw
    for kw in (dict(which=FAKE + 2), dict(x=2 * FAKE + 8), dict(y=4 * FAKE + 2), dict(y=4 * FAKE + 1, yt=1), dict(lora=_lora(r=12)),
               dict(lora=_lora(a=FAKE + 8)), dict(lora=_lora(b=FAKE + 4)), dict(lora=_lora(s=FAKE + 2)), dict(bias=FAKE + 2, wsb=1 << 40)):
        assert mul(**kw) == L.ASF_ERR_MISALIGNED, kw
