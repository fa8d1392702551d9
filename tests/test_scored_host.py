"""Scored attention's arguments that are refused before any launch (no GPU)."""
import ctypes

import pytest

from activation_sparse_ffn_predict_b200 import _lib as L
from activation_sparse_ffn_predict_b200 import build as B

FAKE = 1 << 20          # aligned, never dereferenced: every case fails validation first


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


def _cache(pages=10, page=16, heads=2, dim=64, k=FAKE, v=FAKE, ps=16 * 2 * 64, ts=128, hs=64):
    return L.asf_kv_cache(pages, page, heads, dim, k, v, ps, ts, hs)


def test_scored_attention_refuses(lib):
    c = _cache()
    need = lib.asf_attention_scored_workspace_bytes(ctypes.byref(c), 4, 2, 3, 4)
    assert need > lib.asf_attention_workspace_bytes(ctypes.byref(c), 4, 2, 3)

    def att(R=2, T=3, hq=4, q=FAKE, o=2 * FAKE, scale=1.0, scores=4 * FAKE, S=64, mp=4, ws=8 * FAKE, wsb=need - 1, cache=c):
        return lib.asf_tree_attention_scored(ctypes.byref(cache), FAKE, mp, R, FAKE, FAKE, T, hq, q, FAKE, scale, o, scores, S,
                                             ws, wsb, None)

    assert att() == att(ws=0, wsb=1 << 40) == L.ASF_ERR_WORKSPACE
    for kw in (dict(scores=0), dict(S=0), dict(S=-1), dict(q=0), dict(T=33), dict(scale=float("nan"))):
        assert att(**kw) == L.ASF_ERR_INVALID_ARG, kw
    assert att(scores=4 * FAKE + 2) == L.ASF_ERR_MISALIGNED and att(mp=1 << 27) == L.ASF_ERR_UNSUPPORTED
    for at in (FAKE, 2 * FAKE + 3 * 4 * 64 * 2 - 4, 2 * FAKE - 2 * 2 * 64 * 4 + 4):
        assert att(scores=at, wsb=1 << 40) == L.ASF_ERR_INVALID_ARG
    for bad in ((3, 1, 1, 1), (4, 33, 1, 1), (4, 1, 1, 0), (4, 1, 1, 1 << 27)):
        assert lib.asf_attention_scored_workspace_bytes(ctypes.byref(c), *bad) == 0
    for R in (1, 2):
        for T in (1, 2, 3):
            assert lib.asf_attention_scored_workspace_bytes(ctypes.byref(c), 4, R, T, 2) <= need
