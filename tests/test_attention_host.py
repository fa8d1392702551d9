"""Tree attention's arguments that are refused before any launch (no GPU)."""
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


def test_struct_layout_matches_header():
    assert ctypes.sizeof(L.asf_kv_cache) == 56 and L.asf_kv_cache.k.offset == 16


BAD = [(dict(k=0), L.ASF_ERR_INVALID_ARG), (dict(v=0), L.ASF_ERR_INVALID_ARG), (dict(pages=0), L.ASF_ERR_INVALID_ARG),
       (dict(page=-1), L.ASF_ERR_INVALID_ARG), (dict(heads=0), L.ASF_ERR_INVALID_ARG), (dict(dim=0), L.ASF_ERR_INVALID_ARG),
       (dict(dim=136, hs=136, ts=272), L.ASF_ERR_UNSUPPORTED), (dict(heads=L.ASF_MAX_KV_HEADS + 1), L.ASF_ERR_UNSUPPORTED),
       (dict(dim=60), L.ASF_ERR_MISALIGNED), (dict(ts=132), L.ASF_ERR_MISALIGNED), (dict(k=FAKE + 8), L.ASF_ERR_MISALIGNED),
       (dict(ts=56), L.ASF_ERR_INVALID_ARG), (dict(hs=56), L.ASF_ERR_INVALID_ARG), (dict(ps=-128), L.ASF_ERR_INVALID_ARG)]


@pytest.mark.parametrize("kw,status", BAD)
def test_cache_descriptors_refused(lib, kw, status):
    c = ctypes.byref(_cache(**kw))
    big = 1 << 40
    assert lib.asf_kv_append(c, FAKE, 4, 1, FAKE, FAKE, 1, FAKE, FAKE, FAKE, big, None) == status
    assert lib.asf_tree_attention(c, FAKE, 4, 1, FAKE, FAKE, 1, 4, FAKE, FAKE, 1.0, FAKE, FAKE, big, None) == status
    assert lib.asf_attention_workspace_bytes(c, 4, 1, 1) == 0


def test_arguments_refused(lib):
    c = _cache()
    need = lib.asf_attention_workspace_bytes(ctypes.byref(c), 4, 2, 3)
    assert need > 4096

    def att(table=FAKE, mp=4, R=2, lens=FAKE, begin=FAKE, T=3, hq=4, q=FAKE, anc=FAKE, scale=1.0, o=FAKE, ws=FAKE, wsb=4096):
        return lib.asf_tree_attention(ctypes.byref(c), table, mp, R, lens, begin, T, hq, q, anc, scale, o, ws, wsb, None)

    def app(table=FAKE, mp=4, R=2, lens=FAKE, begin=FAKE, T=3, k=FAKE, v=FAKE, ws=FAKE, wsb=4095):
        return lib.asf_kv_append(ctypes.byref(c), table, mp, R, lens, begin, T, k, v, ws, wsb, None)

    for f in (att, app):
        assert f() == f(ws=0, wsb=1 << 40) == f(ws=FAKE + 64, wsb=1 << 40) == L.ASF_ERR_WORKSPACE
        for kw in (dict(table=0), dict(lens=0), dict(begin=0), dict(mp=0), dict(R=0), dict(R=33), dict(T=0), dict(T=33)):
            assert f(**kw) == L.ASF_ERR_INVALID_ARG, kw
        assert f(mp=1 << 27) == L.ASF_ERR_UNSUPPORTED
        assert f(table=FAKE + 2) == f(lens=FAKE + 1) == f(begin=FAKE + 3) == L.ASF_ERR_MISALIGNED
    for kw in (dict(q=0), dict(anc=0), dict(o=0), dict(hq=3), dict(hq=0), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert att(**kw) == L.ASF_ERR_INVALID_ARG, kw
    assert att(hq=2 * L.ASF_MAX_HEAD_GROUP + 2) == L.ASF_ERR_UNSUPPORTED
    assert att(q=FAKE + 8) == att(o=FAKE + 4) == att(anc=FAKE + 2) == app(k=FAKE + 8) == app(v=FAKE + 2) == L.ASF_ERR_MISALIGNED
    assert app(k=0) == app(v=0) == L.ASF_ERR_INVALID_ARG
    for bad in ((3, 1, 1), (4, 0, 1), (4, 33, 1), (4, 1, 33), (2 * L.ASF_MAX_HEAD_GROUP + 2, 1, 1)):
        assert lib.asf_attention_workspace_bytes(ctypes.byref(c), *bad) == 0


def test_overlaps_are_refused(lib):
    c = ctypes.byref(_cache())
    ws = lib.asf_attention_workspace_bytes(c, 4, 1, 1)
    for o in (FAKE, FAKE + 4 * 64 * 2 - 16):
        assert lib.asf_tree_attention(c, FAKE, 4, 1, FAKE, FAKE, 1, 4, FAKE, FAKE, 1.0, o, FAKE, ws, None) == L.ASF_ERR_INVALID_ARG
    assert lib.asf_attention_workspace_bytes(ctypes.byref(_cache(ps=56)), 4, 1, 1) == 0     # pages over one another
    assert lib.asf_tree_attention(c, FAKE, 4, 1, FAKE, FAKE, 1, 4, FAKE, FAKE, 3e38, FAKE + 4096, FAKE, ws, None) \
        == L.ASF_ERR_INVALID_ARG


def test_workspace_covers_fewer_requests_and_tokens(lib):
    c = ctypes.byref(_cache(heads=8, hs=64, ts=512, ps=8192))
    got = lib.asf_attention_workspace_bytes(c, 64, 4, 32)
    for R in (1, 2, 4):
        for T in (1, 5, 32):
            assert lib.asf_attention_workspace_bytes(c, 64, R, T) <= got
