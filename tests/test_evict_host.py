"""Eviction's arguments that are refused before any launch (no GPU)."""
import ctypes

import pytest

from activation_sparse_ffn_predict_b200 import _lib as L
from activation_sparse_ffn_predict_b200 import build as B

FAKE = 1 << 20          # aligned, never dereferenced: every case fails validation first


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


def test_arguments_refused(lib):
    def ev(table=FAKE, mp=4, R=2, lens=2 * FAKE, sc=3 * FAKE, S=64, keep=32, first=4, recent=8, to=4 * FAKE, mpo=2, lo=5 * FAKE,
           so=6 * FAKE, So=40, kept=7 * FAKE, ws=8 * FAKE, wsb=4095, cache=None):
        c = cache or L.asf_kv_cache(10, 16, 2, 64, 16 * FAKE, 32 * FAKE, 2048, 128, 64)
        return lib.asf_kv_evict(ctypes.byref(c), table, mp, R, lens, sc, S, keep, first, recent, to, mpo, lo, so, So, kept, ws,
                                wsb, None)

    assert ev() == ev(ws=0, wsb=1 << 40) == ev(ws=FAKE + 64, wsb=1 << 40) == L.ASF_ERR_WORKSPACE
    for kw in (dict(table=0), dict(lens=0), dict(sc=0), dict(to=0), dict(lo=0), dict(so=0), dict(kept=0), dict(mp=0), dict(mpo=0),
               dict(R=0), dict(R=33), dict(S=0), dict(keep=0), dict(first=-1), dict(recent=-1), dict(first=25),
               dict(first=1, recent=2 ** 31 - 1), dict(So=31), dict(to=FAKE)):
        assert ev(**kw) == L.ASF_ERR_INVALID_ARG, kw
    for kw in (dict(mp=1 << 27), dict(mpo=1 << 27), dict(S=(1 << 30) + 1)):
        assert ev(**kw) == L.ASF_ERR_UNSUPPORTED, kw
    for n in ("table", "lens", "sc", "to", "lo", "so", "kept"):
        assert ev(**{n: 9 * FAKE + 2}) == L.ASF_ERR_MISALIGNED, n
    rows = 2 * 2 * 4
    for kw in (dict(so=3 * FAKE + rows * 64 - 4), dict(so=3 * FAKE - rows * 40 + 4), dict(kept=3 * FAKE + 4), dict(kept=6 * FAKE),
               dict(lo=2 * FAKE + 4)):
        assert ev(wsb=4096, **kw) == L.ASF_ERR_INVALID_ARG, kw
    assert ev(cache=L.asf_kv_cache(10, 16, 2, 60, FAKE, FAKE, 2048, 128, 64)) == L.ASF_ERR_MISALIGNED


def test_outputs_over_inputs_refused(lib):
    """Each of lens_out, scores_out and kept at the first and the last word of every input, of the cache and of another output."""
    R, heads, mp, mpo, S, So, keep = 2, 2, 4, 2, 64, 40, 32
    c = L.asf_kv_cache(10, 16, heads, 64, 16 * FAKE, 32 * FAKE, 2048, 128, 64)
    rows, span = R * heads * 4, (9 * 2048 + 15 * 128 + 64 + 64) * 2
    place = dict(table=FAKE, lens=2 * FAKE, sc=3 * FAKE, to=4 * FAKE, lo=5 * FAKE, so=6 * FAKE, kept=7 * FAKE)
    size = dict(table=R * mp * 4, lens=R * 4, sc=rows * S, to=R * mpo * 4, lo=R * 4, so=rows * So, kept=rows * keep)

    def ev(wsb=4096, **kw):
        p = dict(place, **kw)
        return lib.asf_kv_evict(ctypes.byref(c), p["table"], mp, R, p["lens"], p["sc"], S, keep, 4, 8, p["to"], mpo, p["lo"], p["so"],
                                So, p["kept"], 8 * FAKE, wsb, None)

    assert ev(wsb=4095) == L.ASF_ERR_WORKSPACE
    for out in ("lo", "so", "kept"):
        for other in place:
            if other != out:
                for at in (place[other], place[other] + size[other] - 4, place[other] - size[out] + 4):
                    assert ev(**{out: at}) == L.ASF_ERR_INVALID_ARG, (out, other)
        for base in (16 * FAKE, 32 * FAKE):
            for at in (base, base + span - 4, base - size[out] + 4):
                assert ev(**{out: at}) == L.ASF_ERR_INVALID_ARG, (out, base)
