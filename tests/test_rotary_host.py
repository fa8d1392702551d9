"""Rotary positions: frequencies, turns, and arguments refused before any launch (no GPU)."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest

from activation_sparse_ffn_predict_b200 import _lib as L
from activation_sparse_ffn_predict_b200 import build as B
from oracle import rotary as O

FAKE = 1 << 20          # aligned, never dereferenced: every case fails validation first
KIND = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


def _freq(lib, rot, base, scaling="none", factor=1.0, original=4096.0):
    out, mul = (ctypes.c_double * (rot // 2))(), ctypes.c_float()
    assert lib.asf_rotary_frequencies(rot, base, KIND[scaling], factor, original, out, ctypes.byref(mul)) == L.ASF_OK
    return np.array(out), mul.value


@pytest.mark.parametrize("rot", [2, 4, 16, 36, 128, 512])
@pytest.mark.parametrize("scaling", list(KIND))
@pytest.mark.parametrize("base,factor,original", [(10000.0, 8.0, 4096.0), (500000.0, 1.0, 2048.0), (100.0, 32.0, 100.0)])
def test_frequencies(lib, rot, scaling, base, factor, original):
    got, mul = _freq(lib, rot, base, scaling, factor, original)
    want, scale = O.frequencies(rot, base, scaling, factor, original)
    assert np.allclose(got, want, rtol=1e-13, atol=0) and abs(mul - scale) <= 2.0 ** -24 * scale


def test_the_scalings_meet_where_they_should(lib):
    plain, _ = _freq(lib, 128, 10000.0)
    ntk, _ = _freq(lib, 128, 10000.0, "ntk", 8.0)
    yarn, mul = _freq(lib, 128, 10000.0, "yarn", 8.0)
    assert ntk[0] == plain[0] and math.isclose(ntk[-1], plain[-1] / 8, rel_tol=1e-12)
    assert yarn[0] == plain[0] and yarn[-1] == plain[-1] / 8 and math.isclose(mul, 1 + 0.1 * math.log(8), rel_tol=1e-7)


@pytest.mark.parametrize("f", [1.0, 0.5, 1e-7, 6.283185307179586, 1e9, -0.25, 0.0, -1e-30, 5e-324])
def test_turns_are_the_nearest_fraction(lib, f):
    out = (ctypes.c_uint64 * 1)()
    assert lib.asf_rotary_turns((ctypes.c_double * 1)(f), 1, out) == L.ASF_OK
    pi = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
    t = Fraction(f) / (2 * pi)
    exact = (t - math.floor(t)) * 2 ** 64
    off = abs(Fraction(out[0]) - exact)
    # half a unit of rounding, and 64 bits of the quotient (2 units in the last place of it)
    bound = Fraction(1, 2) + 2 * max(abs(t), Fraction(1)) * 2
    assert min(off, 2 ** 64 - off) <= bound


def test_host_calls_refuse(lib):
    out, mul, turns = (ctypes.c_double * 4)(), ctypes.c_float(), (ctypes.c_uint64 * 4)()
    f = lambda rot=8, base=1e4, kind=0, factor=2.0, orig=64.0, o=out, m=ctypes.byref(mul): \
        lib.asf_rotary_frequencies(rot, base, kind, factor, orig, o, m)  # noqa: E731
    for kw in (dict(rot=0), dict(rot=7), dict(rot=-2), dict(base=1.0), dict(base=float("nan")), dict(base=float("inf")),
               dict(o=None), dict(m=None), dict(kind=1, factor=0.5), dict(kind=2, factor=float("nan")),
               dict(kind=3, orig=0.0), dict(kind=3, orig=float("inf"))):
        assert f(**kw) == L.ASF_ERR_INVALID_ARG, kw
    assert f(rot=L.ASF_MAX_ROTARY_DIM + 2) == f(kind=4) == f(kind=-1) == L.ASF_ERR_UNSUPPORTED
    assert lib.asf_rotary_turns(None, 1, turns) == lib.asf_rotary_turns(out, 0, turns) == L.ASF_ERR_INVALID_ARG
    assert lib.asf_rotary_turns((ctypes.c_double * 1)(float("nan")), 1, turns) == L.ASF_ERR_INVALID_ARG


def _rot(D=64, rot=64, layout=0, scale=1.0, turns=FAKE):
    return ctypes.byref(L.asf_rotary(D, rot, layout, scale, turns))


def test_struct_layout_matches_header():
    assert ctypes.sizeof(L.asf_rotary) == 24 and L.asf_rotary.turns.offset == 16


BAD = [(dict(D=0), L.ASF_ERR_INVALID_ARG), (dict(rot=0), L.ASF_ERR_INVALID_ARG), (dict(rot=63), L.ASF_ERR_INVALID_ARG),
       (dict(rot=66), L.ASF_ERR_INVALID_ARG), (dict(turns=0), L.ASF_ERR_INVALID_ARG), (dict(turns=FAKE + 4), L.ASF_ERR_MISALIGNED),
       (dict(scale=float("inf")), L.ASF_ERR_INVALID_ARG), (dict(layout=2), L.ASF_ERR_UNSUPPORTED),
       (dict(D=520, rot=64), L.ASF_ERR_UNSUPPORTED)]


@pytest.mark.parametrize("kw,status", BAD)
def test_descriptors_refused(lib, kw, status):
    c = ctypes.byref(L.asf_kv_cache(10, 16, 2, 64, FAKE, FAKE, 2048, 128, 64))
    assert lib.asf_rotary_apply(_rot(**kw), FAKE, 1, 1, 1, 64, 64, FAKE, FAKE, 64, 64, None) == status
    assert lib.asf_rotary_append(_rot(**kw), c, FAKE, 4, 1, FAKE, FAKE, 1, FAKE, 2, FAKE, 128, FAKE, FAKE, 128, FAKE, 128,
                                 FAKE, 4096, None) == status


def test_apply_refuses(lib):
    def app(x=FAKE, dt=1, T=3, heads=2, xt=128, xh=64, pos=FAKE, y=2 * FAKE, yt=128, yh=64, rot=_rot()):
        return lib.asf_rotary_apply(rot, x, dt, T, heads, xt, xh, pos, y, yt, yh, None)

    for kw in (dict(x=0), dict(y=0), dict(pos=0), dict(T=0), dict(T=-1), dict(heads=0), dict(xt=-128), dict(yh=-64),
               dict(yt=64),                                              # y's heads meet
               dict(yh=56), dict(yt=0), dict(yt=120),
               dict(y=FAKE + 16), dict(y=FAKE, xt=256),                  # x and y meet, not as one
               dict(y=FAKE + (2 * 128 + 64 + 64) * 2 - 16)):
        assert app(**kw) == L.ASF_ERR_INVALID_ARG, kw
    assert app(dt=2) == app(heads=L.ASF_MAX_ROTARY_HEADS + 1, yt=1 << 30) == L.ASF_ERR_UNSUPPORTED
    for kw in (dict(x=FAKE + 8), dict(y=2 * FAKE + 4), dict(pos=FAKE + 2), dict(xt=132), dict(xh=4), dict(yt=260), dict(yh=68),
               dict(rot=_rot(D=60, rot=60))):
        assert app(**kw) == L.ASF_ERR_MISALIGNED, kw


def test_append_refuses(lib):
    c = L.asf_kv_cache(10, 16, 2, 64, FAKE, FAKE, 2048, 128, 64)

    def app(table=FAKE, mp=4, R=2, lens=FAKE, begin=FAKE, T=3, pos=FAKE, hq=4, q=FAKE, qs=256, qo=2 * FAKE, k=FAKE, ks=128,
            v=FAKE, vs=128, ws=FAKE, wsb=4095, rot=_rot()):
        return lib.asf_rotary_append(rot, ctypes.byref(c), table, mp, R, lens, begin, T, pos, hq, q, qs, qo, k, ks, v, vs, ws,
                                     wsb, None)

    assert app() == app(ws=0, wsb=1 << 40) == app(ws=FAKE + 64, wsb=1 << 40) == L.ASF_ERR_WORKSPACE
    for kw in (dict(table=0), dict(lens=0), dict(begin=0), dict(mp=0), dict(R=0), dict(R=33), dict(T=0), dict(T=33), dict(pos=0),
               dict(q=0), dict(qo=0), dict(k=0), dict(v=0), dict(hq=0), dict(qs=248), dict(ks=120), dict(vs=0),
               dict(rot=_rot(D=128, rot=64))):
        assert app(**kw) == L.ASF_ERR_INVALID_ARG, kw
    assert app(mp=1 << 27) == app(hq=1 << 18) == L.ASF_ERR_UNSUPPORTED
    for kw in (dict(q=FAKE + 8), dict(qo=FAKE + 2), dict(k=FAKE + 4), dict(v=FAKE + 8), dict(pos=FAKE + 1), dict(qs=260),
               dict(ks=132), dict(vs=129), dict(table=FAKE + 2)):
        assert app(**kw) == L.ASF_ERR_MISALIGNED, kw
    for kw in (dict(qo=FAKE + 16), dict(qo=FAKE, qs=512), dict(q=4 * FAKE, qo=FAKE), dict(q=4 * FAKE, k=8 * FAKE, qo=FAKE + 32)):
        assert app(wsb=4096, **kw) == L.ASF_ERR_INVALID_ARG, kw


def test_turns_are_rounded_once(lib):
    """Half a unit off at most, whatever the size (2^-20 for what the 80 digits here and the 192 bits there leave)."""
    rng = np.random.default_rng(3)
    f = (rng.standard_normal(400) * 2.0 ** rng.integers(-80, 97, 400)).tolist()
    f += [1.0, -1.0, 1e9, -1e9, 2.0 ** 53 + 2, 6.283185307179586, -6.283185307179586, 0.99, np.nextafter(2.0 ** 100, 0), 5e-324, -5e-324, 0.0]
    out = (ctypes.c_uint64 * len(f))()
    assert lib.asf_rotary_turns((ctypes.c_double * len(f))(*f), len(f), out) == L.ASF_OK
    pi = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
    for x, got in zip(f, out):
        t = Fraction(x) / (2 * pi)
        off = abs(got - (t - math.floor(t)) * 2 ** 64)
        assert min(off, 2 ** 64 - off) <= Fraction(1, 2) + Fraction(1, 2 ** 20), x


@pytest.mark.parametrize("f", [2.0 ** 100, -(2.0 ** 100), 1e300, float("inf")])
def test_turns_refuse_what_has_no_fraction_left(lib, f):
    out = (ctypes.c_uint64 * 2)(7, 7)
    assert lib.asf_rotary_turns((ctypes.c_double * 2)(1.0, f), 2, out) == L.ASF_ERR_INVALID_ARG and list(out) == [7, 7]


def test_append_refuses_queries_over_the_cache(lib):
    k, v = 16 * FAKE, 32 * FAKE
    c = L.asf_kv_cache(10, 16, 2, 64, k, v, 2048, 128, 64)
    last, out = (9 * 2048 + 15 * 128 + 64 + 64) * 2, 3 * 4 * 64 * 2

    def app(qo, wsb=4096, q=FAKE):
        return lib.asf_rotary_append(_rot(), ctypes.byref(c), FAKE, 4, 2, FAKE, FAKE, 3, FAKE, 4, q, 256, qo, 2 * FAKE, 128,
                                     4 * FAKE, 128, FAKE, wsb, None)

    for at in (k, v):
        for qo in (at, at + last - 16, at - out + 16):
            assert app(qo) == app(qo, q=qo) == L.ASF_ERR_INVALID_ARG
    assert app(k + last, wsb=4095) == L.ASF_ERR_WORKSPACE
