"""Scored tree attention on the GPU against the float64 oracle.

Tolerance of a key's score, elementwise, with w the rows' weights and big a row's largest
scale sum |q k|: a weight's relative error is twice the absolute error of a score, (D + 16)
2^-23 big of fp32 accumulation and scaling (the largest score's error moves all of the row's
weights), plus 2^-20 for the exponentials, the sums' merge and the addition of the rows and
of the score that was there (2^-24 each, 128 rows and 32 tokens at most in chains of 32);
scores below 2^-100 are zero.
"""
import numpy as np
import pytest
import torch

from oracle import attention as O
from tests.gpu_util import ensure_built
from tests.test_gpu_attention import Case

import activation_sparse_ffn_predict_b200 as A
from activation_sparse_ffn_predict_b200 import _lib as L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def _device(c, S=None, seed=0):
    d = c.device()
    R = len(c.lens)
    S = S or max(1, max(c.lens[r] + c.begin[r + 1] - c.begin[r] for r in range(R)) + 3)
    rng = np.random.default_rng(seed)
    c.old = rng.random((R, c.hkv, S)).astype(np.float32) * np.float32(0.01)
    d["scores"] = torch.from_numpy(c.old.copy()).cuda()
    d["ws"] = A.Workspace.for_attention(d["cache"], c.hkv * c.grp, R, c.T, scored_pages=d["table"].shape[1])
    A.asf_kv_append(d["cache"], d["table"], d["lens"], d["begin"], d["kn"], d["vn"], d["ws"])
    return d


def _run(d, scale=None):
    A.asf_tree_attention_scored(d["cache"], d["table"], d["lens"], d["begin"], d["q"], d["anc"], d["o"], d["scores"], d["ws"],
                                scale=scale)
    return d


def _check(c, d, scale=None, error=0):
    scale = c.D ** -0.5 if scale is None else scale
    k, v = c.k.copy(), c.v.copy()
    O.append(k, v, c.table, c.lens, c.begin, c.kn, c.vn)
    want, err = O.received(k, c.table, c.lens, c.begin, c.q, c.anc, scale, c.old)
    got = d["scores"].cpu().double().numpy()
    tol = 2 * 2.0 ** -23 * err + 2.0 ** -20 * np.abs(want) + 2.0 ** -100
    assert np.isfinite(got).all()
    off = np.abs(got - want) - tol
    assert off.max() <= 0, (off.max(), np.unravel_index(off.argmax(), off.shape))
    for r, n in enumerate(c.lens):                          # behind the request's keys nothing is touched
        m = c.begin[r + 1] - c.begin[r]
        assert np.array_equal(got[r, :, (n + m if m else 0):], c.old[r, :, (n + m if m else 0):])
    plain = torch.full_like(d["o"], 3.0)
    A.asf_tree_attention(d["cache"], d["table"], d["lens"], d["begin"], d["q"], d["anc"], plain, d["ws"], scale=scale)
    assert torch.equal(plain, d["o"]) and A.asf_read_error(d["ws"]) == error


@pytest.mark.parametrize("lens,toks,kw", [
    ([0], [1], {}), ([1], [1], dict(D=8, page=1)), ([0], [32], dict(grp=1)), ([63], [1], dict(D=128)),
    ([64], [1], dict(D=128, hkv=1, grp=1)), ([65, 0, 130], [3, 2, 1], dict(D=80, page=20)),
    ([500], [16], dict(D=128, grp=8)), ([1000, 7], [1, 31], dict(grp=5, page=64)), ([333], [1], dict(hkv=32, grp=1, D=128)),
    ([3000, 1, 0, 2047, 2048], [8, 8, 8, 4, 4], dict(hkv=4, grp=4, D=128)), ([5000], [32], dict(hkv=1, grp=16, D=96, page=256)),
    ([12345], [1], dict(hkv=3, grp=7, D=72, page=7)), (list(range(0, 640, 20)), [1] * 32, dict(hkv=2, grp=1, D=128)),
    ([20000], [2], dict(hkv=1, grp=4, D=128, page=33)), ([4000, 100, 0], [16, 8, 8], dict(hkv=2, grp=128, D=80, page=48)),
    ([1], [32], dict(hkv=1, grp=71, D=64)), ([777, 3], [5, 6], dict(grp=16, D=128, page=8)),
    ([640], [8], dict(hkv=1, grp=9, D=128, page=640)), ([300, 400, 500], [0, 5, 0], dict(D=40)),
    ([2045], [3], dict(hkv=2, grp=4, D=128, page=2048)), ([900], [1], dict(hkv=74, grp=1, D=128, page=1024)),
    ([9000], [1], dict(hkv=1, grp=16, D=128, page=16)), ([9000, 50], [4, 4], dict(hkv=1, grp=8, D=64, page=32)),
    ([200], [12], dict(hkv=2, grp=11, D=64, page=32)), ([5000, 90], [31, 1], dict(hkv=2, grp=128, D=128, page=64)),
    ([3000], [32], dict(hkv=3, grp=7, D=80, page=8)), ([127, 128, 129], [8, 8, 8], dict(hkv=1, grp=16, D=64, page=128)),
    ([260], [9], dict(hkv=1, grp=15, D=72, page=64)), ([100, 100], [16, 16], dict(hkv=1, grp=128, D=128, page=64))])
def test_against_the_definition(lens, toks, kw):
    c = Case(lens, toks, seed=sum(lens) + len(toks), **kw)
    d = _run(_device(c))
    first = d["scores"].clone()
    _check(c, d)
    d["scores"].copy_(torch.from_numpy(c.old))
    _run(d)
    assert torch.equal(d["scores"], first)                  # no order depends on timing
    _run(d)                                                 # a second step over the same prefix adds the same again
    n = c.lens[0]
    if n and c.begin[1]:
        twice = d["scores"][0, :, :n].cpu().double().numpy() - c.old[0, :, :n]
        once = first[0, :, :n].cpu().double().numpy() - c.old[0, :, :n]
        assert np.abs(twice - 2 * once).max() <= 2.0 ** -22 * np.abs(first[0, :, :n].cpu().numpy()).max() * 2
    assert torch.equal(d["scores"][0, :, n:], first[0, :, n:])


@pytest.mark.parametrize("page", [64, 16, 20])
@pytest.mark.parametrize("lens,toks,grp", [([700, 33], [6, 2], 8), ([2000], [8], 2)])
def test_tables_too_wide_to_keep_scores(lens, toks, grp, page):
    """More than 512 MB of scores if they were kept: the keys are read again instead."""
    c = Case(lens, toks, hkv=4, grp=grp, D=128, page=page, seed=17)
    wide = (512 << 20) // (4 * c.T * 4 * grp) // page + 2
    c.table = np.pad(c.table, ((0, 0), (0, wide - c.table.shape[1])))
    d = _run(_device(c))
    _check(c, d)
    assert d["ws"].nbytes > 512 << 20                       # narrower tables on the same workspace do keep theirs
    first = d["scores"].clone()
    d["scores"].copy_(torch.from_numpy(c.old))
    d["table"] = d["table"][:, :wide // 2].contiguous()
    _run(d)
    _check(c, d)
    assert (first - d["scores"]).abs().max() <= 2.0 ** -18 * first.abs().max()


@pytest.mark.parametrize("grp", [2, 16, 40])
def test_the_weights_of_a_step_add_up(grp):
    c = Case([1500, 37], [4, 2], hkv=3, grp=grp, D=128, page=64, seed=2)
    d = _device(c)
    d["scores"].zero_()
    _run(d)
    total = d["scores"].double().sum(-1).cpu().numpy()
    want = np.array([[4 * grp] * 3, [2 * grp] * 3])
    assert np.abs(total - want).max() <= want.max() * 2.0 ** -18    # each row's sum is 1 up to fp32 sums of its weights


@pytest.mark.parametrize("grp,D", [(2, 64), (16, 64), (40, 128)])
def test_large_scores_and_scale(grp, D):
    for scale in (0.5, -0.25):
        c = Case([700], [4], grp=grp, D=D, spread=40.0, seed=3)
        _check(c, _run(_device(c), scale=scale), scale=scale)


@pytest.mark.parametrize("grp", [3, 40])
def test_rows_that_see_nothing(grp):
    c = Case([0, 40], [6, 5], grp=grp, seed=4)
    c.anc[2] = 0
    c.anc[8] = 0
    _check(c, _run(_device(c)))
    c = Case([0], [3], grp=grp, seed=5)
    c.anc[:] = 0
    d = _run(_device(c))
    assert (d["scores"][:, :, :3] == 0).all() and (d["o"] == 0).all()


@pytest.mark.parametrize("grp,page", [(1, 16), (8, 20), (40, 16), (40, 20)])
@pytest.mark.parametrize("n", [0, 50, 700])
def test_what_a_row_does_not_see_does_not_reach_it(n, grp, page):
    """NaN and infinities in drafted tokens' keys and behind the last key: the keys before them get what the sound rows give."""
    c = Case([n], [8], grp=grp, D=64, page=page, seed=n)
    c.anc[:] = [1, 3, 5, 9, 17, 0, 0, 0]                    # no row sees tokens 5, 6 and 7
    for t, val in ((5, np.nan), (6, np.inf), (7, -np.inf)):
        c.kn[t], c.vn[t] = val, val
    if (n + 8) % page:
        c.k[c.table[0][(n + 8) // page], (n + 8) % page:] = np.nan
    d = _device(c)
    _run(d)
    got = d["scores"].cpu().numpy()
    if n == 0:
        assert (got[:, :, 5:8] == 0).all()
    assert np.isfinite(got).all()
    k = c.k.copy()
    O.append(k, c.v.copy(), c.table, c.lens, c.begin, c.kn, c.vn)
    anc = c.anc.copy()
    if n:                                                   # rows 5 to 7 see the prefix alone
        assert (anc[5:] == 0).all()
    want, err = O.received(k, c.table, c.lens, c.begin, c.q, anc, 64 ** -0.5, c.old)
    assert (np.abs(got - want) <= 2.0 ** -22 * err + 2.0 ** -20 * np.abs(want) + 2.0 ** -100).all()


@pytest.mark.parametrize("grp", [2, 40])
def test_a_row_of_nan_spoils_its_own_kv_head_only(grp):
    c = Case([200], [2], grp=grp, page=16, seed=13)
    c.q[0, 0] = np.nan
    got = _run(_device(c))["scores"].cpu().numpy()
    see = [0] + ([1] if c.anc[0] >> 1 & 1 else [])
    assert np.isnan(got[0, 0, :200]).all() and np.isfinite(got[0, 1]).all()
    assert np.isnan(got[0, 0, 200:202][see]).all() and np.isfinite(got[0, 0, 202:]).all()


@pytest.mark.parametrize("grp,page", [(2, 16), (30, 16), (30, 20)])
def test_bad_tables_and_short_scores_are_flagged(grp, page):
    c = Case([100, 30], [2, 3], grp=grp, page=page, seed=9)
    d = _device(c)
    d["table"][0, 1] = c.k.shape[0] + 5
    _run(d)
    assert A.asf_read_error(d["ws"]) == L.ASF_ERR_DEVICE_INDEX
    got = d["scores"].cpu().numpy()
    assert np.array_equal(got[0, :, page:2 * page], c.old[0, :, page:2 * page])    # nobody saw them
    d = _device(c, S=50)                                    # request 0 has 102 keys, the scores hold 50
    pad = torch.full((2, 2, 60), 5.0, device="cuda")
    whole = torch.cat([d["scores"].flatten(), pad.flatten()])
    d["scores"] = whole[:2 * 2 * 50].view(2, 2, 50)
    _run(d)
    assert A.asf_read_error(d["ws"]) == L.ASF_ERR_DEVICE_INDEX
    assert (whole[200:] == 5.0).all()
    k = c.k.copy()
    O.append(k, c.v.copy(), c.table, c.lens, c.begin, c.kn, c.vn)
    old = np.concatenate([c.old, np.zeros((2, 2, 80), np.float32)], 2)
    want, err = O.received(k, c.table, c.lens, c.begin, c.q, c.anc, c.D ** -0.5, old)
    ok = np.abs(d["scores"].cpu().numpy() - want[:, :, :50]) <= (2.0 ** -22 * err + 2.0 ** -20 * np.abs(want) + 2.0 ** -100)[:, :, :50]
    assert ok.all()


def test_strided_and_far_caches():
    page, D, pages = 64, 128, 2 ** 31 // (64 * 128) + 3     # elements behind 2^31
    k = torch.zeros(pages, page, 1, D, dtype=torch.float16, device="cuda")
    v = torch.zeros_like(k)
    for grp in (2, 40):
        c = Case([100], [2], hkv=1, grp=grp, D=D, page=page, seed=8)
        c.table = c.table * 0 + np.arange(c.table.shape[1])
        where = torch.tensor([pages - 1, pages - 3], device="cuda")
        k[where], v[where] = torch.from_numpy(c.k[:2]).cuda(), torch.from_numpy(c.v[:2]).cuda()
        d = _device(c)
        d["cache"], d["table"] = A.KVCache(k, v), where.int()[None].contiguous()
        A.asf_kv_append(d["cache"], d["table"], d["lens"], d["begin"], d["kn"], d["vn"], d["ws"])
        _check(c, _run(d))


def test_streams_and_graphs():
    c = Case([900, 70], [4, 4], grp=8, D=128, page=64, seed=15)
    d = _device(c)
    _run(d)
    torch.cuda.synchronize()
    first = d["scores"].clone()
    d["scores"].copy_(torch.from_numpy(c.old))
    torch.cuda.synchronize()
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g):
        _run(d)
    with torch.cuda.stream(side):
        g.replay()
    side.synchronize()
    assert torch.equal(d["scores"], first)


def test_binding_refuses():
    c = Case([40], [2], grp=2, seed=1)
    d = _device(c)
    good = d["scores"]
    for bad in (good[0], good[:, :1], good.double(), good.cpu(), good.transpose(1, 2).contiguous().transpose(1, 2)):
        d["scores"] = bad
        with pytest.raises(ValueError):
            _run(d)
    d["scores"] = good
    d["ws"] = A.Workspace.for_attention(d["cache"], 4, 1, 2)
    with pytest.raises(A.AsfError):
        _run(d)                                             # a workspace for the plain call alone
