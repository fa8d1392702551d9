"""Tree attention and the append on the GPU against the float64 oracle.

Tolerance, elementwise, with M = sum_p p |v|: the output's rounding 2^-11 |o|,
the weights' rounding to fp16 2^-11 M (their sum stays fp32), and twice the
relative error of a weight, which is the absolute error of its score: (D + 16)
2^-23 max_p scale sum |q k| of fp32 accumulation and scaling, plus 2^-20 for
the exponential and the merges; 2^-24 below fp16's normal range.
"""
import numpy as np
import pytest
import torch

from oracle import attention as O
from tests.gpu_util import ensure_built

import activation_sparse_ffn_predict_b200 as A
from activation_sparse_ffn_predict_b200 import _lib as L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


class Case:
    """Requests of given lengths and tokens, with a random tree each, over shuffled pages."""

    def __init__(self, lens, toks, hkv=2, grp=2, D=64, page=16, seed=0, spread=1.5):
        rng = np.random.default_rng(seed)
        self.rng, self.lens, self.D, self.page, self.hkv, self.grp = rng, list(lens), D, page, hkv, grp
        self.begin = np.concatenate([[0], np.cumsum(toks)]).astype(int)
        T = self.T = int(self.begin[-1])
        need = [-(-(n + m) // page) for n, m in zip(lens, toks)]
        pages = max(1, sum(need)) + 2
        order = rng.permutation(pages)
        self.table = np.zeros((len(lens), max(1, max(need))), int)
        at = 0
        for r, n in enumerate(need):
            self.table[r, :n] = order[at:at + n]
            at += n
        f16 = lambda *s: rng.standard_normal(s).astype(np.float16)  # noqa: E731
        self.k, self.v = f16(pages, page, hkv, D), f16(pages, page, hkv, D)
        self.kn, self.vn = f16(T, hkv, D), f16(T, hkv, D)
        self.q = (rng.standard_normal((T, hkv * grp, D)) * spread).astype(np.float16)
        self.anc = np.zeros(T, np.int64)
        for r in range(len(lens)):
            for t in range(self.begin[r], self.begin[r + 1]):
                up = rng.integers(self.begin[r] - 1, t) if t > self.begin[r] else -1
                self.anc[t] = (1 << t) | (self.anc[up] if up >= self.begin[r] else 0)

    def device(self):
        i32 = lambda a: torch.from_numpy(np.asarray(a).astype(np.uint32).view(np.int32)).cuda()  # noqa: E731
        d = dict(cache=A.KVCache(torch.from_numpy(self.k.copy()).cuda(), torch.from_numpy(self.v.copy()).cuda()),
                 table=i32(self.table), lens=i32(self.lens), begin=i32(self.begin), anc=i32(self.anc))
        for n in ("kn", "vn", "q"):
            d[n] = torch.from_numpy(getattr(self, n)).cuda()
        d["o"] = torch.full_like(d["q"], 7.0)
        d["ws"] = A.Workspace.for_attention(d["cache"], self.hkv * self.grp, len(self.lens), self.T)
        return d

    def run(self, d=None, scale=None, append=True):
        d = d or self.device()
        if append:
            A.asf_kv_append(d["cache"], d["table"], d["lens"], d["begin"], d["kn"], d["vn"], d["ws"])
        A.asf_tree_attention(d["cache"], d["table"], d["lens"], d["begin"], d["q"], d["anc"], d["o"], d["ws"], scale=scale)
        return d

    def check(self, d, scale=None, error=0):
        scale = self.D ** -0.5 if scale is None else scale
        k, v = self.k.copy(), self.v.copy()
        O.append(k, v, self.table, self.lens, self.begin, self.kn, self.vn)
        assert np.array_equal(d["cache"].k.cpu().numpy(), k, equal_nan=True)
        assert np.array_equal(d["cache"].v.cpu().numpy(), v, equal_nan=True)
        o, mass, big = O.tree_attention(k, v, self.table, self.lens, self.begin, self.q, self.anc, scale)
        tol = 2.0 ** -11 * np.abs(o) + (2.0 ** -11 + 2 * (self.D + 16) * 2.0 ** -23 * big + 2.0 ** -20) * mass + 2.0 ** -24
        got = d["o"].cpu().numpy().astype(np.float64)
        assert np.isfinite(got).all()
        off = np.abs(got - o) - tol
        assert off.max() <= 0, (off.max(), np.unravel_index(off.argmax(), off.shape))
        assert A.asf_read_error(d["ws"]) == error


@pytest.mark.parametrize("lens,toks,kw", [
    ([0], [1], {}), ([1], [1], dict(D=8, page=1)), ([0], [32], dict(grp=1)), ([63], [1], dict(D=128)),
    ([64], [1], dict(D=128, hkv=1, grp=1)), ([65, 0, 130], [3, 2, 1], dict(D=80, page=20)),
    ([500], [16], dict(D=128, grp=8)), ([1000, 7], [1, 31], dict(grp=5, page=64)),
    ([3000, 1, 0, 2047, 2048], [8, 8, 8, 4, 4], dict(hkv=4, grp=4, D=128)),
    ([5000], [32], dict(hkv=1, grp=16, D=96, page=256)), ([12345], [1], dict(hkv=3, grp=7, D=72, page=7)),
    (list(range(0, 640, 20)), [1] * 32, dict(hkv=2, grp=1, D=128)),
    ([20000], [2], dict(hkv=1, grp=4, D=128, page=33)), ([9000], [3], dict(hkv=2, grp=11, D=64)),
    ([4000, 100, 0], [16, 8, 8], dict(hkv=2, grp=128, D=80, page=48)), ([1], [32], dict(hkv=1, grp=71, D=64)),
    ([777, 3], [5, 6], dict(grp=16, D=128, page=8)), ([2000], [9], dict(grp=8, D=56, page=128)),
    ([640], [8], dict(hkv=1, grp=9, D=128, page=640)), ([300, 400, 500], [0, 5, 0], dict(D=40))])
def test_against_the_definition(lens, toks, kw):
    c = Case(lens, toks, seed=sum(lens) + len(toks), **kw)
    d = c.run()
    c.check(d)
    first = d["o"].clone()
    d["o"].fill_(0)
    c.run(d)
    assert torch.equal(d["o"], first)                       # no order depends on timing


@pytest.mark.parametrize("lens,toks,kw", [
    ([64], [1], dict(hkv=1, grp=3, page=66)), ([2045], [3], dict(hkv=2, grp=4, D=128, page=2048)),
    ([2046], [3], dict(hkv=2, grp=4, D=128, page=2049)), ([1000], [2], dict(hkv=32, grp=1, D=128, page=1024)),
    ([0], [2], dict(hkv=8, grp=9, page=512)), ([255], [1], dict(hkv=8, grp=32, D=96, page=256)),
    ([3, 300, 0, 129], [2, 1, 0, 4], dict(hkv=2, grp=2, D=40, page=128)), ([70, 1], [1, 1], dict(hkv=40, grp=2, page=64)),
    ([100], [1], dict(hkv=100, grp=2, D=64, page=101)), ([900], [1], dict(hkv=74, grp=1, D=128, page=1024))])
def test_short_requests(lens, toks, kw):
    """Around the sizes at which a cluster takes a request's keys, of 4 or 8 CTAs, some of them without a tile."""
    c = Case(lens, toks, seed=sum(lens) + len(toks), **kw)
    d = c.run()
    c.check(d)
    first = d["o"].clone()
    d["o"].fill_(0)
    c.run(d)
    assert torch.equal(d["o"], first)


@pytest.mark.parametrize("grp,D", [(2, 64), (8, 64), (16, 64), (40, 128)])
def test_large_scores_and_scale(grp, D):
    c = Case([700], [4], grp=grp, D=D, spread=40.0, seed=3)  # one key takes nearly all of the weight
    c.check(c.run(scale=0.5), scale=0.5)
    c.check(c.run(scale=-0.25), scale=-0.25)


@pytest.mark.parametrize("grp", [3, 12])
def test_rows_that_see_nothing_and_rows_behind(grp):
    c = Case([0, 40], [6, 5], grp=grp, seed=4)
    c.anc[2] = 0                                            # no prefix and no own bit
    c.anc[8] = 0                                            # only the prefix
    c.anc[1] |= 1 << 9                                      # a bit of another request: not its token
    c.anc[4] = 1 << 31
    d = c.device()
    pad = torch.full((4,) + d["q"].shape[1:], 5.0, dtype=torch.float16, device="cuda")
    d["q"] = torch.cat([d["q"], pad])
    for n in ("kn", "vn"):
        d[n] = torch.cat([d[n], torch.full((4,) + d[n].shape[1:], 9.0, dtype=torch.float16, device="cuda")])
    d["anc"] = torch.cat([d["anc"], torch.full((4,), -1, dtype=torch.int32, device="cuda")])
    d["o"] = torch.full_like(d["q"], 7.0)
    d["ws"] = A.Workspace.for_attention(d["cache"], 2 * grp, 2, 15)
    c.run(d)
    assert (d["o"][11:] == 7.0).all()                       # tokens behind the last request
    assert (d["o"][2] == 0).all() and (d["o"][4] == 0).all()
    c.anc[1] &= ~(1 << 9)
    c.anc[4] = 0
    d["o"] = d["o"][:11]
    c.check(d)


@pytest.mark.parametrize("grp,D", [(1, 64), (4, 64), (8, 64), (9, 128)])
@pytest.mark.parametrize("page", [16, 20, 64])
@pytest.mark.parametrize("n", [0, 50, 61, 700])
def test_what_a_row_does_not_see_does_not_reach_it(n, grp, D, page):
    """NaN and infinities in drafted tokens' keys and values, and behind the last key."""
    c = Case([n], [8], grp=grp, D=D, page=page, seed=n)
    c.anc[:] = [1, 3, 5, 9, 19, 32, 64, 128]
    for t, val in ((5, np.nan), (6, np.inf), (7, -np.inf)):
        c.kn[t], c.vn[t] = val, val
    c.vn[4, 0, 3] = np.nan
    if (n + 8) % page:                                      # the rest of the last page
        c.k[c.table[0][(n + 8) // page], (n + 8) % page:] = np.nan
        c.v[c.table[0][(n + 8) // page], (n + 8) % page:] = np.inf
    d = c.run()
    got = d["o"].cpu().numpy()
    k, v = c.k.copy(), c.v.copy()
    O.append(k, v, c.table, c.lens, c.begin, c.kn, c.vn)
    o, _, _ = O.tree_attention(k[..., :], v, c.table, c.lens, c.begin, c.q, np.where(np.arange(8) < 4, c.anc, 1), c.D ** -0.5)
    assert np.isfinite(got[:4]).all() and np.allclose(got[:4], o[:4], rtol=4e-3, atol=4e-3)
    assert np.isnan(got[5:]).all()                          # rows that see them
    assert np.isnan(got[4, :grp, 3]).all() and np.isfinite(got[4, grp:]).all()


@pytest.mark.parametrize("grp,page", [(2, 16), (40, 16), (40, 20)])
def test_a_key_of_nan_that_is_seen_is_not_lost(grp, page):
    """Scores that are all NaN for a tile, finite ones after it: NaN, as the softmax has it; the other head is sound."""
    c = Case([200], [2], grp=grp, page=page, seed=13)
    pg, sl = O.positions(c.table[0], page, 64)
    c.k[pg, sl, 0] = np.nan
    got = c.run()["o"].cpu().numpy()
    assert np.isnan(got[:, :grp]).all() and np.isfinite(got[:, grp:]).all()


def test_strides_of_dimensions_of_one():
    c = Case([40], [1], hkv=1, grp=3, page=64, D=64, seed=14)
    d = c.device()
    pages = c.k.shape[0]
    odd = lambda a: torch.as_strided(torch.from_numpy(a).cuda(), (pages, 64, 1, 64), (64 * 64, 64, 1, 1))  # noqa: E731
    d["cache"] = A.KVCache(odd(c.k), odd(c.v))
    c.check(c.run(d))
    one = torch.from_numpy(c.k[:, 0]).cuda()                 # pages of one token, page by page
    kk = torch.as_strided(one, (pages, 1, 1, 64), (64, 1, 1, 1))
    assert A.KVCache(kk, kk).workspace_bytes(1, 1, 1) > 0


@pytest.mark.parametrize("grp,D", [(2, 64), (16, 64), (12, 104)])
def test_strided_caches(grp, D):
    """Pages laid out head by head, and keys and values side by side in one tensor."""
    c = Case([200, 30], [3, 4], hkv=4, grp=grp, D=D, seed=6)
    for make in (lambda a: torch.from_numpy(a).cuda().permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3), None):
        d = c.device()
        if make is not None:
            d["cache"] = A.KVCache(make(c.k), make(c.v))
        else:
            both = torch.stack([torch.from_numpy(c.k), torch.from_numpy(c.v)], 3).cuda()
            d["cache"] = A.KVCache(both[:, :, :, 0], both[:, :, :, 1])
        c.check(c.run(d))


@pytest.mark.parametrize("grp", [2, 40])
def test_offsets_past_32_bits(grp):
    page, D, pages = 64, 128, 2 ** 31 // (64 * 128) + 3     # elements behind 2^31
    k = torch.zeros(pages, page, 1, D, dtype=torch.float16, device="cuda")
    v = torch.zeros_like(k)
    c = Case([100], [2], hkv=1, grp=grp, D=D, page=page, seed=8)
    where = torch.tensor([pages - 1, pages - 3, 0, 1], device="cuda")
    c.table = c.table * 0 + np.arange(c.table.shape[1])
    k[where[:2]], v[where[:2]] = torch.from_numpy(c.k[:2]).cuda(), torch.from_numpy(c.v[:2]).cuda()
    d = c.device()
    small = d["cache"]
    d["cache"], d["table"] = A.KVCache(k, v), where[:2].int()[None].contiguous()
    c.run(d)
    small.k[:2], small.v[:2] = k[where[:2]], v[where[:2]]
    d["cache"] = small
    c.check(d)


@pytest.mark.parametrize("grp", [2, 30])
def test_bad_tables_are_flagged_and_skipped(grp):
    c = Case([40, 30], [2, 3], grp=grp, seed=9)
    d = c.device()
    d["table"][0, 1] = c.k.shape[0] + 5                     # positions 16..31 of request 0
    d["table"][1, 0] = -1
    c.run(d)
    assert A.asf_read_error(d["ws"]) == L.ASF_ERR_DEVICE_INDEX
    o = d["o"].clone()
    # the same with those keys masked by hand: request 0 without 16 keys, request 1 without its first 16
    short = Case([40, 30], [2, 3], grp=grp, seed=9)
    keep = [np.r_[0:16, 32:40], np.r_[16:30]]
    ks, vs = c.k.copy(), c.v.copy()
    O.append(ks, vs, c.table, c.lens, c.begin, c.kn, c.vn)
    for r in range(2):
        pg, sl = O.positions(c.table[r], 16, c.lens[r] + c.begin[r + 1] - c.begin[r])
        idx = np.concatenate([keep[r], np.arange(c.lens[r], len(pg))])
        kk, vv = ks[pg[idx], sl[idx]][None], vs[pg[idx], sl[idx]][None]
        t = slice(c.begin[r], c.begin[r + 1])
        ref, _, _ = O.tree_attention(kk, vv, [[0]], [len(keep[r])], [0, t.stop - t.start], short.q[t],
                                     short.anc[t] >> t.start, 0.125)
        assert np.allclose(o[t].cpu().numpy(), ref, rtol=4e-3, atol=4e-3)
    # lengths and ranges that cannot be: clamped, flagged, nothing written outside
    for lens, begin in (([-5, 30], [0, 2, 5]), ([40, 10 ** 9], [0, 2, 5]), ([40, 30], [0, 7, 3]), ([40, 30], [3, 1, 99]),
                        ([2 ** 31 - 1, 2 ** 31 - 1], [-4, 2, 5])):
        d = c.device()
        d["lens"], d["begin"] = (torch.tensor(x, dtype=torch.int64).int().cuda() for x in (lens, begin))
        c.run(d)
        assert A.asf_read_error(d["ws"]) == L.ASF_ERR_DEVICE_INDEX
    c2 = Case([40, 30], [2, 3], grp=grp, seed=9)
    c2.check(c2.run())                                      # and the next call is sound


def test_accepted_tokens_are_appended_again():
    c = Case([37], [6], seed=10)
    d = c.run()
    keep = [0, 2, 5]                                        # a path of the tree
    d["begin"] = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    A.asf_kv_append(d["cache"], d["table"], d["lens"], d["begin"], d["kn"][keep], d["vn"][keep], d["ws"])
    d["lens"] += 3
    got = d["cache"].k.cpu().numpy()
    pg, sl = O.positions(c.table[0], 16, 40)
    assert np.array_equal(got[pg[37:], sl[37:]], c.kn[keep])


@pytest.mark.parametrize("grp", [2, 20])
def test_graph_replays_with_other_lengths(grp):
    c = Case([900, 0], [4, 4], grp=grp, seed=11)
    d = c.device()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.run(d)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(d)
    for lens in ([900, 0], [10, 0], [333, 0]):
        c.lens = lens
        d["cache"].k.copy_(torch.from_numpy(c.k))
        d["cache"].v.copy_(torch.from_numpy(c.v))
        d["lens"].copy_(torch.tensor(lens))
        graph.replay()
        c.check(d)


def test_python_refusals():
    c = Case([20], [2])
    d = c.device()
    k = d["cache"].k

    def att(**kw):
        a = dict(d, **kw)
        A.asf_tree_attention(a["cache"], a["table"], a["lens"], a["begin"], a["q"], a["anc"], a["o"], a["ws"])

    for bad in (lambda: A.KVCache(k.float(), k.float()), lambda: A.KVCache(k, k[:1]), lambda: A.KVCache(k.cpu(), k.cpu()),
                lambda: A.KVCache(k[..., ::2], k[..., ::2]), lambda: att(q=d["q"].float()), lambda: att(o=d["o"][:1]),
                lambda: att(anc=d["anc"].long()), lambda: att(anc=d["anc"][:1]), lambda: att(lens=d["lens"].cpu()),
                lambda: att(begin=d["begin"][:1]), lambda: att(table=d["table"][0]),
                lambda: A.asf_kv_append(d["cache"], d["table"], d["lens"], d["begin"], d["kn"][:, :1], d["vn"], d["ws"])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: att(q=d["q"][:, :3].contiguous(), o=d["o"][:, :3].contiguous()), lambda: att(o=d["q"]),
                lambda: att(ws=A.Workspace._sized(4096, d["q"].device, None, "test"))):
        with pytest.raises(A.AsfError):
            bad()


@pytest.mark.parametrize("low", [3.5, 4.0])
@pytest.mark.parametrize("grp,hkv,page", [(2, 300, 16), (20, 300, 64), (40, 150, 64), (40, 150, 20), (2, 4, 16), (40, 4, 64)])
def test_many_small_weights_beside_a_large_one(grp, hkv, page, low):
    """The first key takes the weight and has v = 0; 8000 keys 18 or 16 nats below it make the output.

    Many kv heads: one unit has all of a head's keys, four: they are split.  An error of 2^-36 of the
    largest weight per key, v <= 1: 8000 x 2^-36 = 1.2e-7 in all at most, and check() allows
    (2^-11 + 2^-20) mass + 2^-24 = 1.2e-7 beside the output's own rounding (18 nats: mass >= 6e-5)."""
    n = 8000
    c = Case([n], [1], hkv=hkv, grp=grp, D=8, page=page, seed=17)
    c.k[:], c.kn[:], c.q[:] = 0, 0, 0
    c.k[..., 0], c.kn[..., 0], c.q[..., 0] = low, low, 4.0
    c.v[:], c.vn[:] = 0.5 + 0.5 * c.rng.random(c.v.shape), 0.75
    pg, sl = O.positions(c.table[0], page, 1)
    c.k[pg, sl, :, 0], c.v[pg, sl] = 8.0, 0
    c.check(c.run(scale=1.0), scale=1.0)


@pytest.mark.parametrize("grp", [2, 20, 40])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_beyond_24_bits(grp, sign):
    """Equal scores of up to 2^33, where a float's step is wider than the range of the weights: the plain mean of v.

    Equal weights are equal in fp16 too, so that their rounding cancels up to a step of 2^-11 of v."""
    for e in range(12):
        c = Case([500], [1], hkv=2, grp=grp, D=8, seed=e)
        c.k[:], c.kn[:], c.q[:] = 0, 0, 0
        c.k[..., 0], c.kn[..., 0], c.q[..., 0] = 6e4, 6e4, sign * 6e4
        got = c.run(scale=2.0 ** -e)["o"].cpu().numpy().astype(np.float64)
        pg, sl = O.positions(c.table[0], c.page, 500)
        v = np.concatenate([c.v[pg, sl], c.vn]).astype(np.float64)
        ref, mass = (np.repeat(f(v).mean(0)[None], grp, 1).reshape(1, 2 * grp, 8) for f in (np.asarray, np.abs))
        assert (np.abs(got - ref) <= 2.0 ** -11 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -20) * mass + 2.0 ** -24).all()


@pytest.mark.parametrize("lens,toks,kw", [
    ([333], [1], dict(hkv=32, grp=1, D=128)), ([40, 0, 7], [2, 1, 3], dict(hkv=2, grp=4)),
    ([100, 30], [4, 4], dict(hkv=2, grp=16, page=64)), ([700], [5], dict(hkv=1, grp=9, D=80, page=20))])
def test_tables_wider_than_the_requests(lens, toks, kw):
    """Room for 4096 keys and more: the table's width chooses the form, and entries past a request's keys are not read."""
    c = Case(lens, toks, seed=sum(lens), **kw)
    for keys in (512, 1024, 2048, 4096, 70000):
        more = -(-keys // c.page) - c.table.shape[1]
        if more > 0:
            c.table = np.concatenate([c.table, np.full((len(lens), more), 2 ** 31 - 1)], 1)
        c.check(c.run())
