"""Eviction on the GPU against the oracle: all of it is exact."""
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
    """Requests of given lengths over shuffled pages, and fresh pages for what stays."""

    def __init__(self, lens, keep, hkv=2, D=16, page=16, first=0, recent=0, S=None, seed=0, spare=0, values=None):
        rng = np.random.default_rng(seed)
        self.lens, self.keep, self.first, self.recent, self.page = list(lens), keep, first, recent, page
        need, fresh = [-(-max(1, n) // page) for n in lens], [-(-max(1, min(n, keep)) // page) for n in lens]
        pages = sum(need) + sum(fresh) + 2
        order, at = rng.permutation(pages), 0
        self.table, self.table_out = (np.zeros((len(lens), max(m)), np.int32) for m in (need, fresh))
        for t, m in ((self.table, need), (self.table_out, fresh)):
            for r, n in enumerate(m):
                t[r, :n] = order[at:at + n]
                at += n
        self.k, self.v = (rng.integers(-2 ** 15, 2 ** 15, (pages, page, hkv, D)).astype(np.int16) for _ in range(2))   # any bits
        S = S or max(1, max(lens))
        self.scores = np.exp(2 * rng.standard_normal((len(lens), hkv, S))).astype(np.float32)
        if values is not None:
            self.scores = rng.choice(np.array(values, np.float32), self.scores.shape)
        self.S_out = keep + spare

    def device(self):
        cu = lambda a: torch.from_numpy(a.copy()).cuda()  # noqa: E731
        R, hkv = len(self.lens), self.k.shape[2]
        return dict(cache=A.KVCache(cu(self.k).view(torch.float16), cu(self.v).view(torch.float16)), table=cu(self.table),
                    lens=cu(np.array(self.lens, np.int32)), scores=cu(self.scores), table_out=cu(self.table_out),
                    lens_out=torch.full((R,), -7, dtype=torch.int32, device="cuda"),
                    scores_out=torch.full((R, hkv, self.S_out), -7.0, device="cuda"),
                    kept=torch.full((R, hkv, self.keep), -7, dtype=torch.int32, device="cuda"))

    def run(self, d=None, **kw):
        d = d or self.device()
        d.setdefault("ws", A.Workspace.for_eviction(d["cache"]))
        A.asf_kv_evict(d["cache"], d["table"], d["lens"], d["scores"], self.keep, d["table_out"], d["lens_out"], d["scores_out"],
                       d["kept"], d["ws"], first=self.first, recent=self.recent, **kw)
        return d

    def check(self, d, error=0):
        k, v = self.k.copy(), self.v.copy()
        kept, best = O.evict(k, v, self.table, self.lens, self.scores, self.keep, self.first, self.recent, self.table_out)
        assert d["lens_out"].tolist() == [min(n, self.keep) for n in self.lens]
        got, sc = d["kept"].cpu().numpy(), d["scores_out"].cpu().numpy()
        for r in range(len(self.lens)):
            m = min(self.lens[r], self.keep)
            for h in range(k.shape[2]):
                assert np.array_equal(got[r, h, :m], kept[r][h]), (r, h)
                assert np.array_equal(sc[r, h, :m].view(np.int32), best[r][h].view(np.int32))
            assert (got[r, :, m:] == -7).all() and (sc[r, :, m:] == -7.0).all()
        assert np.array_equal(d["cache"].k.cpu().view(torch.int16).numpy(), k)
        assert np.array_equal(d["cache"].v.cpu().view(torch.int16).numpy(), v)
        assert A.asf_read_error(d["ws"]) == error


@pytest.mark.parametrize("lens,keep,kw", [
    ([0], 1, {}), ([1], 1, dict(D=8, page=1)), ([2], 1, dict(hkv=1, page=1)), ([100], 99, dict(D=128)), ([100], 100, {}), ([100], 101, {}),
    ([33, 0, 1, 64], 32, dict(hkv=3, D=80, page=20, first=4, recent=8)), ([500], 100, dict(first=100)), ([500], 100, dict(recent=100)),
    ([500], 100, dict(first=60, recent=40)), ([4000], 1000, dict(hkv=5, first=4, recent=256)), ([4096], 7, {}), ([4097], 4096, {}),
    ([5000, 300, 4999], 2048, dict(hkv=9, D=64, page=64, first=4, recent=100)), ([9001], 4000, dict(hkv=1, D=24, page=7, S=9500)),
    ([513, 512, 511], 256, dict(hkv=2, spare=50)), (list(range(0, 320, 10)), 100, dict(hkv=8, D=8, page=5)),
    ([20000], 19999, dict(hkv=1, D=8, page=256)), ([8191], 1, dict(hkv=2, D=8, page=64, S=8192)),
    # clusters of 4, 2 and 1 CTAs, as many as leave each an SM; 2 where one CTA does not hold the scores
    ([5000, 4097, 30], 700, dict(hkv=9, D=8, page=64)), ([4500] * 3, 100, dict(hkv=20, D=8, page=64, first=1, recent=9)),
    ([4200, 4097], 1000, dict(hkv=50, D=8, page=64)), ([45000, 100], 3, dict(hkv=80, D=8, page=512)), ([5000], 4999, dict(hkv=37, D=8, page=32))])
def test_against_the_definition(lens, keep, kw):
    c = Case(lens, keep, seed=sum(lens) + keep, **kw)
    c.check(c.run())


@pytest.mark.parametrize("n,keep", [(700, 300), (6000, 2500)])
@pytest.mark.parametrize("values", [
    [0.0], [0.0, -0.0, 1.0], [np.inf, -np.inf, 0.0, 1e-45, -1e-45], [np.nan, -np.inf, -1.0], [np.nan], [1.0, 1.0 + 2.0 ** -23, 1.0 - 2.0 ** -24],
    [3e38, -3e38, 2.0, -2.0, 1e-38, np.nan, np.inf]])
def test_ties_and_unusual_scores(n, keep, values):
    c = Case([n], keep, hkv=3, first=3, recent=5, seed=n, values=values)
    c.check(c.run())


@pytest.mark.parametrize("n,hkv", [(66000, 1), (74000, 1), (78000, 2), (81900, 1), (100000, 1), (12200, 60), (13400, 60), (20000, 60), (24600, 20),
                                   (41000, 20), (6100, 100), (6200, 100), (10200, 100)])
def test_shared_memory_of_every_size(n, hkv):
    """Around the sizes from which a kernel has to ask for its shared memory."""
    c = Case([n], 700, hkv=hkv, D=8, page=512, first=4, recent=64, seed=n)
    c.check(c.run())


def test_more_keys_than_shared_memory_holds():
    n = 8 * 40 * 1024 + 12345                                # of a cluster of 8: read again for each digit
    c = Case([n], 5000, hkv=1, D=8, page=4096, first=4, recent=64, seed=1)
    c.check(c.run())


@pytest.mark.parametrize("layout", ["heads first", "one tensor"])
def test_strided_caches(layout):
    c = Case([300, 40], 64, hkv=4, D=64, seed=6)
    d = c.device()
    if layout == "heads first":
        make = lambda a: a.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)  # noqa: E731
        d["cache"] = A.KVCache(make(d["cache"].k), make(d["cache"].v))
    else:
        both = torch.stack([d["cache"].k, d["cache"].v], 3)
        d["cache"] = A.KVCache(both[:, :, :, 0], both[:, :, :, 1])
    c.check(c.run(d))


def test_offsets_past_32_bits():
    page, D, pages = 64, 128, 2 ** 31 // (64 * 128) + 6
    k = torch.zeros(pages, page, 1, D, dtype=torch.float16, device="cuda")
    v = torch.zeros_like(k)
    c = Case([128], 64, hkv=1, D=D, page=page, seed=8)
    d = c.device()
    where = torch.tensor([pages - 1, 5, pages - 4], device="cuda")          # from far to far
    src = [int(i) for i in c.table[0]]
    k[where[:2]], v[where[:2]] = d["cache"].k[src], d["cache"].v[src]
    d["cache"] = A.KVCache(k, v)
    d["table"], d["table_out"] = where[:2].int()[None].contiguous(), where[2:].int()[None].contiguous()
    c.run(d)
    kk, vv = c.k.copy(), c.v.copy()
    O.evict(kk, vv, c.table, c.lens, c.scores, 64, 0, 0, c.table_out)
    assert np.array_equal(k[where[2]].cpu().view(torch.int16).numpy(), kk[c.table_out[0, 0]])
    assert np.array_equal(v[where[2]].cpu().view(torch.int16).numpy(), vv[c.table_out[0, 0]])


def test_shared_pages_stay():
    """Two requests over the same first pages: each evicts to pages of its own."""
    c = Case([160, 144], 50, hkv=2, D=64, seed=11)
    c.table[1, :8] = c.table[0, :8]
    c.check(c.run())


def test_bad_tables_and_lengths_are_flagged():
    c = Case([100, 70], 40, seed=9)
    d = c.device()
    d["table"][0, 2] = c.k.shape[0] + 5
    d["table_out"][1, 1] = -1
    c.run(d)
    assert A.asf_read_error(d["ws"]) == L.ASF_ERR_DEVICE_INDEX
    k, v = c.k.copy(), c.v.copy()
    table, out = np.append(c.table, [[0]] * 2, 1), c.table_out.copy()
    kept, _ = O.evict(c.k.copy(), c.v.copy(), c.table, c.lens, c.scores, 40, 0, 0, c.table_out)
    for r in range(2):                                       # what is left is in its place
        for h in range(2):
            for j, i in enumerate(kept[r][h]):
                if (r == 0 and i // 16 == 2) or (r == 1 and j // 16 == 1):
                    continue
                to, at = (out[r][j // 16], j % 16, h), (table[r][i // 16], i % 16, h)
                k[to], v[to] = k[at], v[at]
    assert np.array_equal(d["cache"].k.cpu().view(torch.int16).numpy(), k)
    assert np.array_equal(d["cache"].v.cpu().view(torch.int16).numpy(), v)
    for lens in ([-3, 70], [100, 10 ** 6], [2 ** 31 - 1, -2 ** 31]):
        d = c.device()
        d["lens"].copy_(torch.tensor(lens))
        c.run(d)
        assert A.asf_read_error(d["ws"]) == L.ASF_ERR_DEVICE_INDEX
        assert d["lens_out"].tolist() == [min(max(n, 0), 40) for n in lens]
    d = c.device()                                           # a new table that is too narrow
    d["table_out"] = d["table_out"][:, :1].contiguous()
    c.run(d)
    assert A.asf_read_error(d["ws"]) == L.ASF_ERR_DEVICE_INDEX


def test_streams_and_graphs():
    c = Case([5000, 800], 600, hkv=2, first=4, recent=50, seed=3)
    d, side = c.device(), torch.cuda.Stream()
    d["ws"] = A.Workspace.for_eviction(d["cache"])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(d)
    with torch.cuda.stream(side):
        g.replay()
    side.synchronize()
    c.check(d)
    c.scores[:] = c.scores[:, ::-1, ::-1]                    # the captured call on new scores, twice
    d["scores"].copy_(torch.from_numpy(c.scores.copy()))
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    c.check(d)


def test_binding_refuses():
    c = Case([100], 40, seed=1)
    d = c.run()
    for name, bad in (("scores", d["scores"][0]), ("scores", d["scores"][:, :1]), ("scores", d["scores"].double()), ("kept", d["kept"].long()),
                      ("kept", d["kept"][:, :, :39]), ("lens_out", d["lens_out"][:0]), ("scores_out", d["scores_out"][:, :1]),
                      ("table_out", d["table_out"][0]), ("table", d["table"].cpu()), ("lens", d["lens"].long())):
        with pytest.raises(ValueError):
            c.run(dict(d, **{name: bad}))
    for name, bad in (("table_out", d["table"]), ("scores_out", d["scores"][:, :, :40].contiguous()[:, :, :39].contiguous()),
                      ("lens_out", d["lens"]), ("scores_out", d["scores"])):
        with pytest.raises(A.AsfError):
            c.run(dict(d, **{name: bad}))


# -------------------------------------------------- the calls together --
@pytest.mark.parametrize("grp", [2, 20])
def test_decode_evict_decode(grp):
    """Rotary append and scored attention for a few steps, an eviction, and attention over what is left: the
    same as over a cache of just those keys."""
    rng = np.random.default_rng(grp)
    hkv, D, page, R, keep, steps = 2, 64, 16, 2, 48, 3
    cu = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    f16 = lambda *s: cu(rng.standard_normal(s).astype(np.float16))  # noqa: E731
    cache = A.KVCache(f16(40, page, hkv, D), f16(40, page, hkv, D))
    table = cu(rng.permutation(40)[:20].reshape(2, 10).astype(np.int32))
    fresh = torch.tensor([p for p in range(40) if p not in table.flatten().tolist()], dtype=torch.int32, device="cuda")[:10].view(2, 5)
    lens, begin = cu(np.array([100, 30], np.int32)), cu(np.array([0, 1, 2], np.int32))
    pos, anc = lens.clone(), cu(np.array([1, 2], np.int32))
    scores = torch.zeros(R, hkv, 160, device="cuda")
    ws = A.Workspace.for_attention(cache, hkv * grp, R, 2, scored_pages=10)
    rot, q, o = A.Rotary(D), torch.empty(2, hkv * grp, D, dtype=torch.float16, device="cuda"), f16(2, hkv * grp, D)

    def step(tab, sc):
        joint = f16(2, hkv * (grp + 2), D)
        A.asf_rotary_append(rot, cache, tab, lens, begin, pos, *[joint[:, :hkv * grp], q], joint[:, hkv * grp:-hkv], joint[:, -hkv:], ws)
        A.asf_tree_attention_scored(cache, tab, lens, begin, q, anc, o, sc, ws)
        lens.add_(1)
        pos.add_(1)

    for _ in range(steps):
        step(table, scores)
    lens_out, kept = torch.empty_like(lens), torch.empty(R, hkv, keep, dtype=torch.int32, device="cuda")
    scores_out = torch.zeros(R, hkv, 80, device="cuda")
    k, v, sc = cache.k.cpu().numpy(), cache.v.cpu().numpy(), scores.cpu().numpy()
    A.asf_kv_evict(cache, table, lens, scores, keep, fresh, lens_out, scores_out, kept, ws, first=2, recent=16)
    O.evict(k, v, table.tolist(), lens.tolist(), sc, keep, 2, 16, fresh.tolist())
    assert np.array_equal(cache.k.cpu().numpy(), k) and np.array_equal(cache.v.cpu().numpy(), v)
    assert lens_out.tolist() == [48, 33]
    lens.copy_(lens_out)
    before = scores_out.cpu().numpy().copy()
    step(fresh, scores_out)                                  # positions go on from the old length
    assert pos.tolist() == [104, 34] and A.asf_read_error(ws) == 0
    k, v = cache.k.cpu().numpy(), cache.v.cpu().numpy()
    at, b = (lens - 1).tolist(), begin.tolist()
    ref, mass, big = O.tree_attention(k, v, fresh.tolist(), at, b, q.cpu().numpy(), np.array([1, 2]), D ** -0.5)
    tol = 2.0 ** -11 * np.abs(ref) + (2.0 ** -11 + 2 * (D + 16) * 2.0 ** -23 * big + 2.0 ** -20) * mass + 2.0 ** -24
    assert (np.abs(o.cpu().double().numpy() - ref) <= tol).all()
    want, err = O.received(k, fresh.tolist(), at, b, q.cpu().numpy(), np.array([1, 2]), D ** -0.5, before)
    assert (np.abs(scores_out.cpu().numpy() - want) <= 2.0 ** -22 * err + 2.0 ** -20 * np.abs(want) + 2.0 ** -100).all()
