"""The attention stage's calls on two streams at once, and two graphs of one workspace each, replayed side by side."""
import numpy as np
import pytest
import torch

from tests.gpu_util import ensure_built
from tests.test_gpu_attention import Case

import activation_sparse_ffn_predict_b200 as A

pytestmark = pytest.mark.gpu


class Step:
    """A turned, scored and adapted step and an eviction over a cache of its own."""

    def __init__(self, seed, grp, page):
        c = self.c = Case([3000, 17], [6, 2], hkv=2, grp=grp, D=128, page=page, seed=seed)
        self.d = c.device()
        torch.manual_seed(seed)
        half = lambda *s: torch.randn(*s, device="cuda").half()  # noqa: E731
        self.hq = 2 * grp
        pages = c.k.shape[0]
        # pages of the eviction behind those of the requests
        self.cache = A.KVCache(torch.cat([self.d["cache"].k, half(80, page, 2, 128)]), torch.cat([self.d["cache"].v, half(80, page, 2, 128)]))
        self.fresh = (pages + torch.arange(80, device="cuda")).int().view(2, 40)
        self.rot, self.pos = A.Rotary(128, 64), torch.arange(8, device="cuda").int() + 70000
        self.qkv, self.q = half(8, self.hq + 4, 128), torch.empty(8, self.hq, 128, device="cuda").half()
        self.o, self.scores = torch.empty_like(self.q), torch.zeros(2, 2, 3100, device="cuda")
        self.keep = 500
        self.lens_out, self.kept = torch.zeros(2, device="cuda").int(), torch.zeros(2, 2, self.keep, device="cuda").int()
        self.left = torch.zeros(2, 2, self.keep, device="cuda")
        self.mat = A.W4Matrix.quantize(half(700, self.hq * 128), 64)
        self.lora = A.LoraSet(half(3, 16, self.hq * 128), half(3, 700, 16))
        self.which, self.y = torch.tensor([0, 1, 2, -1, 0, 0, 1, 2], device="cuda").int(), torch.zeros(8, 700, device="cuda").half()
        self.ws = A.Workspace.for_attention(self.cache, self.hq, 2, 8, scored_pages=self.d["table"].shape[1])
        self.wl = A.Workspace.for_w4(self.mat, 8, lora=self.lora)

    def run(self):
        d, hq = self.d, self.hq
        req = (d["table"], d["lens"], d["begin"])
        A.asf_rotary_append(self.rot, self.cache, *req, self.pos, self.qkv[:, :hq], self.q, self.qkv[:, hq:hq + 2], self.qkv[:, hq + 2:], self.ws)
        self.scores.zero_()
        A.asf_tree_attention_scored(self.cache, *req, self.q, d["anc"], self.o, self.scores, self.ws)
        A.asf_kv_evict(self.cache, d["table"], d["lens"], self.scores, self.keep, self.fresh, self.lens_out, self.left, self.kept, self.ws,
                       first=2, recent=50)
        A.asf_w4_matmul_lora(self.mat, self.lora, self.which, self.o.view(8, -1), self.y, self.wl, relu=True)

    def out(self):
        return [self.q, self.o, self.scores, self.lens_out, self.kept, self.left, self.cache.k, self.cache.v, self.y]

    def clear(self):
        for t in (self.q, self.o, self.scores, self.lens_out, self.kept, self.left, self.y):
            t.zero_()
        for t in (self.cache.k, self.cache.v):
            t[-80:].zero_()


@pytest.mark.parametrize("graphs", [False, True])
def test_side_by_side(graphs):
    ensure_built()
    steps = [Step(1, 4, 16), Step(2, 20, 64)]
    want = []
    for s in steps:
        s.clear()
        s.run()
        torch.cuda.synchronize()
        want.append([t.clone() for t in s.out()])
        assert s.y.abs().max() > 0 and s.kept[0].max() > 500 and (s.scores > 0).any()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    runs = [s.run for s in steps]
    if graphs:
        runs = []
        for s in steps:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                s.run()
            runs.append(g.replay)
    for _ in range(3):
        for s in steps:
            s.clear()
        torch.cuda.synchronize()
        for _ in range(15):
            for st, run in zip(streams, runs):
                with torch.cuda.stream(st):
                    run()
        torch.cuda.synchronize()
        for s, w in zip(steps, want):
            assert all(torch.equal(a, b) for a, b in zip(s.out(), w))
    assert all(A.asf_read_error(w) == 0 for s in steps for w in (s.ws, s.wl))


def test_back_to_back_calls_on_one_workspace():
    """Fifty steps without a wait between them: each sees what the one before has left."""
    ensure_built()
    s = Step(3, 8, 16)
    s.run()
    torch.cuda.synchronize()
    first = [t.clone() for t in s.out()]
    total, again = torch.zeros_like(s.scores), []
    for i in range(50):
        s.pos.add_(1)
        s.pos.sub_(1)                                        # small kernels between the calls
        s.run()
        total += s.scores
        again.append(s.y.clone())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(s.out(), first)) and all(torch.equal(a, first[-1]) for a in again)
    one = np.zeros(total.shape, np.float32)
    for _ in range(50):
        one += first[2].cpu().numpy()
    assert np.array_equal(total.cpu().numpy(), one)
