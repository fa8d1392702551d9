"""The attention stage with rotary positions, scores and adapters, captured with its layers: every stage has the
bits of the single calls, before an eviction and after it."""
import numpy as np
import pytest
import torch

from oracle import attention as O
from tests.gpu_util import ensure_built

import activation_sparse_ffn_predict_b200 as A

pytestmark = pytest.mark.gpu


def _model(layers, B, hkv, grp, D, page, pages, d=512, adapters=True):
    torch.manual_seed(21)
    half = lambda *s: torch.randn(*s, device="cuda").half()  # noqa: E731
    hq = hkv * grp
    caches = [A.KVCache(half(pages, page, hkv, D), half(pages, page, hkv, D)) for _ in range(layers)]
    outs = [A.W4Matrix.quantize(half(d, hq * D) * (hq * D) ** -0.5, 64) for _ in range(layers)]
    loras = [A.LoraSet(half(3, 8 * (l + 1), hq * D) * (hq * D) ** -0.5, half(3, d, 8 * (l + 1)), torch.rand(3, device="cuda"))
             for l in range(layers)] if adapters else None
    ffns = [A.W4FFN.quantize("relu", None, half(700, d) * d ** -0.5, half(700, d) * d ** -0.5, torch.zeros(700, device="cuda"), 64)
            for _ in range(layers)]
    return caches, outs, loras, ffns


@pytest.mark.parametrize("hkv,grp,D,page,R,T", [(2, 4, 64, 16, 2, 5), (1, 16, 80, 20, 1, 6)])
def test_steps_and_an_eviction(hkv, grp, D, page, R, T):
    ensure_built()
    layers, width, d, hq = 2, 12, 512, hkv * grp
    caches, outs, loras, ffns = _model(layers, T, hkv, grp, D, page, 2 * R * width)
    twins = [A.KVCache(c.k.clone(), c.v.clone()) for c in caches]
    rot = A.Rotary(D, D // 2, scaling="yarn", factor=4.0)
    stage = A.AttentionStage(caches, hq, R, width, T, outs, rotary=rot, scored=True, adapters=loras)
    st = A.LayerStack([], ffns, T, mode="dense", attention=stage)
    order = torch.randperm(2 * R * width).int().cuda()
    stage.table.copy_(order[:R * width].view(R, width))
    stage.lens.copy_(torch.tensor([150, 40][:R]))
    stage.begin.copy_(torch.tensor([0, T - 2, T] if R == 2 else [0, T]))
    stage.anc.copy_((2 ** (torch.arange(T) + 1) - 1).int())
    stage.which.copy_((torch.arange(T) % 4 - 1).int())
    stage.pos.copy_(torch.arange(T).int() + 1000)
    stage.q.normal_(), stage.k.normal_(), stage.v.normal_()
    st.capture()                                             # its warm-up runs add to the scores
    assert st.kernel_nodes() == st.launches_per_step()
    stage.scores.zero_()
    scores = stage.scores.clone()

    def by_hand():
        for l in range(layers):
            ws = A.Workspace.for_attention(twins[l], hq, R, T, scored_pages=width)
            q, o = torch.zeros_like(stage.q[l]), torch.zeros_like(stage.q[l])
            x, y = torch.empty(T, d, device="cuda").half(), torch.empty(T, d, device="cuda")
            req = (stage.table, stage.lens, stage.begin)
            A.asf_rotary_append(rot, twins[l], *req, stage.pos, stage.q[l], q, stage.k[l], stage.v[l], ws)
            A.asf_tree_attention_scored(twins[l], *req, q, stage.anc, o, scores[l], ws)
            A.asf_w4_matmul_lora(outs[l], loras[l], stage.which, o.view(T, -1), x, A.Workspace.for_w4(outs[l], T, lora=loras[l]))
            A.asf_w4_sparse_ffn(ffns[l], x, None, None, y, A.Workspace.for_w4(ffns[l], T))
            torch.cuda.synchronize()
            assert torch.equal(x, st.x[l]) and torch.equal(y, st.y[l]) and x.abs().max() > 0
            assert torch.equal(scores[l], stage.scores[l])
            assert torch.equal(twins[l].k, caches[l].k) and torch.equal(twins[l].v, caches[l].v)

    for _ in range(2):
        st.step()
        by_hand()
        stage.lens.add_(stage.begin[1:] - stage.begin[:-1])
        stage.pos.add_(T)
        stage.q.normal_(), stage.k.normal_(), stage.v.normal_()
    fresh = order[R * width:].view(R, width)[:, :8].contiguous()
    keep = 64
    want = torch.zeros(layers, R, hkv, keep, dtype=torch.int32, device="cuda")
    lens, out = torch.empty_like(stage.lens), torch.zeros_like(scores[0])
    for l in range(layers):
        A.asf_kv_evict(twins[l], stage.table, stage.lens, scores[l], keep, fresh, lens, out, want[l], A.Workspace.for_eviction(twins[l]),
                       first=2, recent=20)
        scores[l].copy_(out)
    kept = stage.evict(keep, fresh, first=2, recent=20)
    assert torch.equal(kept, want) and torch.equal(stage.lens, lens) and lens.max() == keep
    assert torch.equal(stage.table[:, :8], fresh) and bool((stage.table[:, 8:] == -1).all()) and torch.equal(stage.scores, scores)
    st.step()                                                # the captured step goes on over what is left
    by_hand()
    assert st.read_error() == 0
    st.release()


def test_stage_refuses_what_does_not_fit():
    ensure_built()
    caches, outs, loras, ffns = _model(2, 1, 2, 2, 64, 16, 8)
    args = (caches, 4, 1, 4, 1)
    for bad in (lambda: A.AttentionStage(*args, outs, rotary=A.Rotary(128)), lambda: A.AttentionStage(*args, adapters=loras),
                lambda: A.AttentionStage(*args, outs, adapters=loras[:1]),
                lambda: A.AttentionStage(*args, outs, adapters=[A.LoraSet(a.A.float(), a.B.float()) for a in loras]),
                lambda: A.AttentionStage(*args, outs).evict(4, torch.zeros(1, 2, dtype=torch.int32, device="cuda")),
                lambda: A.AttentionStage(*args, outs, scored=True).evict(4, torch.zeros(1, 5, dtype=torch.int32, device="cuda")),
                lambda: A.AttentionStage(*args, outs, scored=True).evict(65, torch.zeros(1, 4, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            bad()


@pytest.mark.parametrize("hkv,grp,D,page,turned", [(2, 4, 64, 16, True), (1, 16, 80, 20, True), (3, 8, 128, 64, False)])
def test_drafts_leave_only_what_was_accepted(hkv, grp, D, page, turned):
    """Trees are drafted, some of their tokens accepted: cache and scores are those of decoding the accepted ones, against
    the definition (the tolerance of a key's score is that of tests/test_gpu_scored.py, a rounding more for each
    step that adds to it) and against single calls."""
    ensure_built()
    layers, width, R, T, hq = 2, 12, 2, 8, hkv * grp
    caches, outs, _, ffns = _model(layers, T, hkv, grp, D, page, R * width, adapters=False)
    twins = [A.KVCache(c.k.clone(), c.v.clone()) for c in caches]
    rot = A.Rotary(D, D // 2) if turned else None
    stage = A.AttentionStage(caches, hq, R, width, T, outs, rotary=rot, scored=True, drafts=True)
    st = A.LayerStack([], ffns, T, mode="dense", attention=stage)
    stage.table.copy_(torch.randperm(R * width).int().view(R, width))
    lens, old = [90, 41], torch.rand(stage.scores.shape, device="cuda") * 0.01
    stage.lens.copy_(torch.tensor(lens))
    stage.scores.copy_(old)
    st.capture()
    assert st.kernel_nodes() == st.launches_per_step()
    # (tokens of each request, their parents: -1 the prefix) and what is accepted of them
    trees = [(([-1, 0, 0, 2, 2], [-1, 0, 0]), ([0, 2, 4], [5, 7])), (([-1, -1, 1, 2], [-1, 0, 1, 2]), ([1, 2], [])),
             (([-1], [-1, -1, 1, 2, 2, 0, 0]), ([0], [2, 3, 5]))]
    want, err, step = old.cpu().double().numpy(), np.zeros(old.shape), 0
    table = stage.table.cpu().numpy()
    for parents, accepted in trees:
        begin, anc, depth = [0], [], []
        for tree in parents:
            t0 = begin[-1]
            for i, p in enumerate(tree):
                anc.append((anc[t0 + p] if p >= 0 else 0) | 1 << (t0 + i))
                depth.append(depth[t0 + p] + 1 if p >= 0 else 0)
            begin.append(t0 + len(tree))
        stage.begin.copy_(torch.tensor(begin))
        stage.anc.copy_(torch.tensor(anc))
        stage.pos.copy_(torch.tensor([lens[t >= begin[1]] + d for t, d in enumerate(depth)])) if turned else None
        stage.q.normal_(), stage.k.normal_(), stage.v.normal_()
        before = stage.scores.clone()
        st.step()
        assert torch.equal(stage.scores, before)                             # drafts count for nothing
        stage.accept(accepted)
        for l in range(layers):
            ws = A.Workspace.for_attention(twins[l], hq, R, 1)
            for r in range(R):                                               # token by token
                for i, t in enumerate(accepted[r]):
                    one = lambda x: x[l, t:t + 1].contiguous()  # noqa: E731
                    at = [torch.tensor(v, dtype=torch.int32, device="cuda") for v in (lens, [0, 1, 1] if r == 0 else [0, 0, 1])]
                    at[0][r] += i
                    q = one(stage.q)
                    if turned:
                        A.asf_rotary_append(rot, twins[l], stage.table, *at, stage.pos[t:t + 1], q, q, one(stage.k), one(stage.v), ws)
                    else:
                        A.asf_kv_append(twins[l], stage.table, *at, one(stage.k), one(stage.v), ws)
                    want[l], more = O.received(twins[l].k.cpu().numpy(), table, at[0].tolist(), at[1].tolist(), q.cpu().numpy(),
                                               np.array([1]), D ** -0.5, want[l])
                    err[l] += more
            assert A.asf_read_error(ws) == 0
        lens = [n + len(a) for n, a in zip(lens, accepted)]
        assert stage.lens.tolist() == lens
        step += 1
        got = stage.scores.cpu().double().numpy()
        tol = 2 * 2.0 ** -23 * err + step * 2.0 ** -20 * np.abs(want) + 2.0 ** -100
        for l in range(layers):
            for r in range(R):
                n = lens[r]
                assert (np.abs(got - want) <= tol)[l, r, :, :n].all()
                assert np.array_equal(got[l, r, :, n:], old[l, r, :, n:].cpu().numpy())
                pg, sl = (x.tolist() for x in O.positions(table[r], page, n))
                assert torch.equal(caches[l].k[pg, sl], twins[l].k[pg, sl]) and torch.equal(caches[l].v[pg, sl], twins[l].v[pg, sl])
    assert st.read_error() == 0
    st.release()


def test_accept_refuses():
    ensure_built()
    caches, outs, _, _ = _model(1, 4, 2, 2, 64, 16, 8, adapters=False)
    args = (caches, 4, 2, 4, 4, outs)
    stage = A.AttentionStage(*args, scored=True, drafts=True)
    stage.begin.copy_(torch.tensor([0, 2, 4]))
    stage.table.copy_(torch.arange(8).int().view(2, 4))
    for bad in (lambda: A.AttentionStage(*args, drafts=True), lambda: A.AttentionStage(*args, scored=True).accept([[0], [2]]),
                lambda: stage.accept([[0]]), lambda: stage.accept([[0], [1]]), lambda: stage.accept([[0, 0], [2]]),
                lambda: stage.accept([[-1], []]), lambda: stage.accept([[], [4]])):
        with pytest.raises(ValueError):
            bad()
    stage.accept([[], []])
    assert stage.lens.tolist() == [0, 0] and not stage.scores.any()


def test_capture_leaves_the_scores():
    ensure_built()
    caches, outs, _, ffns = _model(2, 2, 2, 2, 64, 16, 8, adapters=False)
    stage = A.AttentionStage(caches, 4, 1, 8, 2, outs, scored=True)
    st = A.LayerStack([], ffns, 2, mode="dense", attention=stage)
    stage.table.copy_(torch.arange(8).int().view(1, 8))
    stage.lens.fill_(100)
    stage.begin.copy_(torch.tensor([0, 2]))
    stage.anc.copy_(torch.tensor([1, 3]))
    stage.q.normal_(), stage.k.normal_(), stage.v.normal_()
    stage.scores.uniform_()
    before, at = stage.scores.clone(), stage.scores.data_ptr()
    for _ in range(2):                                       # the first time, and in the middle of decoding
        st.capture()
        assert torch.equal(stage.scores, before) and stage.scores.data_ptr() == at
    st.step()
    want = before.clone()
    for l in range(2):
        o, ws = torch.empty_like(stage.q[l]), A.Workspace.for_attention(caches[l], 4, 1, 2, scored_pages=8)
        A.asf_tree_attention_scored(caches[l], stage.table, stage.lens, stage.begin, stage.q[l], stage.anc, o, want[l], ws)
    assert torch.equal(stage.scores, want) and not torch.equal(want, before) and st.read_error() == 0
    st.release()


def test_evict_refuses_a_table_that_keep_does_not_fit():
    ensure_built()
    caches, outs, _, _ = _model(2, 1, 2, 2, 64, 16, 12, adapters=False)
    stage = A.AttentionStage(caches, 4, 1, 8, 1, outs, scored=True)
    table = torch.arange(8).int().view(1, 8).cuda()
    stage.table.copy_(table)
    stage.lens.fill_(120)
    stage.scores.uniform_()
    scores, fresh = stage.scores.clone(), torch.arange(8, 12).int().view(1, 4).cuda()
    for keep, pages in ((17, 1), (64, 3), (65, 4), (128, 4)):
        with pytest.raises(ValueError):
            stage.evict(keep, fresh[:, :pages].contiguous())
        assert torch.equal(stage.table, table) and stage.lens.tolist() == [120] and torch.equal(stage.scores, scores)
    stage.evict(64, fresh)                                   # exactly
    assert stage.lens.tolist() == [64] and A.asf_read_error(stage.ws) == 0


def test_accepting_a_whole_chain_is_a_scored_step():
    """32 tokens (the last one's mask is the sign bit): the same call, so the same bits."""
    ensure_built()
    T, D, page = 32, 64, 16
    caches, outs, _, ffns = _model(2, T, 2, 4, D, page, 16, adapters=False)
    twins = [A.KVCache(c.k.clone(), c.v.clone()) for c in caches]
    stages = [A.AttentionStage(c, 8, 2, 8, T, outs, scored=True, drafts=d) for c, d in ((caches, False), (twins, True))]
    fill = [torch.randn_like(t) for t in (stages[0].q, stages[0].k, stages[0].v)]
    for s in stages:
        s.table.copy_(torch.arange(16).int().view(2, 8))
        s.lens.copy_(torch.tensor([50, 7]))
        s.begin.copy_(torch.tensor([0, 11, 32]))
        s.anc.copy_(torch.tensor([(2 << t) - (1 << (0 if t < 11 else 11)) for t in range(T)]))
        for to, t in zip((s.q, s.k, s.v), fill):
            to.copy_(t)
        st = A.LayerStack([], ffns, T, mode="dense", attention=s)
        st.step()
        if s.drafts:
            s.accept([range(11), range(11, 32)])
            assert s.lens.tolist() == [61, 28]
        assert st.read_error() == 0
    assert torch.equal(stages[0].scores, stages[1].scores) and stages[0].scores.any()
    for a, b in zip(caches, twins):
        assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
