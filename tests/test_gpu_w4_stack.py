"""A decode step of drafted tokens with 4-bit weights, as the layer stack runs
it: append, tree attention, 4-bit output projection, predictor, 4-bit sparse FFN.
Every stage is checked against the float64 oracle on the stage's own input."""
import numpy as np
import pytest
import torch

import oracle as O
import synthetic as S
from oracle import attention as OA
from oracle import w4 as OW
from tests.gpu_util import ensure_built
from tests.test_gpu_attention import Case

import activation_sparse_ffn_predict_b200 as A

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,toks,project,mode,page", [
    ([700], [12], True, "predict", 16), ([90, 0, 33], [1, 2, 1], False, "predict", 16), ([40], [1], True, "dense", 64)])
def test_stack_with_attention_and_w4(lens, toks, project, mode, page):
    ensure_built()
    cfg = S.get("llama2_7b_reglu").with_(d=512, n=1376, r=64, layers=2)
    B, group = sum(toks), 64
    hkv, grp, D = (2, 4, 64) if not project else (3, 2, 80)
    cases = [Case(lens, toks, hkv=hkv, grp=grp, D=D, page=page, seed=l, spread=1.0) for l in range(cfg.layers)]
    preds, ffns, outs, hosts = [], [], [], []
    for l in range(cfg.layers):
        w = S.layer_weights(cfg, l)
        hosts.append(w.numpy())
        d = w.to("cuda")
        preds.append(A.Predictor(d.W1, d.b1, d.W2, d.b2))
        ffns.append(A.W4FFN.quantize(d.act, d.Wg, d.Wu, d.WdT, d.bias, group))
        if project:
            outs.append(A.W4Matrix.quantize(torch.randn(cfg.d, hkv * grp * D, device="cuda") * (12 / (hkv * grp * D)) ** 0.5,
                                            group))
    caches = [A.KVCache(torch.from_numpy(c.k.copy()).cuda(), torch.from_numpy(c.v.copy()).cuda()) for c in cases]
    stage = A.AttentionStage(caches, hkv * grp, len(lens), cases[0].table.shape[1], B, outs if project else None)
    st = A.LayerStack(preds, ffns, B, cfg.tau, mode=mode, attention=stage)
    dev = [c.device() for c in cases]
    for l, d in enumerate(dev):
        stage.q[l].copy_(d["q"])
        stage.k[l].copy_(d["kn"])
        stage.v[l].copy_(d["vn"])
    for n in ("lens", "begin", "anc"):
        getattr(stage, n).copy_(dev[0][n])
        assert torch.equal(dev[0][n], dev[1][n]) or n == "anc"
    table = dev[0]["table"]
    stage.table.copy_(table)
    st.capture()
    assert st.kernel_nodes() == st.launches_per_step()
    for step in range(2):
        st.step()
        torch.cuda.synchronize()
        for l, c in enumerate(cases):
            k, v = c.k.copy(), c.v.copy()
            OA.append(k, v, cases[0].table, c.lens, c.begin, c.kn, c.vn)
            o, mass, _ = OA.tree_attention(k, v, cases[0].table, c.lens, c.begin, c.q, cases[0].anc, D ** -0.5)
            x = st.x[l].double().cpu().numpy()
            if project:
                W = OW.w4_unpack(outs[l].data.cpu().numpy(), hkv * grp * D, group)
                ref, slack = o.reshape(B, -1) @ W.T, mass.reshape(B, -1) @ np.abs(W).T
            else:
                ref, slack = o.reshape(B, -1), mass.reshape(B, -1)
            # attention's own rounding and its weights' (2^-11 each), then x's: 2^-11
            assert np.all(np.abs(x - ref) <= 3 * 2.0 ** -11 * slack + 2.0 ** -11 * np.abs(ref) + 2.0 ** -22)
            h = hosts[l]
            if mode == "predict":
                got = st.idx[l, :int(st.count[l])].cpu().numpy()
                z = O.predictor_logits(h["W1"], h["b1"], h["W2"], h["b2"], x)
                sure = np.abs(z - O.logit(cfg.tau)) > O.predictor_band(h["W1"], h["b1"], h["W2"], h["b2"], x, cfg.tau)
                on = z > O.logit(cfg.tau)
                assert set(np.flatnonzero((on & sure).any(0))) <= set(got) <= set(np.flatnonzero((on | ~sure).any(0)))
            else:
                got = np.arange(cfg.n)
            ref = OW.w4_ffn(h["act"], ffns[l].data.cpu().numpy(), h["bias"], cfg.d, group, x, got)
            y = st.y[l].double().cpu().numpy()
            assert np.abs(y - ref).max() <= 1e-5 * np.abs(ref).max()         # fp32 sums: the fp32 layer's bar
        assert st.read_error() == 0
    st.release()


def test_stack_refuses_what_does_not_fit():
    ensure_built()
    cfg = S.get("tiny_reglu_f32").with_(layers=1)
    w = S.layer_weights(cfg, 0).to("cuda")
    pred = A.Predictor(w.W1, w.b1, w.W2, w.b2)
    ffn, w4 = A.FFN(w.act, w.Wg, w.Wu, w.WdT, w.bias), A.W4FFN.quantize(w.act, w.Wg, w.Wu, w.WdT, w.bias, 32)
    k = torch.zeros(2, 16, 2, 64, dtype=torch.float16, device="cuda")
    stage = A.AttentionStage([A.KVCache(k, k.clone())], 8, 1, 2, 1)
    for bad in (lambda: A.LayerStack([pred] * 2, [ffn, w4], 1), lambda: A.LayerStack([pred], [w4], 1, attention=stage),
                lambda: A.LayerStack([None], [w4], 2, mode="sparse", attention=stage),
                lambda: A.AttentionStage([A.KVCache(k, k.clone())], 8, 1, 2, 1, out=[])):
        with pytest.raises(ValueError):
            bad()
    st = A.LayerStack([pred], [w4], 3)                      # fp32 predictor and 4-bit rows: fp32 x
    assert st.x.dtype == torch.float32
    st.x.normal_()
    st.step()
    got = st.idx[0, :int(st.count[0])].cpu().numpy()
    ref = OW.w4_ffn("reglu", w4.data.cpu().numpy(), w.bias.cpu().numpy(), cfg.d, 32, st.x[0].double().cpu().numpy(), got)
    assert np.abs(st.y[0].cpu().numpy() - ref).max() <= 1e-5 * np.abs(ref).max() and st.read_error() == 0


def test_calls_on_two_streams_at_once():
    """Products and attention side by side, each with its own workspace: the same bits as one after the other."""
    ensure_built()
    torch.manual_seed(3)
    mat = A.W4Matrix.quantize(torch.randn(12000, 4096, device="cuda"), 64)
    x, out = torch.randn(24, 4096, device="cuda").half(), torch.empty(24, 12000, device="cuda")
    ffn = A.W4FFN.quantize("relu", None, torch.randn(900, 2048, device="cuda"), torch.randn(900, 2048, device="cuda"),
                           torch.zeros(900, device="cuda"), 128)
    xf, y = torch.randn(16, 2048, device="cuda").half(), torch.empty(16, 2048, device="cuda")
    c = Case([3000, 17], [20, 2], hkv=4, grp=8, D=128, page=64, seed=5)
    d = c.run()
    wm, wf = A.Workspace.for_w4(mat, 24), A.Workspace.for_w4(ffn, 16)

    def one():
        A.asf_w4_matmul(mat, x, out, wm)
        A.asf_w4_sparse_ffn(ffn, xf, None, None, y, wf)

    one()
    torch.cuda.synchronize()
    want = [t.clone() for t in (out, y, d["o"])]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for t in (out, y, d["o"]):
            t.zero_()
        torch.cuda.synchronize()
        for _ in range(20):
            with torch.cuda.stream(streams[0]):
                one()
            with torch.cuda.stream(streams[1]):
                c.run(d)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (out, y, d["o"])))
    assert A.asf_read_error(wm) == A.asf_read_error(wf) == A.asf_read_error(d["ws"]) == 0


@pytest.mark.parametrize("mode", ["predict", "dense"])
def test_layers_of_different_groups_and_widths(mode):
    """Every later layer needs more workspace than the one before: the same bits as single calls with workspaces of their own."""
    ensure_built()
    torch.manual_seed(12)
    d, B, D, hq, T = 512, 9, 64, 8, 9
    half = lambda *s: torch.randn(*s, device="cuda").half()  # noqa: E731
    preds, ffns, outs, caches = [], [], [], []
    for n, r, group, act in ((600, 64, 128, "relu"), (20000, 96, 64, "relu"), (30000, 160, 32, "reglu")):
        preds.append(A.Predictor(half(r, d) * d ** -0.5, torch.zeros(r, device="cuda"), half(n, r) * r ** -0.5,
                                 torch.full((n,), -0.1, device="cuda")))
        ffns.append(A.W4FFN.quantize(act, half(n, d) * d ** -0.5, half(n, d) * d ** -0.5, half(n, d) * d ** -0.5,
                                     torch.zeros(n, device="cuda"), group))
        outs.append(A.W4Matrix.quantize(half(d, hq * D) * (hq * D) ** -0.5, group))
        caches.append(A.KVCache(half(4, 64, 2, D), half(4, 64, 2, D)))
    assert sorted(f.workspace_bytes(B) for f in ffns) == [f.workspace_bytes(B) for f in ffns]
    stage = A.AttentionStage(caches, hq, 1, 4, B, outs)
    stage.q.normal_(), stage.k.normal_(), stage.v.normal_()
    stage.table.copy_(torch.arange(4)[None])
    stage.lens.fill_(100)
    stage.begin[1] = T
    stage.anc.copy_((2 ** (torch.arange(T) + 1) - 1).int())
    st = A.LayerStack(preds, ffns, B, 0.5, mode=mode, attention=stage)
    assert st.idx.shape == (3, 30000)
    st.capture()
    st.step()
    for l in range(3):
        x, y = torch.empty(B, d, device="cuda").half(), torch.empty(B, d, device="cuda")
        o = torch.empty(B, hq, D, device="cuda").half()
        A.asf_tree_attention(caches[l], stage.table, stage.lens, stage.begin, stage.q[l], stage.anc, o,
                             A.Workspace.for_attention(caches[l], hq, 1, B))
        A.asf_w4_matmul(outs[l], o.view(B, -1), x, A.Workspace.for_w4(outs[l], B))
        assert torch.equal(x, st.x[l]) and x.abs().max() > 0
        idx, cnt = torch.zeros(ffns[l].n, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        if mode == "predict":
            A.asf_predict(preds[l], x, 0.5, idx, cnt, A.Workspace(preds[l], None, B))
            c = int(cnt)
            assert c == int(st.count[l]) > 0 and torch.equal(idx[:c], st.idx[l, :c])
        A.asf_w4_sparse_ffn(ffns[l], x, *((idx, cnt) if mode == "predict" else (None, None)), y,
                            A.Workspace.for_w4(ffns[l], B))
        assert torch.equal(y, st.y[l])
    assert st.read_error() == 0
    st.release()
