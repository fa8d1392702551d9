"""Rotary positions on the GPU against the oracle.

Tolerance, elementwise, with S = scale (|u| + |w|) of the pair: the angle's fraction
of a half turn in fp32, pi 2^-25; sincospi, 2 units in the last place, 2^-23; the
scaled cosine and the two products, a rounding of 2^-24 each; together below 2^-21 S.
Then the output's rounding: half a step, 2^-25 at least in fp16.
"""
import numpy as np
import pytest
import torch

from oracle import attention as OA
from oracle import rotary as O
from tests.gpu_util import ensure_built

import activation_sparse_ffn_predict_b200 as A
from activation_sparse_ffn_predict_b200 import _lib as L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def _check(got, x, pos, rot, layout):
    """got and x: tensors [T, heads, D]."""
    xn = x.cpu().double().numpy()
    want, size = O.turn(xn, pos, rot.frequencies, rot.scale, layout)
    half = torch.finfo(got.dtype).eps / 2
    tol = 2.0 ** -21 * abs(rot.scale) * size + half * np.abs(want) + (2.0 ** -25 if got.dtype == torch.float16 else 0)
    g = got.cpu().double().numpy()
    n = rot.rot_dim
    assert (np.abs(g - want) <= tol)[..., :n].all(), np.abs(g - want)[..., :n].max()
    assert np.array_equal(g[..., n:], xn[..., n:], equal_nan=True)


def _x(T, heads, D, dtype, seed=0):
    return torch.randn(T, heads, D, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("T,heads,D,rot", [
    (1, 1, 8, 8), (1, 1, 8, 2), (1, 72, 128, 128), (3, 5, 80, 36), (33, 7, 64, 16), (1000, 9, 128, 64), (257, 36, 80, 80),
    (5, 130, 72, 6), (2, 3, 512, 512), (7, 1, 512, 2), (4, 2, 512, 510), (2000, 1, 64, 64), (64, 300, 40, 40), (9, 40, 24, 16)])
def test_against_the_definition(T, heads, D, rot, dtype, layout):
    r = A.Rotary(D, rot, layout=layout, scaling="yarn", factor=4.0)
    x = _x(T, heads, D, dtype)
    pos = torch.randint(0, 100000, (T,), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    y = torch.full_like(x, 7.0)
    A.asf_rotary_apply(r, x, pos.cuda(), y)
    _check(y, x, pos.numpy(), r, layout)
    keep = x.clone()
    A.asf_rotary_apply(r, x, pos.cuda(), x)                  # in place: the same bits
    assert torch.equal(x, y)
    _check(x, keep, pos.numpy(), r, layout)


@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_far_and_negative_positions(layout):
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 10 ** 6 + 7, 12345678, -999999937], dtype=torch.int32)
    r = A.Rotary(128, layout=layout, base=500000.0)
    x = _x(len(pos), 4, 128, torch.float32)
    y = torch.empty_like(x)
    A.asf_rotary_apply(r, x, pos.cuda(), y)
    _check(y, x, pos.numpy(), r, layout)
    back = torch.empty_like(x)
    A.asf_rotary_apply(r, y, torch.where(pos == -2 ** 31, pos, -pos).cuda(), back)
    ok = pos != -2 ** 31
    assert (back[ok] - x[ok]).abs().max() < 2 ** -20 * 4 * x.abs().max()   # two turns of 2^-21 (|u| + |w|), |u| + |w| <= 2 max


def test_given_frequencies_and_scale():
    f = [1.0, 0.0, -0.3, 1e-9]
    r = A.Rotary(16, 8, frequencies=f, scale=-2.5)
    assert r.frequencies == f
    x, pos = _x(6, 3, 16, torch.float32), np.arange(6, dtype=np.int32) * 1000
    y = torch.empty_like(x)
    A.asf_rotary_apply(r, x, torch.from_numpy(pos).cuda(), y)
    _check(y, x, pos, r, "half")


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_slices_and_layouts(dtype):
    r = A.Rotary(64, 48)
    joint = _x(50, 24, 64, dtype)
    pos = torch.arange(50, dtype=torch.int32)
    x, before = joint[:, 8:20], joint.clone()
    y = torch.empty(12, 50, 64, dtype=dtype, device="cuda").transpose(0, 1)   # head by head
    A.asf_rotary_apply(r, x, pos.cuda(), y)
    _check(y, x, pos.numpy(), r, "half")
    A.asf_rotary_apply(r, x, pos.cuda(), x)                  # in place in the joint tensor: its other heads stay
    assert torch.equal(x, y) and torch.equal(joint[:, :8], before[:, :8]) and torch.equal(joint[:, 20:], before[:, 20:])
    one = before[:, :1].expand(50, 5, 64)                    # an input whose heads are one and the same
    y = torch.empty(50, 5, 64, dtype=dtype, device="cuda")
    A.asf_rotary_apply(r, one, pos.cuda(), y)
    _check(y, one, pos.numpy(), r, "half")


def test_what_passes_keeps_its_bits():
    r = A.Rotary(32, 12)
    x = _x(4, 3, 32, torch.float16)
    raw = x.view(torch.int16)
    raw[..., 12:] = torch.randint(-2 ** 15, 2 ** 15, raw[..., 12:].shape, device="cuda", dtype=torch.int16)   # NaN among them
    y = torch.empty_like(x)
    A.asf_rotary_apply(r, x, torch.arange(4, dtype=torch.int32, device="cuda"), y)
    assert torch.equal(y.view(torch.int16)[..., 12:], raw[..., 12:])


def test_offsets_past_32_bits():
    r = A.Rotary(128)
    T, big = 3, 2 ** 30 + 64                                 # tokens 2 GB apart
    flat = torch.empty(2 * big + 2 * 128, dtype=torch.float16, device="cuda")
    x = torch.as_strided(flat, (T, 2, 128), (big, 128, 1))
    small = _x(T, 2, 128, torch.float16)
    x.copy_(small)
    pos = torch.tensor([5, 6, 7], dtype=torch.int32)
    A.asf_rotary_apply(r, x, pos.cuda(), x)
    _check(x, small, pos.numpy(), r, "half")


def test_streams_and_graphs():
    r = A.Rotary(128)
    x, pos = _x(40, 8, 128, torch.float16), torch.arange(40, dtype=torch.int32, device="cuda")
    want, y = torch.empty_like(x), torch.empty_like(x)
    A.asf_rotary_apply(r, x, pos, want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        A.asf_rotary_apply(r, x, pos, y)
    side.synchronize()
    assert torch.equal(y, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        A.asf_rotary_apply(r, x, pos, y)
    x2 = _x(40, 8, 128, torch.float16, seed=5)
    x.copy_(x2)
    pos.add_(100)
    g.replay()
    torch.cuda.synchronize()
    _check(y, x2, pos.cpu().numpy(), r, "half")


def test_binding_refuses():
    r = A.Rotary(64)
    x, pos = _x(4, 2, 64, torch.float16), torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (lambda: A.asf_rotary_apply(r, x[..., :32], pos, x[..., :32]), lambda: A.asf_rotary_apply(r, x, pos[:3], x),
                lambda: A.asf_rotary_apply(r, x, pos.long(), x), lambda: A.asf_rotary_apply(r, x, pos, x.float()),
                lambda: A.asf_rotary_apply(r, x.double(), pos, x.double()), lambda: A.asf_rotary_apply(r, x.cpu(), pos, x),
                lambda: A.asf_rotary_apply(r, x.transpose(1, 2)[:, :, :2], pos, x),
                lambda: A.Rotary(64, 63), lambda: A.Rotary(64, 66), lambda: A.Rotary(64, layout="both"),
                lambda: A.Rotary(64, device="cpu"), lambda: A.Rotary(64, frequencies=[1.0])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(A.AsfError):
        A.asf_rotary_apply(r, x, pos, x[:1].expand(4, 2, 64))            # y's tokens meet
    with pytest.raises(A.AsfError):
        A.Rotary(64, base=0.5)


# ------------------------------------------------------------- append --
def _append_case(lens, toks, hkv, grp, D, page, seed=0):
    rng = np.random.default_rng(seed)
    begin = np.concatenate([[0], np.cumsum(toks)]).astype(np.int32)
    need = [-(-(n + m) // page) for n, m in zip(lens, toks)]
    pages = sum(need) + 2
    order, table, at = rng.permutation(pages), np.zeros((len(lens), max(1, max(need))), np.int32), 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n]
        at += n
    T = int(begin[-1])
    f16 = lambda *s: rng.standard_normal(s).astype(np.float16)  # noqa: E731
    return dict(k=f16(pages, page, hkv, D), v=f16(pages, page, hkv, D), qkv=f16(T, hkv * (grp + 2), D), table=table,
                lens=np.array(lens, np.int32), begin=begin, pos=rng.integers(0, 200000, T).astype(np.int32), hq=hkv * grp)


def _run_append(c, rot, joint=True, T=None):
    cu = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    hkv, hq = c["k"].shape[2], c["hq"]
    cache = A.KVCache(cu(c["k"]), cu(c["v"]))
    parts = cu(c["qkv"]).split([hq, hkv, hkv], 1)
    if not joint:
        parts = [p.contiguous() for p in parts]
    out = torch.full_like(parts[0].contiguous(), 7.0) if joint else parts[0]       # in place where q is contiguous
    ws = A.Workspace.for_attention(cache, hq, len(c["lens"]), len(c["pos"]))
    A.asf_rotary_append(rot, cache, cu(c["table"]), cu(c["lens"]), cu(c["begin"]), cu(c["pos"]), parts[0], out, *parts[1:], ws)
    return cache, out, ws


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("joint", [True, False])
@pytest.mark.parametrize("lens,toks,hkv,grp,D,rot,page", [
    ([0], [1], 1, 1, 8, 8, 1), ([33], [1], 8, 8, 128, 128, 16), ([5, 0, 130], [3, 2, 1], 2, 2, 80, 36, 20),
    (list(range(0, 640, 20)), [1] * 32, 8, 8, 128, 64, 16), ([700, 20, 9], [8, 0, 16], 2, 16, 64, 2, 7), ([100], [32], 1, 71, 64, 64, 64)])
def test_append_against_the_definition(lens, toks, hkv, grp, D, rot, page, joint, layout):
    c = _append_case(lens, toks, hkv, grp, D, page, seed=sum(lens))
    r = A.Rotary(D, rot, layout=layout)
    cache, q, ws = _run_append(c, r, joint)
    hq = c["hq"]
    x = torch.from_numpy(c["qkv"])
    _check(q, x[:, :hq], c["pos"], r, layout)
    # the rows that the append writes hold turned keys; every other row, and all values, are kv_append's
    k, v = c["k"].copy(), c["v"].copy()
    got_k = cache.k.cpu()
    for i, n in enumerate(lens):
        for j, t in enumerate(range(c["begin"][i], c["begin"][i + 1])):
            at = (c["table"][i, (n + j) // page], (n + j) % page)
            _check(got_k[at][None], x[t:t + 1, hq:hq + hkv], c["pos"][t:t + 1], r, layout)
            k[at] = got_k[at].numpy()
    OA.append(k.copy(), v, c["table"], c["lens"], c["begin"], c["qkv"][:, hq:hq + hkv], c["qkv"][:, hq + hkv:])
    assert np.array_equal(got_k.numpy(), k) and np.array_equal(cache.v.cpu().numpy(), v)
    assert A.asf_read_error(ws) == 0


def test_append_is_apply_and_kv_append():
    c = _append_case([100, 7], [5, 9], 4, 4, 64, 16, seed=3)
    r = A.Rotary(64, 32, layout="pairs", scaling="ntk", factor=4.0)
    cache, q, ws = _run_append(c, r)
    cu = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    pos, x = cu(c["pos"]), cu(c["qkv"])
    A.asf_rotary_apply(r, x[:, :20], pos, x[:, :20])         # queries and keys
    other = A.KVCache(cu(c["k"]), cu(c["v"]))
    A.asf_kv_append(other, cu(c["table"]), cu(c["lens"]), cu(c["begin"]), x[:, 16:20].contiguous(), x[:, 20:].contiguous(), ws)
    assert torch.equal(q, x[:, :16]) and torch.equal(cache.k, other.k) and torch.equal(cache.v, other.v)


def test_append_leaves_what_is_behind_and_flags_what_is_bad():
    c = _append_case([40, 3], [4, 5], 2, 2, 64, 16, seed=4)
    r = A.Rotary(64)
    c["begin"][:] = [0, 4, 7]                                # tokens 7 and 8 behind the last range
    cache, q, ws = _run_append(c, r)
    assert (q[7:] == 7.0).all() and A.asf_read_error(ws) == 0
    pg, sl = OA.positions(c["table"][1], 16, 8)
    assert np.array_equal(cache.k.cpu().numpy()[pg[6:], sl[6:]], c["k"][pg[6:], sl[6:]])
    c["table"][0, 2] = len(c["k"]) + 9                       # positions 32..47 of request 0
    cache, q, ws = _run_append(c, r)
    assert A.asf_read_error(ws) == L.ASF_ERR_DEVICE_INDEX
    own = np.unique(pg)
    rest = np.setdiff1d(np.arange(len(c["k"])), own)
    assert np.array_equal(cache.k.cpu().numpy()[rest], c["k"][rest])
    _check(q[:7], torch.from_numpy(c["qkv"])[:7, :4], c["pos"][:7], r, "half")
    for bad in (dict(begin=np.array([3, 1, 7], np.int32)), dict(lens=np.array([-5, 3], np.int32)),
                dict(lens=np.array([10 ** 6, 3], np.int32))):
        d = dict(_append_case([40, 3], [4, 5], 2, 2, 64, 16, seed=4), **bad)
        cache, q, ws = _run_append(d, r)
        assert A.asf_read_error(ws) == L.ASF_ERR_DEVICE_INDEX


def test_append_binding_refuses():
    c = _append_case([40], [4], 2, 2, 64, 16)
    cu = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    cache = A.KVCache(cu(c["k"]), cu(c["v"]))
    ws = A.Workspace.for_attention(cache, 4, 1, 4)
    q, k, v = cu(c["qkv"]).split([4, 2, 2], 1)
    req = (cu(c["table"]), cu(c["lens"]), cu(c["begin"]))
    r, pos = A.Rotary(64), cu(c["pos"])
    A.asf_rotary_append(r, cache, *req, pos, q, torch.empty_like(q.contiguous()), k, v, ws)
    for args in ((pos[:2], q, torch.empty(4, 4, 64).half().cuda(), k, v), (pos, q, q, k, v), (pos, q, q.contiguous(), k[:3], v),
                 (pos, q, q.contiguous(), k, v[:, :1]), (pos, q.transpose(0, 1), q.contiguous(), k, v),
                 (pos, q.float(), q.contiguous(), k, v), (pos, q, q.contiguous().cpu(), k, v)):
        with pytest.raises(ValueError):
            A.asf_rotary_append(r, cache, *req, *args, ws)
    with pytest.raises(A.AsfError):
        A.asf_rotary_append(A.Rotary(128), cache, *req, pos, q, q.contiguous(), k, v, ws)
