"""4-bit rows on the GPU against the float64 oracle: the format byte by byte,
the dense product and the sparse FFN.

Tolerances.  Products of a code and an operand are exact, and so are a group's
(c - 8) x terms; what rounds is the fp32 accumulation: a chain of at most 3 x 8
tensor-core steps inside a group (2^-23 of the partial sum each, truncated),
then one fused multiply-add per group (2^-24), then the sums of the splits.
Against sum |w x| =: M, elementwise, |error| <= (24 + groups + 256) 2^-23 M.
"""
import numpy as np
import pytest
import torch

from oracle import w4 as O
from tests.gpu_util import ensure_built

import activation_sparse_ffn_predict_b200 as A
from activation_sparse_ffn_predict_b200 import _lib as L

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def _weights(m, k, seed, std=1.0):
    return (np.random.default_rng(seed).standard_normal((m, k)) * std / np.sqrt(k)).astype(np.float32)


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("m,k,group", [(1, 8, 32), (5, 128, 128), (3, 136, 64), (17, 512, 32), (9, 1000, 32),
                                       (4, 1096, 128), (33, 4096, 64)])
def test_quantize_is_the_definition(m, k, group, dt):
    W = _weights(m, k, k + group)
    W[0] *= 1e-9                                            # scales underflow: zeros
    if m > 2:
        W[1, :k // 2] = 0
        W[2, 0], W[2, k - 1] = 6e4 if dt == "f16" else 4e5, np.nan
    src = torch.from_numpy(W).to(DT[dt]).cuda()
    data = torch.full((m, O.row_bytes(k, group) + 16), 0xAB, dtype=torch.uint8, device="cuda")   # a wider stride
    mat = A.W4Matrix(data, k, group)
    A.asf_w4_quantize(src, mat)
    want = O.w4_pack(src.float().cpu().numpy(), group)
    got = data.cpu().numpy()
    rb = O.row_bytes(k, group)
    nan = np.isnan(want[:, O.padded(k) // 2:].copy().view(np.float16))
    sc = got[:, O.padded(k) // 2:rb].copy().view(np.float16)
    assert np.array_equal(np.isnan(sc), nan)                # a NaN scale may have any NaN's bits
    same = got[:, :rb] == want
    same[:, O.padded(k) // 2:] |= np.repeat(nan, 2, axis=1)
    assert same.all()
    assert (got[:, rb:] == 0xAB).all()                      # behind the row: untouched
    back = torch.empty(m, k, dtype=DT[dt], device="cuda")
    A.asf_w4_dequantize(mat, back)
    ref = O.w4_unpack(got[:, :rb], k, group)
    with np.errstate(over="ignore"):
        assert np.array_equal(back.cpu().numpy(), ref.astype(back.cpu().numpy().dtype), equal_nan=True)


def _check(y, ref, mass, groups):
    y = y.cpu().numpy().astype(np.float64)
    assert np.isfinite(y).all()
    over = np.abs(y - ref) - (24 + groups + 256) * 2.0 ** -23 * mass
    assert over.max() <= 0, (over.max(), np.abs(y - ref).max(), np.abs(ref).max())


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("m,k,group,B", [
    (1, 8, 32, 1), (16, 128, 128, 1), (17, 136, 64, 2), (31, 520, 32, 8), (1003, 1376, 32, 3), (64, 4096, 128, 1),
    (256, 8192, 64, 9), (40, 12288, 128, 17), (129, 2760, 64, 32), (5000, 512, 128, 5), (24, 49152, 128, 32),
    (2500, 4096, 64, 24), (48, 1024, 128, 18),
    (33, 640, 32, 25)])
def test_matmul(m, k, group, B, dt):
    rng = np.random.default_rng(m * k + B)
    rows = O.w4_pack(_weights(m, k, m + k), group)
    x = torch.from_numpy(rng.standard_normal((B, k)).astype(np.float32)).to(DT[dt])
    bias = rng.standard_normal(m).astype(np.float32)
    mat = A.W4Matrix(torch.from_numpy(rows).cuda(), k, group)
    ws = A.Workspace.for_w4(mat, B)
    W = O.w4_unpack(rows, k, group)
    xn = x.double().numpy()
    mass = np.abs(xn) @ np.abs(W).T + np.abs(bias)
    for use_bias, relu in ((False, False), (True, True)):
        y = torch.full((B, m), float("nan"), device="cuda")
        A.asf_w4_matmul(mat, x.cuda(), y, ws, bias=torch.from_numpy(bias).cuda() if use_bias else None, relu=relu)
        ref = xn @ W.T + (bias if use_bias else 0)
        _check(y, np.maximum(ref, 0) if relu else ref, mass, k // group + 1)
        again = torch.full((B, m), float("nan"), device="cuda")
        A.asf_w4_matmul(mat, x.cuda(), again, ws, bias=torch.from_numpy(bias).cuda() if use_bias else None, relu=relu)
        assert torch.equal(y, again)                        # fixed summation order
        half = torch.empty(B, m, device="cuda", dtype=torch.float16)
        A.asf_w4_matmul(mat, x.cuda(), half, ws, bias=torch.from_numpy(bias).cuda() if use_bias else None, relu=relu)
        assert torch.equal(half, y.half())                  # the same sum, rounded once
    assert A.asf_read_error(ws) == 0


@pytest.mark.parametrize("m,k,group,B,pad", [
    (34000, 4096, 128, 1, 0), (20011, 6920, 32, 3, 48), (12345, 12296, 64, 8, 0), (9001, 8712, 32, 13, 16),
    (19000, 4096, 128, 16, 0), (1270, 65536, 64, 16, 0), (5000, 9608, 32, 32, 0), (12000, 4104, 64, 17, 32),
    (100000, 264, 128, 29, 0), (200000, 8, 128, 20, 0), (25000, 2048, 64, 31, 0)])
def test_matmul_of_many_rows(m, k, group, B, pad):
    """fp16 x and enough rows for the product in tensor memory, against float64 products of the dequantised weights."""
    torch.manual_seed(m)
    W = torch.randn(m, k, device="cuda") * torch.exp2(torch.randint(-3, 3, (m, 1), device="cuda").float())
    rb = A.asf_w4_row_bytes(k, group)
    mat = A.W4Matrix(torch.full((m, rb + pad), 0xff, dtype=torch.uint8, device="cuda"), k, group)
    A.asf_w4_quantize(W, mat)
    assert (mat.data[:, rb:] == 0xff).all()
    A.asf_w4_dequantize(mat, W)                             # exact in fp32
    x = torch.randn(B, k, device="cuda").half()
    bias = torch.randn(m, device="cuda")
    ws = A.Workspace.for_w4(mat, B)
    ref, mass = torch.empty(B, m, device="cuda", dtype=torch.float64), torch.empty(B, m, device="cuda", dtype=torch.float64)
    for i in range(0, m, 8192):
        w = W[i:i + 8192].double().t()
        ref[:, i:i + 8192], mass[:, i:i + 8192] = x.double() @ w, x.double().abs() @ w.abs()
    for use_bias, relu in ((False, False), (True, True)):
        kw = dict(bias=bias if use_bias else None, relu=relu)
        want = ref + (bias.double() if use_bias else 0)
        want = want.clamp(min=0) if relu else want
        y, again = (torch.full((B, m), float("nan"), device="cuda") for _ in range(2))
        A.asf_w4_matmul(mat, x, y, ws, **kw)
        _check(y, want.cpu().numpy(), (mass + bias.double().abs()).cpu().numpy(), k // group + 1)
        A.asf_w4_matmul(mat, x, again, ws, **kw)
        assert torch.equal(y, again)
        half = torch.empty(B, m, device="cuda", dtype=torch.float16)
        A.asf_w4_matmul(mat, x, half, ws, **kw)
        assert torch.equal(half, y.half())
    if B > 1:                                               # a token of NaN and infinities is its own affair
        x[B - 1, 0], x[B - 1, k - 1] = float("nan"), float("inf")
        A.asf_w4_matmul(mat, x, again, ws, bias=bias, relu=True)
        assert torch.equal(y[:B - 1], again[:B - 1]) and torch.isnan(again[B - 1]).all()
    assert A.asf_read_error(ws) == 0


def test_matmul_of_many_rows_in_a_graph_on_another_stream():
    m, k, B = 12000, 4104, 24
    mat = A.W4Matrix.quantize(torch.randn(m, k, device="cuda"), 64)
    ws = A.Workspace.for_w4(mat, B)
    x, y = torch.randn(B, k, device="cuda").half(), torch.empty(B, m, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        A.asf_w4_matmul(mat, x, y, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        A.asf_w4_matmul(mat, x, y, ws)
    for seed in range(3):
        x.copy_(torch.randn(B, k))
        graph.replay()
        got = y.clone()
        A.asf_w4_matmul(mat, x, y, ws)
        assert torch.equal(got, y)


def _layer(act, n, d, group, seed):
    mats = 3 if act == "reglu" else 2
    data = np.stack([O.w4_pack(_weights(n, d, seed + i), group) for i in range(mats)], 1)
    bias = (np.random.default_rng(seed).standard_normal(n) * 0.3).astype(np.float32)
    return data, bias


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("act,n,d,group,B,active", [
    ("reglu", 1376, 512, 32, 1, 140), ("relu", 1376, 512, 32, 2, 1), ("reglu", 300, 1096, 64, 8, 0),
    ("relu", 500, 136, 128, 9, 500), ("reglu", 700, 2048, 128, 17, 333), ("relu", 260, 4096, 64, 32, 100),
    ("reglu", 64, 8, 32, 4, 17), ("reglu", 200, 8192, 128, 3, 77), ("relu", 120, 12288, 32, 16, 120),
    ("reglu", 900, 1032, 64, 10, 700), ("relu", 3000, 264, 128, 12, 2900), ("reglu", 130, 4096, 32, 32, 65),
    ("relu", 400, 2560, 64, 30, 129), ("reglu", 257, 264, 128, 25, 256), ("relu", 70, 8, 32, 9, 70)])
def test_sparse_ffn(act, n, d, group, B, active, dt):
    rng = np.random.default_rng(n + d)
    data, bias = _layer(act, n, d, group, n)
    x = torch.from_numpy(rng.standard_normal((B, d)).astype(np.float32)).to(DT[dt])
    ids = np.sort(rng.choice(n, active, replace=False)).astype(np.int32)
    ffn = A.W4FFN(act, torch.from_numpy(data).cuda(), torch.from_numpy(bias).cuda(), d, group)
    ws = A.Workspace.for_w4(ffn, B)
    idx = torch.full((n,), 1 << 30, dtype=torch.int32, device="cuda")       # past the count: never read
    idx[:active] = torch.from_numpy(ids).cuda()
    cnt = torch.tensor([active], dtype=torch.int32, device="cuda")
    y = torch.full((B, d), float("nan"), device="cuda")
    A.asf_w4_sparse_ffn(ffn, x.cuda(), idx, cnt, y, ws)
    _check_ffn(y, act, data, bias, d, group, x.double().numpy(), ids)
    y2 = torch.full((B, d), float("nan"), device="cuda")
    A.asf_w4_sparse_ffn(ffn, x.cuda(), idx, cnt, y2, ws)
    assert torch.equal(y, y2)
    if active == n:                                                           # all neurons: the dense form
        A.asf_w4_sparse_ffn(ffn, x.cuda(), None, None, y2, ws)
        assert torch.equal(y, y2)
    assert A.asf_read_error(ws) == 0


def _check_ffn(y, act, data, bias, d, group, xn, ids):
    """Error of an activation, by the product's bound, then of the sum over them."""
    ref = O.w4_ffn(act, data, bias, d, group, xn, ids)
    y = y.cpu().numpy().astype(np.float64)
    if len(ids) == 0:
        assert (y == 0).all()
        return
    W = O.w4_unpack(data[ids], d, group)
    u = (24 + d // group + 1 + 256) * 2.0 ** -23
    z = [xn @ W[:, i].T + (bias[ids] if i == 0 else 0) for i in range(W.shape[1] - 1)]
    m = [np.abs(xn) @ np.abs(W[:, i]).T + (np.abs(bias[ids]) if i == 0 else 0) for i in range(W.shape[1] - 1)]
    a = np.maximum(z[0], 0)
    da = u * m[0]
    if act == "reglu":
        da = da * np.abs(z[1]) + np.abs(a) * u * m[1] + da * u * m[1]
        a = a * z[1]
    # down: three tensor-core steps of 2^-23 per 16 neurons, and the sums of warps and splits
    v = (3 * len(ids) / 16 + 3 + 300) * 2.0 ** -23
    tol = (da + v * (np.abs(a) + da)) @ np.abs(W[:, -1])
    assert np.isfinite(y).all()
    assert (np.abs(y - ref) - tol).max() <= 0, (np.abs(y - ref).max(), np.abs(ref).max())


@pytest.mark.parametrize("B", [3, 11, 29])
def test_errors_of_the_list_are_flagged_and_skipped(B):
    n, d, group = 96, 256, 64
    data, bias = _layer("reglu", n, d, group, 5)
    x = torch.randn(B, d).half()
    ffn = A.W4FFN("reglu", torch.from_numpy(data).cuda(), torch.from_numpy(bias).cuda(), d, group)
    ws = A.Workspace.for_w4(ffn, B)
    ids = np.array([3, 90, 17, 17, 5], np.int32)                              # any order, one twice
    bad = np.array([3, 90, n, 17, 17, -1, 5], np.int32)
    ys = []
    for lst in (ids, bad):
        idx = torch.zeros(n, dtype=torch.int32, device="cuda")
        idx[:len(lst)] = torch.from_numpy(lst).cuda()
        y = torch.empty(B, d, device="cuda")
        A.asf_w4_sparse_ffn(ffn, x.cuda(), idx, torch.tensor([len(lst)], dtype=torch.int32, device="cuda"), y, ws)
        assert A.asf_read_error(ws) == (0 if lst is ids else L.ASF_ERR_DEVICE_INDEX)
        _check_ffn(y, "reglu", data, bias, d, group, x.double().numpy(), ids)
        ys.append(y)
    idx = torch.arange(n, dtype=torch.int32, device="cuda")
    for count, ref in ((n + 7, np.arange(n)), (-3, np.arange(0))):
        y = torch.empty(B, d, device="cuda")
        A.asf_w4_sparse_ffn(ffn, x.cuda(), idx, torch.tensor([count], dtype=torch.int32, device="cuda"), y, ws)
        assert A.asf_read_error(ws) == L.ASF_ERR_DEVICE_INDEX
        _check_ffn(y, "reglu", data, bias, d, group, x.double().numpy(), ref)


@pytest.mark.parametrize("B", [2, 3, 7, 12, 20])
def test_activations_of_very_different_sizes(B):
    """Activations that grow by 2^40 along the list, tokens 2^12 apart, one token with NaN: the others stay right."""
    n, d, group = 640, 256, 64
    data, bias = _layer("relu", n, d, group, 8)
    rng = np.random.default_rng(B)
    x = (rng.standard_normal((B, d)) * 2.0 ** -(6 * (np.arange(B) % 3))[:, None]).astype(np.float32)
    # rows' scales grow with the neuron
    grow = 2.0 ** np.linspace(-10, 10, n)
    W = [_weights(n, d, 8 + i) * grow[:, None] for i in range(2)]
    data = np.stack([O.w4_pack(w.astype(np.float32), group) for w in W], 1)
    bias = np.zeros(n, np.float32)
    bad = B - 1
    xs = torch.from_numpy(x).cuda()
    xs[bad, 5] = float("nan")
    ffn = A.W4FFN("relu", torch.from_numpy(data).cuda(), torch.from_numpy(bias).cuda(), d, group)
    ws = A.Workspace.for_w4(ffn, B)
    y = torch.empty(B, d, device="cuda")
    A.asf_w4_sparse_ffn(ffn, xs, None, None, y, ws)
    assert torch.isnan(y[bad]).all()
    keep = [b for b in range(B) if b != bad]
    _check_ffn(y[keep], "relu", data, bias, d, group, x[keep].astype(np.float64), np.arange(n))


@pytest.mark.parametrize("B", [2, 4, 8, 16, 32])
@pytest.mark.parametrize("act", ["relu", "reglu"])
def test_a_token_does_not_depend_on_the_others(act, B):
    """Every other token of the batch huge (a padded row that holds anything): the rest give the same bits as beside zeros."""
    n, d, group = 700, 512, 128
    data, bias = _layer(act, n, d, group, 21)
    ffn = A.W4FFN(act, torch.from_numpy(data).cuda(), torch.from_numpy(bias).cuda(), d, group)
    ws = A.Workspace.for_w4(ffn, B)
    rng = np.random.default_rng(B)
    x = rng.standard_normal((B, d)).astype(np.float32)
    ys = []
    for size in (0.0, 6e4):
        x[1::2] = rng.standard_normal(x[1::2].shape).clip(-1, 1) * size
        y = torch.empty(B, d, device="cuda")
        A.asf_w4_sparse_ffn(ffn, torch.from_numpy(x).cuda().half(), None, None, y, ws)
        _check_ffn(y, act, data, bias, d, group, torch.from_numpy(x).half().double().numpy(), np.arange(n))
        ys.append(y[::2].clone())
    assert torch.equal(*ys)


@pytest.mark.parametrize("B", [1, 6, 12])
def test_tiny_activations_beside_large_scales(B):
    """Activations of 2^-115 and down weights of 2^-5, then zero activations and down weights of 2^9."""
    n, d, group = 64, 256, 32
    W = [_weights(n, d, 31 + i) for i in range(2)]
    W[0][32:] = 0
    W[1] *= np.where(np.arange(n) < 32, 2.0 ** -5, 2.0 ** 9)[:, None]
    data = np.stack([O.w4_pack(w.astype(np.float32), group) for w in W], 1)
    bias = np.zeros(n, np.float32)
    x = (np.random.default_rng(B).standard_normal((B, d)) * 2.0 ** -115).astype(np.float32)
    ffn = A.W4FFN("relu", torch.from_numpy(data).cuda(), torch.from_numpy(bias).cuda(), d, group)
    y = torch.empty(B, d, device="cuda")
    A.asf_w4_sparse_ffn(ffn, torch.from_numpy(x).cuda(), None, None, y, A.Workspace.for_w4(ffn, B))
    _check_ffn(y, "relu", data, bias, d, group, x.astype(np.float64), np.arange(n))
    assert (y != 0).any()


def test_a_nan_group_reaches_only_its_rows():
    W = _weights(40, 512, 1)
    W[7, 300] = np.inf
    mat = A.W4Matrix.quantize(torch.from_numpy(W).cuda(), 64)
    y = torch.empty(2, 40, device="cuda")
    A.asf_w4_matmul(mat, torch.randn(2, 512, device="cuda").half(), y, A.Workspace.for_w4(mat, 2))
    assert torch.isnan(y[:, 7]).all() and torch.isfinite(torch.cat([y[:, :7], y[:, 8:]], 1)).all()


def test_matrix_ffn_quantize_and_row_moves():
    """W4FFN.quantize lays rows as described; asf_gather_rows permutes packed neurons."""
    n, d, group = 50, 264, 32
    mats = [_weights(n, d, i) for i in range(3)]
    dev = [torch.from_numpy(m).cuda() for m in mats]
    bias = torch.zeros(n, device="cuda")
    ffn = A.W4FFN.quantize("reglu", *dev, bias, group)
    want = np.stack([O.w4_pack(m, group) for m in mats], 1)
    assert np.array_equal(ffn.data.cpu().numpy(), want)
    perm = torch.randperm(n).int().cuda()
    out = torch.empty_like(ffn.data)
    A.asf_gather_rows(ffn.data, out, perm)
    assert np.array_equal(out.cpu().numpy(), want[perm.cpu().numpy()])


def test_graph_streams_and_shared_workspace():
    """A captured call, replayed with new inputs; two shapes in turn on one workspace; a side stream."""
    a = A.W4Matrix.quantize(torch.from_numpy(_weights(300, 4096, 1)).cuda(), 128)
    b = A.W4Matrix.quantize(torch.from_numpy(_weights(4096, 304, 2)).cuda(), 32)
    ws = max((A.Workspace.for_w4(m, 8) for m in (a, b)), key=lambda w: w.nbytes)
    x = torch.zeros(8, 4096, device="cuda", dtype=torch.float16)
    h, y = torch.empty(8, 300, device="cuda"), torch.empty(8, 4096, device="cuda")
    hp = torch.zeros(8, 304, device="cuda")

    def both():
        A.asf_w4_matmul(a, x, h, ws, relu=True)
        hp[:, :300].copy_(h)
        A.asf_w4_matmul(b, hp, y, ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for seed in range(3):
        torch.manual_seed(seed)
        x.copy_(torch.randn(8, 4096))
        graph.replay()
        got = y.clone()
        y.zero_()
        both()
        assert torch.equal(got, y) and float(got.abs().max()) > 0


def test_python_refusals():
    mat = A.W4Matrix.quantize(torch.randn(32, 256, device="cuda"), 64)
    ws = A.Workspace.for_w4(mat, 2)
    x, y = torch.randn(2, 256, device="cuda"), torch.empty(2, 32, device="cuda")
    for bad in (lambda: A.asf_w4_matmul(mat, x.cpu(), y, ws), lambda: A.asf_w4_matmul(mat, x, y.cpu(), ws),
                lambda: A.asf_w4_matmul(mat, x.bfloat16(), y, ws), lambda: A.asf_w4_matmul(mat, x[:, :128], y, ws),
                lambda: A.asf_w4_matmul(mat, x.t().contiguous().t(), y, ws), lambda: A.asf_w4_matmul(mat, x, y.double(), ws),
                lambda: A.asf_w4_matmul(mat, x, y[:1], ws), lambda: A.asf_w4_matmul(mat, x, y, ws, bias=y[0, :5]),
                lambda: A.W4Matrix(mat.data.int(), 256, 64), lambda: A.W4Matrix(mat.data, 1024, 64),
                lambda: A.W4Matrix.quantize(x.bfloat16(), 64), lambda: A.asf_w4_dequantize(mat, y),
                lambda: A.W4FFN("reglu", mat.data[None], y[0], 256, 64)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(A.AsfError):
        A.asf_w4_matmul(mat, torch.randn(33, 256, device="cuda"), torch.empty(33, 32, device="cuda"), ws)


@pytest.mark.parametrize("dt", ["f32", "f16"])
@pytest.mark.parametrize("act,group", [("relu", 32), ("reglu", 64), ("reglu", 128)])
@pytest.mark.parametrize("B", [1, 3, 7, 12, 20])
def test_an_infinite_activation(B, act, group, dt):
    """One neuron's activation overflows (fp32: for token 0 by its x, fp16: for all by the bias): infinities of the down
    weights' signs, NaN where a weight is 0, and the other tokens unharmed.  fp32: a later neuron of the same warp, eight
    tiles of 32 on, is token 0's only other active one, 2^40."""
    n, d, j, later = 300, 264, 10, 261
    rng = np.random.default_rng(B)
    W = [_weights(n, d, 50 + i) for i in range(3 if act == "reglu" else 2)]
    for w in W[:-1]:
        w[:, 8:16] = 0
        w[j, 8], w[later, 9] = 2.0 ** 18, 2.0 ** 10
    data = np.stack([O.w4_pack(w, group) for w in W], 1)
    bias = np.zeros(n, np.float32)
    x = rng.standard_normal((B, d)).astype(np.float32)
    x[:, 8:16] = 0
    if dt == "f32":
        x[0] = 0
        x[0, 8], x[0, 9] = 2.0 ** 115, 2.0 ** 30
    else:
        bias[j] = np.inf
        x[:, 8] = 1
    xt = torch.from_numpy(x).to(DT[dt])
    ffn = A.W4FFN(act, torch.from_numpy(data).cuda(), torch.from_numpy(bias).cuda(), d, group)
    ws = A.Workspace.for_w4(ffn, B)
    y = torch.empty(B, d, device="cuda")
    A.asf_w4_sparse_ffn(ffn, xt.cuda(), None, None, y, ws)
    hit = [0] if dt == "f32" else list(range(B))
    down = O.w4_unpack(data[j, -1], d, group)
    with np.errstate(invalid="ignore"):
        want = np.inf * down
    assert np.isnan(want).any() and (want == np.inf).any() and (want == -np.inf).any()
    got = y.cpu().numpy()
    assert all(np.array_equal(got[b], want.astype(np.float32), equal_nan=True) for b in hit)
    rest = [b for b in range(B) if b not in hit]
    if rest:
        _check_ffn(y[rest], act, data, bias, d, group, xt.double().numpy()[rest], np.arange(n))
    assert A.asf_read_error(ws) == 0


@pytest.mark.parametrize("m,k,group,B", [(62017, 1032, 128, 32), (61449, 2568, 32, 9), (125001, 1032, 64, 25)])
def test_matmul_with_several_tiles_under_a_ticket(m, k, group, B):
    """fp32 x too wide for a CTA, so that k is split, and more row tiles than tickets: units of two and three tiles."""
    torch.manual_seed(m)
    W = torch.randn(m, k, device="cuda")
    mat = A.W4Matrix.quantize(W, group)
    A.asf_w4_dequantize(mat, W)
    x, bias = torch.randn(B, k, device="cuda"), torch.randn(m, device="cuda")
    ws = A.Workspace.for_w4(mat, B)
    ref, mass = torch.empty(B, m, device="cuda", dtype=torch.float64), torch.empty(B, m, device="cuda", dtype=torch.float64)
    for i in range(0, m, 8192):
        w = W[i:i + 8192].double().t()
        ref[:, i:i + 8192], mass[:, i:i + 8192] = x.double() @ w, x.double().abs() @ w.abs()
    want = (ref + bias.double()).clamp(min=0).cpu().numpy()
    ys = [torch.full((B, m), float("nan"), device="cuda") for _ in range(3)]
    for y in ys:
        A.asf_w4_matmul(mat, x, y, ws, bias=bias, relu=True)
        _check(y, want, (mass + bias.double().abs()).cpu().numpy(), k // group + 1)
        assert torch.equal(y, ys[0]) and not ws.buf[64:4096].any()           # the tickets are zero again
    assert A.asf_read_error(ws) == 0


@pytest.mark.parametrize("act,n,active,d,B", [("reglu", 31001, 30999, 1032, 32), ("relu", 62100, 61990, 1032, 25)])
def test_sparse_ffn_with_several_tiles_under_a_ticket(act, n, active, d, B):
    """The same over a list, in no order; its names and biases are read again for a unit's earlier tiles."""
    torch.manual_seed(n)
    group, mats = 128, 3 if act == "reglu" else 2
    W = [torch.randn(n, d, device="cuda") / d ** 0.5 for _ in range(mats)]
    bias = torch.randn(n, device="cuda") * 0.3
    ffn = A.W4FFN.quantize(act, W[0] if mats == 3 else None, W[-2], W[-1], bias, group)
    back = torch.empty(n * mats, d, device="cuda")
    A.asf_w4_dequantize(A.W4Matrix(ffn.data.view(n * mats, -1), d, group), back)
    idx = torch.randperm(n, device="cuda").int()
    cnt = torch.tensor([active], dtype=torch.int32, device="cuda")
    x = torch.randn(B, d, device="cuda")
    rows = [w.double() for w in back.view(n, mats, d)[idx[:active].long()].unbind(1)]
    b, xd, u = bias[idx[:active].long()].double(), x.double(), (24 + d // group + 1 + 256) * 2.0 ** -23
    a = (xd @ rows[0].t() + b).clamp(min=0)
    da = u * (xd.abs() @ rows[0].abs().t() + b.abs())
    if act == "reglu":
        up, dup = xd @ rows[1].t(), u * (xd.abs() @ rows[1].abs().t())
        a, da = a * up, da * up.abs() + a * dup + da * dup
    v = (3 * active / 16 + 3 + 300) * 2.0 ** -23
    ref, tol = a @ rows[-1], (da + v * (a.abs() + da)) @ rows[-1].abs()
    ws = A.Workspace.for_w4(ffn, B)
    ys = [torch.full((B, d), float("nan"), device="cuda") for _ in range(3)]
    for y in ys:
        A.asf_w4_sparse_ffn(ffn, x, idx, cnt, y, ws)
        assert ((y.double() - ref).abs() <= tol).all()
        assert torch.equal(y, ys[0]) and not ws.buf[64:4096].any()
    assert A.asf_read_error(ws) == 0
