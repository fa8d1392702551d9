"""The 4-bit product with adapters on the GPU against float64.

Tolerances, elementwise.  The product has its own, (24 + groups + 256) 2^-23 of sum |w x| + |bias|.
The adapter's share, of M = s |B| |A| |x|: A x is a chain of 8 ceil(k / 1024) fused steps at most, a
tree of 5 and 8 warps; times s, a chain of 8 and a tree of 5, and one addition to the product: each
2^-24 of what it adds to, 64 of them beside the first chain being more than enough.
"""
import numpy as np
import pytest
import torch

from tests.gpu_util import ensure_built

import activation_sparse_ffn_predict_b200 as A
from activation_sparse_ffn_predict_b200 import _lib as L

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


class Case:
    def __init__(self, m, k, B, rank, adapters, dt="f16", group=128, which=None, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed + m + k)
        normal = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.m, self.k, self.B, self.group = m, k, B, group
        self.mat = A.W4Matrix.quantize(normal(m, k) / k ** 0.5, group)
        self.W = torch.empty(m, k, device="cuda")
        A.asf_w4_dequantize(self.mat, self.W)                # exact in fp32
        self.x = normal(B, k).to(DT[dt])
        self.lora = A.LoraSet((normal(adapters, rank, k) / k ** 0.5).to(DT[dt]), (normal(adapters, m, rank) / rank ** 0.5).to(DT[dt]),
                              torch.rand(adapters, generator=g, device="cuda") * 4 - 2)
        self.bias = normal(m)
        w = torch.randint(-1, adapters, (B,), generator=g, device="cuda").tolist() if which is None else which
        self.which = torch.tensor(w, dtype=torch.int32, device="cuda")
        self.ws = A.Workspace.for_w4(self.mat, B, lora=self.lora)

    def run(self, half=False, bias=False, relu=False, lora=None, which=None, x=None):
        y = torch.full((self.B, self.m), float("nan"), device="cuda", dtype=torch.float16 if half else torch.float32)
        A.asf_w4_matmul_lora(self.mat, lora or self.lora, self.which if which is None else which, self.x if x is None else x, y,
                             self.ws, bias=self.bias if bias else None, relu=relu)
        return y

    def want(self, bias=False, relu=False, scale=True):
        """(y, tolerance) in float64."""
        x, w = self.x.double(), self.W.double()
        y, tol = x @ w.t(), x.abs() @ w.abs().t()
        if bias:
            y, tol = y + self.bias.double(), tol + self.bias.double().abs()
        tol = (24 + self.k // self.group + 257 + 1) * 2.0 ** -23 * tol
        steps = 8 * -(-self.k // 1024) + 64
        for b, a in enumerate(self.which.tolist()):
            if a < 0:
                continue
            d, u, s = self.lora.A[a].double(), self.lora.B[a].double(), float(self.lora.scale[a]) if scale else 1.0
            y[b] += s * (u @ (d @ x[b]))
            tol[b] += steps * 2.0 ** -24 * abs(s) * (u.abs() @ (d.abs() @ x[b].abs()))
        return (y.clamp(min=0) if relu else y), tol

    def check(self):
        for bias, relu in ((False, False), (True, True)):
            y = self.run(bias=bias, relu=relu)
            want, tol = self.want(bias, relu)
            assert torch.isfinite(y).all()
            off = (y.double() - want).abs() - tol
            assert off.max() <= 0, (float(off.max()), int(off.argmax()))
            assert torch.equal(y, self.run(bias=bias, relu=relu))               # fixed summation order
            assert torch.equal(self.run(True, bias, relu), y.half())            # the same sum, rounded once
        assert A.asf_read_error(self.ws) == 0


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("m,k,B,rank,adapters,group", [
    (1, 8, 1, 8, 1, 32), (129, 136, 2, 8, 2, 64), (1003, 1376, 3, 16, 5, 32), (64, 4096, 1, 16, 8, 128), (300, 8192, 9, 24, 3, 64),
    (40, 12288, 17, 32, 1, 128), (500, 2760, 32, 64, 24, 64), (257, 512, 32, 256, 4, 128), (4096, 256, 8, 128, 32, 128),
    (24, 65536, 5, 8, 2, 128), (1000, 1000, 31, 40, 7, 32), (128, 2048, 4, 16, 2, 128)])
def test_against_the_definition(m, k, B, rank, adapters, group, dt):
    Case(m, k, B, rank, adapters, dt, group).check()


@pytest.mark.parametrize("B,rank,adapters", [(1, 16, 3), (16, 64, 16), (32, 16, 5)])
def test_products_large_enough_for_tensor_memory(B, rank, adapters):
    Case(34000, 4096, B, rank, adapters, seed=1).check()


@pytest.mark.parametrize("which", [[-1] * 9, [2] * 9, [0, 1, 2, 0, 1, 2, 0, 1, 2], [-1, 0, -5, 0, -1, 0, 1, 1, -2], [2, 1, 0, -1, -1, -1, -1, -1, 0]])
def test_who_shares_an_adapter(which):
    c = Case(700, 1024, 9, 16, 3, which=which, seed=3)
    c.check()
    plain = torch.empty(9, 700, device="cuda")
    A.asf_w4_matmul(c.mat, c.x, plain, c.ws)
    y, none = c.run(), torch.tensor([w < 0 for w in which], device="cuda")
    assert torch.equal(y[none], plain[none])                 # a token without an adapter: the product's bits


def test_a_token_does_not_depend_on_the_others():
    c = Case(300, 2048, 13, 24, 6, which=[b % 6 for b in range(13)], seed=4)
    first = c.run()
    for which in ([3] * 13, [3 if b == 3 else -1 for b in range(13)], [3] + [b % 2 for b in range(1, 13)]):
        which[3] = 3
        assert torch.equal(c.run(which=torch.tensor(which, dtype=torch.int32, device="cuda"))[3], first[3])
    x = c.x.clone()
    x[9] = float("nan")                                      # shares adapter 3 with token 3
    x[5, 0], x[6, 1] = float("inf"), float("-inf")
    y = c.run(x=x)
    sound = [b for b in range(13) if b not in (5, 6, 9)]
    assert torch.equal(y[sound], first[sound]) and torch.isnan(y[9]).all()


def test_no_scale_and_padded_ranks():
    c = Case(200, 512, 6, 16, 3, seed=5)
    unit = A.LoraSet(c.lora.A, c.lora.B)
    want, tol = c.want(scale=False)
    assert ((c.run(lora=unit).double() - want).abs() <= tol).all()
    pad = A.LoraSet(torch.cat([c.lora.A, torch.zeros(3, 8, 512).half().cuda()], 1), torch.cat([c.lora.B, torch.zeros(3, 200, 8).half().cuda()], 2),
                    c.lora.scale)
    c.ws = A.Workspace.for_w4(c.mat, 6, lora=pad)
    want, tol = c.want()
    assert ((c.run(lora=pad).double() - want).abs() <= tol).all()


def test_bad_adapters_are_flagged_and_none():
    c = Case(300, 512, 5, 8, 2, which=[0, 2, 1, 2 ** 31 - 1, -2 ** 31], seed=6)
    y, plain = c.run(bias=True, relu=True), torch.empty(5, 300, device="cuda")
    assert A.asf_read_error(c.ws) == L.ASF_ERR_DEVICE_INDEX
    A.asf_w4_matmul(c.mat, c.x, plain, c.ws, bias=c.bias, relu=True)
    assert torch.equal(y[[1, 3, 4]], plain[[1, 3, 4]]) and not torch.equal(y[0], plain[0])


def test_infinite_and_large_values():
    c = Case(128, 256, 3, 8, 2, dt="f32", which=[0, 1, 0], seed=7)
    x = c.x * torch.tensor([1e20, 1.0, 1e-20], device="cuda")[:, None]
    y = c.run(x=x)
    c.x = x
    want, tol = c.want()
    assert ((y.double() - want).abs() <= tol).all()


def test_streams_and_graphs():
    c = Case(4096, 4096, 8, 16, 4, seed=8)
    want = c.run(bias=True)
    torch.cuda.synchronize()
    y, g, side = torch.empty_like(want), torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(side):
        A.asf_w4_matmul_lora(c.mat, c.lora, c.which, c.x, y, c.ws, bias=c.bias)
    side.synchronize()
    assert torch.equal(y, want)
    with torch.cuda.graph(g):
        for _ in range(3):                                   # calls one behind the other on one workspace
            A.asf_w4_matmul_lora(c.mat, c.lora, c.which, c.x, y, c.ws, bias=c.bias)
    c.x.copy_(torch.randn_like(c.x))
    c.which.copy_(c.which.flip(0))
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, c.run(bias=True)) and not torch.equal(y, want)


def test_binding_refuses():
    c = Case(64, 256, 4, 8, 2, seed=9)
    y = torch.empty(4, 64, device="cuda")
    for bad in (lambda: A.LoraSet(c.lora.A[0], c.lora.B), lambda: A.LoraSet(c.lora.A, c.lora.B[:1]), lambda: A.LoraSet(c.lora.A, c.lora.B.float()),
                lambda: A.LoraSet(c.lora.A.cpu(), c.lora.B), lambda: A.LoraSet(c.lora.A, c.lora.B, c.lora.scale[:1]),
                lambda: A.LoraSet(c.lora.A, c.lora.B, c.lora.scale.double()), lambda: A.LoraSet(c.lora.A.transpose(1, 2), c.lora.B),
                lambda: c.run(which=c.which[:3]), lambda: c.run(which=c.which.long()), lambda: c.run(which=c.which.cpu()),
                lambda: c.run(x=c.x.float()), lambda: c.run(x=c.x[:, :128])):
        with pytest.raises(ValueError):
            bad()
    other = A.LoraSet(c.lora.A[:, :, :128].contiguous(), c.lora.B)
    with pytest.raises(A.AsfError):
        c.run(lora=other)
    c.ws = A.Workspace.for_w4(c.mat, 4)
    with pytest.raises(A.AsfError):
        c.run()                                              # a workspace for the plain product alone
    with pytest.raises(A.AsfError):
        A.Workspace.for_w4(c.mat, 4, lora=other)


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("m,rank", [(4096, 48), (4096, 96), (1003, 80), (2000, 112), (4096, 240), (700, 64)])
def test_the_adapters_share_does_not_depend_on_the_batch(m, rank, dt):
    """Over weights of zero, so that the product is zero for every number of tokens: a token's bits alone, with another,
    and as one of 8 and of 32, whose calls lay out rows of B in other tiles."""
    c = Case(m, 256, 32, rank, 8, dt, 128, which=[b % 8 for b in range(32)], seed=11)
    c.mat = A.W4Matrix.quantize(torch.zeros(m, 256, device="cuda"), 128)
    want = c.run(bias=True)
    x, which = c.x, c.which
    for first, B in ((0, 1), (7, 1), (2, 2), (0, 8), (5, 8), (1, 31)):
        c.B, c.x, c.which = B, x[first:first + B].contiguous(), which[first:first + B].contiguous()
        assert torch.equal(c.run(bias=True), want[first:first + B]), (first, B)


@pytest.mark.parametrize("B,rank", [(8, 64), (21, 128), (22, 128), (32, 88), (32, 96), (32, 256)])
def test_the_up_steps_grid_is_resident_at_once(B, rank):
    """Its CTAs take equal runs, so one that waits for another to end would double the time."""
    from cuda.bindings import driver as cu
    c = Case(20000, 64, B, rank, B, group=64, which=list(range(B)), seed=13)
    c.run()
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g):
        y = c.run()
    graph = cu.CUgraph(init_value=g.raw_cuda_graph())
    nodes = cu.cuGraphGetNodes(graph, cu.cuGraphGetNodes(graph, 0)[2])[1]
    kernels = [n for n in nodes if cu.cuGraphNodeGetType(n)[1] == cu.CUgraphNodeType.CU_GRAPH_NODE_TYPE_KERNEL]
    up = [p for p in (cu.cuGraphKernelNodeGetParams(n)[1] for n in kernels) if p.sharedMemBytes == 4 * 16384 + B * rank * 4]
    assert len(up) == 1
    dev = torch.cuda.get_device_properties(0)
    each = up[0].sharedMemBytes + 1024 + (4 * 8 + 2 * 32 * 4)          # its own static part, and the system's
    assert -(-up[0].gridDimX // dev.multi_processor_count) * each <= dev.shared_memory_per_multiprocessor
    g.instantiate()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, c.run())
