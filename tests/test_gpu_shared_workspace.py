"""One split workspace for calls of every kind and size.

A workspace is zeroed once and calls in one stream may share it, whatever their shapes: the counters
of one call must not lie where another one left partial sums.  The products here differ in tile count
(4 to 324) and in ranges; every ordered pair of them runs through one buffer, with D preset to NaN,
and has to give the bits it gives with a workspace of its own, which are within the operator's bound
of the 64-bit product.
"""
import numpy as np
import pytest
import torch

import lowbit_ref as R
import sparse_matrix_multiply_amd as mm
from gpu_helpers import dev, env

pytestmark = pytest.mark.gpu

KIB = 1024


def gen(seed):
    return torch.Generator(device=dev()).manual_seed(seed)


def normal(g, rows, cols, scale=1.0):
    return (torch.randn((rows, cols), generator=g, device=dev()) * scale).to(torch.bfloat16)


class Dense:
    def __init__(self, M, N, K, seed, forced=None):
        g = gen(seed)
        self.A, self.B = normal(g, M, K), normal(g, N, K)
        self.env, self.terms = forced or {}, K
        self.ref, self.S = self.A.double() @ self.B.double().t(), self.A.double().abs() @ self.B.double().abs().t()
        with env(**self.env):
            self.bytes = mm.workspace_bytes(mm.BF16, M, N, K)

    def __call__(self, D, ws):
        with env(**self.env):
            mm.gemm_dense(self.A, self.B, D, workspace=ws)


class Sparse:
    def __init__(self, M, N, K, seed):
        g = gen(seed)
        A, self.B, self.K, self.terms = normal(g, M, K), normal(g, N, K), K, K
        keep = torch.zeros((M, K // 4, 4), dtype=torch.bool, device=dev())
        keep.scatter_(2, A.float().abs().view(M, K // 4, 4).topk(2, dim=2).indices, True)
        A = torch.where(keep.view(M, K), A, torch.zeros_like(A))
        self.Ac, self.idx = torch.empty((M, K // 2), dtype=A.dtype, device=dev()), torch.empty((M, K // 32), dtype=torch.int32, device=dev())
        mm.sparse24_compress(A, self.Ac, self.idx)
        self.ref, self.S = A.double() @ self.B.double().t(), A.double().abs() @ self.B.double().abs().t()
        self.bytes = mm.workspace_bytes(mm.BF16, M, N, K, sparse=True)

    def __call__(self, D, ws):
        mm.gemm_sparse24(self.Ac, self.idx, self.B, D, K=self.K, workspace=ws)


class Weight4:
    def __init__(self, M, N, K, seed):
        g = gen(seed)
        self.A, W, self.terms = normal(g, M, K), normal(g, N, K, K ** -0.5), K
        self.Wq, self.SW = torch.empty((N, K // 2), dtype=torch.uint8, device=dev()), torch.empty((K // 128, N), dtype=torch.int32, device=dev())
        mm.w4_quantize(W, self.Wq, self.SW)
        n = torch.stack((self.Wq & 15, self.Wq >> 4), -1).view(N, -1, 128).double()
        w = self.SW.t()
        s, z = (w & ~255).contiguous().view(torch.float32).double().unsqueeze(-1), (w & 255).double().unsqueeze(-1)
        self.ref = self.A.double() @ ((n - z) * s).view(N, K).t()
        self.S = self.A.double().abs() @ ((n + z) * s).view(N, K).t()
        self.bytes = mm.w4_workspace_bytes(M, N, K)

    def __call__(self, D, ws):
        mm.gemm_w4(self.A, self.Wq, self.SW, D, workspace=ws)


class Gradient:
    def __init__(self, M, N, K, seed):
        g = gen(seed)
        self.dY, X, self.terms = normal(g, M, N), normal(g, M, K), M
        self.Xq, self.SX = torch.empty((M, K), dtype=torch.float8_e4m3fn, device=dev()), torch.empty((K // 128, M), dtype=torch.int32, device=dev())
        mm.mx8_quantize(X, self.Xq, self.SX)
        V = torch.empty((M, K), device=dev())
        mm.mx8_dequantize(self.Xq, self.SX, V)
        self.ref, self.S = self.dY.double().t() @ V.double(), self.dY.double().abs().t() @ V.double().abs()
        self.bytes = mm.mx8_wgrad_workspace_bytes(M, N, K)

    def __call__(self, D, ws):
        mm.gemm_mx8_wgrad(self.dY, self.Xq, self.SX, D, workspace=ws)


def run(op, ws):
    D = torch.full(op.ref.shape, float("nan"), device=dev())
    op(D, ws)
    return D


def alone(op):
    """The bits of `op` with a workspace of its own, checked against the 64-bit product."""
    assert op.bytes > 0, "the product has to split"
    D = run(op, torch.zeros(op.bytes, dtype=torch.uint8, device=dev()))
    assert ((D.double() - op.ref).abs() <= 2 * (op.terms + 32) * R.U32 * op.S).all()
    return D


def test_products_of_every_kind_share_one_workspace():
    ops = [Weight4(64, 4096, 4096, 1),           # 32 tiles of 64 x 128, 8 ranges
           Weight4(64, 11008, 4096, 2),          # 86 tiles, 2 ranges: another projection of the same model
           Weight4(100, 512, 2048, 3),           # 4 tiles of 128 x 128
           Gradient(2048, 1024, 2048, 4),        # 128 tiles of 128 x 128, 4 ranges
           Gradient(1024, 1024, 4096, 5),        # 256 tiles, 2 ranges
           Gradient(4096, 32, 512, 6),           # 4 tiles of 32 x 128
           Dense(512, 512, 16384, 7),            # 64 tiles of 64 x 64, 4 ranges
           Dense(1024, 512, 8192, 8),            # 128 tiles, 2 ranges
           Dense(256, 256, 8192, 9),             # 16 tiles, 8 ranges
           Sparse(1024, 512, 8192, 10),
           Dense(1100, 1100, 256, 11, dict(MMAC_SPLITK=2, MMAC_TILE=64))]    # 324 tiles, forced
    want = [alone(op) for op in ops]
    ws = torch.zeros(max(op.bytes for op in ops), dtype=torch.uint8, device=dev())
    for i, first in enumerate(ops):
        for j, second in enumerate(ops):
            for k, op in ((i, first), (j, second)):
                D = run(op, ws)
                assert torch.equal(D, want[k]), f"operator {k} (pair {i}, {j}): {int(D.isnan().sum())} NaN"
                assert int(torch.count_nonzero(ws[:KIB])) == 0, f"operator {k} left counters"


def test_the_workspace_is_shared_by_replayed_graphs_too():
    ops = [Weight4(64, 4096, 4096, 21), Gradient(1024, 1024, 4096, 22), Weight4(64, 11008, 4096, 23), Dense(1024, 512, 8192, 24)]
    want = [alone(op) for op in ops]
    ws = torch.zeros(max(op.bytes for op in ops), dtype=torch.uint8, device=dev())
    Ds = [torch.empty(op.ref.shape, device=dev()) for op in ops]
    graphs = []
    for op, D in zip(ops, Ds):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            op(D, ws)
        graphs.append(graph)
    for order in ((0, 1, 2, 3), (3, 2, 1, 0), (2, 0, 3, 1)):
        for D in Ds:
            D.fill_(float("nan"))
        for k in order:
            graphs[k].replay()
        assert torch.equal(run(ops[order[0]], ws), want[order[0]])      # eager, in between
        torch.cuda.synchronize()
        for k in order:
            assert torch.equal(Ds[k], want[k]), f"operator {k} in {order}"


@pytest.mark.parametrize("order", [(0, 1, 0, 2, 1), (2, 1, 0, 1, 2)])
def test_static_scratch_is_shared_by_shapes(order):
    """mmac_gemm_dense_static keeps one array for all shapes: 64, 128 and 16 tiles.  Small integers, so that every
    order of summation gives the same bits."""
    problems = []
    for M, N, K in ((512, 512, 16384), (1024, 512, 8192), (256, 256, 8192)):
        g = np.random.default_rng(M + K)
        A, B = (torch.from_numpy(g.integers(-4, 5, s)).to(dev()) for s in ((M, K), (N, K)))
        assert mm.workspace_bytes(mm.BF16, M, N, K) > 0
        problems.append((A.to(torch.bfloat16), B.to(torch.bfloat16), A.double() @ B.double().t()))
    for k in order:
        A, B, ref = problems[k]
        D = torch.full(ref.shape, float("nan"), device=dev())
        mm.gemm_dense_static(A, B, D)
        assert torch.equal(D.double(), ref), f"{tuple(ref.shape)}: {int(D.isnan().sum())} NaN"
