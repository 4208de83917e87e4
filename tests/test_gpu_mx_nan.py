"""GPU tests of blocks that are marked as NaN (exponent 255) in the block-scaled products: NaN in every output whose sum holds such a
block, whatever its elements, and nowhere else; and so from the quantizer that marks them to the products' outputs."""
import numpy as np
import pytest
import torch

import oracle
import sparse_matrix_multiply_amd as mm
from gpu_helpers import dev, env
from test_gpu_grouped import OUT, run_mx_codes
from test_gpu_mx import FP6_PAIRS, PAIRS, fp4_problem, fp6_problem, mx_problem, run_fp4, run_fp6, run_mx
from test_gpu_norm import rng

pytestmark = pytest.mark.gpu


def mark(g, ea, eb):
    """255 in a few blocks of some rows of A and columns of B; which outputs are NaN then."""
    rows, cols = g.choice(len(ea), 3, replace=False), g.choice(len(eb), 4, replace=False)
    for e, some in ((ea, rows), (eb, cols)):
        for i in some:
            e[i, g.integers(0, e.shape[1])] = 255
    bad = np.zeros((len(ea), len(eb)), bool)
    bad[rows], bad[:, cols] = True, True
    return bad


def check(D, bad):
    assert np.array_equal(torch.isnan(D.float()).cpu().numpy(), bad)


@pytest.mark.parametrize("tile", [16, 64, 128, 1282])
@pytest.mark.parametrize("kb", ["e4m3", "fp4"])
@pytest.mark.parametrize("out", list(OUT))
@pytest.mark.parametrize("zeros", [False, True])
def test_grouped(tile, kb, out, zeros, monkeypatch):
    monkeypatch.setenv("MMAC_TILE", str(tile))
    g = rng("nan", tile, kb, out, zeros)
    K, M, N = 416, 150, 100                                                       # three whole strips and one block
    ca, cb = g.integers(0, 0x40, (M, K)) + 128 * g.integers(0, 2, (M, K)), g.integers(0, 8 if kb == "fp4" else 0x40, (N, K))
    ea, eb = g.integers(120, 130, (M, K // 32)), g.integers(120, 130, (N, K // 32))
    bad = mark(g, ea, eb)
    if zeros:
        ca[np.repeat(ea == 255, 32, 1)], cb[np.repeat(eb == 255, 32, 1)] = 0, 0
    got, _, _ = run_mx_codes(ca, ea, cb, eb, kb, OUT[out])
    assert np.array_equal(np.isnan(got), bad)


@pytest.mark.parametrize("tile", [2561, 1282, 128, 64])
@pytest.mark.parametrize("ta,tb", PAIRS + [(oracle.FP4, oracle.FP4)] + FP6_PAIRS)
def test_dense(ta, tb, tile):
    M, N, K = 150, 100, 416
    seed = tile + 11 * ta + tb
    if ta == oracle.FP4:
        A, B, SA, SB = fp4_problem(M, N, K, seed, 120, 130)
    elif (ta, tb) in FP6_PAIRS:
        A, B, SA, SB = fp6_problem(M, N, K, seed, 120, 130)
    else:
        A, B, SA, SB, _ = mx_problem(ta, tb, M, N, K, seed, lo=120, hi=130)
    bad = mark(rng("dense", seed), SA, SB)
    with env(MMAC_TILE=tile):
        if ta == oracle.FP4:
            D = run_fp4(A, SA, B, SB)
        elif (ta, tb) in FP6_PAIRS:
            D = run_fp6(ta, tb, A, SA, B, SB, pad=24)                            # rows of 448 elements
        else:
            D = run_mx(ta, tb, A, SA, B, SB, 1.0, 0.0, None)
    check(D, bad)


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float32])
def test_from_the_quantizer_to_the_outputs(t):
    """A NaN or an infinity in a weight shows in its outputs, of fp32 and of 16 bits, in the grouped and in the dense product."""
    g = rng("quantizer")
    M, N, K = 40, 100, 416
    w, x = g.standard_normal((N, K)), g.standard_normal((M, K))
    w[3, 70], w[50, 0], w[99, 415] = np.nan, np.inf, -np.inf
    W, X = (torch.from_numpy(v).to(dev()).to(t) for v in (w, x))
    q, s = torch.empty(1, N, K // 2, dtype=torch.uint8, device=dev()), torch.empty(1, 4, N, dtype=torch.int32, device=dev())
    mm.mx4_quantize(W, q[0], s[0])
    a, sa = torch.empty(M, K, dtype=torch.float8_e4m3fn, device=dev()), torch.empty(4, M, dtype=torch.int32, device=dev())
    mm.mx8_quantize(X, a, sa)
    bad = np.zeros((M, N), bool)
    bad[:, [3, 50, 99]] = True
    o = torch.tensor([0, M], dtype=torch.int32, device=dev())
    for out in (torch.float32, torch.bfloat16):
        D = torch.empty(M, N, dtype=out, device=dev())
        mm.gemm_grouped_mx(a, sa, o, q, s, D, b_type=mm.FP4_E2M1)
        check(D, bad)
        a4, s4 = torch.empty(M, K // 2, dtype=torch.uint8, device=dev()), torch.empty(4, M, dtype=torch.int32, device=dev())
        mm.mx4_quantize(X, a4, s4)
        mm.gemm_mx(a4, s4, q[0], s[0], D, a_type=mm.FP4_E2M1, b_type=mm.FP4_E2M1)
        check(D, bad)
