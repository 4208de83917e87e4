"""GPU tests of the low-bit operands against their 64-bit references (lowbit_ref.py).

Stored forms (codes, scale words, elements, exponents) must match bit for bit, the range
checks' guard cells stay untouched.  Products: with S the sum of the magnitudes of
what the kernel adds up and u = 2^-24, fp32 sums of n terms are within 2 (n + c) u S element by
element (each addition rounds once, doubled for an accumulator that truncates; c counts
the roundings of the scale, the zero point's term, the joins of up to 16 partial sums
and the epilogue: 32 covers them), and 8 u sqrt(n) normwise as for the other products here;
a 16-bit output adds half a step, eps / 2 of its value (and half the smallest subnormal).
Integer inputs with power-of-two scales make every sum exact: those must match bit for bit.
"""
import numpy as np
import pytest
import torch

import lowbit_ref as R
import sparse_matrix_multiply_amd as mm
from gpu_helpers import dev

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ELEMENTS = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2, "int8": torch.int8}


def rng(*key):
    """A generator of its own for every case, the same on every run."""
    return np.random.default_rng([int.from_bytes(str(k).encode(), "little") % (1 << 32) for k in key])


def pitched(x, t, pad=0):
    """Host float64 matrix -> device tensor of type t whose row pitch is a multiple of 16 bytes; the padding is NaN."""
    x = torch.from_numpy(np.ascontiguousarray(x))
    rows, cols = x.shape
    per = 16 // torch.empty((), dtype=t).element_size()
    ld = max(per, -(-cols // per) * per + pad * per)
    buf = torch.full((rows, ld), float("nan"), dtype=t, device=dev())
    buf[:, :cols] = x.to(dev()).to(t)
    return buf[:, :cols]


def exact(x):
    """Device tensor -> float64 host array."""
    return x.double().cpu().numpy()


def rounded(x, t):
    return torch.from_numpy(np.ascontiguousarray(x)).to(t).double().numpy()


def guarded(rows, cols, dtype, ld, fill):
    """(buffer, view): one guard row above and below and guard columns after each row."""
    buf = torch.full((rows + 2, ld), fill, dtype=dtype, device=dev())
    return buf, buf[1:rows + 1, :cols]


def check_guards(buf, rows, cols, fill):
    host = buf.cpu()
    assert (host[0] == fill).all() and (host[rows + 1] == fill).all() and (host[:, cols:] == fill).all(), "guard cells"


# ---- 4-bit weights: the quantizer ----------------------------------------------------------------

def run_w4_quantize(W, t, group, q_type, symmetric):
    N, K = W.shape
    Wd = pitched(W, t, pad=1)
    rb, G = -(-K // 32) * 16, R.n_groups(K, group)
    cbuf, Wq = guarded(N, rb, torch.uint8, rb + 16, 0xA5)
    sbuf, SW = guarded(G, N, torch.int32, N + 3, -7)
    mm.w4_quantize(Wd, Wq, SW, group=group, q_type=q_type, symmetric=symmetric)
    torch.cuda.synchronize()
    check_guards(cbuf, N, rb, 0xA5)
    check_guards(sbuf, G, N, -7)
    return Wq, SW, exact(Wd)


FORMS = [(R.U4, True), (R.U4, False), (R.FP4, True)]


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("q_type,symmetric", FORMS)
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("N,K", [(1, 1), (3, 31), (33, 127), (65, 300), (37, 2305)])
def test_w4_quantize_bits(t, q_type, symmetric, group, N, K):
    W = rng(N, K, group, q_type).standard_normal((N, K)) * 0.02
    Wq, SW, W = run_w4_quantize(W, TYPES[t], group, q_type, symmetric)
    codes, s, z = R.w4_quantize(W, group, q_type, symmetric)
    assert np.array_equal(SW.cpu().numpy(), R.scale_words(s, z))
    assert np.array_equal(Wq.cpu().numpy(), R.pack_codes(codes))


@pytest.mark.parametrize("q_type,symmetric", FORMS)
@pytest.mark.parametrize("group", [0, 32, 128])
def test_w4_quantize_special_groups(q_type, symmetric, group):
    """Zeros, ties on every middle, one-sided groups, tiny and huge ranges, NaN and infinities."""
    g = rng(q_type, group, symmetric)
    K = 256
    W = g.standard_normal((16, K))
    W[0] = 0.0
    W[1] = g.integers(-14, 15, K) / 2.0                  # quotients on the middles (scale 1 when 7 is there)
    W[1, ::32] = 7.0
    W[2] = g.integers(-24, 25, K) / 4.0
    W[2, ::32] = 6.0
    W[3] = g.integers(0, 31, K) / 2.0
    W[3, ::32] = 15.0
    W[4] = np.abs(W[4]) + 1
    W[5] = -np.abs(W[5]) - 1
    W[6] *= 2.0 ** -126                                  # scales below the smallest normal
    W[7] *= 2.0 ** -120
    W[8] = g.choice([-3e38, 3e38], K)                    # hi - lo passes fp32
    W[9] *= 1e37
    W[10, 40] = np.nan
    W[11, 200] = np.inf
    W[12, 0] = -np.inf
    W[13] = -0.0
    W[14] = 2.0 ** -149
    Wq, SW, W = run_w4_quantize(W, torch.float32, group, q_type, symmetric)
    codes, s, z = R.w4_quantize(W, group, q_type, symmetric)
    assert np.array_equal(SW.cpu().numpy(), R.scale_words(s, z))
    assert np.array_equal(Wq.cpu().numpy(), R.pack_codes(codes))


# ---- 4-bit weights: the product ------------------------------------------------------------------

def w4_problem(M, N, K, group, q_type, t, integers=False, key=0):
    """A (float64, exact in t), codes, scales and zero points."""
    g = rng(M, N, K, group, q_type, t, integers, key)
    G = R.n_groups(K, group)
    codes = g.integers(0, 16, (N, K))
    z = g.integers(0, 16, (N, G)) if q_type == R.U4 else np.zeros((N, G), np.int64)
    if integers:
        A = g.integers(-4, 5, (M, K)).astype(np.float64)
        s = 2.0 ** g.integers(-2, 3, (N, G))
    else:
        A = rounded(g.standard_normal((M, K)), TYPES[t])
        s = R.round16(np.abs(g.standard_normal((N, G))) * 0.01 + 1e-4)
    return A, codes, s, z


def w4_tensors(codes, s, z, fill=15, garbage=True):
    """Codes and words on the device; nibbles past K `fill`, words past N and K NaN scales."""
    Wq = torch.from_numpy(R.pack_codes(codes, fill)).to(dev())
    buf = torch.full((Wq.shape[0], Wq.shape[1] + 32), 0xFF, dtype=torch.uint8, device=dev())
    buf[:, :Wq.shape[1]] = Wq
    words = torch.from_numpy(R.scale_words(s, z)).to(dev())
    wbuf = torch.full((words.shape[0], words.shape[1] + 5), 0x7fc0000f, dtype=torch.int32, device=dev())
    wbuf[:, :words.shape[1]] = words
    return buf[:, :Wq.shape[1]], wbuf[:, :words.shape[1]]


def check_sum(D, ref, S, n, t=torch.float32, what=""):
    """The bounds of the module's docstring; `ref` and S already carry the epilogue's terms."""
    D = exact(D)
    assert np.isfinite(D).all(), what
    half = 0.0 if t == torch.float32 else torch.finfo(t).eps / 2
    tiny = 2.0 ** -25 if t == torch.float16 else 0.0
    diff = np.abs(D - ref)
    bound = 2 * (n + 32) * R.U32 * S
    assert (diff <= bound + half * (np.abs(ref) + bound) + tiny).all(), f"{what}: {(diff / np.maximum(S, 1e-300)).max():.3e}"
    allowed = 8 * R.U32 * np.sqrt(n + 32) * np.linalg.norm(S) + half * np.linalg.norm(ref) + tiny * np.sqrt(ref.size)
    assert np.linalg.norm(diff) <= allowed, f"{what}: normwise {np.linalg.norm(diff):.3e} > {allowed:.3e}"


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("q_type", [R.U4, R.FP4])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 33, 256), (2, 16, 31), (3, 100, 600), (8, 17, 2305), (9, 40, 255),
                                   (16, 50, 1030), (17, 31, 700), (32, 16, 33), (33, 130, 513), (64, 70, 96),
                                   (130, 200, 1160)])
def test_gemm_w4_matches_reference(t, q_type, group, M, N, K):
    A, codes, s, z = w4_problem(M, N, K, group, q_type, t)
    Wq, SW = w4_tensors(codes, s, z)
    ref, S = R.gemm_w4(A, codes, s, z, group, q_type)
    buf, D = guarded(M, N, torch.float32, N + 5, -77.0)
    mm.gemm_w4(pitched(A, TYPES[t], 1), Wq, SW, D, group=group, q_type=q_type, workspace=mm.w4_workspace(M, N, K))
    torch.cuda.synchronize()
    check_sum(D, ref, S, K, what=f"{t} {q_type} {group} {M}x{N}x{K}")
    check_guards(buf, M, N, -77.0)


@pytest.mark.parametrize("q_type", [R.U4, R.FP4])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("M,N,K", [(1, 64, 4096), (7, 48, 1000), (16, 100, 520), (40, 36, 1290), (300, 260, 640)])
def test_gemm_w4_small_integers_exact(q_type, group, M, N, K):
    """|a| <= 4, codes and zero points below 16, scales 1/4 .. 4: sums stay below 2^20 in steps of 2^-3."""
    A, codes, s, z = w4_problem(M, N, K, group, q_type, "bf16", integers=True)
    Wq, SW = w4_tensors(codes, s, z, fill=9)
    ref, _ = R.gemm_w4(A, codes, s, z, group, q_type)
    for t in ("bf16", "fp16"):
        D = torch.full((M, N), float("nan"), device=dev())
        mm.gemm_w4(pitched(A, TYPES[t]), Wq, SW, D, group=group, q_type=q_type, workspace=mm.w4_workspace(M, N, K))
        assert np.array_equal(exact(D), ref), t


@pytest.mark.parametrize("t,q_type", [("bf16", R.U4), ("fp16", R.U4), ("bf16", R.FP4)])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("K", [96, 650])
def test_gemm_w4_widest_tile(t, q_type, group, K):
    """Enough 128 x 256 tiles (13 x 16) for the widest kernel, ragged at every edge."""
    M, N = 1601, 3900
    assert mm.w4_workspace_bytes(M, N, K) == 0
    A, codes, s, z = w4_problem(M, N, K, group, q_type, t)
    Wq, SW = w4_tensors(codes, s, z)
    ref, S = R.gemm_w4(A, codes, s, z, group, q_type)
    buf, D = guarded(M, N, torch.float32, N + 5, -77.0)
    mm.gemm_w4(pitched(A, TYPES[t], 1), Wq, SW, D, group=group, q_type=q_type)
    torch.cuda.synchronize()
    check_sum(D, ref, S, K, what=f"{t} {q_type} {group} {K}")
    check_guards(buf, M, N, -77.0)


@pytest.mark.parametrize("M,N,K", [(40, 200, 4100), (64, 1000, 2048), (200, 300, 3000)])
def test_gemm_w4_split_sums_are_deterministic(M, N, K):
    """With a workspace K is cut into ranges: the same bits on every run, the counters back at zero, and the unsplit
    call's result within both sums' bounds."""
    A, codes, s, z = w4_problem(M, N, K, 128, R.U4, "bf16")
    Wq, SW = w4_tensors(codes, s, z)
    Ad, ws = pitched(A, torch.bfloat16), mm.w4_workspace(M, N, K)
    assert ws is not None
    ref, S = R.gemm_w4(A, codes, s, z, 128, R.U4)
    first = None
    for _ in range(4):
        D = torch.full((M, N), float("nan"), device=dev())
        mm.gemm_w4(Ad, Wq, SW, D, workspace=ws)
        check_sum(D, ref, S, K)
        first = D if first is None else first
        assert torch.equal(D, first)
        assert int(ws[:256].view(torch.int32).abs().max()) == 0, "counters"
    D = torch.empty((M, N), device=dev())
    mm.gemm_w4(Ad, Wq, SW, D)
    check_sum(D, ref, S, K)
    mm.gemm_w4(Ad, Wq, SW, D, workspace=ws[:ws.numel() // 2])      # too small: unsplit
    check_sum(D, ref, S, K)


@pytest.mark.parametrize("M", [3, 20, 140])
@pytest.mark.parametrize("out", ["fp32", "bf16", "fp16"])
def test_gemm_w4_epilogue(M, out):
    """alpha, beta * C, bias, ReLU and the output type; C and D strided, and D the same buffer as C."""
    N, K, o = 77, 300, TYPES[out]
    A, codes, s, z = w4_problem(M, N, K, 64, R.U4, "bf16")
    g = rng(M, out)
    C, bias = rounded(g.standard_normal((M, N)), o), g.standard_normal(N).astype(np.float32)
    ref, S = R.gemm_w4(A, codes, s, z, 64, R.U4)
    ref = np.maximum(1.25 * ref - 0.5 * C + bias, 0)
    S = 1.25 * S + 0.5 * np.abs(C) + np.abs(bias)
    Wq, SW = w4_tensors(codes, s, z)
    buf, D = guarded(M, N, o, N + 3, -77.0)
    args = dict(group=64, alpha=1.25, beta=-0.5, bias=torch.from_numpy(bias).to(dev()), act=mm.ACT_RELU,
                workspace=mm.w4_workspace(M, N, K))
    Ad = pitched(A, torch.bfloat16)
    mm.gemm_w4(Ad, Wq, SW, D, C=pitched(C, o, 2), **args)
    check_sum(D, ref, S, K, o)
    check_guards(buf, M, N, -77.0)
    D.copy_(torch.from_numpy(C).to(dev()).to(o))
    mm.gemm_w4(Ad, Wq, SW, D, C=D, **args)
    check_sum(D, ref, S, K, o, "in place")


@pytest.mark.parametrize("M", [2, 70])
def test_gemm_w4_fp8_outputs_saturate(M):
    N, K = 33, 128
    A, codes, s, z = w4_problem(M, N, K, 128, R.FP4, "bf16", integers=True)
    Wq, SW = w4_tensors(codes, s, z)
    ref, _ = R.gemm_w4(A, codes, s, z, 128, R.FP4)
    for t, top in ((torch.float8_e4m3fn, 448.0), (torch.float8_e5m2, 57344.0)):
        D = torch.empty((M, N), dtype=t, device=dev())
        mm.gemm_w4(pitched(A, torch.bfloat16), Wq, SW, D, q_type=mm.FP4_E2M1)
        want = torch.from_numpy(np.clip(ref, -top, top)).float().to(t)
        assert np.array_equal(exact(D), want.double().numpy())


@pytest.mark.parametrize("M", [1, 16, 33, 100])
def test_gemm_w4_empty_sum_and_sizes(M):
    """K == 0 gives beta * C; M == 0 and N == 0 write nothing."""
    C = torch.randn(M, 8, device=dev())
    D = torch.full((M, 8), float("nan"), device=dev())
    A = torch.empty((M, 8), dtype=torch.bfloat16, device=dev())[:, :0]
    Wq, SW = torch.empty((8, 16), dtype=torch.uint8, device=dev()), torch.empty((1, 8), dtype=torch.int32, device=dev())
    mm.gemm_w4(A, Wq, SW, D, group=0, beta=2.0, C=C)
    assert torch.equal(D, 2 * C)
    mm.gemm_w4(torch.empty((0, 32), dtype=torch.bfloat16, device=dev()), Wq, SW, D[:0], group=0)
    mm.gemm_w4(torch.empty((M, 32), dtype=torch.bfloat16, device=dev()), Wq[:0], SW[:, :0], D[:, :0], group=0)
    torch.cuda.synchronize()


@pytest.mark.parametrize("M", [5, 16, 48, 160])
@pytest.mark.parametrize("q_type", [R.U4, R.FP4])
def test_gemm_w4_non_finite_values_stay_in_their_row_and_column(M, q_type):
    N, K = 50, 400
    A, codes, s, z = w4_problem(M, N, K, 128, q_type, "bf16", integers=True)
    s[7, 1] = np.nan
    A[1, 399], A[M - 1, 0] = np.nan, np.inf
    with np.errstate(invalid="ignore"):
        ref, _ = R.gemm_w4(A, codes, s, z, 128, q_type)
    Wq, SW = w4_tensors(codes, s, z)
    D = torch.empty((M, N), device=dev())
    mm.gemm_w4(pitched(A, torch.bfloat16), Wq, SW, D, q_type=q_type, workspace=mm.w4_workspace(M, N, K))
    D = exact(D)
    clean = np.ones((M, N), bool)
    clean[[1, M - 1]] = False
    clean[:, 7] = False
    assert np.array_equal(D[clean], ref[clean])
    assert not np.isfinite(D[~clean]).any()


# ---- 8-bit activations ---------------------------------------------------------------------------

def run_mx8_quantize(X, t, q):
    M, K = X.shape
    Xd = pitched(X, t, pad=1)
    kp = -(-K // 32) * 32
    qbuf, Xq8 = guarded(M, kp, torch.uint8, kp + 16, 0x5A)
    sbuf, SX = guarded(-(-K // 128), M, torch.int32, M + 3, -7)
    Xq = Xq8.view(ELEMENTS[q])
    mm.mx8_quantize(Xd, Xq, SX)
    torch.cuda.synchronize()
    check_guards(qbuf, M, kp, 0x5A)
    check_guards(sbuf, SX.shape[0], M, -7)
    return Xq8.cpu().numpy(), SX.cpu().numpy(), exact(Xd)


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("q", list(ELEMENTS))
@pytest.mark.parametrize("M,K", [(1, 1), (3, 31), (33, 33), (40, 256), (70, 1000), (5, 2049)])
def test_mx8_quantize_bits(t, q, M, K):
    g = rng(t, q, M, K)
    X = g.standard_normal((M, K)) * np.exp(g.uniform(-9, 9, (M, 1)))
    X[g.random((M, K)) < 0.02] *= 300
    X = np.clip(X, -60000, 60000)
    X[0, :K // 2] = 0
    got, words, X = run_mx8_quantize(X, TYPES[t], q)
    codes, e = R.mx8_quantize(X, q)
    assert np.array_equal(words, R.sx_words(e))
    assert np.array_equal(got, (codes & 255).astype(np.uint8))


@pytest.mark.parametrize("q", list(ELEMENTS))
def test_mx8_quantize_borders(q):
    """Block maxima on and just past the type's largest value, ties, subnormals, the ends of fp32, both zeros."""
    g = rng(q)
    top = R.TOP[q]
    X = np.zeros((12, 64))
    up = lambda v: float(np.nextafter(np.float32(v), np.float32(np.inf)))   # noqa: E731
    X[0, 0], X[0, 32] = top, up(top)
    X[1, 0], X[1, 32] = -top * 2.0 ** 100, -up(top * 2.0 ** 100)
    X[2] = g.integers(-300, 300, 64) / 256.0
    X[2, ::32] = top / 64
    X[3] = g.standard_normal(64) * 2.0 ** -126
    X[4] = 2.0 ** -149
    X[5] = g.choice([-1, 1], 64) * float(np.finfo(np.float32).max)
    X[6] = -0.0
    X[7, 3] = 1e-30
    X[8] = (np.arange(64) + 0.5) / 32
    X[9] = g.standard_normal(64) * 2.0 ** -118
    X[10, ::2] = -0.0
    X[10, 1] = 3.0
    got, words, X = run_mx8_quantize(X, torch.float32, q)
    codes, e = R.mx8_quantize(X, q)
    assert np.array_equal(words, R.sx_words(e))
    assert np.array_equal(got, (codes & 255).astype(np.uint8))


@pytest.mark.parametrize("t", list(TYPES))
def test_mx8_quantize_non_finite(t):
    """E4M3: NaN for both; E5M2 keeps infinities; neither changes the rest of its block.  I8: the block is NaN."""
    X = rng(t).standard_normal((4, 96))
    X[0, 5], X[1, 40], X[2, 70], X[2, 71] = np.nan, np.inf, -np.inf, np.nan
    clean = np.where(np.isfinite(X), X, 0)
    for q in ELEMENTS:
        got, words, Xr = run_mx8_quantize(X, TYPES[t], q)
        codes, e = R.mx8_quantize(rounded(clean, TYPES[t]), q)
        if q == "int8":
            for i, b in ((0, 0), (1, 1), (2, 2)):
                e[i, b] = 255
                codes[i, 32 * b:32 * b + 32] = 0
            assert np.array_equal(got, (codes & 255).astype(np.uint8))
        else:
            finite = np.isfinite(Xr)
            assert np.array_equal(got[finite], codes[finite].astype(np.uint8))
            v = R.mx8_values(got.astype(np.int64), e, q)
            assert np.isnan(v[0, 5]) and np.isnan(v[2, 71])
            assert np.isnan(v[1, 40]) if q == "e4m3" else v[1, 40] == np.inf and v[2, 70] == -np.inf
        assert np.array_equal(words, R.sx_words(e))


def all_values(q):
    """Every code with every exponent: 256 rows (exponent) x 256 codes."""
    codes = np.tile(np.arange(256), (256, 1))
    e = np.tile(np.arange(256)[:, None], (1, 8))
    return (codes.astype(np.int8).astype(np.int64) if q == "int8" else codes), e


def put_mx8(codes, e, q, fill=255):
    Xq = torch.from_numpy((codes & 255).astype(np.uint8)).to(dev()).view(ELEMENTS[q])
    return Xq, torch.from_numpy(R.sx_words(e, fill)).to(dev())


def finite_rounded(v, t):
    """float64 -> t to nearest even with finite values saturating, as float64."""
    top = float(torch.finfo(t).max)
    r = torch.from_numpy(np.clip(np.where(np.isfinite(v), v, 0), -top, top)).to(t).double().numpy()
    return np.where(np.isfinite(v), r, v)


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("q", list(ELEMENTS))
def test_mx8_dequantize_every_value(t, q):
    codes, e = all_values(q)
    Xq, SX = put_mx8(codes, e, q)
    X = torch.empty((256, 256), dtype=TYPES[t], device=dev())
    mm.mx8_dequantize(Xq, SX, X)
    with np.errstate(over="ignore"):
        want = finite_rounded(R.mx8_values(codes, e, q), TYPES[t])
    assert np.array_equal(exact(X), want, equal_nan=True)


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("M,K", [(1, 1), (3, 31), (34, 200), (65, 1000)])
def test_mx8_dequantize_ragged(t, M, K):
    g = rng(t, M, K)
    for q in ELEMENTS:
        codes, e = R.mx8_quantize(g.standard_normal((M, K)).astype(np.float32).astype(np.float64), q)
        Xq, SX = put_mx8(codes, e, q)
        per = 16 // torch.empty((), dtype=TYPES[t]).element_size()
        buf, X = guarded(M, K, TYPES[t], -(-K // per) * per + per, -77.0)
        mm.mx8_dequantize(Xq, SX, X)
        torch.cuda.synchronize()
        assert np.array_equal(exact(X), finite_rounded(R.mx8_values(codes, e, q)[:, :K], TYPES[t]))
        check_guards(buf, M, K, -77.0)


@pytest.mark.parametrize("qx,qw", [("e4m3", "e4m3"), ("e5m2", "e4m3")])
def test_mx8_matrices_feed_the_block_scaled_product(qx, qw):
    """What mx8_quantize stores is gemm_mx's operand: their product against the stored values in 64 bits (that
    instruction's own bound, 2^-13 of the magnitudes' sum, added)."""
    M, N, K = 70, 100, 320
    g = rng(qx, qw)
    X, W = rounded(g.standard_normal((M, K)), torch.bfloat16), rounded(g.standard_normal((N, K)) / 18, torch.bfloat16)
    parts = []
    for x, q in ((X, qx), (W, qw)):
        rows = x.shape[0]
        Xq = torch.empty((rows, K), dtype=ELEMENTS[q], device=dev())
        SX = torch.empty((3, -(-rows // 4) * 4), dtype=torch.int32, device=dev())[:, :rows]
        mm.mx8_quantize(pitched(x, torch.bfloat16), Xq, SX)
        codes, e = R.mx8_quantize(x, q)
        parts.append((Xq, SX, R.mx8_values(codes, e, q)))
    D = torch.empty((M, N), device=dev())
    (Xq, SX, x), (Wq, SW, w) = parts
    mm.gemm_mx(Xq, SX, Wq, SW, D)
    S = np.abs(x) @ np.abs(w).T
    assert (np.abs(exact(D) - x @ w.T) <= (2 * (K + 32) * R.U32 + 2.0 ** -13) * S).all()


# ---- weight gradient -----------------------------------------------------------------------------

def wgrad_problem(M, N, K, t, q, key=0):
    g = rng(M, N, K, t, q, key)
    Y = rounded(g.standard_normal((M, N)), TYPES[t])
    X = g.standard_normal((M, K)) * np.exp(g.uniform(-3, 3, (1, K)))
    codes, e = R.mx8_quantize(X.astype(np.float32).astype(np.float64), q)
    return Y, codes, e


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("q", list(ELEMENTS))
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (5, 7, 33), (64, 32, 128), (65, 33, 130), (300, 64, 257), (511, 65, 96),
                                   (1000, 130, 300), (2113, 20, 260)])
def test_wgrad_matches_reference(t, q, M, N, K):
    Y, codes, e = wgrad_problem(M, N, K, t, q)
    Xq, SX = put_mx8(codes, e, q)
    V = R.mx8_values(codes, e, q)[:, :K]
    # fp16: elements below its normal range are rounded to its subnormals, half a step of 2^-24 each
    slack = (np.abs(Y).T @ np.ones_like(V)) * 2.0 ** -25 if t == "fp16" else 0.0
    ref, S = Y.T @ V, np.abs(Y).T @ np.abs(V)
    for ws in (None, mm.mx8_wgrad_workspace(M, N, K)):
        buf, D = guarded(N, K, torch.float32, K + 5, -77.0)
        mm.gemm_mx8_wgrad(pitched(Y, TYPES[t], 1), Xq, SX, D, workspace=ws)
        torch.cuda.synchronize()
        check_sum(D, ref, S + slack / (2 * (M + 32) * R.U32), M, what=f"{t} {q} {M}x{N}x{K}")
        check_guards(buf, N, K, -77.0)
        if ws is not None:
            assert int(ws[:4 * 1024].view(torch.int32)[:((N + 31) // 32) * ((K + 127) // 128)].abs().max()) == 0, "counters"


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("q", list(ELEMENTS))
def test_wgrad_of_the_identity_is_the_input(t, q):
    """dY = 1 on the diagonal: D is X in dY's type, for every code (but those of NaN and infinity) and every exponent."""
    codes, e = all_values(q)
    V = R.mx8_values(codes, e, q)
    ok = np.isfinite(V)
    codes = np.where(ok, codes, 0)
    e = np.where(e == 255, 127, e)
    with np.errstate(over="ignore", invalid="ignore"):
        want = torch.from_numpy(R.mx8_values(codes, e, q)).to(TYPES[t]).double().numpy()
    keep = np.isfinite(want).all(1)                 # rows whose values all fit the type
    codes, e = np.where(keep[:, None], codes, 0), np.where(keep[:, None], e, 127)
    want = np.where(keep[:, None], want, 0)
    # products and sums of fp32 subnormals may be flushed: below bf16's normal range compare to that
    small = np.abs(want) < 2.0 ** -126
    Xq, SX = put_mx8(codes, e, q)
    D = torch.empty((256, 256), device=dev())
    mm.gemm_mx8_wgrad(torch.eye(256, dtype=TYPES[t], device=dev()), Xq, SX, D)
    D = exact(D)
    assert np.array_equal(D[~small], want[~small])
    assert (np.abs(D[small]) <= 2.0 ** -126).all()


@pytest.mark.parametrize("t,q", [("bf16", "e4m3"), ("bf16", "int8"), ("fp16", "e5m2")])
@pytest.mark.parametrize("M", [100, 201])
def test_wgrad_widest_tile(t, q, M):
    """Enough 256 x 256 tiles (14 x 15) for the widest kernel, ragged at every edge."""
    N, K = 3500, 3601
    assert mm.mx8_wgrad_workspace_bytes(M, N, K) == 0
    Y, codes, e = wgrad_problem(M, N, K, t, q)
    Xq, SX = put_mx8(codes, e, q)
    V = R.mx8_values(codes, e, q)[:, :K]
    slack = (np.abs(Y).T @ np.ones_like(V)) * 2.0 ** -25 if t == "fp16" else 0.0
    buf, D = guarded(N, K, torch.float32, K + 5, -77.0)
    mm.gemm_mx8_wgrad(pitched(Y, TYPES[t], 1), Xq, SX, D)
    torch.cuda.synchronize()
    check_sum(D, Y.T @ V, np.abs(Y).T @ np.abs(V) + slack / (2 * (M + 32) * R.U32), M)
    check_guards(buf, N, K, -77.0)


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("q", list(ELEMENTS))
def test_wgrad_non_finite_values_stay_in_their_columns(t, q):
    M, N, K = 130, 33, 200
    Y, codes, e = wgrad_problem(M, N, K, t, q)
    e[129, 3] = 255
    bad = np.zeros(K, bool)
    bad[96:128] = True
    if q != "int8":
        codes[5, 170] = 0x7f if q == "e4m3" else 0xfc     # NaN, -infinity
        bad[170] = True
    Xq, SX = put_mx8(codes, e, q)
    D = torch.empty((N, K), device=dev())
    mm.gemm_mx8_wgrad(pitched(Y, TYPES[t]), Xq, SX, D)
    D = exact(D)
    assert not np.isfinite(D[:, bad]).any() and np.isfinite(D[:, ~bad]).all()


def test_wgrad_nan_block_and_elements():
    """e = 255 makes its block NaN, a NaN element its column of D; other columns stay clean."""
    M, N, K = 70, 40, 160
    Y, codes, e = wgrad_problem(M, N, K, "bf16", "e4m3")
    clean = R.mx8_values(codes, e, "e4m3")
    e[3, 2] = 255
    codes[69, 7] = 0x7f
    Xq, SX = put_mx8(codes, e, "e4m3")
    D = torch.empty((N, K), device=dev())
    mm.gemm_mx8_wgrad(pitched(Y, torch.bfloat16), Xq, SX, D)
    D = exact(D)
    bad = np.zeros(K, bool)
    bad[64:96], bad[7] = True, True
    assert np.isnan(D[:, bad]).all()
    ref, S = Y.T @ clean, np.abs(Y).T @ np.abs(clean)
    assert (np.abs(D - ref)[:, ~bad] <= 2 * (M + 32) * R.U32 * S[:, ~bad]).all()


@pytest.mark.parametrize("out", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("N", [24, 60, 150])
def test_wgrad_accumulates(out, N):
    """alpha, beta * C, in place, 16-bit outputs; the same bits on every run."""
    M, K, o = 700, 200, TYPES[out]
    Y, codes, e = wgrad_problem(M, N, K, "bf16", "e4m3")
    C = rounded(rng(out, N).standard_normal((N, K)) * 10, o)
    V = R.mx8_values(codes, e, "e4m3")[:, :K]
    ref, S = 0.5 * (Y.T @ V) + 2.0 * C, 0.5 * (np.abs(Y).T @ np.abs(V)) + 2.0 * np.abs(C)
    Xq, SX = put_mx8(codes, e, "e4m3")
    Yd, ws = pitched(Y, torch.bfloat16), mm.mx8_wgrad_workspace(M, N, K)
    first = None
    for _ in range(3):
        D = torch.from_numpy(C).to(dev()).to(o)
        mm.gemm_mx8_wgrad(Yd, Xq, SX, D, alpha=0.5, beta=2.0, C=D, workspace=ws)
        check_sum(D, ref, S, M, o)
        first = D.clone() if first is None else first
        assert torch.equal(D, first)


def test_wgrad_without_rows():
    D = torch.full((8, 40), float("nan"), device=dev())
    C = torch.randn(8, 40, device=dev())
    Y = torch.empty((0, 8), dtype=torch.bfloat16, device=dev())
    Xq, SX = torch.empty((0, 64), dtype=torch.int8, device=dev()), torch.empty((1, 0), dtype=torch.int32, device=dev())
    mm.gemm_mx8_wgrad(Y, Xq, SX, D, beta=-1.5, C=C)
    assert torch.equal(D, -1.5 * C)
    mm.gemm_mx8_wgrad(Y, Xq, SX, D)
    assert (D == 0).all()


# ---- together ------------------------------------------------------------------------------------

def adapter_step(buf, stream=None):
    """One step of a low-rank adapter (B @ A) on a frozen 4-bit weight: y = x W^T + (x A^T) B^T, the input kept in 8
    bits, and the gradients of both factors for a given dy."""
    mm.gemm_w4(buf["x"], buf["Wq"], buf["SW"], buf["y"], workspace=buf["ws4"], stream=stream)
    mm.gemm_dense(buf["x"], buf["A"], buf["h"], stream=stream)
    mm.gemm_dense(buf["h"], buf["B"], buf["y"], beta=1.0, C=buf["y"], stream=stream)
    mm.mx8_quantize(buf["x"], buf["xq"], buf["sx"], stream=stream)
    mm.mx8_quantize(buf["h"], buf["hq"], buf["sh"], stream=stream)
    mm.gemm_layout(buf["dy"], buf["B"], buf["dh"], trans_b=True, stream=stream)
    mm.gemm_mx8_wgrad(buf["dy"], buf["hq"], buf["sh"], buf["dB"], workspace=buf["wsB"], stream=stream)
    mm.gemm_mx8_wgrad(buf["dh"], buf["xq"], buf["sx"], buf["dA"], workspace=buf["wsA"], stream=stream)


def adapter_buffers(M=200, N=320, K=512, r=32, seed=0):
    g = torch.Generator().manual_seed(seed)
    d, bf = dev(), torch.bfloat16
    rand = lambda *s: torch.randn(*s, generator=g).to(d)   # noqa: E731
    W = (rand(N, K) / K ** 0.5).to(bf)
    b = dict(x=rand(M, K).to(bf), A=(rand(r, K) / K ** 0.5).to(bf), B=(rand(N, r) / 6).to(bf), dy=rand(M, N).to(bf), W=W,
             Wq=torch.empty((N, K // 2), dtype=torch.uint8, device=d), SW=torch.empty((K // 128, N), dtype=torch.int32, device=d),
             y=torch.empty((M, N), device=d), h=torch.empty((M, r), dtype=bf, device=d),
             xq=torch.empty((M, K), dtype=torch.float8_e4m3fn, device=d), sx=torch.empty((K // 128, M), dtype=torch.int32, device=d),
             hq=torch.empty((M, r), dtype=torch.int8, device=d), sh=torch.empty((1, M), dtype=torch.int32, device=d),
             dh=torch.empty((M, r), dtype=bf, device=d), dA=torch.empty((r, K), device=d), dB=torch.empty((N, r), device=d),
             ws4=mm.w4_workspace(M, N, K), wsA=mm.mx8_wgrad_workspace(M, r, K), wsB=mm.mx8_wgrad_workspace(M, N, r))
    mm.w4_quantize(W, b["Wq"], b["SW"])
    return b


def test_adapter_step_against_the_formulas():
    """Forward and both gradients of the step in 64 bits.  The stored input is within half a step of its 8-bit type of
    the true one (e4m3: 2^-4 of the value or 2^-10 of the block's scale; int8: half its scale), so each gradient is
    within sum |dy| times that, plus the products' own bounds."""
    b = adapter_buffers()
    adapter_step(b)
    x, A, B, dy, h, dh = (exact(b[k]) for k in ("x", "A", "B", "dy", "h", "dh"))
    M, K = x.shape
    codes, s, z = R.w4_quantize(exact(b["W"]), 128, R.U4, False)
    y, S = R.gemm_w4(x, codes, s, z, 128, R.U4)
    y, S = y + h @ B.T, S + np.abs(h) @ np.abs(B).T
    check_sum(b["y"], y, S, K + 32)
    check_sum(b["dh"], dy @ B, np.abs(dy) @ np.abs(B), dy.shape[1], torch.bfloat16)
    qx, ex = R.mx8_quantize(x, "e4m3")
    qh, eh = R.mx8_quantize(h, "int8")
    vx, vh = R.mx8_values(qx, ex, "e4m3"), R.mx8_values(qh, eh, "int8")
    check_sum(b["dA"], dh.T @ vx, np.abs(dh).T @ np.abs(vx), M)
    check_sum(b["dB"], dy.T @ vh, np.abs(dy).T @ np.abs(vh), M)
    scale_x = np.repeat(np.ldexp(1.0, ex - 127), 32, 1)
    scale_h = np.repeat(np.ldexp(1.0, eh - 127), 32, 1)
    off_x, off_h = np.maximum(np.abs(x) * 2.0 ** -4, scale_x * 2.0 ** -10), scale_h * 0.5
    assert (np.abs(vx - x) <= off_x).all() and (np.abs(vh - h) <= off_h).all()
    for got, dl, v, true, off in ((b["dA"], dh, vx, x, off_x), (b["dB"], dy, vh, h, off_h)):
        own = 2 * (M + 32) * R.U32 * (np.abs(dl).T @ np.abs(v))
        assert (np.abs(exact(got) - dl.T @ true) <= np.abs(dl).T @ off + own).all()


def test_wgrad_against_differences():
    """L(W) = sum(dY * (X W^T)) is linear in W: (L(W + E) - L(W - E)) / 2 for a unit step E of one entry is that entry
    of the gradient.  With small integers every product is exact, so both must agree bit for bit."""
    M, N, K = 96, 40, 64
    g = rng("differences")
    X, Y, W = (g.integers(-3, 4, shape).astype(np.float64) for shape in ((M, K), (M, N), (N, K)))
    codes, e = R.mx8_quantize(X, "int8")
    Xq, SX = put_mx8(codes, e, "int8")
    D = torch.empty((N, K), device=dev())
    mm.gemm_mx8_wgrad(pitched(Y, torch.bfloat16), Xq, SX, D)
    Xd, Yd, out = pitched(X, torch.bfloat16), torch.from_numpy(Y).to(dev()), torch.empty((M, N), device=dev())

    def loss(Wh):
        mm.gemm_dense(Xd, pitched(Wh, torch.bfloat16), out)
        return float((out.double() * Yd).sum())

    for n, k in ((0, 0), (39, 63), (17, 5), (8, 40)):
        E = np.zeros_like(W)
        E[n, k] = 1
        assert (loss(W + E) - loss(W - E)) / 2 == float(D[n, k])


def test_captured_step_replays_like_the_eager_one():
    """The whole step in one captured graph, replayed with changed inputs, eager steps (with workspaces of their own)
    and synchronisations in between."""
    b, eager = adapter_buffers(seed=1), adapter_buffers(seed=1)
    names = ("y", "h", "dh", "dA", "dB")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        adapter_step(b)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        adapter_step(b)
    g = torch.Generator().manual_seed(9)
    for rep in range(4):
        for k in ("x", "dy"):
            new = torch.randn(b[k].shape, generator=g).to(dev()).to(torch.bfloat16)
            b[k].copy_(new)
            eager[k].copy_(new)
        for k in names:
            b[k].fill_(float("nan"))
        adapter_step(eager)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k in names + ("xq", "sx", "hq", "sh"):
            w = lambda v: v.contiguous().view(torch.uint8)   # noqa: E731
            assert torch.equal(w(b[k]), w(eager[k])), f"replay {rep}: {k}"


def test_two_streams_at_once():
    """Steps on two streams, each with its own buffers and workspaces, give what they give alone."""
    bufs = [adapter_buffers(seed=s) for s in (3, 4)]
    want = []
    for b in bufs:
        adapter_step(b)
        torch.cuda.synchronize()
        want.append({k: b[k].clone() for k in ("y", "dA", "dB")})
    streams = [torch.cuda.Stream() for _ in bufs]
    for _ in range(5):
        for b, s in zip(bufs, streams):
            adapter_step(b, stream=s)
    torch.cuda.synchronize()
    for b, w in zip(bufs, want):
        for k in w:
            assert torch.equal(b[k], w[k])


def test_matrices_beyond_four_gib():
    """Codes and elements whose offsets pass 32 bits: the last rows come out as they do alone."""
    rows, K, last = (1 << 19) + 133, 8192, 133
    d = dev()
    # 8-bit: quantize rows past the 4 GiB border of X's 8 GiB and Xq's 4 GiB
    X = torch.zeros((rows, K), dtype=torch.bfloat16, device=d)
    g = torch.Generator(device=d).manual_seed(5)
    X[-last:] = torch.randn((last, K), generator=g, device=d).to(torch.bfloat16)
    Xq = torch.empty((rows, K), dtype=torch.float8_e4m3fn, device=d)
    SX = torch.empty((K // 128, rows), dtype=torch.int32, device=d)
    mm.mx8_quantize(X, Xq, SX)
    q1, s1 = torch.empty((last, K), dtype=torch.float8_e4m3fn, device=d), torch.empty((K // 128, last), dtype=torch.int32, device=d)
    mm.mx8_quantize(X[-last:], q1, s1)
    assert torch.equal(Xq[-last:].view(torch.uint8), q1.view(torch.uint8)) and torch.equal(SX[:, -last:].contiguous(), s1)
    X.fill_(1.0)
    mm.mx8_dequantize(Xq, SX, X)
    x1 = torch.empty((last, K), dtype=torch.bfloat16, device=d)
    mm.mx8_dequantize(q1, s1, x1)
    assert torch.equal(X[-last:], x1)
    # its gradient: only the last rows of dY are not zero
    N = 16
    dY = torch.zeros((rows, N), dtype=torch.bfloat16, device=d)
    dY[-last:] = torch.randn((last, N), generator=g, device=d).to(torch.bfloat16)
    D, D1 = torch.empty((N, K), device=d), torch.empty((N, K), device=d)
    mm.gemm_mx8_wgrad(dY, Xq, SX, D, workspace=mm.mx8_wgrad_workspace(rows, N, K))
    mm.gemm_mx8_wgrad(dY[-last:].contiguous(), q1, s1, D1)
    y, v = dY[-last:].double(), x1.double()
    S = y.abs().t() @ v.abs()
    assert ((D.double() - D1.double()).abs() <= 4 * (last + 32) * R.U32 * S).all()
    del X, Xq, SX, dY
    # 4-bit: 2^20 + 133 rows of 4096 bytes of codes
    rows = (1 << 20) + last
    Wq = torch.zeros((rows, K // 2), dtype=torch.uint8, device=d)
    SW = torch.zeros((1, rows), dtype=torch.int32, device=d)
    W = torch.randn((last, K), generator=g, device=d).to(torch.bfloat16)
    mm.w4_quantize(W, Wq[-last:], SW[:, -last:], group=0)
    for M in (2, 40):
        A = torch.randn((M, K), generator=g, device=d).to(torch.bfloat16)
        D = torch.empty((M, rows), device=d)
        mm.gemm_w4(A, Wq, SW, D, group=0, workspace=mm.w4_workspace(M, rows, K))
        D1 = torch.empty((M, last), device=d)
        mm.gemm_w4(A, Wq[-last:], SW[:, -last:], D1, group=0)
        # the same sums, perhaps in another order: 2 (K + 32) u of them, twice
        ref = D1.double()
        bound = 4 * (K + 32) * R.U32 * 32 * (A.double().abs() @ W.double().abs().t())
        assert ((D[:, -last:].double() - ref).abs() <= bound).all()
        assert (D[:, :-last] == 0).all()


# ---- finite elements past dY's type ----------------------------------------------------------------

@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("q", list(ELEMENTS))
def test_wgrad_reads_what_the_dequantizer_restores(t, q):
    """dY = 1 on the diagonal, every finite code with every exponent: D is what mx8_dequantize gives in dY's type, at
    its ends too (finite elements saturate)."""
    codes, e = all_values(q)
    codes = np.where(np.isfinite(R.mx8_values(codes, np.full_like(e, 127), q)), codes, 0)
    e = np.where(e == 255, 127, e)
    want = finite_rounded(R.mx8_values(codes, e, q), TYPES[t])
    Xq, SX = put_mx8(codes, e, q)
    X, D = torch.empty((256, 256), dtype=TYPES[t], device=dev()), torch.empty((256, 256), device=dev())
    mm.mx8_dequantize(Xq, SX, X)
    mm.gemm_mx8_wgrad(torch.eye(256, dtype=TYPES[t], device=dev()), Xq, SX, D)
    assert np.array_equal(exact(X), want)
    D = exact(D)
    small = np.abs(want) < 2.0 ** -126                     # fp32 subnormals may be flushed
    assert np.array_equal(D[~small], want[~small])
    assert (np.abs(D[small]) <= 2.0 ** -126).all()


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("q", list(ELEMENTS))
@pytest.mark.parametrize("N", [1, 40, 200])
def test_wgrad_saturates_next_to_infinities_and_nan(t, q, N):
    """One row: each column of D is dY times one element.  Blocks at the border of the type's range and past it, every
    code in each; infinities and NaN of the element type, and of a block (e = 255), stay."""
    border = {"e4m3": {"fp16": 135, "bf16": 247}, "e5m2": {"fp16": 128, "bf16": 240}, "int8": {"fp16": 136, "bf16": 248}}[q][t]
    exps = np.array([127, border - 1, border, border + 1, 254, 255])
    K = 256 * len(exps)
    codes = np.tile(np.arange(256), len(exps))[None]
    codes = codes.astype(np.int8).astype(np.int64) if q == "int8" else codes
    e = np.repeat(exps, 8)[None]
    v = finite_rounded(R.mx8_values(codes, e, q), TYPES[t])
    Xq, SX = put_mx8(codes, e, q)
    y = 2.0 ** -np.arange(N)[None] * (-1.0) ** np.arange(N) if N <= 2 else 2.0 ** -(np.arange(N)[None] % 5) * (-1.0) ** np.arange(N)
    D = torch.empty((N, K), device=dev())
    mm.gemm_mx8_wgrad(pitched(y, TYPES[t]), Xq, SX, D, workspace=mm.mx8_wgrad_workspace(1, N, K))
    with np.errstate(invalid="ignore"):
        assert np.array_equal(exact(D), y.T @ v if np.isfinite(v).all() else y.T * v, equal_nan=True)


@pytest.mark.parametrize("q", list(ELEMENTS))
def test_wgrad_of_the_largest_fp16_activations_is_finite(q):
    """fp16 inputs up to 65504 round up to 65536 in 8 bits; the gradient sees 65504 there, in the widest tiles too."""
    M, N, K = 70, 3500, 3601
    g = rng(q)
    X = g.choice([-65504.0, 65504.0, 63488.0, 61440.0, 1000.0], (M, K))
    X[:, ::7] = 65504.0
    Xq = torch.empty((M, -(-K // 32) * 32), dtype=ELEMENTS[q], device=dev())
    SX = torch.empty((-(-K // 128), M), dtype=torch.int32, device=dev())
    mm.mx8_quantize(pitched(X, torch.float16), Xq, SX)
    codes, e = R.mx8_quantize(X, q)
    V = np.clip(R.mx8_values(codes, e, q)[:, :K], -65504, 65504)
    assert (np.abs(R.mx8_values(codes, e, q)) > 65504).any()
    Y = rounded(g.standard_normal((M, N)), torch.float16)
    D = torch.empty((N, K), device=dev())
    mm.gemm_mx8_wgrad(pitched(Y, torch.float16), Xq, SX, D)
    check_sum(D, Y.T @ V, np.abs(Y).T @ np.abs(V), M)


# ---- the zero points' term of many rows --------------------------------------------------------------

def bf16_rest(x):
    """x less its nearest bf16 value."""
    return x - rounded(x, torch.bfloat16)


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("M,N", [(40, 150), (130, 200), (1601, 3900)])
def test_gemm_w4_long_row_sums_exact(t, group, M, N):
    """Group sums of A of 19 bits with a large mean, under large zero points: as bf16 terms they need all three.  Four
    elements of 65280 (8 significant bits) and odd ones up to 255 in each group: sum |a| over K stays below 2^19.2, times
    15 below 2^24, so that every sum is exact in fp32 and the result must match bit for bit."""
    width = group if group else 128                 # whole rows are summed in chunks of 128
    K = 2 * width + 16
    g = rng(t, group, M, N)
    A = 2.0 * g.integers(0, 128, (M, K)) + 1
    for k in range(0, 2 * width, width):
        for i in range(M):
            A[i, k + g.permutation(width)[:5]] = 65280, 65280, 65280, 65280, 2      # an odd sum
    A[::3] *= -1
    assert np.abs(A).sum(1).max() * 15 < 2 ** 24 and (rounded(A, TYPES[t]) == A).all()
    for k in range(0, 2 * width, width):            # what the third term is for
        assert (bf16_rest(bf16_rest(A[:, k:k + width].sum(1))) != 0).mean() > 0.5
    G = R.n_groups(K, group)
    codes, z, s = g.integers(0, 16, (N, K)), g.integers(11, 16, (N, G)), 2.0 ** g.integers(-2, 1, (N, G))
    if group:
        s[:] = s[:, :1]                             # one scale per row, so that the groups' total is exact too
    ref, _ = R.gemm_w4(A, codes, s, z, group, R.U4)
    Wq, SW = w4_tensors(codes, s, z)
    D = torch.full((M, N), float("nan"), device=dev())
    mm.gemm_w4(pitched(A, TYPES[t]), Wq, SW, D, group=group, workspace=mm.w4_workspace(M, N, K))
    assert np.array_equal(exact(D), ref)


@pytest.mark.parametrize("q_type", [R.U4, R.FP4])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("M", [1, 20, 40, 130])
def test_gemm_w4_fp16_subnormals_exact(q_type, group, M):
    """A of multiples of 2^-24 below fp16's normal range (|a| <= 200 units): sums below 2^24 units, bit for bit."""
    N, K = 70, 300
    _, codes, s, z = w4_problem(M, N, K, group, q_type, "fp16", integers=True)
    A = rng(M, group, q_type).integers(-200, 201, (M, K)) * 2.0 ** -24
    ref, _ = R.gemm_w4(A, codes, s, z, group, q_type)
    Wq, SW = w4_tensors(codes, s, z)
    D = torch.full((M, N), float("nan"), device=dev())
    mm.gemm_w4(pitched(A, torch.float16), Wq, SW, D, group=group, q_type=q_type, workspace=mm.w4_workspace(M, N, K))
    assert np.array_equal(exact(D), ref)


# ---- paths of large and odd calls ----------------------------------------------------------------------

@pytest.mark.parametrize("N", [20, 60, 150])
@pytest.mark.parametrize("t,top", [(torch.float8_e4m3fn, 448.0), (torch.float8_e5m2, 57344.0)])
def test_wgrad_fp8_outputs_saturate(N, t, top):
    """Small integers, so that the sum is exact and only the output rounds."""
    M, K = 300, 160
    g = rng(N, top)
    X, Y = g.integers(-4, 5, (M, K)).astype(np.float64), g.integers(-4, 5, (M, N)).astype(np.float64)
    C = rounded(g.integers(-200, 201, (N, K)).astype(np.float64), t)
    codes, e = R.mx8_quantize(X, "int8")
    Xq, SX = put_mx8(codes, e, "int8")
    ref = 64 * (Y.T @ X) + 2 * C
    assert (np.abs(ref) > top).any() == (top == 448.0)
    D = torch.from_numpy(C).to(dev()).to(t)
    mm.gemm_mx8_wgrad(pitched(Y, torch.bfloat16), Xq, SX, D, alpha=64.0, beta=2.0, C=D, workspace=mm.mx8_wgrad_workspace(M, N, K))
    assert np.array_equal(exact(D), torch.from_numpy(np.clip(ref, -top, top)).float().to(t).double().numpy())


@pytest.mark.parametrize("q_type,symmetric", FORMS)
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_w4_quantize_long_rows_that_hold_non_finite_values(q_type, symmetric, bad):
    """Rows of several passes of a workgroup (2048 elements each), the value in the first, a middle and the last one."""
    W = rng(q_type, symmetric, str(bad)).standard_normal((5, 7000))
    W[0, 3], W[1, 2047], W[2, 3000], W[3, 6999] = bad, bad, bad, bad
    Wq, SW, W = run_w4_quantize(W, torch.float32, 0, q_type, symmetric)
    codes, s, z = R.w4_quantize(W, 0, q_type, symmetric)
    assert np.isnan(s[:4]).all() and np.isfinite(s[4]).all()
    assert np.array_equal(SW.cpu().numpy(), R.scale_words(s, z))
    assert np.array_equal(Wq.cpu().numpy(), R.pack_codes(codes))


@pytest.mark.parametrize("group", [0, 32, 64, 128])
def test_gemm_w4_nan_scales_in_the_widest_tile(group):
    """NaN groups, one row of W in a group that ends short, and non-finite rows of A: nothing else changes."""
    M, N, K = 1601, 3900, 160
    A, codes, s, z = w4_problem(M, N, K, group, R.U4, "bf16", integers=True)
    ref, _ = R.gemm_w4(A, codes, s, z, group, R.U4)
    s[7, 0] = s[3899, -1] = s[300, s.shape[1] // 2] = np.nan
    A[130, 159], A[1600, 0] = np.nan, np.inf
    clean = np.ones((M, N), bool)
    clean[[130, 1600]] = False
    clean[:, [7, 300, 3899]] = False
    Wq, SW = w4_tensors(codes, s, z)
    D = torch.empty((M, N), device=dev())
    mm.gemm_w4(pitched(A, torch.bfloat16), Wq, SW, D, group=group)
    D = exact(D)
    assert np.array_equal(D[clean], ref[clean])
    assert not np.isfinite(D[~clean]).any()


def test_more_units_than_workgroups():
    """The grids stop at 2^20 workgroups: what comes after is their second turn.  Rows of 8 elements, 32 per unit (one
    per unit in the whole-row quantizer)."""
    d = dev()
    rows, K = (32 << 20) + 77, 8
    g = torch.Generator(device=d).manual_seed(11)
    X = torch.randn((rows, K), generator=g, device=d).to(torch.bfloat16)
    last = slice(rows - 200, rows)                      # on both sides of the border
    Xq, SX = torch.zeros((rows, 32), dtype=torch.float8_e4m3fn, device=d), torch.zeros((1, rows), dtype=torch.int32, device=d)
    mm.mx8_quantize(X, Xq, SX)
    codes, e = R.mx8_quantize(exact(X[last]), "e4m3")
    assert np.array_equal(SX[:, last].cpu().numpy(), R.sx_words(e))
    assert np.array_equal(Xq[last].view(torch.uint8).cpu().numpy(), (codes & 255).astype(np.uint8))
    back = torch.full((rows, K), float("nan"), dtype=torch.bfloat16, device=d)
    mm.mx8_dequantize(Xq, SX, back)
    assert np.array_equal(exact(back[last]), finite_rounded(R.mx8_values(codes, e, "e4m3")[:, :K], torch.bfloat16))
    assert not back.isnan().any()
    del Xq, SX, back
    for group, n in ((32, rows), (0, (1 << 20) + 77)):
        Wq, SW = torch.zeros((n, 16), dtype=torch.uint8, device=d), torch.zeros((1, n), dtype=torch.int32, device=d)
        mm.w4_quantize(X[:n], Wq, SW, group=group)
        codes, s, z = R.w4_quantize(exact(X[n - 200:n]), group, R.U4, False)
        assert np.array_equal(SW[:, n - 200:].cpu().numpy(), R.scale_words(s, z))
        assert np.array_equal(Wq[n - 200:].cpu().numpy(), R.pack_codes(codes))
        assert int((SW == 0).sum()) == 0
