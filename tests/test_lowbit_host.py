"""Host-side checks of the low-bit entry points (no GPU needed, no compute call).

include/mmac_lowbit.h and the library agree; every argument error is reported before
any GPU work (the pointers passed here are fake); the binding refuses tensors that do not
fit the call; the workspace plans; and the 64-bit references agree with each other.
"""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import lowbit_ref as R
import sparse_matrix_multiply_amd as mm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20          # a fake, 16-byte aligned "device pointer": never dereferenced here
OK, INV, UNS, MIS = mm.OK, mm.ERR_INVALID_ARG, mm.ERR_UNSUPPORTED, mm.ERR_MISALIGNED


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(mm.LIB_PATH):
        from sparse_matrix_multiply_amd import build
        build.build()
    return mm.lib()


def test_header_and_library_agree(L):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "mmac_lowbit.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(mmac_[a-z0-9_]+)\s*\(", text)))
    assert names == ["mmac_gemm_mx8_wgrad", "mmac_gemm_mx8_wgrad_workspace_bytes", "mmac_gemm_w4",
                     "mmac_gemm_w4_workspace_bytes", "mmac_mx8_dequantize", "mmac_mx8_quantize", "mmac_w4_quantize"]
    for name in names:
        assert hasattr(L, name), name


def w4(**kw):
    a = dict(q_type=mm.U4, group=32, codes=P, pitch=32, words=P, ldw=64)
    a.update(kw)
    return mm.W4(*[a[k] for k in ("q_type", "group", "codes", "pitch", "words", "ldw")])


W4_ERRORS = [
    (dict(q_type=mm.I8), UNS), (dict(q_type=0), UNS), (dict(group=16), UNS), (dict(group=-1), UNS),
    (dict(group=256), UNS), (dict(codes=None), INV), (dict(words=None), INV), (dict(pitch=16), INV),
    (dict(pitch=-32), INV), (dict(pitch=40), MIS), (dict(codes=P + 8), MIS), (dict(words=P + 2), MIS),
    (dict(pitch=(1 << 23) + 16), UNS), (dict(ldw=63), INV), (dict(ldw=0), INV), (dict(ldw=1 << 28), UNS),
    (dict(ldw=(1 << 63) - 1), UNS), (dict(pitch=(1 << 63) - 16), UNS),
]


def quantize(L, q=None, **kw):
    a = dict(t=mm.BF16, sym=0, N=64, K=64, W=P, ld=64)
    a.update(kw)
    return L.mmac_w4_quantize(a["t"], a["sym"], a["N"], a["K"], a["W"], a["ld"],
                              ctypes.byref(q if q is not None else w4()), None)


@pytest.mark.parametrize("kw,code", [
    (dict(t=mm.I8), UNS), (dict(t=mm.FP8_E4M3), UNS), (dict(N=-1), INV), (dict(K=1 << 31), INV), (dict(W=None), INV),
    (dict(sym=2), INV), (dict(ld=63), INV), (dict(ld=65), MIS), (dict(W=P + 4), MIS), (dict(ld=(1 << 22) + 8), UNS),
    (dict(ld=(1 << 63) - 1), UNS), (dict(t=mm.F32, ld=66), MIS),
])
def test_w4_quantize_argument_errors(L, kw, code):
    assert quantize(L, **kw) == code


@pytest.mark.parametrize("kw,code", W4_ERRORS)
def test_w4_matrix_errors(L, kw, code):
    assert quantize(L, w4(**kw)) == code
    assert gemm(L, w4(**kw)) == code


def test_w4_quantize_other_refusals(L):
    assert quantize(L, w4(q_type=mm.FP4_E2M1), sym=0) == UNS
    assert L.mmac_w4_quantize(mm.BF16, 0, 64, 64, P, 64, None, None) == INV
    for kw in (dict(N=0), dict(K=0, W=None)):
        assert quantize(L, **kw) == OK


def gemm(L, q=None, **kw):
    a = dict(t=mm.BF16, M=4, N=64, K=64, alpha=1.0, A=P, lda=64, beta=0.0, C=None, ldc=64, D=P, ldd=64, ep=None,
             ws=None, n=0)
    a.update(kw)
    return L.mmac_gemm_w4(a["t"], a["M"], a["N"], a["K"], a["alpha"], a["A"], a["lda"],
                          ctypes.byref(q if q is not None else w4()), a["beta"], a["C"], a["ldc"], a["D"], a["ldd"],
                          None if a["ep"] is None else ctypes.byref(a["ep"]), a["ws"], a["n"], None)


OUT_ERRORS = [
    (dict(D=None), INV), (dict(ldd=63), INV), (dict(beta=1.0), INV), (dict(beta=1.0, C=P, ldc=10), INV),
    (dict(beta=1.0, C=P, ldc=72), INV), (dict(alpha=float("nan")), INV), (dict(beta=float("inf"), C=P), INV),
    (dict(alpha=1e39), INV), (dict(D=P + 2), MIS), (dict(beta=1.0, C=P + 1), MIS), (dict(ldd=1 << 22), UNS),
    (dict(ws=P, n=-1), INV), (dict(ws=P + 8, n=1 << 20), MIS),
    (dict(ep=mm.Epilogue(9, 0, None)), INV), (dict(ep=mm.Epilogue(0, 7, None)), INV),
]


@pytest.mark.parametrize("kw,code", OUT_ERRORS + [
    (dict(t=mm.F32), UNS), (dict(t=mm.I8), UNS), (dict(M=-1), INV), (dict(N=1 << 31), INV), (dict(A=None), INV),
    (dict(lda=60), INV), (dict(lda=68), MIS), (dict(A=P + 8), MIS), (dict(lda=1 << 23), UNS),
    (dict(ep=mm.Epilogue(1, 0, P + 2)), MIS),
])
def test_gemm_w4_argument_errors(L, kw, code):
    assert gemm(L, **kw) == code


def test_gemm_w4_empty_is_a_no_op(L):
    assert gemm(L, M=0) == OK
    assert gemm(L, N=0) == OK
    assert L.mmac_gemm_w4(mm.BF16, 4, 64, 64, 1.0, P, 64, None, 0.0, None, 64, P, 64, None, None, 0, None) == INV


def mx8(L, entry, **kw):
    a = dict(x=mm.BF16, q=mm.FP8_E4M3, M=64, K=64, X=P, ldx=64, Xq=P, ldq=64, SX=P, lds=64)
    a.update(kw)
    if entry == "mmac_mx8_quantize":
        return L.mmac_mx8_quantize(a["x"], a["q"], a["M"], a["K"], a["X"], a["ldx"], a["Xq"], a["ldq"], a["SX"], a["lds"], None)
    return L.mmac_mx8_dequantize(a["q"], a["x"], a["M"], a["K"], a["Xq"], a["ldq"], a["SX"], a["lds"], a["X"], a["ldx"], None)


@pytest.mark.parametrize("entry", ["mmac_mx8_quantize", "mmac_mx8_dequantize"])
@pytest.mark.parametrize("kw,code", [
    (dict(x=mm.I8), UNS), (dict(q=mm.BF16), UNS), (dict(q=mm.FP4_E2M1), UNS), (dict(M=-1), INV), (dict(K=1 << 31), INV),
    (dict(X=None), INV), (dict(Xq=None), INV), (dict(SX=None), INV), (dict(ldx=60), INV), (dict(ldx=68), MIS),
    (dict(K=63, ldq=48), INV), (dict(K=33, ldx=40, ldq=48), INV), (dict(ldq=72), MIS), (dict(X=P + 2), MIS),
    (dict(Xq=P + 8), MIS), (dict(SX=P + 2), MIS), (dict(lds=63), INV), (dict(ldx=1 << 22 | 8), UNS),
    (dict(ldq=(1 << 23) + 16), UNS), (dict(lds=1 << 29), UNS), (dict(lds=(1 << 63) - 1), UNS),
])
def test_mx8_argument_errors(L, entry, kw, code):
    assert mx8(L, entry, **kw) == code


@pytest.mark.parametrize("entry", ["mmac_mx8_quantize", "mmac_mx8_dequantize"])
def test_mx8_empty_is_a_no_op(L, entry):
    assert mx8(L, entry, M=0) == OK
    assert mx8(L, entry, K=0, X=None, Xq=None, SX=None) == OK


def wgrad(L, **kw):
    a = dict(t=mm.BF16, q=mm.FP8_E4M3, M=64, N=64, K=64, alpha=1.0, Y=P, ldy=64, Xq=P, ldq=64, SX=P, lds=64, beta=0.0,
             C=None, ldc=64, D=P, ldd=64, ep=None, ws=None, n=0)
    a.update(kw)
    return L.mmac_gemm_mx8_wgrad(a["t"], a["q"], a["M"], a["N"], a["K"], a["alpha"], a["Y"], a["ldy"], a["Xq"], a["ldq"],
                                 a["SX"], a["lds"], a["beta"], a["C"], a["ldc"], a["D"], a["ldd"],
                                 None if a["ep"] is None else ctypes.byref(a["ep"]), a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,code", OUT_ERRORS + [
    (dict(t=mm.F32), UNS), (dict(q=mm.BF16), UNS), (dict(M=-1), INV), (dict(K=1 << 31), INV), (dict(Y=None), INV),
    (dict(Xq=None), INV), (dict(SX=None), INV), (dict(ldy=60), INV), (dict(ldy=68), MIS), (dict(Y=P + 4), MIS),
    (dict(ldq=48), INV), (dict(ldq=72), MIS), (dict(lds=60), INV), (dict(SX=P + 1), MIS), (dict(lds=1 << 29), UNS),
    (dict(ep=mm.Epilogue(0, 1, None)), UNS), (dict(ep=mm.Epilogue(0, 0, P)), UNS),
    (dict(N=1 << 30, K=1 << 20, ldy=1 << 30, ldq=1 << 20, ldd=1 << 20), UNS),
])
def test_wgrad_argument_errors(L, kw, code):
    assert wgrad(L, **kw) == code


def test_wgrad_empty_is_a_no_op(L):
    assert wgrad(L, N=0) == OK
    assert wgrad(L, K=0, Xq=None, SX=None) == OK


def test_workspace_plans(L):
    assert mm.mx8_wgrad_workspace_bytes(0, 64, 64) == 0
    assert mm.mx8_wgrad_workspace_bytes(8192, 32, 8192) > 0
    assert mm.mx8_wgrad_workspace_bytes(8192, 8192, 8192) == 0
    assert mm.mx8_wgrad_workspace_bytes(-1, 64, 64) == 0
    assert mm.w4_workspace_bytes(0, 64, 64) == 0
    assert mm.w4_workspace_bytes(-1, 64, 64) == 0


def test_binding_checks_before_any_launch():
    A = torch.zeros((4, 64), dtype=torch.bfloat16)
    Wq, SW = torch.zeros((32, 32), dtype=torch.uint8), torch.zeros((1, 32), dtype=torch.int32)
    D = torch.zeros((4, 32))
    W = torch.zeros((32, 64), dtype=torch.bfloat16)
    for kw in (dict(Wq=torch.zeros((32, 16), dtype=torch.uint8)), dict(Wq=torch.zeros((32, 32), dtype=torch.int16)),
               dict(SW=torch.zeros((1, 31), dtype=torch.int32)), dict(SW=torch.zeros((1, 32), dtype=torch.int64)),
               dict(group=32), dict(D=torch.zeros((4, 31))), dict(D=torch.zeros((4, 32), dtype=torch.float64)),
               dict(C=torch.zeros((3, 32)), beta=1.0), dict(bias=torch.zeros(31)), dict(A=torch.zeros((4, 64), dtype=torch.int32)),
               dict(a_type=mm.F32), dict(D=torch.zeros((1, 32)).expand(4, 32)), {}):
        args = dict(A=A, Wq=Wq, SW=SW, D=D)
        args.update(kw)
        with pytest.raises(ValueError):         # {}: host memory
            mm.gemm_w4(**args)
    for kw in (dict(Wq=torch.zeros((31, 32), dtype=torch.uint8)), dict(SW=torch.zeros((0, 32), dtype=torch.int32)), {}):
        args = dict(W=W, Wq=Wq, SW=SW)
        args.update(kw)
        with pytest.raises(ValueError):
            mm.w4_quantize(**args)
    X, Xq, SX = torch.zeros((4, 64)), torch.zeros((4, 64), dtype=torch.int8), torch.zeros((1, 4), dtype=torch.int32)
    for kw in (dict(Xq=torch.zeros((4, 48), dtype=torch.int8)), dict(Xq=torch.zeros((4, 64), dtype=torch.uint8)),
               dict(SX=torch.zeros((1, 3), dtype=torch.int32)), dict(SX=torch.zeros((1, 4), dtype=torch.int16)),
               dict(X=torch.zeros((4, 64), dtype=torch.float64)), {}):
        args = dict(X=X, Xq=Xq, SX=SX)
        args.update(kw)
        with pytest.raises(ValueError):
            mm.mx8_quantize(**args)
        with pytest.raises(ValueError):
            mm.mx8_dequantize(**args)
    dY, G = torch.zeros((4, 16), dtype=torch.bfloat16), torch.zeros((16, 64))
    for kw in (dict(dY=torch.zeros((3, 16), dtype=torch.bfloat16)), dict(D=torch.zeros((15, 64))),
               dict(D=torch.zeros((16, 128))), dict(C=torch.zeros((16, 63)), beta=1.0),
               dict(Xq=torch.zeros((4, 64), dtype=torch.uint8)), {}):
        args = dict(dY=dY, Xq=Xq, SX=SX, D=G)
        args.update(kw)
        with pytest.raises(ValueError):
            mm.gemm_mx8_wgrad(**args)


# ---- the references themselves ----

def test_reference_tables_against_torch():
    for pos, t in ((R.E4M3_POS, torch.float8_e4m3fn), (R.E5M2_POS, torch.float8_e5m2)):
        got = torch.arange(len(pos), dtype=torch.uint8).view(t).float().double().numpy()
        assert np.array_equal(got, pos)
        x = np.concatenate([pos, (pos[:-1] + pos[1:]) / 2, np.random.default_rng(0).uniform(0, pos[-1], 500)]).astype(np.float32)
        code = torch.from_numpy(x).to(t).view(torch.uint8).numpy()
        assert np.array_equal(code, R.rne_codes(x.astype(np.float64), pos))


@pytest.mark.parametrize("symmetric", [False, True])
@pytest.mark.parametrize("q_type", [R.U4, R.FP4])
def test_reference_quantizer_is_within_half_a_step(q_type, symmetric):
    if q_type == R.FP4 and not symmetric:
        return
    W = np.random.default_rng(1).standard_normal((7, 100)).astype(np.float32).astype(np.float64)
    codes, s, z = R.w4_quantize(W, 32, q_type, symmetric)
    V = R.w4_values(codes, s, z, 32, q_type)
    gi = R.group_index(100, 32)
    # half of the widest step (U4: 1; E2M1: 2), and the scale's own rounding (2^-17 of the largest value); not
    # symmetric: the zero point's rounding moves both ends by half a step more
    step = s[:, gi] * (1.0 if q_type == R.FP4 else 0.5 if symmetric else 1.0)
    assert (np.abs(V - W) <= step * (1 + 2.0 ** -12)).all()
    assert np.array_equal(R.unpack_codes(R.pack_codes(codes, 9), 100), codes)


def test_split_plans_agree_on_where_partial_tiles_begin(L):
    """Low-bit calls of every size share a workspace: 1 KiB of counters, at most 256, then the partial tiles."""
    tile = 64 * 128 * 4
    assert mm.w4_workspace_bytes(64, 4096, 4096) == 1024 + 32 * 8 * tile
    assert mm.w4_workspace_bytes(64, 11008, 4096) == 1024 + 86 * 2 * tile
    assert mm.w4_workspace_bytes(100, 512, 2048) == 1024 + 4 * 8 * 2 * tile
    assert mm.mx8_wgrad_workspace_bytes(2048, 1024, 2048) == 1024 + 128 * 4 * 2 * tile
    assert mm.mx8_wgrad_workspace_bytes(1024, 1024, 4096) == 1024 + 256 * 2 * 2 * tile
    for M, N, K in ((33, 1 << 17, 8192), (64, 1 << 15, 512), (128, 1 << 16, 4096), (8192, 1 << 15, 8192)):
        for n in (mm.w4_workspace_bytes(M, N, K), mm.mx8_wgrad_workspace_bytes(K, M, N)):
            assert n == 0 or (n - 1024) % (32 * 128 * 4) == 0 and n <= 1024 + 512 * 4 * tile


def test_outputs_are_floating_and_c_has_their_type():
    """The sums are fp32: an int32 D would hold their bit patterns, an int32 C would be read as some."""
    A, dY = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros((4, 16), dtype=torch.bfloat16)
    Wq, SW = torch.zeros((32, 32), dtype=torch.uint8), torch.zeros((1, 32), dtype=torch.int32)
    Xq, SX = torch.zeros((4, 64), dtype=torch.int8), torch.zeros((1, 4), dtype=torch.int32)
    for d, c, message in ((torch.int32, None, "D has dtype torch.int32"), (torch.int32, torch.int32, "D has dtype torch.int32"),
                          (torch.int16, None, "D has dtype torch.int16"), (torch.float64, None, "D has dtype torch.float64"),
                          (torch.float32, torch.int32, "C has dtype torch.int32"), (torch.bfloat16, torch.float16, "C has dtype torch.float16"),
                          (torch.float16, torch.float32, "C has dtype torch.float32"), (torch.float32, torch.float32, "in GPU memory")):
        def pair(rows, cols):
            return torch.zeros((rows, cols), dtype=d), None if c is None else torch.zeros((rows, cols), dtype=c)
        D, C = pair(4, 32)
        with pytest.raises(ValueError, match=message):
            mm.gemm_w4(A, Wq, SW, D, beta=1.0 if c else 0.0, C=C)
        D, C = pair(16, 64)
        with pytest.raises(ValueError, match=message):
            mm.gemm_mx8_wgrad(dY, Xq, SX, D, beta=1.0 if c else 0.0, C=C)


class Reached(Exception):
    """A call passed every check of the binding."""


@pytest.fixture
def no_library(monkeypatch):
    """Host tensors count as device ones, and the library's entries raise Reached: a check that is missing shows."""
    class Entries:
        def __getattr__(self, name):
            def call(*args):
                raise Reached(name)
            return call
    monkeypatch.setattr(mm, "lib", lambda: Entries())
    monkeypatch.setattr(mm, "_stream_of", lambda stream, *tensors: 0)


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def i8(*shape):
    return torch.zeros(shape, dtype=torch.int8)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


# entry -> (arguments that pass, [(changed arguments, the message)])
BINDING = {
    "w4_quantize": (lambda: dict(W=bf16(32, 64), Wq=u8(32, 32), SW=i32(1, 32)), [
        (lambda: dict(Wq=u8(31, 32)), r"Wq has shape \(31, 32\)"), (lambda: dict(Wq=u8(32, 31)), r"Wq has shape \(32, 31\)"),
        (lambda: dict(Wq=u8(1, 32).expand(32, 32)), "Wq: rows .* overlap"), (lambda: dict(Wq=u8(32, 64)[:, ::2]), "Wq: expected a contiguous"),
        (lambda: dict(Wq=torch.zeros(32, 32, dtype=torch.int16)), "Wq must hold bytes"), (lambda: dict(SW=i32(0, 32)), r"SW has shape \(0, 32\)"),
        (lambda: dict(group=32), r"SW has shape \(1, 32\), expected \(2, >= 32\)"), (lambda: dict(SW=i32(1, 31)), r"SW has shape \(1, 31\)"),
        (lambda: dict(SW=torch.zeros(1, 32)), "SW must hold 32-bit"), (lambda: dict(W=torch.zeros(32, 64, dtype=torch.float64)), "expected a float16, bfloat16"),
        (lambda: dict(W=bf16(1, 64).expand(32, 64)), "W: rows .* overlap"), (lambda: dict(W=bf16(64, 32).t()), "W: expected a contiguous"),
        (lambda: dict(w_type=mm.F32), "2-byte elements for type code 10")]),
    "gemm_w4": (lambda: dict(A=bf16(4, 64), Wq=u8(32, 32), SW=i32(1, 32), D=torch.zeros(4, 32)), [
        (lambda: dict(Wq=u8(32, 16)), r"Wq has shape \(32, 16\)"), (lambda: dict(Wq=torch.zeros(32, 32, dtype=torch.int16)), "Wq must hold bytes"),
        (lambda: dict(SW=i32(1, 31)), r"SW has shape \(1, 31\)"), (lambda: dict(SW=torch.zeros(1, 32, dtype=torch.int64)), "SW must hold 32-bit"),
        (lambda: dict(group=32), r"SW has shape \(1, 32\), expected \(2"), (lambda: dict(D=torch.zeros(4, 31)), r"D has shape \(4, 31\)"),
        (lambda: dict(D=torch.zeros(3, 32)), r"D has shape \(3, 32\)"), (lambda: dict(D=torch.zeros(1, 32).expand(4, 32)), "D: rows .* overlap"),
        (lambda: dict(D=torch.zeros(32, 4).t()), "D: expected a contiguous"), (lambda: dict(C=torch.zeros(3, 32), beta=1.0), r"C has shape \(3, 32\)"),
        (lambda: dict(C=torch.zeros(1, 32).expand(4, 32), beta=1.0), "C: rows .* overlap"), (lambda: dict(bias=torch.zeros(31)), "bias must be"),
        (lambda: dict(bias=bf16(32)), "bias must be"), (lambda: dict(bias=torch.zeros(64)[::2]), "bias must be"),
        (lambda: dict(A=i32(4, 64)), "expected a float16, bfloat16"), (lambda: dict(a_type=mm.F32), "2-byte elements for type code 10"),
        (lambda: dict(A=bf16(1, 64).expand(4, 64)), "A: rows .* overlap"), (lambda: dict(A=bf16(64, 4).t()), "A: expected a contiguous"),
        (lambda: dict(d_type=mm.OUT_BF16), "D has 4-byte elements"), (lambda: dict(workspace=u8(64, 64)[:, :32]), "workspace must be contiguous")]),
    "mx8_quantize": (lambda: dict(X=torch.zeros(4, 40), Xq=i8(4, 64), SX=i32(1, 4)), [
        (lambda: dict(Xq=i8(4, 48)), r"Xq has shape \(4, 48\)"), (lambda: dict(Xq=i8(3, 64)), r"Xq has shape \(3, 64\)"),
        (lambda: dict(Xq=u8(4, 64)), "Xq must hold"), (lambda: dict(Xq=bf16(4, 64)), "Xq must hold"), (lambda: dict(SX=i32(1, 3)), r"SX has shape \(1, 3\)"),
        (lambda: dict(SX=i32(0, 4)), r"SX has shape \(0, 4\)"), (lambda: dict(SX=torch.zeros(1, 4, dtype=torch.int16)), "SX must hold 32-bit"),
        (lambda: dict(X=torch.zeros(4, 40, dtype=torch.float64)), "expected a float16, bfloat16"), (lambda: dict(Xq=i8(1, 64).expand(4, 64)), "Xq: rows .* overlap")]),
    "gemm_mx8_wgrad": (lambda: dict(dY=bf16(4, 16), Xq=i8(4, 64), SX=i32(1, 4), D=torch.zeros(16, 64)), [
        (lambda: dict(dY=bf16(3, 16)), r"Xq has shape \(4, 64\), expected \(3"), (lambda: dict(D=torch.zeros(15, 64)), r"D has shape \(15, 64\)"),
        (lambda: dict(D=torch.zeros(16, 128)), r"Xq has shape \(4, 64\), expected \(4, >= 128\)"), (lambda: dict(C=torch.zeros(16, 63), beta=1.0), r"C has shape \(16, 63\)"),
        (lambda: dict(Xq=u8(4, 64)), "Xq must hold"), (lambda: dict(SX=i32(1, 3)), r"SX has shape \(1, 3\)"),
        (lambda: dict(dY=torch.zeros(4, 16, dtype=torch.float64)), "expected a float16, bfloat16"), (lambda: dict(D=torch.zeros(1, 64).expand(16, 64)), "D: rows .* overlap"),
        (lambda: dict(workspace=u8(64, 64)[:, :32]), "workspace must be contiguous")]),
}
BINDING["mx8_dequantize"] = BINDING["mx8_quantize"]


@pytest.mark.parametrize("entry", list(BINDING))
def test_each_check_of_the_binding(entry, no_library):
    """Arguments that fit reach the library, and each that does not raises its own message before that."""
    fits, changes = BINDING[entry]
    with pytest.raises(Reached):
        getattr(mm, entry)(**fits())
    for change, message in changes:
        with pytest.raises(ValueError, match=message):
            getattr(mm, entry)(**{**fits(), **change()})


@pytest.mark.parametrize("entry", list(BINDING))
def test_the_binding_refuses_host_memory(entry):
    with pytest.raises(ValueError, match="every tensor must be in GPU memory"):
        getattr(mm, entry)(**BINDING[entry][0]())
