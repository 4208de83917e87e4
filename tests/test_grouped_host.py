"""Host-side checks of the grouped products' entry points (no GPU needed, no compute call): the header and the library
agree, every argument error is reported before any GPU work (the pointers passed here are fake), and the binding refuses
tensors that do not fit the call."""
import ctypes
import os
import re

import pytest
import torch

import sparse_matrix_multiply_amd as mm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20          # a fake, 16-byte aligned "device pointer": never dereferenced here
OK, INV, UNS, MIS = mm.OK, mm.ERR_INVALID_ARG, mm.ERR_UNSUPPORTED, mm.ERR_MISALIGNED
BIG = (1 << 63) - 1


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(mm.LIB_PATH):
        from sparse_matrix_multiply_amd import build
        build.build()
    return mm.lib()


def test_header_and_library_agree(L):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "mmac_grouped.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(mmac_[a-z0-9_]+)\s*\(", text)))
    assert names == ["mmac_gemm_grouped", "mmac_gemm_grouped_mx", "mmac_gemm_grouped_wgrad"]
    for name in names:
        assert hasattr(L, name), name


def call(f, a):
    return f(*[ctypes.byref(v) if isinstance(v, mm.Epilogue) else v for v in a.values()], None)


def grouped(L, **kw):
    a = dict(t=mm.BF16, trans=0, G=4, M=16, N=64, K=128, alpha=1.0, A=P, lda=128, off=P, B=P, ldb=128, sb=64 * 128, beta=0.0,
             C=None, ldc=0, D=P, ldd=64, ep=None)
    a.update(kw)
    return call(L.mmac_gemm_grouped, a)


def grouped_mx(L, **kw):
    a = dict(ta=mm.FP8_E4M3, tb=mm.FP4_E2M1, G=4, M=16, N=64, K=128, alpha=1.0, A=P, lda=128, SA=P, ldsa=16, off=P, B=P,
             ldb=128, sb=64 * 128, SB=P, ldsb=64, ssb=64, beta=0.0, C=None, ldc=0, D=P, ldd=64, ep=None)
    a.update(kw)
    return call(L.mmac_gemm_grouped_mx, a)


def wgrad(L, **kw):
    a = dict(t=mm.BF16, G=4, M=16, N=64, K=128, alpha=1.0, dY=P, ldy=64, X=P, ldx=128, off=P, beta=0.0, C=None, ldc=0, sc=0,
             D=P, ldd=128, sd=64 * 128, ep=None)
    a.update(kw)
    return call(L.mmac_gemm_grouped_wgrad, a)


OUT = [
    (dict(D=None), INV), (dict(ldd=1), INV), (dict(beta=1.0), INV), (dict(alpha=float("nan")), INV),
    (dict(beta=float("inf"), C=P, ldc=128), INV), (dict(alpha=1e39), INV), (dict(D=P + 2), MIS), (dict(ldd=1 << 22), UNS),
    (dict(beta=1.0, C=P, ldc=10), INV), (dict(ep=mm.Epilogue(9, 0, None)), INV), (dict(ep=mm.Epilogue(0, 7, None)), INV),
    (dict(G=-1), INV), (dict(G=1 << 31), INV), (dict(G=(1 << 30) + 1), UNS), (dict(M=-1), INV), (dict(N=1 << 31), INV), (dict(K=-1), INV), (dict(off=None), INV), (dict(off=P + 2), MIS),
]


@pytest.mark.parametrize("kw,code", OUT + [
    (dict(t=mm.F32), UNS), (dict(t=mm.I8), UNS), (dict(trans=2), INV), (dict(A=None), INV), (dict(B=None), INV),
    (dict(lda=120), INV), (dict(lda=132), MIS), (dict(A=P + 8), MIS), (dict(lda=1 << 23), UNS), (dict(ldb=120), INV),
    (dict(B=P + 4), MIS), (dict(sb=64 * 128 - 8), INV), (dict(sb=64 * 128 + 4), MIS), (dict(sb=BIG), INV), (dict(sb=-8), INV),
    (dict(trans=1, ldb=60, sb=1 << 20), INV), (dict(trans=1, ldb=64, sb=127 * 64), INV), (dict(ep=mm.Epilogue(1, 0, P + 2)), MIS),
    (dict(beta=1.0, C=P, ldc=128, ldd=64), INV),
    (dict(trans=1, K=1 << 12, lda=1 << 12, ldb=1 << 19, sb=1 << 32), UNS),
])
def test_gemm_grouped_argument_errors(L, kw, code):
    assert grouped(L, **kw) == code


@pytest.mark.parametrize("kw,code", OUT + [
    (dict(ta=mm.BF16), UNS), (dict(ta=mm.FP4_E2M1), UNS), (dict(tb=mm.I8), UNS), (dict(tb=mm.FP6_E2M3), UNS), (dict(K=100), INV),
    (dict(A=None), INV), (dict(SA=None), INV), (dict(B=None), INV), (dict(SB=None), INV), (dict(lda=112), INV), (dict(lda=136), MIS),
    (dict(ldb=127), INV), (dict(ldb=129), MIS), (dict(ldb=144), MIS), (dict(sb=64 * 128 + 16), MIS), (dict(sb=64 * 128 - 32), INV),
    (dict(sb=64 * 128 + 1), MIS), (dict(ldsa=15), INV), (dict(SA=P + 2), MIS), (dict(ldsa=1 << 30), UNS), (dict(ldsb=63), INV), (dict(ssb=60), INV), (dict(SB=P + 1), MIS),
    (dict(ldsb=1 << 30, ssb=1 << 31), UNS), (dict(B=P + 8), MIS), (dict(tb=mm.FP8_E4M3, ldb=136, sb=64 * 136), MIS),
])
def test_gemm_grouped_mx_argument_errors(L, kw, code):
    assert grouped_mx(L, **kw) == code


@pytest.mark.parametrize("kw,code", [x for x in OUT if x[0].get("ldd") != 1 << 22] + [
    (dict(ldd=1 << 22, sd=1 << 30), UNS), (dict(t=mm.F32), UNS), (dict(dY=None), INV), (dict(X=None), INV), (dict(ldy=60), INV),
    (dict(ldy=68), MIS), (dict(dY=P + 2), MIS), (dict(ldx=120), INV), (dict(X=P + 8), MIS), (dict(ldx=1 << 23), UNS),
    (dict(sd=64 * 128 - 1), INV), (dict(sd=-1), INV), (dict(beta=1.0, C=2 * P, ldc=128, sc=64 * 128 - 1), INV),
    (dict(beta=1.0, C=P, ldc=128, sc=64 * 128 + 8), INV), (dict(ep=mm.Epilogue(0, 1, None)), UNS), (dict(ep=mm.Epilogue(0, 0, P)), UNS),
])
def test_gemm_grouped_wgrad_argument_errors(L, kw, code):
    assert wgrad(L, **kw) == code


def test_matrices_without_elements_have_any_pitch(L):
    """As torch has them: rows of nothing lie one element apart, no rows any number of elements."""
    assert grouped(L, M=0, K=100, lda=100, ldb=104) == OK
    assert grouped(L, G=0, K=100, lda=104, ldb=100) == OK
    assert grouped(L, N=0, trans=1, ldb=1, sb=1, ldd=1) == OK
    assert grouped(L, N=0, ldd=1, sb=0) == OK
    assert wgrad(L, N=0, ldy=1, sd=0) == OK and wgrad(L, K=0, ldx=1, ldd=1, sd=0) == OK


# On a machine without a GPU the launch itself is what fails: the call was not refused.
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers are fake: the calls would run")


@no_gpu
@pytest.mark.parametrize("kw", [
    dict(G=384, M=65536, N=2048, K=7168), dict(G=256, M=300, N=1100, K=7168, ep=mm.Epilogue(2, 0, None)), dict(G=300_000, M=300_000, N=16, K=16),
    dict(G=100_000, M=300, N=1000, K=1000, ep=mm.Epilogue(2, 0, None)), dict(G=60_000, M=300, N=1000, K=1000),
])
def test_wgrad_of_many_tiles_is_not_refused(L, kw):
    """Matrices that fit the GPU's memory: any of the tiles' grids that fits will do."""
    N, K = kw["N"], kw["K"]
    assert wgrad(L, ldy=-(-N // 8) * 8, ldx=-(-K // 8) * 8, ldd=K, sd=N * K, **kw) == mm.ERR_HIP


@no_gpu
@pytest.mark.parametrize("kw", [
    dict(G=16384, M=1 << 20, N=8192, K=64), dict(G=80_000, M=80_000, N=2048, K=16), dict(G=270_000, M=270_000, N=2048, K=8),
    dict(G=16384, M=1 << 20, N=8192, K=64, trans=1), dict(G=4096, M=16384, N=16384, K=4096, tb=mm.FP4_E2M1),
    dict(G=300_000, M=300_000, N=2048, K=32, tb=mm.FP8_E4M3), dict(G=1000, M=2 << 20, N=16384, K=64), dict(G=1, M=1 << 21, N=32768, K=64),
])
def test_forward_of_many_tiles_is_not_refused(L, kw):
    kw = dict(kw)
    N, K = kw["N"], kw["K"]
    if "tb" in kw:
        assert grouped_mx(L, lda=K, ldb=K, sb=N * K, ldsa=kw["M"], ldsb=N, ssb=-(-K // 128) * N, ldd=N, **kw) == mm.ERR_HIP
    else:
        assert grouped(L, lda=K, ldb=N if kw.get("trans") else K, sb=N * K, ldd=N, **kw) == mm.ERR_HIP


def test_empty_is_a_no_op(L):
    for kw in (dict(G=0), dict(M=0), dict(N=0)):
        assert grouped(L, A=None, B=None, D=None, off=None, **kw) == OK
        assert grouped_mx(L, A=None, B=None, SA=None, SB=None, D=None, off=None, **kw) == OK
    for kw in (dict(G=0), dict(N=0), dict(K=0)):
        assert wgrad(L, dY=None, X=None, off=None, D=None, **kw) == OK


def z(*shape, t=torch.bfloat16):
    return torch.zeros(*shape, dtype=t)


def off(n=4, t=torch.int32):
    return torch.zeros(n + 1, dtype=t)


E4, U8, I32 = torch.float8_e4m3fn, torch.uint8, torch.int32


@pytest.mark.parametrize("f,words", [
    (lambda: mm.gemm_grouped(z(16, 128), off(), z(4, 64, 128), z(16, 64)), "GPU memory"),
    (lambda: mm.gemm_grouped(z(16, 128), off(), z(64, 128), z(16, 64)), "one matrix per group"),
    (lambda: mm.gemm_grouped(z(16, 128), off(), z(4, 64, 120), z(16, 64)), "B has shape"),
    (lambda: mm.gemm_grouped(z(16, 128), off(), z(4, 64, 128), z(16, 64), trans_b=True), "B has shape"),
    (lambda: mm.gemm_grouped(z(16, 128), off(), z(4, 64, 128, t=torch.float16), z(16, 64)), "B has dtype"),
    (lambda: mm.gemm_grouped(z(16, 128), off(3), z(4, 64, 128), z(16, 64)), "offsets must be"),
    (lambda: mm.gemm_grouped(z(16, 128), off(t=torch.int64), z(4, 64, 128), z(16, 64)), "offsets has dtype"),
    (lambda: mm.gemm_grouped(z(16, 128), off(), z(4, 64, 128), z(15, 64)), "D has shape"),
    (lambda: mm.gemm_grouped(z(16, 128), off(), z(4, 64, 128), z(16, 64, t=torch.int32)), "D has dtype"),
    (lambda: mm.gemm_grouped(z(16, 128), off(), z(4, 64, 128), z(16, 64), beta=1.0, C=z(16, 64, t=torch.float16)), "C has dtype"),
    (lambda: mm.gemm_grouped(z(16, 128), off(), z(4, 64, 128), z(16, 64), bias=z(64, t=torch.float32)), "bias must be"),
    (lambda: mm.gemm_grouped(z(16, 128), off(), z(1, 64, 128).expand(4, 64, 128), z(16, 64)), "overlap"),
    (lambda: mm.gemm_grouped(z(16, 128), off(), z(4, 1, 128).expand(4, 64, 128), z(16, 64)), "overlap"),
    (lambda: mm.gemm_grouped(z(16, 128), off(), z(4, 128, 64).transpose(1, 2), z(16, 64)), "contiguous last"),
    (lambda: mm.gemm_grouped_wgrad(z(16, 64), z(16, 128), off(), z(4, 64, 128)), "GPU memory"),
    (lambda: mm.gemm_grouped_wgrad(z(16, 64), z(15, 128), off(), z(4, 64, 128)), "X has shape"),
    (lambda: mm.gemm_grouped_wgrad(z(16, 64), z(16, 128), off(), z(64, 128)), "one matrix per group"),
    (lambda: mm.gemm_grouped_wgrad(z(16, 64), z(16, 128), off(), z(4, 64, 120)), "D has shape"),
    (lambda: mm.gemm_grouped_wgrad(z(16, 64), z(16, 128), off(), z(4, 64, 128), C=z(3, 64, 128)), "C has shape"),
    (lambda: mm.gemm_grouped_mx(z(16, 128, t=E4), z(1, 16, t=I32), off(), z(4, 64, 128, t=E4), z(4, 1, 64, t=I32), z(16, 64)), "GPU memory"),
    (lambda: mm.gemm_grouped_mx(z(16, 128, t=E4), z(1, 16, t=I32), off(), z(4, 64, 64, t=U8), z(4, 1, 64, t=I32), z(16, 64)), "8-bit elements"),
    (lambda: mm.gemm_grouped_mx(z(16, 128), z(1, 16, t=I32), off(), z(4, 64, 128, t=E4), z(4, 1, 64, t=I32), z(16, 64)), "8-bit elements"),
    (lambda: mm.gemm_grouped_mx(z(16, 128, t=E4), z(1, 15, t=I32), off(), z(4, 64, 128, t=E4), z(4, 1, 64, t=I32), z(16, 64)), "SA has shape"),
    (lambda: mm.gemm_grouped_mx(z(16, 128, t=E4), z(1, 16, t=I32), off(), z(4, 64, 128, t=E4), z(4, 1, 63, t=I32), z(16, 64)), "SB has shape"),
    (lambda: mm.gemm_grouped_mx(z(16, 128, t=E4), z(1, 16), off(), z(4, 64, 128, t=E4), z(4, 1, 64, t=I32), z(16, 64)), "scale words"),
    (lambda: mm.gemm_grouped_mx(z(16, 128, t=E4), z(1, 16, t=I32), off(), z(4, 64, 60, t=U8), z(4, 1, 64, t=I32), z(16, 64), b_type=mm.FP4_E2M1), "B has shape"),
])
def test_binding_refuses(L, f, words):
    with pytest.raises(ValueError, match=words):
        f()
