"""Host-side checks of the RMS norm and 4-bit quantizer entry points (no GPU needed, no compute call): the headers and
the library agree, every argument error is reported before any GPU work (the pointers passed here are fake), and the
binding refuses tensors that do not fit the call."""
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


@pytest.mark.parametrize("header,names", [
    ("mmac_norm.h", ["mmac_rmsnorm", "mmac_rmsnorm_grad", "mmac_rmsnorm_grad_workspace_bytes"]),
    ("mmac_mx4.h", ["mmac_mx4_quantize"]),
])
def test_header_and_library_agree(L, header, names):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    assert sorted(set(re.findall(r"\b(mmac_[a-z0-9_]+)\s*\(", text))) == names
    for name in names:
        assert hasattr(L, name), name


def norm(L, **kw):
    a = dict(x=mm.BF16, w=mm.BF16, y=mm.BF16, M=4, N=64, X=P, ldx=64, R=None, ldr=0, W=P, eps=1e-6, H=None, ldh=0, Y=2 * P,
             ldy=64, SY=None, lds=0, rstd=None)
    a.update(kw)
    return L.mmac_rmsnorm(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=mm.I8), UNS), (dict(w=mm.F16), UNS), (dict(y=mm.F32), UNS), (dict(y=mm.I8), UNS), (dict(x=mm.F32, w=mm.BF16, y=mm.F32), UNS),
    (dict(M=-1), INV), (dict(N=1 << 31), INV), (dict(X=None), INV), (dict(W=None), INV), (dict(Y=None), INV),
    (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(eps=float("inf")), INV), (dict(eps=1e39), INV),
    (dict(ldx=63), INV), (dict(ldx=68), MIS), (dict(X=P + 8), MIS), (dict(ldx=(1 << 22) + 8), UNS), (dict(ldx=BIG), UNS),
    (dict(R=3 * P, ldr=63), INV), (dict(R=3 * P + 2, ldr=64), MIS), (dict(H=3 * P, ldh=60), INV), (dict(H=3 * P, ldh=65), MIS),
    (dict(ldy=63), INV), (dict(Y=2 * P + 4), MIS), (dict(W=P + 8), MIS), (dict(rstd=P + 2), MIS),
    (dict(H=P, ldh=72), INV), (dict(R=3 * P, ldr=64, H=3 * P, ldh=72), INV), (dict(Y=P, ldy=72), INV), (dict(Y=P, H=P, ldh=64), INV), (dict(H=2 * P, ldh=64), INV), (dict(R=2 * P, ldr=64), INV),
    (dict(y=mm.FP8_E4M3), INV), (dict(y=mm.FP8_E4M3, SY=P, lds=3), INV), (dict(y=mm.FP8_E4M3, SY=P + 2, lds=4), MIS),
    (dict(y=mm.FP8_E4M3, SY=P, lds=1 << 30), UNS), (dict(y=mm.BF8_E5M2, SY=P, lds=4, ldy=72), MIS),
    (dict(y=mm.FP8_E4M3, SY=P, lds=4, N=70, ldx=72, ldy=80), INV), (dict(y=mm.FP8_E4M3, SY=P, lds=4, Y=P), INV),
])
def test_rmsnorm_argument_errors(L, kw, code):
    assert norm(L, **kw) == code


def test_rmsnorm_empty_is_a_no_op(L):
    assert norm(L, M=0, X=None, W=None, Y=None) == OK
    assert norm(L, N=0, X=None, W=None, Y=None) == OK
    assert norm(L, N=0, y=mm.FP8_E4M3, X=None, W=None, Y=None, SY=None, lds=4) == OK


def grad(L, **kw):
    a = dict(x=mm.BF16, w=mm.F32, M=4, N=64, dY=P, lddy=64, H=2 * P, ldh=64, W=P, rstd=P, dH=None, lddh=0, dX=3 * P, lddx=64,
             dW=None, ws=None, n=0)
    a.update(kw)
    return L.mmac_rmsnorm_grad(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=mm.FP8_E4M3), UNS), (dict(w=mm.F16), UNS), (dict(M=-1), INV), (dict(N=-1), INV), (dict(dY=None), INV), (dict(H=None), INV),
    (dict(W=None), INV), (dict(rstd=None), INV), (dict(dX=None), INV), (dict(lddy=60), INV), (dict(ldh=60), INV), (dict(lddx=60), INV),
    (dict(dH=P, lddh=60), INV), (dict(lddy=68), MIS), (dict(H=P + 8), MIS), (dict(dX=3 * P + 2), MIS), (dict(W=P + 4), MIS),
    (dict(rstd=P + 1), MIS), (dict(lddx=1 << 23), UNS), (dict(dX=P, lddx=72), INV), (dict(dH=4 * P, lddh=64, dX=4 * P, lddx=72), INV),
    (dict(dX=2 * P), INV), (dict(n=-1), INV), (dict(dW=P + 8, ws=P, n=1 << 30), MIS), (dict(dW=P, ws=P + 8, n=1 << 30), MIS),
    (dict(dW=P), INV), (dict(dW=P, ws=P, n=1024), INV), (dict(M=0, dW=P), INV),
])
def test_rmsnorm_grad_argument_errors(L, kw, code):
    assert grad(L, **kw) == code


def test_rmsnorm_grad_empty_and_workspace(L):
    none = dict(dY=None, H=None, W=None, rstd=None, dX=None)
    assert grad(L, M=0, **none) == OK
    assert grad(L, N=0, dW=P, **none) == OK
    assert mm.rmsnorm_grad_workspace_bytes(4, 0) == 0 and mm.rmsnorm_grad_workspace_bytes(-1, 4) == 0
    for M, N in ((0, 8), (1, 8), (5000, 64), (1 << 30, 4096)):
        n = mm.rmsnorm_grad_workspace_bytes(M, N)
        assert n >= 1024 + 4 * N and (n - 1024) % (4 * N) == 0 and n <= 1024 + 512 * 4 * N
        assert grad(L, M=M, N=N, lddy=N, ldh=N, lddx=N, dW=P, ws=P, n=n - 1) == INV


def quantize(L, **kw):
    a = dict(t=mm.BF16, M=64, K=64, X=P, ldx=64, Xq=P, pitch=32, SX=P, lds=64)
    a.update(kw)
    return L.mmac_mx4_quantize(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(t=mm.I8), UNS), (dict(t=mm.FP8_E4M3), UNS), (dict(M=-1), INV), (dict(K=1 << 31), INV), (dict(X=None), INV),
    (dict(Xq=None), INV), (dict(SX=None), INV), (dict(ldx=63), INV), (dict(ldx=65), MIS), (dict(X=P + 4), MIS),
    (dict(pitch=16), INV), (dict(pitch=40), MIS), (dict(Xq=P + 8), MIS), (dict(pitch=(1 << 23) + 16), UNS), (dict(lds=63), INV),
    (dict(lds=1 << 30), UNS), (dict(SX=P + 2), MIS), (dict(ldx=BIG), UNS),
])
def test_mx4_quantize_argument_errors(L, kw, code):
    assert quantize(L, **kw) == code


def test_mx4_quantize_empty_is_a_no_op(L):
    assert quantize(L, M=0, X=None, Xq=None, SX=None) == OK
    assert quantize(L, K=0, X=None, Xq=None, SX=None) == OK


def test_matrices_without_elements_have_any_pitch(L):
    """As torch has them: rows of nothing lie one element apart, no rows any number of elements."""
    assert norm(L, M=0, N=33, ldx=33, ldy=33) == OK
    assert grad(L, M=0, N=33, lddy=33, ldh=33, lddx=33) == OK
    assert quantize(L, M=0, K=33, ldx=33, pitch=33) == OK
    assert norm(L, N=0, ldx=1, R=P, ldr=1, H=2 * P, ldh=1, Y=3 * P, ldy=1) == OK
    assert norm(L, N=0, ldx=1, y=mm.BF8_E5M2, ldy=1, SY=P, lds=4) == OK
    assert grad(L, N=0, lddy=1, ldh=1, dH=P, lddh=1, lddx=1, dW=P) == OK
    assert quantize(L, K=0, ldx=1, pitch=1) == OK


B16, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def z(*shape, t=B16):
    return torch.zeros(*shape, dtype=t)


@pytest.mark.parametrize("call,words", [
    (lambda: mm.rmsnorm(z(4, 64), z(64), z(4, 64)), "GPU memory"),
    (lambda: mm.rmsnorm(z(4, 64), z(63), z(4, 64)), "w must be"),
    (lambda: mm.rmsnorm(z(4, 64), z(64, t=torch.float16), z(4, 64)), "w has dtype"),
    (lambda: mm.rmsnorm(z(4, 64), z(64), z(4, 64, t=F32)), "Y has dtype"),
    (lambda: mm.rmsnorm(z(4, 64), z(64), z(4, 65)), "Y has shape"),
    (lambda: mm.rmsnorm(z(4, 64), z(64), z(4, 64, t=E4)), "needs SY"),
    (lambda: mm.rmsnorm(z(4, 64), z(64), z(4, 64), SY=z(1, 4, t=torch.int32)), "8-bit Y"),
    (lambda: mm.rmsnorm(z(4, 64), z(64), z(4, 64, t=E4), SY=z(1, 3, t=torch.int32)), "SX has shape"),
    (lambda: mm.rmsnorm(z(4, 64), z(64), z(4, 64), residual=z(4, 64, t=F32)), "residual has dtype"),
    (lambda: mm.rmsnorm(z(4, 64), z(64), z(4, 64), H=z(5, 64)), "H has shape"),
    (lambda: mm.rmsnorm(z(4, 64), z(64), z(4, 64), rstd=z(4)), "rstd has dtype"),
    (lambda: mm.rmsnorm(z(64, 4).t(), z(64), z(4, 64)), "contiguous last"),
    (lambda: mm.rmsnorm(z(1, 64).expand(4, 64), z(64), z(4, 64)), "overlap"),
    (lambda: mm.rmsnorm(z(4, 64, t=E4), z(64), z(4, 64)), "expected a float16"),
    (lambda: mm.rmsnorm_grad(z(4, 64), z(4, 64), z(64), z(4, t=F32), z(4, 64)), "GPU memory"),
    (lambda: mm.rmsnorm_grad(z(4, 64), z(4, 64, t=F32), z(64), z(4, t=F32), z(4, 64)), "H has dtype"),
    (lambda: mm.rmsnorm_grad(z(4, 64), z(4, 64), z(64), z(5, t=F32), z(4, 64)), "rstd must be"),
    (lambda: mm.rmsnorm_grad(z(4, 64), z(4, 64), z(64), z(4, t=F32), z(4, 64), dW=z(64)), "dW has dtype"),
    (lambda: mm.rmsnorm_grad(z(4, 64), z(4, 64), z(64), z(4, t=F32), z(4, 64), dH=z(4, 60)), "dH has shape"),
    (lambda: mm.rmsnorm_grad(z(4, 64), z(4, 64), z(64), z(4, t=F32), z(4, 64), workspace=z(8, 4).t()), "contiguous"),
    (lambda: mm.mx4_quantize(z(4, 64), z(4, 32, t=torch.uint8), z(1, 4, t=torch.int32)), "GPU memory"),
    (lambda: mm.mx4_quantize(z(4, 64), z(4, 32), z(1, 4, t=torch.int32)), "two elements each"),
    (lambda: mm.mx4_quantize(z(4, 64), z(4, 31, t=torch.uint8), z(1, 4, t=torch.int32)), "Xq has shape"),
    (lambda: mm.mx4_quantize(z(4, 64), z(4, 32, t=torch.uint8), z(1, 4, t=F32)), "scale words"),
])
def test_binding_refuses(L, call, words):
    with pytest.raises(ValueError, match=words):
        call()
