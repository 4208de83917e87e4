"""Python binding of libmmac: tiled dense and 4:2-sparse GEMM for MI355X (gfx950).

Thin ctypes layer over the C ABI in include/mmac.h, mmac_lowbit.h, mmac_mx4.h,
mmac_norm.h and mmac_grouped.h, with the same entry points.  It only marshals arguments: torch tensors provide device memory and
the current HIP stream; every step of the computation runs in the library's
HIP kernels.  If libmmac.so is missing, importing the binding succeeds but the
first call raises -- there is no fallback path.

Tensor conventions (element strides; the last dimension must be contiguous):
    A   M x K  row-major             (torch dtype gives the element type)
    B   N x K  (the K x N matrix B stored column-major)
    C,D M x N  float32 (int32 for int8 inputs); with floating inputs also
               bfloat16, float16, float8_e4m3fn or float8_e5m2 (the epilogue
               variants: D's dtype picks the output type, C has D's dtype),
               plus an optional fp32 bias of N values and ReLU
    Ac  M x K/2, idx M x ceil(K/32) int32/uint32 words
    4-bit weights   codes N x 16 ceil(K/32) uint8, scale words groups x N int32
    8-bit activations   elements M x 32 ceil(K/32) (float8_e4m3fn, float8_e5m2 or int8),
               scale words ceil(K/128) x M int32
    4-bit block-scaled rows   M x 16 ceil(K/32) uint8, scale words as above
    products grouped by expert   B groups x N x K (or K x N), bias groups x N, offsets groups + 1 int32
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmmac.so")

F16, BF16, I8, FP8_E4M3, BF8_E5M2, FP4_E2M1, FP6_E2M3, BF6_E3M2 = 1, 2, 3, 4, 5, 6, 7, 8
U4, F32 = 9, 10
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_MISALIGNED, ERR_HIP, ERR_SCRATCH = 0, 1, 2, 3, 4, 5

OUT_ACC, OUT_BF16, OUT_F16, OUT_FP8_E4M3, OUT_BF8_E5M2 = 0, 1, 2, 3, 4
ACT_NONE, ACT_RELU = 0, 1
OUT_OF = {torch.float32: OUT_ACC, torch.int32: OUT_ACC, torch.bfloat16: OUT_BF16, torch.float16: OUT_F16,
          torch.float8_e4m3fn: OUT_FP8_E4M3, torch.float8_e5m2: OUT_BF8_E5M2}

DTYPE_OF = {torch.float16: F16, torch.bfloat16: BF16, torch.int8: I8,
            torch.float8_e4m3fn: FP8_E4M3, torch.float8_e5m2: BF8_E5M2}
TORCH_OF = {v: k for k, v in DTYPE_OF.items()}

_lib = None


class Epilogue(ctypes.Structure):
    """mmac_epilogue_t."""
    _fields_ = [("d_type", ctypes.c_int32), ("act", ctypes.c_int32), ("bias", ctypes.c_void_p)]


class W4(ctypes.Structure):
    """mmac_w4_t."""
    _fields_ = [("q_type", ctypes.c_int32), ("group", ctypes.c_int32), ("codes", ctypes.c_void_p),
                ("pitch", ctypes.c_int64), ("words", ctypes.c_void_p), ("ldw", ctypes.c_int64)]


class MmacError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__(f"{what}: {string(status)}")


def lib():
    """The loaded libmmac.so (raises if it was never built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run `python -m sparse_matrix_multiply_amd.build` first")
        L = ctypes.CDLL(LIB_PATH)
        i64, dbl, vp, i32 = ctypes.c_int64, ctypes.c_double, ctypes.c_void_p, ctypes.c_int
        L.mmac_gemm_dense.restype = i32
        L.mmac_gemm_dense.argtypes = [i32, i32, i64, i64, i64, dbl, vp, i64, vp, i64, dbl, vp, i64, vp, i64, vp]
        L.mmac_sparse24_compress.restype = i32
        L.mmac_sparse24_compress.argtypes = [i32, i64, i64, vp, i64, vp, i64, vp, i64, vp, vp]
        L.mmac_sparse24_prune_compress.restype = i32
        L.mmac_sparse24_prune_compress.argtypes = [i32, i64, i64, vp, i64, vp, i64, vp, i64, vp, vp]
        L.mmac_gemm_sparse24.restype = i32
        L.mmac_gemm_sparse24.argtypes = [i32, i32, i64, i64, i64, dbl, vp, i64, vp, i64, vp, i64, dbl, vp, i64,
                                         vp, i64, vp]
        ep = ctypes.POINTER(Epilogue)
        L.mmac_gemm_dense_ep.restype = i32
        L.mmac_gemm_dense_ep.argtypes = [i32, i32, i64, i64, i64, dbl, vp, i64, vp, i64, dbl, vp, i64, vp, i64, ep, vp]
        L.mmac_gemm_sparse24_ep.restype = i32
        L.mmac_gemm_sparse24_ep.argtypes = [i32, i32, i64, i64, i64, dbl, vp, i64, vp, i64, vp, i64, dbl, vp, i64,
                                            vp, i64, ep, vp]
        L.mmac_gemm_dense_ws.restype = i32
        L.mmac_gemm_dense_ws.argtypes = [i32, i32, i64, i64, i64, dbl, vp, i64, vp, i64, dbl, vp, i64, vp, i64, ep,
                                         vp, i64, vp]
        L.mmac_gemm_dense_static.restype = i32
        L.mmac_gemm_dense_static.argtypes = [i32, i32, i64, i64, i64, dbl, vp, i64, vp, i64, dbl, vp, i64, vp, i64,
                                             ep, vp]
        L.mmac_gemm_sparse24_ws.restype = i32
        L.mmac_gemm_sparse24_ws.argtypes = [i32, i32, i64, i64, i64, dbl, vp, i64, vp, i64, vp, i64, dbl, vp, i64,
                                            vp, i64, ep, vp, i64, vp]
        L.mmac_gemm_dense_mx.restype = i32
        L.mmac_gemm_dense_mx.argtypes = [i32, i32, i64, i64, i64, dbl, vp, i64, vp, i64, vp, i64, vp, i64, dbl, vp,
                                         i64, vp, i64, ep, vp]
        L.mmac_gemm_dense_layout.restype = i32
        L.mmac_gemm_dense_layout.argtypes = [i32, i32, i32, i32, i64, i64, i64, dbl, vp, i64, vp, i64, dbl, vp, i64,
                                             vp, i64, ep, vp]
        L.mmac_gemm_workspace_bytes.restype = i64
        L.mmac_gemm_workspace_bytes.argtypes = [i32, i64, i64, i64, i32]
        w4 = ctypes.POINTER(W4)
        L.mmac_w4_quantize.restype = i32
        L.mmac_w4_quantize.argtypes = [i32, i32, i64, i64, vp, i64, w4, vp]
        L.mmac_gemm_w4.restype = i32
        L.mmac_gemm_w4.argtypes = [i32, i64, i64, i64, dbl, vp, i64, w4, dbl, vp, i64, vp, i64, ep, vp, i64, vp]
        L.mmac_gemm_w4_workspace_bytes.restype = i64
        L.mmac_gemm_w4_workspace_bytes.argtypes = [i64, i64, i64]
        L.mmac_mx8_quantize.restype = i32
        L.mmac_mx8_quantize.argtypes = [i32, i32, i64, i64, vp, i64, vp, i64, vp, i64, vp]
        L.mmac_mx8_dequantize.restype = i32
        L.mmac_mx8_dequantize.argtypes = [i32, i32, i64, i64, vp, i64, vp, i64, vp, i64, vp]
        L.mmac_gemm_mx8_wgrad.restype = i32
        L.mmac_gemm_mx8_wgrad.argtypes = [i32, i32, i64, i64, i64, dbl, vp, i64, vp, i64, vp, i64, dbl, vp, i64, vp,
                                          i64, ep, vp, i64, vp]
        L.mmac_gemm_mx8_wgrad_workspace_bytes.restype = i64
        L.mmac_gemm_mx8_wgrad_workspace_bytes.argtypes = [i64, i64, i64]
        L.mmac_mx4_quantize.restype = i32
        L.mmac_mx4_quantize.argtypes = [i32, i64, i64, vp, i64, vp, i64, vp, i64, vp]
        L.mmac_rmsnorm.restype = i32
        L.mmac_rmsnorm.argtypes = [i32, i32, i32, i64, i64, vp, i64, vp, i64, vp, dbl, vp, i64, vp, i64, vp, i64, vp, vp]
        L.mmac_rmsnorm_grad.restype = i32
        L.mmac_rmsnorm_grad.argtypes = [i32, i32, i64, i64, vp, i64, vp, i64, vp, vp, vp, i64, vp, i64, vp, vp, i64, vp]
        L.mmac_rmsnorm_grad_workspace_bytes.restype = i64
        L.mmac_rmsnorm_grad_workspace_bytes.argtypes = [i64, i64]
        L.mmac_gemm_grouped.restype = i32
        L.mmac_gemm_grouped.argtypes = [i32, i32, i64, i64, i64, i64, dbl, vp, i64, vp, vp, i64, i64, dbl, vp, i64, vp,
                                        i64, ep, vp]
        L.mmac_gemm_grouped_mx.restype = i32
        L.mmac_gemm_grouped_mx.argtypes = [i32, i32, i64, i64, i64, i64, dbl, vp, i64, vp, i64, vp, vp, i64, i64, vp, i64,
                                           i64, dbl, vp, i64, vp, i64, ep, vp]
        L.mmac_gemm_grouped_wgrad.restype = i32
        L.mmac_gemm_grouped_wgrad.argtypes = [i32, i64, i64, i64, i64, dbl, vp, i64, vp, i64, vp, dbl, vp, i64, i64, vp,
                                              i64, i64, ep, vp]
        L.mmac_status_string.restype = ctypes.c_char_p
        L.mmac_status_string.argtypes = [i32]
        _lib = L
    return _lib


def string(status):
    return lib().mmac_status_string(int(status)).decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _ld(t):
    """Row pitch (elements) of a 2-D tensor whose last dimension is contiguous and whose rows do not
    overlap (a broadcast or overlapping view would make the kernels write past or over its rows)."""
    st, sh = t.stride(), t.shape
    if len(sh) != 2 or (st[1] != 1 and sh[1] > 1):
        raise ValueError("expected a 2-D tensor with a contiguous last dimension")
    if sh[0] > 1 and st[0] < sh[1]:
        raise ValueError(f"rows of a {tuple(sh)} tensor with row stride {st[0]} overlap")
    return max(st[0], sh[1], 1)


def _shape(t, rows, cols, name, min_cols=False):
    """Check that a 2-D tensor has `rows` rows and `cols` columns (at least `cols` with min_cols)."""
    if t is None:
        return
    if t.dim() != 2 or t.shape[0] != rows or (t.shape[1] < cols if min_cols else t.shape[1] != cols):
        want = f"({rows}, {'>= ' if min_cols else ''}{cols})"
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {want}")


def _same_device(*tensors):
    """Every tensor given lives on one CUDA device (the library's kernels address them all)."""
    devs = {t.device for t in tensors if t is not None}
    if any(d.type != "cuda" for d in devs):
        raise ValueError("every tensor must be in GPU memory")
    if len(devs) > 1:
        raise ValueError(f"tensors on different devices: {sorted(str(d) for d in devs)}")


def _bias(bias, N):
    if bias is not None and (bias.dtype != torch.float32 or bias.dim() != 1 or bias.numel() < N or
                             (bias.numel() > 1 and bias.stride(0) != 1)):
        raise ValueError(f"bias must be a contiguous float32 vector of at least N = {N} values")


# The current stream's handle without building a Stream object (a few microseconds per call, which
# is as long as a small GEMM): torch's own accessor where it has one.
_raw_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_current_stream is not None:
            return ctypes.c_void_p(_raw_current_stream(torch.cuda.current_device()))
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype(t, given):
    return given if given is not None else DTYPE_OF[t.dtype]


def _check(status, what):
    if status != OK:
        raise MmacError(status, what)


def _epilogue(D, bias, act, d_type, C=None):
    """The mmac_epilogue_t of a call, or None for the plain call.  D (and C) must have the element
    size of the output type the call writes."""
    if d_type is None:
        if D.dtype not in OUT_OF:
            raise ValueError(f"D has dtype {D.dtype}; expected one of {sorted(str(t) for t in OUT_OF)}")
        d_type = OUT_OF[D.dtype]
    size = {OUT_ACC: 4, OUT_BF16: 2, OUT_F16: 2, OUT_FP8_E4M3: 1, OUT_BF8_E5M2: 1}.get(d_type)
    for t, name in ((D, "D"), (C, "C")):
        if size is not None and t is not None and t.element_size() != size:
            raise ValueError(f"{name} has {t.element_size()}-byte elements; the output type writes {size}")
    if d_type == OUT_ACC and bias is None and act == ACT_NONE:
        return None
    return Epilogue(d_type, act, None if bias is None else bias.data_ptr())


def workspace_bytes(a_type, M, N, K, sparse=False):
    """Bytes of workspace the split-K calls use for this product (0: they would not split)."""
    return int(lib().mmac_gemm_workspace_bytes(int(a_type), M, N, K, 1 if sparse else 0))


def workspace(a_type, M, N, K, sparse=False, device=None):
    """A zeroed workspace tensor for the split-K calls (None if they would not split)."""
    n = workspace_bytes(a_type, M, N, K, sparse)
    if n == 0:
        return None
    return torch.zeros(n, dtype=torch.uint8, device=device if device is not None else torch.device("cuda"))


def gemm_dense(A, B, D, alpha=1.0, beta=0.0, C=None, a_type=None, b_type=None, stream=None, bias=None,
               act=ACT_NONE, d_type=None, workspace=None):
    """D = alpha * A @ B + beta * C with A M x K (row-major) and B given as its N x K transpose.
    With bias (N fp32 values), act or a bfloat16 / float16 D (d_type overrides what D's dtype
    says) this is mmac_gemm_dense_ep: D = round(act(alpha * A @ B + beta * C + bias)); with a
    workspace tensor (see workspace()) it is mmac_gemm_dense_ws, which may split K."""
    M, K = A.shape
    N = B.shape[0]
    _shape(B, N, K, "B")
    _shape(D, M, N, "D")
    _shape(C, M, N, "C")
    _bias(bias, N)
    _same_device(A, B, C, D, bias, workspace)
    ta, tb = _dtype(A, a_type), _dtype(B, b_type)
    args = (ta, tb, M, N, K, float(alpha), _ptr(A), _ld(A), _ptr(B), _ld(B), float(beta),
            _ptr(C), _ld(C) if C is not None else 0, _ptr(D), _ld(D))
    ep = _epilogue(D, bias, act, d_type, C)
    if workspace is not None:
        _check(lib().mmac_gemm_dense_ws(*args, None if ep is None else ctypes.byref(ep), _ptr(workspace),
                                        workspace.numel() * workspace.element_size(), _stream(stream)),
               "mmac_gemm_dense_ws")
    elif ep is None:
        _check(lib().mmac_gemm_dense(*args, _stream(stream)), "mmac_gemm_dense")
    else:
        _check(lib().mmac_gemm_dense_ep(*args, ctypes.byref(ep), _stream(stream)), "mmac_gemm_dense_ep")
    return D


def _compress_shapes(A, Ac, idx, bad_groups):
    M, K = A.shape
    _shape(Ac, M, K // 2, "Ac")
    _shape(idx, M, (K + 31) // 32, "idx")
    if idx.element_size() != 4:
        raise ValueError("idx must hold 32-bit words")
    if bad_groups is not None and (bad_groups.numel() < 1 or bad_groups.element_size() != 4):
        raise ValueError("bad_groups must hold at least one 32-bit counter")
    _same_device(A, Ac, idx, bad_groups)


def gemm_dense_static(A, B, D, alpha=1.0, beta=0.0, C=None, a_type=None, b_type=None, stream=None, bias=None,
                      act=ACT_NONE, d_type=None):
    """gemm_dense with split-K through the library's fixed scratch array (mmac_gemm_dense_static):
    no workspace argument, nothing allocated."""
    M, K = A.shape
    N = B.shape[0]
    _shape(B, N, K, "B")
    _shape(D, M, N, "D")
    _shape(C, M, N, "C")
    _bias(bias, N)
    _same_device(A, B, C, D, bias)
    ta, tb = _dtype(A, a_type), _dtype(B, b_type)
    ep = _epilogue(D, bias, act, d_type, C)
    _check(lib().mmac_gemm_dense_static(ta, tb, M, N, K, float(alpha), _ptr(A), _ld(A), _ptr(B), _ld(B), float(beta),
                                        _ptr(C), _ld(C) if C is not None else 0, _ptr(D), _ld(D),
                                        None if ep is None else ctypes.byref(ep), _stream(stream)),
           "mmac_gemm_dense_static")
    return D


def sparse24_compress(A, Ac, idx, bad_groups=None, a_type=None, stream=None):
    """Compress a 4:2 A (M x K) into Ac (M x K/2) and idx (M x ceil(K/32) words)."""
    M, K = A.shape
    _compress_shapes(A, Ac, idx, bad_groups)
    ta = _dtype(A, a_type)
    st = lib().mmac_sparse24_compress(ta, M, K, _ptr(A), _ld(A), _ptr(Ac), _ld(Ac), _ptr(idx), _ld(idx),
                                      _ptr(bad_groups), _stream(stream))
    _check(st, "mmac_sparse24_compress")
    return Ac, idx


def sparse24_prune_compress(A, Ac, idx, bad_groups=None, a_type=None, stream=None):
    """Prune a dense A (M x K) to 4:2 by magnitude (two largest |a| per group of four) and
    compress it into Ac (M x K/2) and idx (M x ceil(K/32) words), in one pass."""
    M, K = A.shape
    _compress_shapes(A, Ac, idx, bad_groups)
    ta = _dtype(A, a_type)
    st = lib().mmac_sparse24_prune_compress(ta, M, K, _ptr(A), _ld(A), _ptr(Ac), _ld(Ac), _ptr(idx), _ld(idx),
                                            _ptr(bad_groups), _stream(stream))
    _check(st, "mmac_sparse24_prune_compress")
    return Ac, idx


def gemm_sparse24(Ac, idx, B, D, K=None, alpha=1.0, beta=0.0, C=None, a_type=None, b_type=None, stream=None,
                  bias=None, act=ACT_NONE, d_type=None, workspace=None):
    """D = alpha * A @ B + beta * C with A given compressed (Ac, idx); K is the dense K.
    bias / act / a 16-bit D select mmac_gemm_sparse24_ep and a workspace mmac_gemm_sparse24_ws,
    as in gemm_dense."""
    M = Ac.shape[0]
    N, KB = B.shape
    K = KB if K is None else K
    _shape(Ac, M, K // 2, "Ac")
    _shape(B, N, K, "B")
    _shape(idx, M, (K + 31) // 32, "idx", min_cols=True)
    if idx.element_size() != 4:
        raise ValueError("idx must hold 32-bit words")
    _shape(D, M, N, "D")
    _shape(C, M, N, "C")
    _bias(bias, N)
    _same_device(Ac, idx, B, C, D, bias, workspace)
    ta, tb = _dtype(Ac, a_type), _dtype(B, b_type)
    args = (ta, tb, M, N, K, float(alpha), _ptr(Ac), _ld(Ac), _ptr(idx), _ld(idx), _ptr(B), _ld(B), float(beta),
            _ptr(C), _ld(C) if C is not None else 0, _ptr(D), _ld(D))
    ep = _epilogue(D, bias, act, d_type, C)
    if workspace is not None:
        _check(lib().mmac_gemm_sparse24_ws(*args, None if ep is None else ctypes.byref(ep), _ptr(workspace),
                                           workspace.numel() * workspace.element_size(), _stream(stream)),
               "mmac_gemm_sparse24_ws")
    elif ep is None:
        _check(lib().mmac_gemm_sparse24(*args, _stream(stream)), "mmac_gemm_sparse24")
    else:
        _check(lib().mmac_gemm_sparse24_ep(*args, ctypes.byref(ep), _stream(stream)), "mmac_gemm_sparse24_ep")
    return D


def gemm_mx(A, SA, B, SB, D, alpha=1.0, beta=0.0, C=None, a_type=None, b_type=None, stream=None, bias=None,
            act=ACT_NONE, d_type=None):
    """Block-scaled (MX) GEMM: D = alpha * (A, SA) @ (B, SB) + beta * C.  A M x K and B N x K fp8;
    SA and SB the E8M0 scale words (ceil(K/128) x >= M and ceil(K/128) x >= N int32 tensors,
    four block exponents per word, see include/mmac.h).  For FP4_E2M1, A and B are uint8 tensors
    of packed pairs (M x K/2, N x K/2); for FP6_E2M3 / BF6_E3M2 uint8 tensors of packed
    elements, four per three bytes (M x 3K/4, N x 3K/4).  Epilogue arguments as in gemm_dense."""
    M, K = A.shape
    N = B.shape[0]
    ta, tb = _dtype(A, a_type), _dtype(B, b_type)

    def elems(nbytes, t):                      # elements in nbytes stored bytes of type t
        if t == FP4_E2M1:
            return nbytes * 2
        if t in (FP6_E2M3, BF6_E3M2):
            if nbytes % 3:
                raise ValueError("packed FP6 rows and pitches must be whole multiples of 3 bytes")
            return nbytes // 3 * 4
        return nbytes

    K, lda, ldb = elems(K, ta), elems(_ld(A), ta), elems(_ld(B), tb)
    if elems(B.shape[1], tb) != K:
        raise ValueError(f"B has {elems(B.shape[1], tb)} elements per row, A has {K}")
    _shape(SA, (K + 127) // 128, M, "SA", min_cols=True)
    _shape(SB, (K + 127) // 128, N, "SB", min_cols=True)
    if SA.element_size() != 4 or SB.element_size() != 4:
        raise ValueError("SA and SB must hold 32-bit scale words")
    _shape(D, M, N, "D")
    _shape(C, M, N, "C")
    _bias(bias, N)
    _same_device(A, SA, B, SB, C, D, bias)
    ep = _epilogue(D, bias, act, d_type, C)
    st = lib().mmac_gemm_dense_mx(ta, tb, M, N, K, float(alpha), _ptr(A), lda, _ptr(SA), _ld(SA), _ptr(B), ldb,
                                  _ptr(SB), _ld(SB), float(beta), _ptr(C), _ld(C) if C is not None else 0, _ptr(D),
                                  _ld(D), None if ep is None else ctypes.byref(ep), _stream(stream))
    _check(st, "mmac_gemm_dense_mx")
    return D


def gemm_layout(A, B, D, trans_a=False, trans_b=False, alpha=1.0, beta=0.0, C=None, a_type=None, b_type=None,
                stream=None, bias=None, act=ACT_NONE, d_type=None):
    """D = alpha * op(A) @ op(B) + beta * C for every dense type pair.  trans_a: A is given as its K x M
    transpose (M contiguous); trans_b: B is given as K x N (N contiguous).  Otherwise A is M x K and
    B is N x K as in gemm_dense."""
    M = A.shape[1] if trans_a else A.shape[0]
    K = A.shape[0] if trans_a else A.shape[1]
    N = B.shape[1] if trans_b else B.shape[0]
    if (B.shape[0] if trans_b else B.shape[1]) != K:
        raise ValueError(f"B has shape {tuple(B.shape)}, which does not hold K = {K} for this layout")
    _shape(D, M, N, "D")
    _shape(C, M, N, "C")
    _bias(bias, N)
    _same_device(A, B, C, D, bias)
    ta, tb = _dtype(A, a_type), _dtype(B, b_type)
    ep = _epilogue(D, bias, act, d_type, C)
    st = lib().mmac_gemm_dense_layout(ta, tb, int(bool(trans_a)), int(bool(trans_b)), M, N, K, float(alpha), _ptr(A),
                                      _ld(A), _ptr(B), _ld(B), float(beta), _ptr(C), _ld(C) if C is not None else 0,
                                      _ptr(D), _ld(D), None if ep is None else ctypes.byref(ep), _stream(stream))
    _check(st, "mmac_gemm_dense_layout")
    return D


# ---- low-bit operands (include/mmac_lowbit.h) ----------------------------------------------------
# A product for one token takes a few microseconds, as long as a call takes on the host: the checks
# below look at every tensor once, and pass addresses as plain integers.

def _rows_of(t, rows, cols, name, wider=False):
    """_shape and _ld in one: checks a 2-D tensor and returns its row pitch in elements."""
    sh = t.shape
    if len(sh) != 2 or sh[0] != rows or (sh[1] < cols if wider else sh[1] != cols):
        raise ValueError(f"{name} has shape {tuple(sh)}, expected ({rows}, {'>= ' if wider else ''}{cols})")
    pitch, step = t.stride()
    width = sh[1]
    if step != 1 and width > 1:
        raise ValueError(f"{name}: expected a contiguous last dimension")
    if pitch < width:
        if rows > 1:
            raise ValueError(f"{name}: rows of a {tuple(sh)} tensor with row stride {pitch} overlap")
        pitch = width
    return pitch if pitch > 0 else 1


def _stream_of(stream, *tensors):
    """The stream of a call, whose tensors must all live on the current CUDA device, the one it belongs to."""
    device = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError(f"tensors on different devices: {sorted({str(x.device) for x in tensors if x is not None})}")
    if device < 0:
        raise ValueError("every tensor must be in GPU memory")
    if device != torch._C._cuda_getDevice():
        raise ValueError(f"tensors on cuda:{device}, but the current device is cuda:{torch.cuda.current_device()}")
    if stream is not None:
        if stream.device_index != device:
            raise ValueError(f"tensors on cuda:{device}, the stream on cuda:{stream.device_index}")
        return stream.cuda_stream
    if _raw_current_stream is not None:
        return _raw_current_stream(device)
    return torch.cuda.current_stream().cuda_stream


def _input_type(t, given):
    """Type code of an unquantized matrix."""
    if given is not None:
        if t.element_size() != {F32: 4, F16: 2, BF16: 2}.get(given, t.element_size()):
            raise ValueError(f"a tensor of {t.element_size()}-byte elements for type code {given}")
        return given
    code = _INPUT_OF.get(t.dtype)
    if code is None:
        raise ValueError(f"expected a float16, bfloat16 or float32 tensor, got {t.dtype}")
    return code


_INPUT_OF = {torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32}
# dtypes of codes and elements, and of scale words
_BYTES = {torch.uint8, torch.int8, torch.float8_e4m3fn, torch.float8_e5m2}
_WORDS = {torch.int32, torch.uint32}


def _out(D, C, bias, act, d_type):
    """_epilogue of the products below, whose sums are floating: without a d_type, D is of a floating type and C of D's."""
    if d_type is not None:
        return _epilogue(D, bias, act, d_type, C)
    code = OUT_OF.get(D.dtype)
    if code is None or D.dtype is torch.int32:
        raise ValueError(f"D has dtype {D.dtype}; expected float32, bfloat16, float16, float8_e4m3fn or float8_e5m2")
    if C is not None and C.dtype is not D.dtype:
        raise ValueError(f"C has dtype {C.dtype}; expected D's, {D.dtype}")
    if code == OUT_ACC and bias is None and act == ACT_NONE:
        return None
    return Epilogue(code, act, None if bias is None else bias.data_ptr())


def _w4(Wq, SW, N, K, group, q_type):
    """The mmac_w4_t of a weight matrix."""
    if Wq.dtype not in _BYTES:
        raise ValueError("Wq must hold bytes, two codes each")
    if SW.dtype not in _WORDS:
        raise ValueError("SW must hold 32-bit scale words")
    pitch = _rows_of(Wq, N, (K + 31) // 32 * 16, "Wq", True)
    ldw = _rows_of(SW, (K + group - 1) // group if group > 0 else 1, N, "SW", True)
    return W4(q_type, group, Wq.data_ptr(), pitch if pitch > 16 else 16, SW.data_ptr(), ldw)


def _mx8(Xq, SX, M, K, q_type):
    """Checks an mx8 matrix; returns its element type's code and both pitches."""
    if q_type is None:
        q_type = DTYPE_OF.get(Xq.dtype)
    if Xq.dtype not in _BYTES or q_type is None:
        raise ValueError(f"Xq must hold float8_e4m3fn, float8_e5m2 or int8 elements, got {Xq.dtype}")
    if SX.dtype not in _WORDS:
        raise ValueError("SX must hold 32-bit scale words")
    return (q_type, _rows_of(Xq, M, (K + 31) // 32 * 32, "Xq", True), _rows_of(SX, (K + 127) // 128, M, "SX", True))


def _workspace_tensor(nbytes, device):
    if nbytes == 0:
        return None
    return torch.zeros(nbytes, dtype=torch.uint8, device=device if device is not None else torch.device("cuda"))


def _workspace_args(workspace):
    if workspace is None:
        return None, 0
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def w4_quantize(W, Wq, SW, group=128, q_type=U4, symmetric=False, w_type=None, stream=None):
    """Weights W (N x K, float16, bfloat16 or float32) to 4-bit codes Wq (N x 16 ceil(K/32) uint8) and
    scale words SW (groups x N int32), one per `group` (32, 64, 128; 0: whole rows) elements of a
    row, rounded to nearest.  q_type U4 (symmetric: zero point 8) or FP4_E2M1 (symmetric)."""
    N, K = W.shape
    q = _w4(Wq, SW, N, K, group, q_type)
    _check(lib().mmac_w4_quantize(_input_type(W, w_type), 1 if symmetric or q_type == FP4_E2M1 else 0, N, K,
                                  W.data_ptr(), _rows_of(W, N, K, "W"), ctypes.byref(q), _stream_of(stream, W, Wq, SW)),
           "mmac_w4_quantize")
    return Wq, SW


def w4_workspace_bytes(M, N, K):
    """Bytes of workspace gemm_w4 uses for this product (0: it would not split)."""
    return int(lib().mmac_gemm_w4_workspace_bytes(M, N, K))


def w4_workspace(M, N, K, device=None):
    """A zeroed workspace tensor for gemm_w4 (None if it would not split)."""
    return _workspace_tensor(w4_workspace_bytes(M, N, K), device)


def gemm_w4(A, Wq, SW, D, group=128, q_type=U4, alpha=1.0, beta=0.0, C=None, a_type=None, stream=None, bias=None,
            act=ACT_NONE, d_type=None, workspace=None):
    """D = round(act(alpha * A @ W.T + beta * C + bias)) with A M x K (float16 or bfloat16) and the weight W (N x K)
    as w4_quantize stores it.  Epilogue arguments as in gemm_dense; with a workspace (see w4_workspace())
    K may be split."""
    M, K = A.shape
    N = Wq.shape[0]
    ldd = _rows_of(D, M, N, "D")
    ldc = _rows_of(C, M, N, "C") if C is not None else 0
    if bias is not None:
        _bias(bias, N)
    q = _w4(Wq, SW, N, K, group, q_type)
    ep = _out(D, C, bias, act, d_type)
    ws, nbytes = _workspace_args(workspace)
    _check(lib().mmac_gemm_w4(_input_type(A, a_type), M, N, K, alpha, A.data_ptr(), _rows_of(A, M, K, "A"),
                              ctypes.byref(q), beta, C.data_ptr() if C is not None else None, ldc, D.data_ptr(), ldd,
                              None if ep is None else ctypes.byref(ep), ws, nbytes,
                              _stream_of(stream, A, Wq, SW, C, D, bias, workspace)), "mmac_gemm_w4")
    return D


def mx8_quantize(X, Xq, SX, x_type=None, q_type=None, stream=None):
    """Activations X (M x K, float16, bfloat16 or float32) to 8-bit elements Xq (M x 32 ceil(K/32),
    float8_e4m3fn, float8_e5m2 or int8) and scale words SX (ceil(K/128) x M int32): the operand
    form of gemm_mx, and of gemm_mx8_wgrad."""
    M, K = X.shape
    tq, ldq, lds = _mx8(Xq, SX, M, K, q_type)
    _check(lib().mmac_mx8_quantize(_input_type(X, x_type), tq, M, K, X.data_ptr(), _rows_of(X, M, K, "X"), Xq.data_ptr(),
                                   ldq, SX.data_ptr(), lds, _stream_of(stream, X, Xq, SX)), "mmac_mx8_quantize")
    return Xq, SX


def mx8_dequantize(Xq, SX, X, q_type=None, x_type=None, stream=None):
    """The activations that (Xq, SX) stand for, rounded to X's type; X gives M and K."""
    M, K = X.shape
    tq, ldq, lds = _mx8(Xq, SX, M, K, q_type)
    _check(lib().mmac_mx8_dequantize(tq, _input_type(X, x_type), M, K, Xq.data_ptr(), ldq, SX.data_ptr(), lds,
                                     X.data_ptr(), _rows_of(X, M, K, "X"), _stream_of(stream, X, Xq, SX)),
           "mmac_mx8_dequantize")
    return X


def mx8_wgrad_workspace_bytes(M, N, K):
    """Bytes of workspace gemm_mx8_wgrad uses for this product (0: it would not split)."""
    return int(lib().mmac_gemm_mx8_wgrad_workspace_bytes(M, N, K))


def mx8_wgrad_workspace(M, N, K, device=None):
    """A zeroed workspace tensor for gemm_mx8_wgrad (None if it would not split)."""
    return _workspace_tensor(mx8_wgrad_workspace_bytes(M, N, K), device)


def gemm_mx8_wgrad(dY, Xq, SX, D, alpha=1.0, beta=0.0, C=None, y_type=None, q_type=None, stream=None, d_type=None,
                   workspace=None):
    """Weight gradient D = alpha * dY.T @ X + beta * C (N x K) from the gradient dY (M x N, float16 or bfloat16) of a
    linear layer's output and its input as mx8_quantize stored it; D gives K."""
    M, N = dY.shape
    K = D.shape[1]
    ldd = _rows_of(D, N, K, "D")
    ldc = _rows_of(C, N, K, "C") if C is not None else 0
    tq, ldq, lds = _mx8(Xq, SX, M, K, q_type)
    ep = _out(D, C, None, ACT_NONE, d_type)
    ws, nbytes = _workspace_args(workspace)
    _check(lib().mmac_gemm_mx8_wgrad(_input_type(dY, y_type), tq, M, N, K, alpha, dY.data_ptr(),
                                     _rows_of(dY, M, N, "dY"), Xq.data_ptr(), ldq, SX.data_ptr(), lds, beta,
                                     C.data_ptr() if C is not None else None, ldc, D.data_ptr(), ldd,
                                     None if ep is None else ctypes.byref(ep), ws, nbytes,
                                     _stream_of(stream, dY, Xq, SX, C, D, workspace)), "mmac_gemm_mx8_wgrad")
    return D


def mx4_quantize(X, Xq, SX, x_type=None, stream=None):
    """Rows X (M x K, float16, bfloat16 or float32) to packed FP4 (E2M1) elements Xq (M x 16 ceil(K/32) bytes) and scale
    words SX (ceil(K/128) x M int32): the operand form of gemm_mx (K % 32 == 0) and of gemm_grouped_mx's weights."""
    M, K = X.shape
    if Xq.dtype not in _BYTES:
        raise ValueError("Xq must hold bytes, two elements each")
    if SX.dtype not in _WORDS:
        raise ValueError("SX must hold 32-bit scale words")
    _check(lib().mmac_mx4_quantize(_input_type(X, x_type), M, K, X.data_ptr(), _rows_of(X, M, K, "X"), Xq.data_ptr(),
                                   max(_rows_of(Xq, M, (K + 31) // 32 * 16, "Xq", True), 16), SX.data_ptr(),
                                   _rows_of(SX, (K + 127) // 128, M, "SX", True), _stream_of(stream, X, Xq, SX)),
           "mmac_mx4_quantize")
    return Xq, SX


# ---- RMS norm (include/mmac_norm.h) --------------------------------------------------------------

def _vector(t, n, name, other=torch.float32):
    """The address of a contiguous vector of n float32 (or `other`) values."""
    dtype = t.dtype
    if dtype is not torch.float32 and dtype is not other:
        raise ValueError(f"{name} has dtype {dtype}; expected {' or '.join(sorted({'torch.float32', str(other)}))}")
    if t.shape != (n,) or (n > 1 and t.stride() != (1,)):
        raise ValueError(f"{name} must be a contiguous vector of {n} values")
    return t.data_ptr()


def _same_type(t, X, name):
    if t.dtype is not X.dtype:
        raise ValueError(f"{name} has dtype {t.dtype}; expected {X.dtype}")


def rmsnorm(X, w, Y, eps=1e-6, residual=None, H=None, rstd=None, SY=None, stream=None):
    """Y = h * r * w with h = X (+ residual, rounded to X's type), r = 1 / sqrt(mean(h^2) + eps) per row of X (M x N,
    float16, bfloat16 or float32); w of X's type or float32.  Y of X's type, or 8-bit elements (M x 32 ceil(N/32),
    float8_e4m3fn or float8_e5m2) with their scale words SY (ceil(N/128) x M int32), the operand form of gemm_mx, gemm_grouped_mx
    and gemm_mx8_wgrad.  H (h itself, may be X or residual) and rstd (r, M float32) are written when given."""
    M, N = X.shape
    dtype = X.dtype
    tx = _input_type(X, None)
    lds = ldr = ldh = 0
    at_r = at_h = at_s = None
    if Y.dtype is dtype:
        ty, ldy = tx, _rows_of(Y, M, N, "Y")
        if SY is not None:
            raise ValueError("SY goes with an 8-bit Y")
    elif Y.dtype is torch.float8_e4m3fn or Y.dtype is torch.float8_e5m2:
        if SY is None:
            raise ValueError("an 8-bit Y needs SY")
        ty, ldy, lds = _mx8(Y, SY, M, N, None)
        at_s = SY.data_ptr()
    else:
        raise ValueError(f"Y has dtype {Y.dtype}; expected {dtype}, float8_e4m3fn or float8_e5m2")
    if residual is not None:
        _same_type(residual, X, "residual")
        ldr, at_r = _rows_of(residual, M, N, "residual"), residual.data_ptr()
    if H is not None:
        _same_type(H, X, "H")
        ldh, at_h = _rows_of(H, M, N, "H"), H.data_ptr()
    at_w = _vector(w, N, "w", dtype)
    _check(lib().mmac_rmsnorm(tx, _INPUT_OF[w.dtype], ty, M, N, X.data_ptr(), _rows_of(X, M, N, "X"), at_r, ldr, at_w, eps,
                              at_h, ldh, Y.data_ptr(), ldy, at_s, lds, _vector(rstd, M, "rstd") if rstd is not None else None,
                              _stream_of(stream, X, w, Y, residual, H, rstd, SY)), "mmac_rmsnorm")
    return Y


def rmsnorm_grad_workspace_bytes(M, N):
    """Bytes of workspace rmsnorm_grad needs for dW."""
    return int(lib().mmac_rmsnorm_grad_workspace_bytes(M, N))


def rmsnorm_grad_workspace(M, N, device=None):
    """A workspace tensor for rmsnorm_grad with dW."""
    return _workspace_tensor(rmsnorm_grad_workspace_bytes(M, N), device)


def rmsnorm_grad(dY, H, w, rstd, dX, dW=None, dH=None, workspace=None, stream=None):
    """Gradients of rmsnorm from that of Y and the forward pass's h and r: dX (that of X and of the residual, dH added, the
    gradient that reaches h on the residual stream; dX may be dY or dH) and dW (N float32; needs a
    workspace, see rmsnorm_grad_workspace())."""
    M, N = dY.shape
    for t, name in ((H, "H"), (dX, "dX"), (dH, "dH")):
        if t is not None:
            _same_type(t, dY, name)
    at_w = _vector(w, N, "w", dY.dtype)
    ws, nbytes = _workspace_args(workspace)
    _check(lib().mmac_rmsnorm_grad(_input_type(dY, None), _INPUT_OF[w.dtype], M, N, dY.data_ptr(), _rows_of(dY, M, N, "dY"),
                                   H.data_ptr(), _rows_of(H, M, N, "H"), at_w, _vector(rstd, M, "rstd"),
                                   dH.data_ptr() if dH is not None else None,
                                   _rows_of(dH, M, N, "dH") if dH is not None else 0, dX.data_ptr(),
                                   _rows_of(dX, M, N, "dX"), _vector(dW, N, "dW") if dW is not None else None, ws, nbytes,
                                   _stream_of(stream, dY, H, w, rstd, dX, dW, dH, workspace)), "mmac_rmsnorm_grad")
    return dX


# ---- products grouped by expert (include/mmac_grouped.h) -------------------------------------------

def _groups_of(t, groups, rows, cols, name, wider=False):
    """Checks a groups x rows x cols tensor; returns the strides of its rows and of its groups."""
    sh = t.shape
    if len(sh) != 3 or sh[0] != groups or sh[1] != rows or (sh[2] < cols if wider else sh[2] != cols):
        raise ValueError(f"{name} has shape {tuple(sh)}, expected ({groups}, {rows}, {'>= ' if wider else ''}{cols})")
    stride, pitch, step = t.stride()
    width = sh[2]
    if step != 1 and width > 1:
        raise ValueError(f"{name}: expected a contiguous last dimension")
    if pitch < width:
        if rows > 1:
            raise ValueError(f"{name}: rows of a {tuple(sh)} tensor with row stride {pitch} overlap")
        pitch = width
    if groups > 1 and stride < (rows - 1) * pitch + width:
        raise ValueError(f"{name}: groups of a {tuple(sh)} tensor with strides {tuple(t.stride())} overlap")
    return (pitch if pitch > 0 else 1), stride


def _offsets(offsets, groups):
    if offsets.dtype is not torch.int32:
        raise ValueError(f"offsets has dtype {offsets.dtype}; expected torch.int32")
    if offsets.shape != (groups + 1,) or (groups and offsets.stride() != (1,)):
        raise ValueError(f"offsets must be a contiguous vector of {groups + 1} values")
    return offsets.data_ptr()


def _group_bias(bias, groups, N):
    if bias is not None and (bias.dtype != torch.float32 or tuple(bias.shape) != (groups, N) or not bias.is_contiguous()):
        raise ValueError(f"bias must be a contiguous float32 tensor of shape ({groups}, {N})")


def gemm_grouped(A, offsets, B, D, trans_b=False, alpha=1.0, beta=0.0, C=None, a_type=None, stream=None, bias=None,
                 act=ACT_NONE, d_type=None):
    """For the rows of each group g, offsets[g] .. offsets[g+1] - 1 (int32, in GPU memory): D = round(act(alpha * A @ B[g].T
    + beta * C + bias[g])), A M x K (float16 or bfloat16), B groups x N x K of the same type.  trans_b: B is
    groups x K x N and the product is with B[g] itself: with a forward product's weights, the gradient of its input.
    Rows of no group are neither read nor written.  Epilogue arguments as in gemm_dense, bias groups x N."""
    M, K = A.shape
    if B.dim() != 3:
        raise ValueError(f"B has shape {tuple(B.shape)}, expected one matrix per group")
    _same_type(B, A, "B")
    groups, N = B.shape[0], B.shape[2 if trans_b else 1]
    ldb, stride_b = _groups_of(B, groups, K if trans_b else N, N if trans_b else K, "B")
    ldd = _rows_of(D, M, N, "D")
    ldc = _rows_of(C, M, N, "C") if C is not None else 0
    _group_bias(bias, groups, N)
    ep = _out(D, C, bias, act, d_type)
    _check(lib().mmac_gemm_grouped(_input_type(A, a_type), 1 if trans_b else 0, groups, M, N, K, alpha, A.data_ptr(),
                                   _rows_of(A, M, K, "A"), _offsets(offsets, groups), B.data_ptr(), ldb, stride_b, beta,
                                   C.data_ptr() if C is not None else None, ldc, D.data_ptr(), ldd,
                                   None if ep is None else ctypes.byref(ep),
                                   _stream_of(stream, A, offsets, B, C, D, bias)), "mmac_gemm_grouped")
    return D


def gemm_grouped_mx(A, SA, offsets, B, SB, D, alpha=1.0, beta=0.0, C=None, a_type=None, b_type=None, stream=None,
                    bias=None, act=ACT_NONE, d_type=None):
    """gemm_grouped from block-scaled operands: A M x K (float8_e4m3fn or float8_e5m2) with its scale words SA (ceil(K/128)
    x >= M int32), B groups x N x K of one of these types, or (b_type FP4_E2M1) groups x N x K/2 uint8 of packed pairs,
    with SB groups x ceil(K/128) x >= N.  K % 32 == 0."""
    M, K = A.shape
    if B.dim() != 3:
        raise ValueError(f"B has shape {tuple(B.shape)}, expected one matrix per group")
    groups, N = B.shape[0], B.shape[1]
    ta, tb = _dtype(A, a_type), _dtype(B, b_type) if b_type is not None or B.dtype in DTYPE_OF else None
    if tb is None or B.dtype not in _BYTES or A.dtype not in _BYTES:
        raise ValueError(f"A and B must hold 8-bit elements or packed FP4 (b_type), got {A.dtype} and {B.dtype}")
    per = 2 if tb == FP4_E2M1 else 1
    ldb, stride_b = _groups_of(B, groups, N, K // per, "B")
    if SA.dtype not in _WORDS or SB.dtype not in _WORDS:
        raise ValueError("SA and SB must hold 32-bit scale words")
    strips = (K + 127) // 128
    ldsa = _rows_of(SA, strips, M, "SA", True)
    ldsb, stride_sb = _groups_of(SB, groups, strips, N, "SB", True)
    ldd = _rows_of(D, M, N, "D")
    ldc = _rows_of(C, M, N, "C") if C is not None else 0
    _group_bias(bias, groups, N)
    ep = _out(D, C, bias, act, d_type)
    _check(lib().mmac_gemm_grouped_mx(ta, tb, groups, M, N, K, alpha, A.data_ptr(), _rows_of(A, M, K, "A"), SA.data_ptr(),
                                      ldsa, _offsets(offsets, groups), B.data_ptr(), ldb * per, stride_b * per, SB.data_ptr(),
                                      ldsb, stride_sb, beta, C.data_ptr() if C is not None else None, ldc, D.data_ptr(), ldd,
                                      None if ep is None else ctypes.byref(ep),
                                      _stream_of(stream, A, SA, offsets, B, SB, C, D, bias)), "mmac_gemm_grouped_mx")
    return D


def gemm_grouped_wgrad(dY, X, offsets, D, alpha=1.0, beta=0.0, C=None, y_type=None, stream=None, d_type=None):
    """Weight gradients of a grouped product: D[g] = alpha * dY[rows of g].T @ X[rows of g] + beta * C[g] (groups x N x K)
    with dY M x N and X M x K (float16 or bfloat16).  A group without rows gives beta * C[g]."""
    M, N = dY.shape
    K = X.shape[1]
    _same_type(X, dY, "X")
    if D.dim() != 3:
        raise ValueError(f"D has shape {tuple(D.shape)}, expected one matrix per group")
    groups = D.shape[0]
    ldd, stride_d = _groups_of(D, groups, N, K, "D")
    ldc, stride_c = _groups_of(C, groups, N, K, "C") if C is not None else (0, 0)
    ep = _out(D, C, None, ACT_NONE, d_type)
    _check(lib().mmac_gemm_grouped_wgrad(_input_type(dY, y_type), groups, M, N, K, alpha, dY.data_ptr(),
                                         _rows_of(dY, M, N, "dY"), X.data_ptr(), _rows_of(X, M, K, "X"),
                                         _offsets(offsets, groups), beta, C.data_ptr() if C is not None else None, ldc,
                                         stride_c, D.data_ptr(), ldd, stride_d, None if ep is None else ctypes.byref(ep),
                                         _stream_of(stream, dY, X, offsets, C, D)), "mmac_gemm_grouped_wgrad")
    return D


def raw_call(name, *args):
    """Call a C entry point with raw arguments (pointers as ints); returns the status."""
    return getattr(lib(), name)(*args)
