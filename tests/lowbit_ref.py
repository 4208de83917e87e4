"""References of the low-bit operands in 64 bits (numpy; no code of the library), and the layouts that
include/mmac_lowbit.h defines, written from their definitions."""
import numpy as np

U4, FP4 = 9, 6
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)
U32 = 2.0 ** -24

# element types: largest value and all finite non-negative values in code order (code = index)
E4M3_POS = np.array([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][:127])
E5M2_POS = np.array([m * 2.0 ** -16 if e == 0 else (4 + m) * 2.0 ** (e - 17) for e in range(31) for m in range(4)])
TOP = {"e4m3": 448.0, "e5m2": 57344.0, "int8": 127.0}


def rne_codes(a, table):
    """Index of the table value (ascending, from 0) nearest to a >= 0, ties to the even index."""
    hi = np.clip(np.searchsorted(table, a), 1, len(table) - 1)
    lo = hi - 1
    d_lo, d_hi = a - table[lo], table[hi] - a
    return np.where((d_hi < d_lo) | ((d_hi == d_lo) & (hi % 2 == 0)), hi, lo)


def group_index(K, group):
    return np.zeros(K, np.int64) if group == 0 else np.arange(K) // group


def n_groups(K, group):
    return 1 if group == 0 else -(-K // group)


def round16(s):
    """Non-negative values rounded to 16 significant bits, ties to even."""
    m, e = np.frexp(s)
    return np.ldexp(np.round(m * 65536), e - 16)


def w4_quantize(W, group, q_type, symmetric):
    """W float64 (N x K), its values exact in fp32 -> codes (N x K), scales and zero points (N x groups)."""
    N, K = W.shape
    G = n_groups(K, group)
    gi = group_index(K, group)
    s, z = np.zeros((N, G)), np.zeros((N, G), np.int64)
    codes = np.zeros((N, K), np.int64)
    steps = 6 if q_type == FP4 else 7 if symmetric else 15
    with np.errstate(all="ignore"):
        for g in range(G):
            w = W[:, gi == g]
            finite = np.isfinite(w).all(1)
            hi, lo = np.maximum(w.max(1), 0), np.minimum(w.min(1), 0)
            if q_type == FP4 or symmetric:
                r = np.abs(w).max(1)
            else:
                r = (hi.astype(np.float32) - lo.astype(np.float32)).astype(np.float64)
            sg = (r / steps).astype(np.float32).astype(np.float64)
            finite &= np.isfinite(sg)
            sg = np.where(sg < 2.0 ** -126, 0.0, round16(sg))
            zg = np.full(N, 8 if q_type == U4 and symmetric else 0)
            live = finite & (sg > 0)
            div = np.where(live, sg, 1.0)
            if q_type == U4 and not symmetric:
                zg = np.where(live, np.clip(np.round(-np.where(live, lo, 0) / div), 0, 15), 0).astype(np.int64)
            x = np.where(live[:, None], w, 0.0) / div[:, None]
            if q_type == FP4:
                c = rne_codes(np.abs(x), E2M1) + 8 * (x < 0)
            else:
                c = np.clip(np.round(x).astype(np.int64) + zg[:, None], 0, 15)
            codes[:, gi == g] = c
            s[:, g], z[:, g] = np.where(finite, sg, np.nan), zg
    return codes, s, z


def pack_codes(codes, fill=0):
    """N x K codes -> N x 16 ceil(K/32) bytes; nibbles past K are `fill`."""
    N, K = codes.shape
    c = np.full((N, -(-K // 32) * 32), fill, np.uint8)
    c[:, :K] = codes
    return c[:, 0::2] | (c[:, 1::2] << 4)


def unpack_codes(b, K):
    c = np.empty((b.shape[0], 2 * b.shape[1]), np.int64)
    c[:, 0::2], c[:, 1::2] = b & 15, b >> 4
    return c[:, :K]


def scale_words(s, z):
    """N x groups scales (16 significant bits) and zero points -> groups x N words."""
    u = np.where(np.isnan(s), np.uint32(0x7fc00000), s.astype(np.float32).view(np.uint32))
    return np.ascontiguousarray((u | z.astype(np.uint32)).T).view(np.int32)


def w4_values(codes, s, z, group, q_type):
    gi = group_index(codes.shape[1], group)
    if q_type == FP4:
        v = np.where(codes >= 8, -1.0, 1.0) * E2M1[codes & 7]
        return v * s[:, gi]
    return (codes - z[:, gi]) * s[:, gi]


def gemm_w4(A, codes, s, z, group, q_type):
    """(A @ W^T, the sum of the magnitudes that the kernel adds up: U4 forms sum a n - z sum a)."""
    gi = group_index(codes.shape[1], group)
    if q_type == FP4:
        mags = E2M1[codes & 7] * s[:, gi]
    else:
        mags = (codes + z[:, gi]) * s[:, gi]
    return A @ w4_values(codes, s, z, group, q_type).T, np.abs(A) @ mags.T


def mx8_quantize(X, t):
    """X float64 (M x K, finite, exact in fp32) -> codes (M x Kp int; int8 values, fp8 bits) and exponents (M x ceil(K/32))."""
    M, K = X.shape
    x = np.zeros((M, -(-K // 32) * 32))
    x[:, :K] = X
    b = x.reshape(M, -1, 32)
    top = np.abs(b).max(2)
    e = np.full(top.shape, 1, np.int64)
    for i, v in np.ndenumerate(top):       # the smallest exponent whose power of two holds the block
        if v == 0:
            e[i] = 127
            continue
        k = int(np.floor(np.log2(v / TOP[t]))) - 1
        while TOP[t] * 2.0 ** k < v:
            k += 1
        e[i] = max(k + 127, 1)
    y = np.ldexp(b, (127 - e)[:, :, None])
    if t == "int8":
        q = np.round(y).astype(np.int64)
    else:
        q = rne_codes(np.abs(y), E4M3_POS if t == "e4m3" else E5M2_POS) + 128 * (np.signbit(y))
    return q.reshape(M, -1), e


def mx8_values(q, e, t):
    """Codes and exponents -> float64 values (NaN codes and e = 255 are NaN)."""
    if t == "int8":
        v = q.astype(np.float64)
    else:
        pos = E4M3_POS if t == "e4m3" else E5M2_POS
        n = len(pos)
        full = np.concatenate([pos, [np.nan] if t == "e4m3" else [np.inf, np.nan, np.nan, np.nan]])
        assert len(full) == 128 and n in (127, 124)
        v = np.where(q >= 128, -1.0, 1.0) * full[q & 127]
    s = np.ldexp(1.0, e - 127)
    s[e == 255] = np.nan
    return (v.reshape(v.shape[0], -1, 32) * s[:, :, None]).reshape(v.shape[0], -1)


def sx_words(e, fill=127):
    """M x blocks exponents -> ceil(blocks/4) x M words; bytes past the blocks are `fill`."""
    M, nb = e.shape
    full = np.full((M, -(-nb // 4) * 4), fill, np.uint8)
    full[:, :nb] = e
    return np.ascontiguousarray(full.view("<u4").reshape(M, -1).T).view(np.int32)
