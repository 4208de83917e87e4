// C ABI of the products grouped by expert: argument validation on the host, choice of the tile, launch on the
// caller's stream.  The public contract is in include/mmac_grouped.h.
#include <algorithm>
#include <cstdlib>

#include "abi_check.h"
#include "grouped.h"
#include "mmac_grouped.h"

using namespace mmac;

namespace {

constexpr int64_t kMaxGroups = 1 << 30;   // the search for a tile counts them in 32 bits, 256 at a time

int forced_tile() {
    const char *s = std::getenv("MMAC_TILE");
    switch (s ? std::atoi(s) : 0) {
    case 256: return GROUP_256;
    case 1282: return GROUP_128x256;
    case 128: return GROUP_128;
    case 64: return GROUP_64;
    case 32: return GROUP_32;
    case 16: return GROUP_16;
    default: return -1;
    }
}

// Tiles of a product whose rows are spread evenly over the groups that can have some.
int64_t even_tiles(int64_t groups, int64_t M, int64_t N, GroupTile t) {
    const int64_t n = std::min(groups, M), rows = (M + n - 1) / n;
    return n * ((rows + group_rows(t) - 1) / group_rows(t)) * ((N + group_cols(t) - 1) / group_cols(t));
}

// Tiles, measured in us (bf16, 16-bit outputs, M spread evenly; G groups of r rows, N x K weights; a tile's rows x columns).
// Few rows, streamed weights: 16 or 32 rows x 16 columns, eight waves on K, win where tiles of 64 x 64 would leave compute
// units idle (2 x 4096 x 4096: 16 against 32) or K is long (16 groups of 1: 113 against 121), and lose elsewhere (64 x 2 x 2048^2: 141
// against 129).  K up to 1024 or too few tiles of 128 rows: 64 x 64 (32 x 64 x 2048 x 1024: 33 against 41).  Up to 64 rows:
// 128 x 128 (16 x 32 x 4096^2: 130 against 157 in 64 x 64).  Up to 384 rows: 128 x 256 (16 x 256 x 4096^2: 213, in 256 x 256
// 226); beyond, 256 x 256 (16 x 512 x 4096^2: 331, in 128 x 256 339; 8 x 1024 x 1024 x 2048, 128 tiles: 55, 62), where there are enough.
GroupTile forward_tile(int64_t groups, int64_t M, int64_t N, int64_t K) {
    const int64_t rows = (M + groups - 1) / groups, small = even_tiles(groups, M, N, GROUP_64);
    if ((rows <= 8 && K >= 4096) || (rows <= 32 && small <= 256)) return rows <= 16 ? GROUP_16 : GROUP_32;
    if (rows <= 16 || (rows <= 64 && K <= 1024)) return GROUP_64;
    if (rows >= 384 && even_tiles(groups, M, N, GROUP_256) >= 128) return GROUP_256;
    if (rows > 64 && even_tiles(groups, M, N, GROUP_128x256) >= 192) return GROUP_128x256;
    return even_tiles(groups, M, N, GROUP_128) >= 192 ? GROUP_128 : GROUP_64;
}
// Weights read as K x N rows (K: the sum).  128 x 128, two workgroups a compute unit, up to 512 rows (16 x 128 x 4096^2: 184 against 208 in
// 256 x 256; 8 x 512 x 8192 x 2048: 299 against 258), 64 x 64 for short sums or too few tiles (11 x 163, 1452 columns, K 6313: 113
// against 142; K 2048, 2048 columns: 16 x 128, 256 tiles, 38 against 40; 24 x 128, 384 of them, 54 against 41).
GroupTile input_tile(int64_t groups, int64_t M, int64_t N, int64_t K) {
    const int64_t rows = (M + groups - 1) / groups;
    if (rows >= 512 && even_tiles(groups, M, N, GROUP_256) >= 192) return GROUP_256;
    if ((rows <= 64 && K <= 1024) || even_tiles(groups, M, N, GROUP_128) < 384) return GROUP_64;
    return GROUP_128;
}
// Block-scaled: a 128 x 128 tile's stages are small enough for two or three workgroups a compute unit (FP4 weights, 4 x 2048 x 4096^2:
// 142 against 164 in 128 x 256; 16 x 64: 51 against 47; 16 x 16: 39 against 31).  16 rows x 32 columns also for up to 32 rows and few
// tiles (kernel time, 8 x 32 x 1024 x 2048 E4M3, 128 tiles of 64 x 64: 7.9 against 11.5; 4 x 32 x 4096 x 2048 FP4, 256 of them: 11.6
// against 11.3).  64 x 64 for short sums of groups that a tile of 128 rows would leave half empty (FP4, N 4096, K 1024: 16 x 64 12.6,
// 16 in 128 x 256; 16 x 128 20.6 against 17.3; 4 x 2048 67 against 51 in 128 x 128) or too few of those.
GroupTile mx_tile(int64_t groups, int64_t M, int64_t N, int64_t K) {
    const int64_t rows = (M + groups - 1) / groups, small = even_tiles(groups, M, N, GROUP_64);
    if ((rows <= 8 && (K > 2048 || small <= 256)) || (rows <= 32 && small <= 128)) return GROUP_16;
    if ((rows <= 64 && K <= 1152) || even_tiles(groups, M, N, GROUP_128) < 256) return GROUP_64;
    return rows <= 128 && even_tiles(groups, M, N, GROUP_128x256) >= 192 ? GROUP_128x256 : GROUP_128;
}

// Weight gradients (us; a group's D is N x K, its sum M / groups rows long).  64 x 64, four or five workgroups a compute unit, hide
// short sums' latencies and lose least at the edges (49 x 1109 x 1775 bf16 from 20 rows each, tiles 0.86 full: 178, in 256 x 256 237;
// 7 x 1965 x 1924 fp32 from 4: 42 against 63).  256 x 256 for long sums that fill their tiles (4 x 4096^2 from 2048 rows: 290 against
// 441; 4 x 1850^2 from 1024, 0.82 full: 46 against 55; 8 x 1300^2 from 512, 0.72 full: 54 against 42) and, where they fill them better
// still, for many large matrices in 16 bits (16 x 4096^2 from 32 rows: 204 against 241; 24 x 2700^2 from 64, 0.92 full: 154 against 171);
// those in fp32, whose C and D take the time, in 128 x 128 (440, 473 in 256 x 256).
GroupTile wgrad_tile(int64_t groups, int64_t M, int64_t N, int64_t K, int64_t tiles, bool fp32) {
    const int64_t rows = M / groups;
    const double filled = (double)groups * N * K / (65536.0 * tiles);   // share of the 256 x 256 tiles that is D
    if (rows >= 512 && tiles >= 192 && filled >= 0.8) return GROUP_256;
    if (tiles >= 1024 && filled >= 0.91) return fp32 ? GROUP_128 : GROUP_256;
    return GROUP_64;
}

// A launch counts its threads in 32 bits; half of that is enough here.
bool grid_fits(int64_t blocks, GroupTile t) { return blocks <= INT32_MAX / group_threads(t); }

// The most tiles that M rows in `groups` groups can make: n groups with rows, all but one row of each spread evenly
// (a half tile counts as one).
int64_t most_tiles(int64_t groups, int64_t M, int rows, int64_t columns) {
    const int64_t n = std::min(groups, M);
    return (n + (M - n) / rows) * columns;
}

// What the products share: dimensions, alpha ... D and the epilogue, offsets.
mmac_status_t check_common(int64_t groups, int64_t M, int64_t N, int64_t K, const int32_t *offsets) {
    if (bad_dim(groups) || bad_dim(M) || bad_dim(N) || bad_dim(K)) return MMAC_ERR_INVALID_ARG;
    if (groups > kMaxGroups) return MMAC_ERR_UNSUPPORTED;
    if (groups > 0 && M > 0 && N > 0 && !offsets) return MMAC_ERR_INVALID_ARG;
    return aligned(offsets, 4) ? MMAC_OK : MMAC_ERR_MISALIGNED;
}

// Matrices of `rows` rows of `cols` elements, pitch ld, one per group, `stride` elements apart; `per` elements a byte.
mmac_status_t check_stride(int64_t groups, int64_t rows, int64_t cols, int64_t ld, int64_t stride, int align) {
    if (groups <= 1 || rows <= 0 || cols <= 0) return MMAC_OK;
    if (stride < (rows - 1) * ld + cols || stride > INT64_MAX / 8 / groups) return MMAC_ERR_INVALID_ARG;
    return stride % align ? MMAC_ERR_MISALIGNED : MMAC_OK;
}

GemmParams make_params(int64_t M, int64_t N, int64_t K, double alpha, const void *A, int64_t a_pitch, const void *B,
                       int64_t b_pitch, double beta, const void *C, int64_t ldc, void *D, int64_t ldd,
                       const mmac_epilogue_t &ep) {
    GemmParams p{};
    p.A = static_cast<const uint8_t *>(A);
    p.a_pitch = a_pitch;
    p.B = static_cast<const uint8_t *>(B);
    p.b_pitch = b_pitch;
    p.D = D;
    p.ldd = ldd;
    p.M = (int)M;
    p.N = (int)N;
    p.K = (int)K;
    p.alpha = (float)alpha;
    p.beta = (float)beta;
    p.use_c = p.beta != 0.0f;
    p.C = p.use_c ? C : nullptr;
    p.ldc = p.use_c ? ldc : 0;
    // fp32 C starts the sum only where that scales nothing by beta / alpha (see GemmParams)
    if (p.use_c && ep.d_type == MMAC_OUT_ACC && (p.alpha == p.beta || p.alpha == 1.0f)) {
        p.fold_c = 1;
        p.c_scale = p.alpha == p.beta ? 1.0f : p.beta;
    }
    const int es = out_size(ep.d_type);
    p.vec_d = aligned(D, 16) && (ldd * es) % 16 == 0;
    p.vec_c = p.use_c && aligned(C, 16) && (ldc * es) % 16 == 0;
    p.d_type = ep.d_type;
    p.act = ep.act;
    p.bias = ep.bias;
    p.group_m = 8;
    p.splits = 1;
    p.kt_per_split = 0x7fffffff;
    return p;
}

constexpr GroupTile kMxLargest = GROUP_128x256;   // of the block-scaled products

// Tile counts of the forward products and their grid.  Where that is too large to launch, larger tiles up to `largest` take the
// place of t; false if none fits.
bool set_grid(GemmParams &p, int64_t groups, GroupTile &t, GroupTile largest, int64_t &grid) {
    for (;;) {
        const int cols = largest == kMxLargest && t == GROUP_16 ? kMxRowsCols : group_cols(t);
        const int64_t tn = (p.N + (int64_t)cols - 1) / cols;
        grid = (most_tiles(groups, p.M, group_rows(t), tn) + 7) / 8 * 8 + 8;   // either kind of tile may leave some XCDs one short
        if (grid_fits(grid, t)) {
            p.tiles_n = (int)tn;
            p.tiles_m = 0;   // differs by group
            return true;
        }
        if (t >= largest) return false;
        t = t < GROUP_64 ? GROUP_64 : t == GROUP_64 ? GROUP_128 : largest;
    }
}

}  // namespace

extern "C" {

mmac_status_t mmac_gemm_grouped(mmac_dtype_t a_type, int trans_b, int64_t groups, int64_t M, int64_t N, int64_t K,
                                double alpha, const void *A, int64_t lda, const int32_t *offsets, const void *B,
                                int64_t ldb, int64_t stride_b, double beta, const void *C, int64_t ldc, void *D,
                                int64_t ldd, const mmac_epilogue_t *ep_in, void *stream) {
    const mmac_epilogue_t ep = epilogue_of(ep_in);
    if (!is_16bit(a_type)) return MMAC_ERR_UNSUPPORTED;
    if (trans_b != 0 && trans_b != 1) return MMAC_ERR_INVALID_ARG;
    mmac_status_t st = check_common(groups, M, N, K, offsets);
    if (st != MMAC_OK) return st;
    const bool empty = groups == 0 || M == 0 || N == 0;
    if (!empty && K > 0 && (!A || !B)) return MMAC_ERR_INVALID_ARG;
    const int64_t b_rows = trans_b ? K : N, b_cols = trans_b ? N : K;
    if (K > 0) {   // else neither is read
        st = check_matrix(A, lda, M, K, 2);
        if (st == MMAC_OK) st = check_matrix(B, ldb, groups * b_rows, b_cols, 2);
        if (st == MMAC_OK) st = check_stride(groups, b_rows, b_cols, ldb, stride_b, 8);
    }
    if (st == MMAC_OK) st = check_out(groups > 0 ? M : 0, N, alpha, beta, C, ldc, D, ldd, ep);
    if (st != MMAC_OK) return st;
    if (trans_b && K * ldb * 2 >= ((int64_t)1 << 31)) return MMAC_ERR_UNSUPPORTED;
    if (empty) return MMAC_OK;

    const int forced = forced_tile();
    GroupTile t = forced >= 0 ? (GroupTile)forced : trans_b ? input_tile(groups, M, N, K) : forward_tile(groups, M, N, K);
    if (trans_b && (t == GROUP_16 || t == GROUP_32)) t = GROUP_64;
    GemmParams p = make_params(M, N, K, alpha, A, lda * 2, B, ldb * 2, beta, C, ldc, D, ldd, ep);
    Groups g{};
    g.offsets = offsets;
    g.count = (int)groups;
    g.rows = (int)M;
    g.b_stride = groups > 1 ? stride_b * 2 : 0;
    g.bias_stride = N;
    int64_t grid;
    if (!set_grid(p, groups, t, GROUP_256, grid)) return MMAC_ERR_UNSUPPORTED;
    return launched(launch_gemm_grouped(a_type, trans_b != 0, t, p, g, grid, static_cast<hipStream_t>(stream)));
}

mmac_status_t mmac_gemm_grouped_mx(mmac_dtype_t a_type, mmac_dtype_t b_type, int64_t groups, int64_t M, int64_t N,
                                   int64_t K, double alpha, const void *A, int64_t lda, const uint32_t *SA,
                                   int64_t ldsa, const int32_t *offsets, const void *B, int64_t ldb, int64_t stride_b,
                                   const uint32_t *SB, int64_t ldsb, int64_t stride_sb, double beta, const void *C,
                                   int64_t ldc, void *D, int64_t ldd, const mmac_epilogue_t *ep_in, void *stream) {
    const mmac_epilogue_t ep = epilogue_of(ep_in);
    const auto fp8 = [](int t) { return t == MMAC_FP8_E4M3 || t == MMAC_BF8_E5M2; };
    if (!fp8(a_type) || (!fp8(b_type) && b_type != MMAC_FP4_E2M1)) return MMAC_ERR_UNSUPPORTED;
    mmac_status_t st = check_common(groups, M, N, K, offsets);
    if (st != MMAC_OK) return st;
    if (K % 32) return MMAC_ERR_INVALID_ARG;
    const bool empty = groups == 0 || M == 0 || N == 0;
    if (!empty && K > 0 && (!A || !SA || !B || !SB)) return MMAC_ERR_INVALID_ARG;
    const int per = b_type == MMAC_FP4_E2M1 ? 2 : 1;   // elements a byte
    const int64_t strips = (K + 127) / 128;
    if (K > 0) {   // else none of the four is read
        if (ldb < K || ldb < 1) return MMAC_ERR_INVALID_ARG;
        if (ldb % per || stride_b % per) return MMAC_ERR_MISALIGNED;
        st = check_matrix(A, lda, M, K, 1);
        if (st == MMAC_OK) st = check_matrix(B, ldb / per, groups * N, K / per, 1);
        if (st == MMAC_OK) st = check_stride(groups, N, K, ldb, stride_b, 16 * per);
        if (st == MMAC_OK) st = check_words(SA, ldsa, strips, M);
        if (st == MMAC_OK) st = check_words(SB, ldsb, strips, N);
        if (st == MMAC_OK) st = check_stride(groups, strips, N, ldsb, stride_sb, 1);
    }
    if (st == MMAC_OK) st = check_out(groups > 0 ? M : 0, N, alpha, beta, C, ldc, D, ldd, ep);
    if (st != MMAC_OK) return st;
    if (empty) return MMAC_OK;

    const int forced = forced_tile();
    GroupTile t = forced >= 0 ? (GroupTile)forced : mx_tile(groups, M, N, K);
    if (t == GROUP_32) t = GROUP_16;
    if (t == GROUP_256) t = kMxLargest;   // the 256 x 256 tile has no registers left for the scale words
    GemmParams p = make_params(M, N, K, alpha, A, lda, B, ldb / per, beta, C, ldc, D, ldd, ep);
    p.sa = SA;
    p.ldsa = ldsa;
    p.sb = SB;
    p.ldsb = ldsb;
    p.scale_rows = (int)strips;
    Groups g{};
    g.offsets = offsets;
    g.count = (int)groups;
    g.rows = (int)M;
    g.b_stride = groups > 1 ? stride_b / per : 0;
    g.sb_stride = groups > 1 ? stride_sb : 0;
    g.bias_stride = N;
    int64_t grid;
    if (!set_grid(p, groups, t, kMxLargest, grid)) return MMAC_ERR_UNSUPPORTED;
    return launched(launch_gemm_grouped_mx(a_type, b_type, t, p, g, grid, static_cast<hipStream_t>(stream)));
}

mmac_status_t mmac_gemm_grouped_wgrad(mmac_dtype_t y_type, int64_t groups, int64_t M, int64_t N, int64_t K,
                                      double alpha, const void *dY, int64_t ldy, const void *X, int64_t ldx,
                                      const int32_t *offsets, double beta, const void *C, int64_t ldc,
                                      int64_t stride_c, void *D, int64_t ldd, int64_t stride_d,
                                      const mmac_epilogue_t *ep_in, void *stream) {
    const mmac_epilogue_t ep = epilogue_of(ep_in);
    if (!is_16bit(y_type)) return MMAC_ERR_UNSUPPORTED;
    if (bad_dim(groups) || bad_dim(M) || bad_dim(N) || bad_dim(K)) return MMAC_ERR_INVALID_ARG;
    if (groups > kMaxGroups) return MMAC_ERR_UNSUPPORTED;
    const bool empty = groups == 0 || N == 0 || K == 0;
    if (!empty && (!offsets || (M > 0 && (!dY || !X)))) return MMAC_ERR_INVALID_ARG;
    mmac_status_t st = check_out(groups > 0 ? N : 0, K, alpha, beta, C, ldc, D, ldd, ep);
    if (st != MMAC_OK) return st;
    if (ep.act != MMAC_ACT_NONE || ep.bias) return MMAC_ERR_UNSUPPORTED;
    st = check_matrix(dY, ldy, M, N, 2);
    if (st == MMAC_OK) st = check_matrix(X, ldx, M, K, 2);
    if (st == MMAC_OK) st = check_stride(groups, N, K, ldd, stride_d, 1);
    if (st == MMAC_OK && beta != 0.0) st = check_stride(groups, N, K, ldc, stride_c, 1);
    if (st != MMAC_OK) return st;
    if (C == D && beta != 0.0 && groups > 1 && stride_c != stride_d) return MMAC_ERR_INVALID_ARG;
    if (!aligned(offsets, 4)) return MMAC_ERR_MISALIGNED;
    if (empty) return MMAC_OK;

    const auto per = [&](GroupTile t) { return ((N + group_rows(t) - 1) / group_rows(t)) * ((K + group_cols(t) - 1) / group_cols(t)); };
    const int forced = forced_tile();
    GroupTile t = forced >= 0 ? (GroupTile)forced : wgrad_tile(groups, M, N, K, groups * per(GROUP_256), ep.d_type == MMAC_OUT_ACC);
    if (t == GROUP_16 || t == GROUP_32) t = GROUP_64;
    // so many tiles that only larger ones can be launched
    while (t != GROUP_256 && !grid_fits(wgrad_blocks(per(t), groups), t)) t = t == GROUP_64 ? GROUP_128 : GROUP_256;
    if (!grid_fits(wgrad_blocks(per(t), groups), t)) return MMAC_ERR_UNSUPPORTED;
    if (M == 0) ldy = ldx = 8;   // nothing is read
    GemmParams p = make_params(N, K, 0, alpha, dY, ldy * 2, X, ldx * 2, beta, C, ldc, D, ldd, ep);
    p.tiles_m = (int)((N + group_rows(t) - 1) / group_rows(t));
    p.tiles_n = (int)((K + group_cols(t) - 1) / group_cols(t));
    const int es = out_size(ep.d_type);
    Groups g{};
    g.offsets = offsets;
    g.count = (int)groups;
    g.rows = (int)M;
    g.d_stride = groups > 1 ? stride_d * es : 0;
    g.c_stride = groups > 1 ? stride_c * es : 0;
    // every group's matrix has to allow 16-byte accesses
    p.vec_d = p.vec_d && g.d_stride % 16 == 0;
    p.vec_c = p.vec_c && g.c_stride % 16 == 0;
    g.span = (int)((((int64_t)1 << 31) - 1) / (std::max(ldy, ldx) * 2) / 64 * 64);   // at least 192: pitches are at most 8 MiB
    return launched(launch_gemm_grouped_wgrad(y_type, t, p, g, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
