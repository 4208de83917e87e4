// C ABI of the low-bit operands: argument validation on the host, kernel
// selection, launch on the caller's stream.  The public contract is in
// include/mmac_lowbit.h and include/mmac_mx4.h.
#include <algorithm>
#include <cstdint>

#include "abi_check.h"
#include "lowbit.h"
#include "mmac_lowbit.h"
#include "mmac_mx4.h"

using namespace mmac;

namespace {

int64_t groups_of(int64_t K, int group) { return group == 0 ? 1 : (K + group - 1) / group; }

mmac_status_t check_w4(const mmac_w4_t *q, int64_t N, int64_t K) {
    if (!q) return MMAC_ERR_INVALID_ARG;
    if (q->q_type != MMAC_U4 && q->q_type != MMAC_FP4_E2M1) return MMAC_ERR_UNSUPPORTED;
    if (q->group != 0 && q->group != 32 && q->group != 64 && q->group != 128) return MMAC_ERR_UNSUPPORTED;
    if (N > 0 && K > 0 && (!q->codes || !q->words)) return MMAC_ERR_INVALID_ARG;
    if (q->pitch < (K + 31) / 32 * 16) return MMAC_ERR_INVALID_ARG;
    if (q->pitch > kMaxPitchBytes) return MMAC_ERR_UNSUPPORTED;
    if (!aligned(q->codes, 16) || q->pitch % 16) return MMAC_ERR_MISALIGNED;
    return check_words(q->words, q->ldw, groups_of(K, q->group), N);
}

OutParams out_params(double alpha, double beta, const void *C, int64_t ldc, void *D, int64_t ldd,
                     const mmac_epilogue_t &ep) {
    OutParams o{};
    o.alpha = (float)alpha;
    o.beta = (float)beta;
    o.use_c = o.beta != 0.0f;
    o.C = o.use_c ? C : nullptr;
    o.ldc = o.use_c ? ldc : 0;
    o.D = D;
    o.ldd = ldd;
    o.d_type = ep.d_type;
    o.act = ep.act;
    o.bias = ep.bias;
    return o;
}

// `chunks` chunks of the summed axis cut into at most `want` ranges, none empty.  The partial tiles lie behind the
// workspace's first KiB, whose 256 counters are enough for every plan below.
struct SplitPlan {
    int splits, per_split;
    int64_t bytes;
};
SplitPlan plan(int64_t tiles, int64_t tile_bytes, int64_t chunks, int64_t want) {
    want = tiles * 4 > kSplitCounterBytes ? 1 : std::max<int64_t>(1, std::min(want, chunks));
    SplitPlan s{};
    s.per_split = (int)std::max<int64_t>(1, (chunks + want - 1) / want);
    s.splits = (int)std::max<int64_t>(1, (chunks + s.per_split - 1) / s.per_split);
    if (s.splits > 1) s.bytes = kSplitCounterBytes + tiles * s.splits * tile_bytes;
    return s;
}
SplitParams apply(const SplitPlan &s, int64_t chunks, void *ws, int64_t ws_bytes) {
    if (s.splits < 2 || !ws || ws_bytes < s.bytes) return SplitParams{1, (int)chunks, nullptr, nullptr};
    return SplitParams{s.splits, s.per_split, static_cast<uint32_t *>(ws), static_cast<uint8_t *>(ws) + kSplitCounterBytes};
}

// 4-bit products of more than 32 rows: the largest tile that still gives a workgroup to most of the 256 compute
// units; then, if tiles of 128 columns leave units idle, up to 8 K ranges of at least two chunks.  Measured with U4,
// groups of 128, N = K = 8192: 64 rows 28 us in 64 x 128 tiles and 4 ranges (60 us in 64 x 256 tiles and 8), 512 rows
// 103 us in 128 x 128 tiles (111 in 128 x 256 and 2 ranges), 2048 rows 312 us in 128 x 256 tiles.
W4Tile w4_tile(int64_t M, int64_t N) {
    const auto tiles = [&](W4Tile t) { return ((M + w4_rows(t) - 1) / w4_rows(t)) * ((N + w4_cols(t) - 1) / w4_cols(t)); };
    if (M <= 64) return W4_64x128;
    return tiles(W4_128x256) >= 192 ? W4_128x256 : W4_128x128;
}
SplitPlan plan_w4(int64_t M, int64_t N, int64_t K) {
    if (M <= 32 || N == 0 || K == 0) return SplitPlan{1, 1, 0};
    const W4Tile t = w4_tile(M, N);
    const int64_t tiles = ((M + w4_rows(t) - 1) / w4_rows(t)) * ((N + w4_cols(t) - 1) / w4_cols(t));
    const int64_t chunks = (K + kW4Chunk - 1) / kW4Chunk;
    return plan(tiles, w4_rows(t) * w4_cols(t) * 4, chunks, std::min<int64_t>({8, 256 / tiles, chunks / 2}));
}

// Weight gradient: 256 x 256 tiles where they occupy most compute units, else narrower ones (two or more workgroups
// fit a unit) with M cut into at most 8 ranges of at least four chunks until there are two workgroups per unit.
// Measured with 256, 512 and 1024 workgroups in all (M 8192, bf16 x E4M3): N 32, K 8192 32, 26 and 31 us; N 256, K 4096
// 53, 47 and 68 us; and N 64, K 4096 with 8 ranges 26 us, with 16 30 us: more ranges write and read more partial sums.
WgradTile wgrad_tile(int64_t N, int64_t K) {
    if (N <= 32) return WGRAD_32x128;
    if (N <= 64) return WGRAD_64x128;
    return ((N + 255) / 256) * ((K + 255) / 256) >= 192 ? WGRAD_256x256 : WGRAD_128x128;
}
SplitPlan plan_wgrad(int64_t M, int64_t N, int64_t K) {
    if (M == 0 || N == 0 || K == 0) return SplitPlan{1, 1, 0};
    const WgradTile t = wgrad_tile(N, K);
    if (t == WGRAD_256x256) return SplitPlan{1, 1, 0};
    const int64_t tiles = ((N + wgrad_rows(t) - 1) / wgrad_rows(t)) * ((K + wgrad_cols(t) - 1) / wgrad_cols(t));
    const int64_t chunks = (M + kWgradChunk - 1) / kWgradChunk;
    return plan(tiles, wgrad_rows(t) * wgrad_cols(t) * 4, chunks, std::min<int64_t>({8, 512 / tiles, chunks / 4}));
}

}  // namespace

extern "C" {

mmac_status_t mmac_w4_quantize(mmac_dtype_t w_type, int symmetric, int64_t N, int64_t K, const void *W, int64_t ldw_in,
                               const mmac_w4_t *q, void *stream) {
    if (!is_input(w_type)) return MMAC_ERR_UNSUPPORTED;
    if (bad_dim(N) || bad_dim(K) || (symmetric != 0 && symmetric != 1)) return MMAC_ERR_INVALID_ARG;
    if (N > 0 && K > 0 && !W) return MMAC_ERR_INVALID_ARG;
    mmac_status_t st = check_w4(q, N, K);
    if (st != MMAC_OK) return st;
    if (q->q_type == MMAC_FP4_E2M1 && !symmetric) return MMAC_ERR_UNSUPPORTED;
    st = check_rows(W, ldw_in, K, elem_size(w_type));
    if (st != MMAC_OK) return st;
    if (N == 0 || K == 0) return MMAC_OK;
    W4QuantParams p{};
    p.W = static_cast<const uint8_t *>(W);
    p.w_pitch = ldw_in * elem_size(w_type);
    p.codes = static_cast<uint8_t *>(q->codes);
    p.pitch = q->pitch;
    p.words = q->words;
    p.ldw = q->ldw;
    p.N = (int)N;
    p.K = (int)K;
    return launched(launch_w4_quantize(w_type, q->q_type, symmetric != 0, q->group, p, static_cast<hipStream_t>(stream)));
}

mmac_status_t mmac_gemm_w4(mmac_dtype_t a_type, int64_t M, int64_t N, int64_t K, double alpha, const void *A,
                           int64_t lda, const mmac_w4_t *W, double beta, const void *C, int64_t ldc, void *D,
                           int64_t ldd, const mmac_epilogue_t *ep_in, void *workspace, int64_t workspace_bytes,
                           void *stream) {
    const mmac_epilogue_t ep = epilogue_of(ep_in);
    if (!is_16bit(a_type)) return MMAC_ERR_UNSUPPORTED;
    if (bad_dim(M) || bad_dim(N) || bad_dim(K) || (M > 0 && N > 0 && K > 0 && !A)) return MMAC_ERR_INVALID_ARG;
    mmac_status_t st = check_w4(W, N, K);
    if (st != MMAC_OK) return st;
    st = check_rows(A, lda, K, 2);
    if (st != MMAC_OK) return st;
    st = check_out(M, N, alpha, beta, C, ldc, D, ldd, ep);
    if (st != MMAC_OK) return st;
    if (workspace_bytes < 0) return MMAC_ERR_INVALID_ARG;
    if (workspace && !aligned(workspace, 16)) return MMAC_ERR_MISALIGNED;
    if (M == 0 || N == 0) return MMAC_OK;
    W4Params p{};
    p.A = static_cast<const uint8_t *>(A);
    p.a_pitch = lda * 2;
    p.codes = static_cast<const uint8_t *>(W->codes);
    p.pitch = W->pitch;
    p.words = W->words;
    p.ldw = W->ldw;
    p.groups = (int)groups_of(K, W->group);
    p.group = W->group;
    p.M = (int)M;
    p.N = (int)N;
    p.K = (int)K;
    p.out = out_params(alpha, beta, C, ldc, D, ldd, ep);
    if (M <= 32) return launched(launch_gemm_w4_rows(a_type, W->q_type, p, static_cast<hipStream_t>(stream)));
    p.tile = w4_tile(M, N);

    const int64_t tm = (M + w4_rows(p.tile) - 1) / w4_rows(p.tile), tn = (N + w4_cols(p.tile) - 1) / w4_cols(p.tile);
    if (tm * tn > INT32_MAX / 1024) return MMAC_ERR_UNSUPPORTED;   // the grid, up to 512 threads each
    p.tiles_m = (int)tm;
    p.tiles_n = (int)tn;
    p.split = apply(plan_w4(M, N, K), (K + kW4Chunk - 1) / kW4Chunk, workspace, workspace_bytes);
    return launched(launch_gemm_w4_tiled(a_type, W->q_type, p, static_cast<hipStream_t>(stream)));
}

int64_t mmac_gemm_w4_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (bad_dim(M) || bad_dim(N) || bad_dim(K)) return 0;
    return plan_w4(M, N, K).bytes;
}

static mmac_status_t check_mx8(int x_type, int q_type, int64_t M, int64_t K, const void *X, int64_t ldx, const void *Xq,
                               int64_t ldq, const uint32_t *SX, int64_t lds) {
    if (!is_input(x_type) || !is_mx8(q_type)) return MMAC_ERR_UNSUPPORTED;
    if (bad_dim(M) || bad_dim(K)) return MMAC_ERR_INVALID_ARG;
    if (M > 0 && K > 0 && (!X || !Xq || !SX)) return MMAC_ERR_INVALID_ARG;
    mmac_status_t st = check_rows(X, ldx, K, elem_size(x_type));
    if (st == MMAC_OK) st = check_rows(Xq, ldq, (K + 31) / 32 * 32, 1);
    if (st == MMAC_OK) st = check_words(SX, lds, (K + 127) / 128, M);
    return st;
}
static Mx8Params mx8_params(int x_type, int64_t M, int64_t K, const void *X, int64_t ldx, const void *Xq, int64_t ldq,
                            const uint32_t *SX, int64_t lds) {
    Mx8Params p{};
    p.X = static_cast<const uint8_t *>(X);
    p.x_pitch = ldx * elem_size(x_type);
    p.Xq = static_cast<const uint8_t *>(Xq);
    p.q_pitch = ldq;
    p.SX = SX;
    p.lds = lds;
    p.M = (int)M;
    p.K = (int)K;
    return p;
}

mmac_status_t mmac_mx8_quantize(mmac_dtype_t x_type, mmac_dtype_t q_type, int64_t M, int64_t K, const void *X,
                                int64_t ldx, void *Xq, int64_t ldq, uint32_t *SX, int64_t lds, void *stream) {
    const mmac_status_t st = check_mx8(x_type, q_type, M, K, X, ldx, Xq, ldq, SX, lds);
    if (st != MMAC_OK || M == 0 || K == 0) return st;
    return launched(launch_mx8_quantize(x_type, q_type, mx8_params(x_type, M, K, X, ldx, Xq, ldq, SX, lds),
                                        static_cast<hipStream_t>(stream)));
}

mmac_status_t mmac_mx8_dequantize(mmac_dtype_t q_type, mmac_dtype_t x_type, int64_t M, int64_t K, const void *Xq,
                                  int64_t ldq, const uint32_t *SX, int64_t lds, void *X, int64_t ldx, void *stream) {
    const mmac_status_t st = check_mx8(x_type, q_type, M, K, X, ldx, Xq, ldq, SX, lds);
    if (st != MMAC_OK || M == 0 || K == 0) return st;
    return launched(launch_mx8_dequantize(q_type, x_type, mx8_params(x_type, M, K, X, ldx, Xq, ldq, SX, lds),
                                          static_cast<hipStream_t>(stream)));
}

mmac_status_t mmac_mx4_quantize(mmac_dtype_t x_type, int64_t M, int64_t K, const void *X, int64_t ldx, void *Xq,
                                int64_t pitch, uint32_t *SX, int64_t lds, void *stream) {
    if (!is_input(x_type)) return MMAC_ERR_UNSUPPORTED;
    if (bad_dim(M) || bad_dim(K)) return MMAC_ERR_INVALID_ARG;
    if (M > 0 && K > 0 && (!X || !Xq || !SX)) return MMAC_ERR_INVALID_ARG;
    mmac_status_t st = check_matrix(X, ldx, M, K, elem_size(x_type));
    if (st == MMAC_OK) st = check_matrix(Xq, pitch, M, (K + 31) / 32 * 16, 1);
    if (st == MMAC_OK) st = check_words(SX, lds, (K + 127) / 128, M);
    if (st != MMAC_OK || M == 0 || K == 0) return st;
    return launched(launch_mx4_quantize(x_type, mx8_params(x_type, M, K, X, ldx, Xq, pitch, SX, lds),
                                        static_cast<hipStream_t>(stream)));
}

mmac_status_t mmac_gemm_mx8_wgrad(mmac_dtype_t y_type, mmac_dtype_t q_type, int64_t M, int64_t N, int64_t K,
                                  double alpha, const void *dY, int64_t ldy, const void *Xq, int64_t ldq,
                                  const uint32_t *SX, int64_t lds, double beta, const void *C, int64_t ldc, void *D,
                                  int64_t ldd, const mmac_epilogue_t *ep_in, void *workspace, int64_t workspace_bytes,
                                  void *stream) {
    const mmac_epilogue_t ep = epilogue_of(ep_in);
    if (!is_16bit(y_type) || !is_mx8(q_type)) return MMAC_ERR_UNSUPPORTED;
    if (bad_dim(M) || bad_dim(N) || bad_dim(K)) return MMAC_ERR_INVALID_ARG;
    if (M > 0 && K > 0 && N > 0 && (!dY || !Xq || !SX)) return MMAC_ERR_INVALID_ARG;
    mmac_status_t st = check_out(N, K, alpha, beta, C, ldc, D, ldd, ep);
    if (st != MMAC_OK) return st;
    if (ep.act != MMAC_ACT_NONE || ep.bias) return MMAC_ERR_UNSUPPORTED;
    st = check_rows(dY, ldy, N, 2);
    if (st == MMAC_OK) st = check_rows(Xq, ldq, (K + 31) / 32 * 32, 1);
    if (st == MMAC_OK) st = check_words(SX, lds, (K + 127) / 128, M);
    if (st != MMAC_OK) return st;
    if (workspace_bytes < 0) return MMAC_ERR_INVALID_ARG;
    if (workspace && !aligned(workspace, 16)) return MMAC_ERR_MISALIGNED;
    if (N == 0 || K == 0) return MMAC_OK;
    WgradParams p{};
    p.Y = static_cast<const uint8_t *>(dY);
    p.y_pitch = ldy * 2;
    p.Xq = static_cast<const uint8_t *>(Xq);
    p.q_pitch = ldq;
    p.SX = SX;
    p.lds = lds;
    p.M = (int)M;
    p.N = (int)N;
    p.K = (int)K;
    p.tile = wgrad_tile(N, K);
    const int64_t bn = wgrad_rows(p.tile), bk = wgrad_cols(p.tile), tn = (N + bn - 1) / bn, tk = (K + bk - 1) / bk;
    if (tn * tk > INT32_MAX / 1024) return MMAC_ERR_UNSUPPORTED;   // the grid, up to 512 threads each and 8 ranges
    p.tiles_n = (int)tn;
    p.tiles_k = (int)tk;
    p.out = out_params(alpha, beta, C, ldc, D, ldd, ep);
    p.split = apply(plan_wgrad(M, N, K), (M + kWgradChunk - 1) / kWgradChunk, workspace, workspace_bytes);
    return launched(launch_gemm_mx8_wgrad(y_type, q_type, p, static_cast<hipStream_t>(stream)));
}

int64_t mmac_gemm_mx8_wgrad_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (bad_dim(M) || bad_dim(N) || bad_dim(K)) return 0;
    return plan_wgrad(M, N, K).bytes;
}

}  // extern "C"
