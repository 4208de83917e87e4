// C ABI of the RMS norm: argument validation on the host, launch on the caller's stream.  The public contract is in
// include/mmac_norm.h.
#include "abi_check.h"
#include "mmac_norm.h"
#include "norm.h"

using namespace mmac;

namespace {

mmac_status_t check_types(int x_type, int w_type, int64_t M, int64_t N) {
    if (!is_input(x_type) || (w_type != x_type && w_type != MMAC_F32)) return MMAC_ERR_UNSUPPORTED;
    return bad_dim(M) || bad_dim(N) ? MMAC_ERR_INVALID_ARG : MMAC_OK;
}

// Floats of the partial sums of dW, behind the first KiB of a workspace that others may share.
int64_t grad_bytes(int64_t M, int64_t N) { return kSplitCounterBytes + norm_grad_parts(M, N) * N * 4; }

}  // namespace

extern "C" {

mmac_status_t mmac_rmsnorm(mmac_dtype_t x_type, mmac_dtype_t w_type, mmac_dtype_t y_type, int64_t M, int64_t N,
                           const void *X, int64_t ldx, const void *residual, int64_t ldr, const void *w, double eps,
                           void *H, int64_t ldh, void *Y, int64_t ldy, uint32_t *SY, int64_t lds, float *rstd,
                           void *stream) {
    const int es = elem_size(x_type);
    const bool low = y_type == MMAC_FP8_E4M3 || y_type == MMAC_BF8_E5M2;
    mmac_status_t st = check_types(x_type, w_type, M, N);
    if (st != MMAC_OK) return st;
    if (y_type != x_type && !low) return MMAC_ERR_UNSUPPORTED;
    if (!std::isfinite(eps) || eps < 0.0 || eps > (double)FLT_MAX) return MMAC_ERR_INVALID_ARG;
    if (M > 0 && N > 0 && (!X || !w || !Y || (low && !SY))) return MMAC_ERR_INVALID_ARG;
    st = check_matrix(X, ldx, M, N, es);
    if (st == MMAC_OK && residual) st = check_matrix(residual, ldr, M, N, es);
    if (st == MMAC_OK && H) st = check_matrix(H, ldh, M, N, es);
    if (st == MMAC_OK) st = check_matrix(Y, ldy, M, low ? (N + 31) / 32 * 32 : N, low ? 1 : es);
    if (st == MMAC_OK && low) st = check_words(SY, lds, (N + 127) / 128, M);
    if (st != MMAC_OK) return st;
    // outputs in an input's place
    if (H && ((H == X && ldh != ldx) || (H == residual && ldh != ldr) || H == Y)) return MMAC_ERR_INVALID_ARG;
    if (Y && ((Y == X && (low || ldy != ldx)) || Y == residual)) return MMAC_ERR_INVALID_ARG;
    if (!aligned(w, 16) || !aligned(rstd, 4)) return MMAC_ERR_MISALIGNED;
    if (M == 0 || N == 0) return MMAC_OK;
    NormParams p{};
    p.X = static_cast<const uint8_t *>(X);
    p.x_pitch = ldx * es;
    p.R = static_cast<const uint8_t *>(residual);
    p.r_pitch = residual ? ldr * es : 0;
    p.w = w;
    p.H = static_cast<uint8_t *>(H);
    p.h_pitch = H ? ldh * es : 0;
    p.Y = static_cast<uint8_t *>(Y);
    p.y_pitch = ldy * (low ? 1 : es);
    p.SY = SY;
    p.lds = lds;
    p.rstd = rstd;
    p.M = M;
    p.N = (int)N;
    p.eps = (float)eps;
    return launched(launch_rmsnorm(x_type, w_type, y_type, p, static_cast<hipStream_t>(stream)));
}

mmac_status_t mmac_rmsnorm_grad(mmac_dtype_t x_type, mmac_dtype_t w_type, int64_t M, int64_t N, const void *dY,
                                int64_t lddy, const void *H, int64_t ldh, const void *w, const float *rstd,
                                const void *dH, int64_t lddh, void *dX, int64_t lddx, float *dW, void *workspace,
                                int64_t workspace_bytes, void *stream) {
    const int es = elem_size(x_type);
    mmac_status_t st = check_types(x_type, w_type, M, N);
    if (st != MMAC_OK) return st;
    if (workspace_bytes < 0 || (M > 0 && N > 0 && (!dY || !H || !w || !rstd || !dX))) return MMAC_ERR_INVALID_ARG;
    st = check_matrix(dY, lddy, M, N, es);
    if (st == MMAC_OK) st = check_matrix(H, ldh, M, N, es);
    if (st == MMAC_OK && dH) st = check_matrix(dH, lddh, M, N, es);
    if (st == MMAC_OK) st = check_matrix(dX, lddx, M, N, es);
    if (st != MMAC_OK) return st;
    if (dX && ((dX == dY && lddx != lddy) || (dX == dH && lddx != lddh) || dX == H)) return MMAC_ERR_INVALID_ARG;
    if (!aligned(w, 16) || !aligned(rstd, 4) || !aligned(dW, 16) || !aligned(workspace, 16)) return MMAC_ERR_MISALIGNED;
    if (N == 0 || (M == 0 && !dW)) return MMAC_OK;
    if (dW && (!workspace || workspace_bytes < grad_bytes(M, N))) return MMAC_ERR_INVALID_ARG;
    NormGradParams p{};
    p.dY = static_cast<const uint8_t *>(dY);
    p.dy_pitch = lddy * es;
    p.H = static_cast<const uint8_t *>(H);
    p.h_pitch = ldh * es;
    p.w = w;
    p.rstd = rstd;
    p.dH = static_cast<const uint8_t *>(dH);
    p.dh_pitch = dH ? lddh * es : 0;
    p.dX = static_cast<uint8_t *>(dX);
    p.dx_pitch = lddx * es;
    p.dW = dW;
    p.partials = dW ? reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + kSplitCounterBytes) : nullptr;
    p.M = M;
    p.N = (int)N;
    return launched(launch_rmsnorm_grad(x_type, w_type, p, static_cast<hipStream_t>(stream)));
}

int64_t mmac_rmsnorm_grad_workspace_bytes(int64_t M, int64_t N) {
    if (bad_dim(M) || bad_dim(N) || N == 0) return 0;
    return grad_bytes(M, N);
}

}  // extern "C"
