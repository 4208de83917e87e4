// RMS norm, forward: h = x + residual, y = h * rstd * w with rstd = (mean(h^2) + eps)^(-1/2), in one pass over memory.
//
// A row of N elements is held in registers by T threads with V groups of eight elements each (T = 64: one wave per
// row, four rows a workgroup; 256 to 1024: a workgroup per row), so x and the residual are read once, h and y
// written once.  Rows longer than 32768 are walked twice, the second time from the caches.
// Sums, rstd and the products of y are fp32; y itself is rounded once, to its output type.
//
// HBM bounds it, but for rows of up to 256, which leave lanes of their wave without elements (2^20 x 128 331 us, 3.2 TB/s; 2^18 x 256
// 111, 4.8): 8192^2 bf16 with a residual to E4M3 moves 472 MB in 91 us (5.2 TB/s; a large copy reaches 5.0).  256 threads with four
// groups and the weight read again for every row took 112 us, before the weight stayed in registers and 16-bit values were
// converted in pairs.  One row of 4096 takes 2.8 us, all of it latency: the weight is loaded with the row (5.4 us when
// it was loaded after the sum).  Consecutive rows run on one XCD, so their scale words, 4 bytes a row in each line, meet
// in its L2: the bytes written are the outputs' own (203 MB).
#include <algorithm>

#include "mx_block.h"
#include "norm.h"
#include "rows.h"

namespace mmac {

// y's eight elements of columns e0 .. e0 + 7 from h's, into the row of Y: OT 0 for X's type, or the 8-bit type.
template <int XT, int OT>
struct NormOut {
    const NormParams &p;
    int64_t row;
    RowOf<XT> y;
    uint8_t *q;
    int kp, strips;
    __device__ __forceinline__ NormOut(const NormParams &p_, int64_t row_)
        : p(p_), row(row_), y(p_.Y, row_, OT ? 0 : p_.y_pitch, OT ? 0 : p_.N), q(p_.Y + row_ * p_.y_pitch),
          kp((p_.N + 31) / 32 * 32), strips((p_.N + 127) / 128) {}
    __device__ __forceinline__ void put(const float (&h)[8], const float (&w)[8], float rstd, int e0) const {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = h[i] * rstd * w[i];
        if constexpr (OT == 0) {
            const Raw8<XT> r = pack8<XT>(v);
            y.template store<0>(r, e0);
            if (p.N & 7)
                if (e0 == (p.N & ~7)) y.store_short(r, e0, p.N & 7);
        } else {
            if (p.N & 31) {   // a row may end inside the block: nothing behind it counts, whatever rstd is
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = e0 + i < p.N ? v[i] : 0.0f;
            }
            float s[8];
            bool odd;
            const int e = scale_block<OT>(v, s, odd), l16 = threadIdx.x & 15;
            const u32x2 b = to_elements<OT>(s, odd);
            if (e0 < kp) *reinterpret_cast<u32x2 *>(q + e0) = b;
            const uint32_t word = scale_word_of(e, l16);
            if (l16 == 0 && (e0 >> 7) < strips) p.SY[(int64_t)(e0 >> 7) * p.lds + row] = word;
        }
    }
};

template <int WT>
__device__ __forceinline__ Raw8<WT> load_weight(const void *at, int e0, int N) {
    const RowOf<WT> r(at, 0, 0, N);
    Raw8<WT> x = load_raw8<WT, 0>(r.whole, e0);
    if (N & 7)
        if (e0 == (N & ~7)) r.load_short(x, e0, N & 7);
    return x;
}

// h's eight elements at e0 from x's and the residual's, as they are kept: rounded to X's type.
template <int XT>
__device__ __forceinline__ void add_residual(float (&h)[8], const Raw8<XT> &x, const Raw8<XT> &r) {
    float sum[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] = element<XT>(x, i) + element<XT>(r, i);
    elements<XT>(pack8<XT>(sum), h);
}

template <int XT, int WT, int OT, int T, int V>
__global__ __launch_bounds__(T < 256 ? 256 : T) void rmsnorm_kernel(NormParams p, int64_t units) {
    constexpr int ROWS = T < 256 ? 256 / T : 1;
    __shared__ float red[2][T / 64];
    const int t = threadIdx.x % T, sub = __builtin_amdgcn_readfirstlane(threadIdx.x / T);
    const int N = p.N;
    const XcdPart part(units);
    // the weight too stays in registers, from before the first row on, where they suffice
    constexpr bool KEEP = V <= 2;
    Raw8<WT> wr[V];
    if constexpr (KEEP) {
#pragma unroll
        for (int v = 0; v < V; ++v) wr[v] = load_weight<WT>(p.w, (v * T + t) * 8, N);
    }
    int turn = 0;
    for (int64_t u = blockIdx.x >> 3; u < part.count; u += gridDim.x >> 3) {
        const int64_t row = (part.first + u) * ROWS + sub;
        if (ROWS > 1 && row >= p.M) return;   // waves of their own
        const RowOf<XT> x(p.X, row, p.x_pitch, N), r(p.R ? p.R : p.X, row, p.R ? p.r_pitch : p.x_pitch, N);
        Raw8<XT> xr[V], rr[V];
#pragma unroll
        for (int v = 0; v < V; ++v) xr[v] = load_raw8<XT, 0>(x.whole, (v * T + t) * 8);
        if (p.R) {
#pragma unroll
            for (int v = 0; v < V; ++v) rr[v] = load_raw8<XT, 0>(r.whole, (v * T + t) * 8);
        }
        if (N & 7) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if ((v * T + t) * 8 == (N & ~7)) {
                    x.load_short(xr[v], N & ~7, N & 7);
                    if (p.R) r.load_short(rr[v], N & ~7, N & 7);
                }
        }
        float h[V][8], sum = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (p.R) add_residual<XT>(h[v], xr[v], rr[v]);
            else elements<XT>(xr[v], h[v]);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fmaf(h[v][i], h[v][i], sum);
        }
        if (p.H) {
            const RowOf<XT> hr(p.H, row, p.h_pitch, N);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int e0 = (v * T + t) * 8;
                const Raw8<XT> o = pack8<XT>(h[v]);
                hr.template store<0>(o, e0);
                if (N & 7)
                    if (e0 == (N & ~7)) hr.store_short(o, e0, N & 7);
            }
        }
        sum = row_sum<T>(sum, red[turn]);
        turn ^= 1;   // the other words next time: this row's may still be read
        const float rstd = 1.0f / sqrtf(sum / (float)N + p.eps);
        if (p.rstd && t == 0) p.rstd[row] = rstd;
        const NormOut<XT, OT> out(p, row);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float w[8];
            if constexpr (KEEP) elements<WT>(wr[v], w);
            else elements<WT>(load_weight<WT>(p.w, (v * T + t) * 8, N), w);
            out.put(h[v], w, rstd, (v * T + t) * 8);
        }
    }
}

// Rows of any length, 8192 columns at a time: h is formed twice (or read back where it is kept, since it may
// have taken the place of x or the residual).
template <int XT, int WT, int OT>
__global__ __launch_bounds__(1024) void rmsnorm_long_kernel(NormParams p, int64_t units) {
    constexpr int T = 1024;
    __shared__ float red[2][T / 64];
    const int t = threadIdx.x, N = p.N;
    const XcdPart part(units);
    int turn = 0;
    for (int64_t u = blockIdx.x >> 3; u < part.count; u += gridDim.x >> 3) {
        const int64_t row = part.first + u;
        const RowOf<XT> x(p.X, row, p.x_pitch, N), r(p.R ? p.R : p.X, row, p.R ? p.r_pitch : p.x_pitch, N);
        const RowOf<XT> hr(p.H ? p.H : p.Y, row, p.H ? p.h_pitch : 0, p.H ? N : 0);
        const auto form = [&](float(&h)[8], int e0) {
            Raw8<XT> a = load_raw8<XT, 0>(x.whole, e0), b = load_raw8<XT, 0>(r.whole, e0);
            if (N & 7)
                if (e0 == (N & ~7)) {
                    x.load_short(a, e0, N & 7);
                    r.load_short(b, e0, N & 7);
                }
            if (p.R) add_residual<XT>(h, a, b);
            else elements<XT>(a, h);
        };
        float sum = 0.0f;
        for (int e0 = t * 8; e0 < N; e0 += T * 8) {
            float h[8];
            form(h, e0);
            if (p.H) {
                const Raw8<XT> o = pack8<XT>(h);
                hr.template store<0>(o, e0);
                if (N & 7)
                    if (e0 == (N & ~7)) hr.store_short(o, e0, N & 7);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fmaf(h[i], h[i], sum);
        }
        sum = row_sum<T>(sum, red[turn]);
        turn ^= 1;
        const float rstd = 1.0f / sqrtf(sum / (float)N + p.eps);
        if (p.rstd && t == 0) p.rstd[row] = rstd;
        const NormOut<XT, OT> out(p, row);
        // every lane of the sixteen that share a scale word comes along
        for (int e0 = t * 8; e0 < (N + 127) / 128 * 128; e0 += T * 8) {
            float h[8], w[8];
            if (p.H) {   // what this thread has stored
                Raw8<XT> a = load_raw8<XT, 0>(hr.whole, e0);
                if (N & 7)
                    if (e0 == (N & ~7)) hr.load_short(a, e0, N & 7);
                elements<XT>(a, h);
            } else {
                form(h, e0);
            }
            elements<WT>(load_weight<WT>(p.w, e0, N), w);
            out.put(h, w, rstd, e0);
        }
    }
}

template <int XT, int WT, int OT>
static hipError_t launch_as(const NormParams &p, hipStream_t s) {
    // workgroups that fit the 256 compute units at a time, several rounds of them
    const auto grid = [](int64_t units) { return dim3((unsigned)std::min<int64_t>((units + 7) / 8 * 8, 8192)); };
    const int64_t four = (p.M + 3) / 4;
    if (p.N <= 512) hipLaunchKernelGGL((rmsnorm_kernel<XT, WT, OT, 64, 1>), grid(four), dim3(256), 0, s, p, four);
    else if (p.N <= 1024) hipLaunchKernelGGL((rmsnorm_kernel<XT, WT, OT, 64, 2>), grid(four), dim3(256), 0, s, p, four);
    else if (p.N <= 2048) hipLaunchKernelGGL((rmsnorm_kernel<XT, WT, OT, 256, 1>), grid(p.M), dim3(256), 0, s, p, p.M);
    else if (p.N <= 4096) hipLaunchKernelGGL((rmsnorm_kernel<XT, WT, OT, 256, 2>), grid(p.M), dim3(256), 0, s, p, p.M);
    else if (p.N <= 8192) hipLaunchKernelGGL((rmsnorm_kernel<XT, WT, OT, 512, 2>), grid(p.M), dim3(512), 0, s, p, p.M);
    else if (p.N <= 16384) hipLaunchKernelGGL((rmsnorm_kernel<XT, WT, OT, 1024, 2>), grid(p.M), dim3(1024), 0, s, p, p.M);
    else if (p.N <= 32768) hipLaunchKernelGGL((rmsnorm_kernel<XT, WT, OT, 1024, 4>), grid(p.M), dim3(1024), 0, s, p, p.M);
    else hipLaunchKernelGGL((rmsnorm_long_kernel<XT, WT, OT>), grid(p.M), dim3(1024), 0, s, p, p.M);
    return hipGetLastError();
}
template <int XT, int WT>
static hipError_t by_output(int y, const NormParams &p, hipStream_t s) {
    switch (y) {
    case XT: return launch_as<XT, WT, 0>(p, s);
    case DT_E4M3: return launch_as<XT, WT, DT_E4M3>(p, s);
    case DT_E5M2: return launch_as<XT, WT, DT_E5M2>(p, s);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_rmsnorm(int x, int w, int y, const NormParams &p, hipStream_t s) {
    if (w != x && w != DT_F32) return hipErrorInvalidValue;
    switch (x) {
    case DT_F16: return w == DT_F32 ? by_output<DT_F16, DT_F32>(y, p, s) : by_output<DT_F16, DT_F16>(y, p, s);
    case DT_BF16: return w == DT_F32 ? by_output<DT_BF16, DT_F32>(y, p, s) : by_output<DT_BF16, DT_BF16>(y, p, s);
    case DT_F32: return by_output<DT_F32, DT_F32>(y, p, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace mmac
