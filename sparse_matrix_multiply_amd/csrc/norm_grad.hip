// RMS norm, backward.  With xhat = h * rstd and v = w * dy, each row's gradient is
//   dx = rstd * (v - xhat * mean(v * xhat)) + dh,
// and the weight's is the sum over the rows of dy * xhat.
//
// A row is held by T threads, as in the forward pass.  Every workgroup walks rows and adds up dy * xhat of its columns
// in registers (fp32); each leaves one row of partial sums behind, and a second kernel adds those up in their order,
// so the result does not depend on timing.
//
// HBM bounds it: 8192^2 bf16 with dh moves 537 MB, and 34 MB of partial sums, in 103 us (5.2 TB/s), 4 of them the second kernel.  T is large
// and V small (8 or 16 elements a thread) because a thread holds the weight and its sums besides the row; 512 workgroups are two per
// compute unit, so one reads while the other adds up.  Rows of more than 8192: 16 elements a thread fill the 128 registers that 1024
// threads leave (6 to 14 spilled, 86 for fp32), reloaded once a row: 4096 x 16384 121 us in bf16 (4.4 TB/s), 249 in fp32.  Past 16384
// the partial sums go through memory with every row, as many bytes again: 2048 x 32768 bf16 272 us, 108 without dW and dh.
// Rows of up to 256 leave most of a wave's lanes without elements: 2^20 x 128 489 us (2.2 TB/s), 2^18 x 256 143 (3.8).
#include <algorithm>

#include "norm.h"
#include "rows.h"

namespace mmac {

template <int WT>
__device__ __forceinline__ void load_weight8(float (&w)[8], const void *at, int e0, int N) {
    const RowOf<WT> r(at, 0, 0, N);
    Raw8<WT> x = load_raw8<WT, 0>(r.whole, e0);
    if (N & 7)
        if (e0 == (N & ~7)) r.load_short(x, e0, N & 7);
    elements<WT>(x, w);
}

// A row of partial sums, eight columns a thread.
__device__ __forceinline__ void store_sums(float *row, const float (&a)[8], int e0, int N) {
    const RowOf<DT_F32> r(row, 0, 0, N);
    const Raw8<DT_F32> x = pack8<DT_F32>(a);
    r.store<0>(x, e0);
    if (N & 7)
        if (e0 == (N & ~7)) r.store_short(x, e0, N & 7);
}

template <int XT, int WT, int T, int V>
__global__ __launch_bounds__(T < 256 ? 256 : T) void rmsnorm_grad_kernel(NormGradParams p) {
    constexpr int ROWS = T < 256 ? 256 / T : 1;
    __shared__ float red[2][T / 64];
    __shared__ float sums[ROWS > 1 ? ROWS - 1 : 1][V][ROWS > 1 ? T * 8 : 1];
    const int t = threadIdx.x % T, sub = __builtin_amdgcn_readfirstlane(threadIdx.x / T);
    const int N = p.N;
    const float inv = 1.0f / (float)N;
    float w[V][8], dw[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        load_weight8<WT>(w[v], p.w, (v * T + t) * 8, N);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[v][i] = 0.0f;
    }
    int turn = 0;
    for (int64_t row = (int64_t)blockIdx.x * ROWS + sub; row < p.M; row += (int64_t)gridDim.x * ROWS) {
        const RowOf<XT> y(p.dY, row, p.dy_pitch, N), h(p.H, row, p.h_pitch, N);
        const RowOf<XT> g(p.dH ? p.dH : p.dY, row, p.dH ? p.dh_pitch : p.dy_pitch, N), x(p.dX, row, p.dx_pitch, N);
        Raw8<XT> yr[V], hr[V], gr[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            yr[v] = load_raw8<XT, 0>(y.whole, (v * T + t) * 8);
            hr[v] = load_raw8<XT, 0>(h.whole, (v * T + t) * 8);
            if (p.dH) gr[v] = load_raw8<XT, 0>(g.whole, (v * T + t) * 8);
        }
        const float rstd = p.rstd[row];
        if (N & 7) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if ((v * T + t) * 8 == (N & ~7)) {
                    y.load_short(yr[v], N & ~7, N & 7);
                    h.load_short(hr[v], N & ~7, N & 7);
                    if (p.dH) g.load_short(gr[v], N & ~7, N & 7);
                }
        }
        float dot = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float xhat = element<XT>(hr[v], i) * rstd, dy = element<XT>(yr[v], i);
                dw[v][i] = fmaf(dy, xhat, dw[v][i]);
                dot = fmaf(dy * w[v][i], xhat, dot);
            }
        dot = row_sum<T>(dot, red[turn]) * inv;
        turn ^= 1;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e0 = (v * T + t) * 8;
            float d[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float xhat = element<XT>(hr[v], i) * rstd;
                d[i] = rstd * fmaf(-xhat, dot, element<XT>(yr[v], i) * w[v][i]);
                if (p.dH) d[i] += element<XT>(gr[v], i);
            }
            const Raw8<XT> o = pack8<XT>(d);
            x.template store<0>(o, e0);
            if (N & 7)
                if (e0 == (N & ~7)) x.store_short(o, e0, N & 7);
        }
    }
    if (!p.dW) return;
    if constexpr (ROWS > 1) {   // the workgroup's waves, in their order
        if (sub > 0) {
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int i = 0; i < 8; ++i) sums[sub - 1][v][i * T + t] = dw[v][i];
        }
        __syncthreads();
        if (sub > 0) return;
        for (int s = 0; s < ROWS - 1; ++s)
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int i = 0; i < 8; ++i) dw[v][i] += sums[s][v][i * T + t];
    }
#pragma unroll
    for (int v = 0; v < V; ++v) store_sums(p.partials + (int64_t)blockIdx.x * N, dw[v], (v * T + t) * 8, N);
}

// Rows of any length, 8192 columns at a time; the partial sums stay in memory between rows.
template <int XT, int WT>
__global__ __launch_bounds__(1024) void rmsnorm_grad_long_kernel(NormGradParams p) {
    constexpr int T = 1024;
    __shared__ float red[2][T / 64];
    const int t = threadIdx.x, N = p.N;
    const float inv = 1.0f / (float)N;
    int turn = 0;
    float *sums = p.dW ? p.partials + (int64_t)blockIdx.x * N : nullptr;
    for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
        const RowOf<XT> y(p.dY, row, p.dy_pitch, N), h(p.H, row, p.h_pitch, N);
        const RowOf<XT> g(p.dH ? p.dH : p.dY, row, p.dH ? p.dh_pitch : p.dy_pitch, N), x(p.dX, row, p.dx_pitch, N);
        const float rstd = p.rstd[row];
        const auto get = [&](const RowOf<XT> &r, float(&f)[8], int e0) {
            Raw8<XT> a = load_raw8<XT, 0>(r.whole, e0);
            if (N & 7)
                if (e0 == (N & ~7)) r.load_short(a, e0, N & 7);
            elements<XT>(a, f);
        };
        float dot = 0.0f;
        for (int e0 = t * 8; e0 < N; e0 += T * 8) {
            float dy[8], hh[8], w[8];
            get(y, dy, e0);
            get(h, hh, e0);
            load_weight8<WT>(w, p.w, e0, N);
#pragma unroll
            for (int i = 0; i < 8; ++i) dot = fmaf(dy[i] * w[i], hh[i] * rstd, dot);
        }
        dot = row_sum<T>(dot, red[turn]) * inv;
        turn ^= 1;
        for (int e0 = t * 8; e0 < N; e0 += T * 8) {
            float dy[8], hh[8], w[8], d[8], gg[8], a[8];
            get(y, dy, e0);
            get(h, hh, e0);
            load_weight8<WT>(w, p.w, e0, N);
            if (p.dH) get(g, gg, e0);
            const bool first = row == blockIdx.x;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float xhat = hh[i] * rstd;
                d[i] = rstd * fmaf(-xhat, dot, dy[i] * w[i]);
                if (p.dH) d[i] += gg[i];
                a[i] = 0.0f;
                if (sums && !first && e0 + i < N) a[i] = sums[e0 + i];   // this thread's own
                a[i] = fmaf(dy[i], xhat, a[i]);
            }
            const Raw8<XT> o = pack8<XT>(d);
            x.template store<0>(o, e0);
            if (N & 7)
                if (e0 == (N & ~7)) x.store_short(o, e0, N & 7);
            if (sums) store_sums(sums, a, e0, N);
        }
    }
}

// dW = the sum of `parts` rows of partial sums in their order: 64 columns a workgroup, whose 16 waves take
// consecutive parts of the rows.
__global__ __launch_bounds__(1024) void norm_weight_sum_kernel(const float *partials, float *dW, int N, int parts) {
    __shared__ float red[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t column = (int64_t)blockIdx.x * 64 + lane;
    const int per = (parts + 15) / 16, first = min(wave * per, parts), end = min(first + per, parts);
    float sum = 0.0f;
    if (column < N) {
        const float *at = partials + column;
#pragma unroll 8
        for (int i = first; i < end; ++i) sum += at[(int64_t)i * N];
    }
    red[wave][lane] = sum;
    __syncthreads();
    if (wave == 0 && column < N) {
        for (int w = 1; w < 16; ++w) sum += red[w][lane];
        dW[column] = sum;
    }
}

int norm_grad_parts(int64_t M, int64_t N) {
    const int64_t rows = N <= 1024 ? 4 : 1;
    return (int)std::max<int64_t>(1, std::min<int64_t>((M + rows - 1) / rows, 512));
}

template <int XT, int WT>
static hipError_t launch_as(const NormGradParams &p, hipStream_t s) {
    // without rows there are no partial sums, and nothing to read: only dW, which is zero, is written
    const int parts = p.M > 0 ? norm_grad_parts(p.M, p.N) : 0;
    const dim3 grid(parts);
    if (parts == 0) {}
    else if (p.N <= 512) hipLaunchKernelGGL((rmsnorm_grad_kernel<XT, WT, 64, 1>), grid, dim3(256), 0, s, p);
    else if (p.N <= 1024) hipLaunchKernelGGL((rmsnorm_grad_kernel<XT, WT, 64, 2>), grid, dim3(256), 0, s, p);
    else if (p.N <= 2048) hipLaunchKernelGGL((rmsnorm_grad_kernel<XT, WT, 256, 1>), grid, dim3(256), 0, s, p);
    else if (p.N <= 4096) hipLaunchKernelGGL((rmsnorm_grad_kernel<XT, WT, 512, 1>), grid, dim3(512), 0, s, p);
    else if (p.N <= 8192) hipLaunchKernelGGL((rmsnorm_grad_kernel<XT, WT, 1024, 1>), grid, dim3(1024), 0, s, p);
    else if (p.N <= 16384) hipLaunchKernelGGL((rmsnorm_grad_kernel<XT, WT, 1024, 2>), grid, dim3(1024), 0, s, p);
    else hipLaunchKernelGGL((rmsnorm_grad_long_kernel<XT, WT>), grid, dim3(1024), 0, s, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !p.dW) return e;
    hipLaunchKernelGGL(norm_weight_sum_kernel, dim3((p.N + 63) / 64), dim3(1024), 0, s, p.partials, p.dW, p.N, parts);
    return hipGetLastError();
}

hipError_t launch_rmsnorm_grad(int x, int w, const NormGradParams &p, hipStream_t s) {
    if (w != x && w != DT_F32) return hipErrorInvalidValue;
    switch (x) {
    case DT_F16: return w == DT_F32 ? launch_as<DT_F16, DT_F32>(p, s) : launch_as<DT_F16, DT_F16>(p, s);
    case DT_BF16: return w == DT_F32 ? launch_as<DT_BF16, DT_F32>(p, s) : launch_as<DT_BF16, DT_BF16>(p, s);
    case DT_F32: return launch_as<DT_F32, DT_F32>(p, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace mmac
