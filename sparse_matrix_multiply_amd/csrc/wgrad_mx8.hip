// Weight gradient from an 8-bit input: D = alpha * dY^T * X + beta * C, dY M x N in 16
// bits, X M x K as 8-bit elements with a power-of-two scale per 32 along K.
//
// The sum runs over the rows m, so both operands are stored with the summed axis
// outermost, and X's scales change along it: they cannot be taken out of the sum
// and have to be applied to the elements.  An element has at most 8 significant
// bits and its scale is a power of two, so the product is exact in bf16 (in fp16
// within its range): X is brought to dY's type on its way from memory to LDS, and the
// sum itself runs on the 32 x 32 matrix instructions with fp32 accumulators.
//
// A workgroup owns a BN x 128 tile of D (BN rows: columns of dY) and walks a range of M
// in chunks of 64 rows.  dY's part of a chunk is copied straight into LDS; X's goes
// through registers, where its conversion costs one instruction per two
// elements.  Two LDS stages: while one chunk is multiplied the next is in flight.
// Fragments are read with the transposing LDS reads, as the summed axis is outermost.
//
// With few tiles M is cut into ranges; each writes its partial tile to the
// workspace, and the one that arrives last adds them in range order.
#include "gemm_tiled.h"
#include "lowbit.h"

namespace mmac {

template <int DT>
__device__ __forceinline__ f32x16 mma32(const i32x4 &a, const i32x4 &b, f32x16 c) {
    if constexpr (DT == DT_BF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// XOR of the 16-byte unit number in row r of an LDS tile with U units of 16-bit elements per row: the four rows
// that one transposing read meets lie in different quarters of the banks.
template <int U>
__device__ __forceinline__ constexpr uint32_t tr_swz(uint32_t r) { return (r % 4) * (U >= 16 ? 4 : U / 4); }

// Fragment of step s of the 32 columns n0 .. n0 + 31 of an LDS tile of MN-element rows (rows: the summed axis):
// lane half g holds rows 16 s + 8 g .. + 7 of its column.  Of a group of 16 lanes, lane l addresses
// row k0 + l / 4, columns n + 4 (l mod 4) .. + 3, and lane i receives rows k0 .. k0 + 3 of column n + i.
template <int MN>
__device__ __forceinline__ i32x4 tr_frag(const uint8_t *tile, int n0, int s, int lane) {
    constexpr int U = MN / 8;
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    const int h = lane >> 4, l = lane & 15;
    const int n = n0 + 16 * (h & 1) + 4 * (l & 3);
    i32x4 f;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const int k = 16 * s + 8 * (h >> 1) + 4 * c + (l >> 2);
        const uint8_t *at = tile + k * (MN * 2) + (((uint32_t)(n >> 3) ^ tr_swz<U>(k)) << 4) + (n & 7) * 2;
        const i32x2 w = __builtin_bit_cast(i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)at));
        f[2 * c] = w[0];
        f[2 * c + 1] = w[1];
    }
    return f;
}

// Sixteen elements of one block -> sixteen DT values (32 bytes), scaled.
template <int DT, int QT>
__device__ __forceinline__ void scaled16(const i32x4 &q, uint32_t e, i32x4 (&o)[2]) {
    const float scale = __builtin_bit_cast(float, e == 255 ? 0x7fc00000u : e == 0 ? 0x00400000u : e << 23);
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        int lo, hi;
        const int v = q[d];
        if constexpr (QT == DT_I8) {
            const float f0 = (float)(int8_t)v * scale, f1 = (float)(int8_t)(v >> 8) * scale,
                        f2 = (float)(int8_t)(v >> 16) * scale, f3 = (float)(v >> 24) * scale;
            if constexpr (DT == DT_BF16) {
                lo = __builtin_bit_cast(int, bf16x2{(__bf16)f0, (__bf16)f1});
                hi = __builtin_bit_cast(int, bf16x2{(__bf16)f2, (__bf16)f3});
            } else {
                lo = __builtin_bit_cast(int, f16x2{(_Float16)f0, (_Float16)f1});
                hi = __builtin_bit_cast(int, f16x2{(_Float16)f2, (_Float16)f3});
            }
        } else {
            // two elements per conversion: fp32 pair, scaled, then rounded to DT
            const auto a = QT == DT_E4M3 ? __builtin_amdgcn_cvt_pk_f32_fp8(v, false) : __builtin_amdgcn_cvt_pk_f32_bf8(v, false);
            const auto b = QT == DT_E4M3 ? __builtin_amdgcn_cvt_pk_f32_fp8(v, true) : __builtin_amdgcn_cvt_pk_f32_bf8(v, true);
            const float f0 = a[0] * scale, f1 = a[1] * scale, f2 = b[0] * scale, f3 = b[1] * scale;
            if constexpr (DT == DT_BF16) {
                lo = __builtin_bit_cast(int, bf16x2{(__bf16)f0, (__bf16)f1});
                hi = __builtin_bit_cast(int, bf16x2{(__bf16)f2, (__bf16)f3});
            } else {
                lo = __builtin_bit_cast(int, f16x2{(_Float16)f0, (_Float16)f1});
                hi = __builtin_bit_cast(int, f16x2{(_Float16)f2, (_Float16)f3});
            }
        }
        o[d >> 1][2 * (d & 1)] = lo;
        o[d >> 1][2 * (d & 1) + 1] = hi;
    }
}

template <int DT, int QT, int BN, int WN, int WK>
__global__ __launch_bounds__(256) void gemm_mx8_wgrad_kernel(WgradParams p) {
    constexpr int BK = kWgradCols, MC = kWgradChunk, NT = 256;
    static_assert(WN * WK * 64 == NT, "four waves");
    constexpr int TN = BN / WN / 32, TK = BK / WK / 32;
    constexpr int UY = BN / 8, UX = BK / 8;                 // 16-byte units per LDS row
    constexpr int YP = MC * UY / NT;                        // copy instructions of dY per chunk
    constexpr int Y_BYTES = MC * BN * 2, X_BYTES = MC * BK * 2, STAGE = Y_BYTES + X_BYTES;
    constexpr int XU = MC * BK / 16 / NT;                   // 16-element units of X per thread
    __shared__ __attribute__((aligned(16))) uint8_t smem[2 * STAGE];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave / WK, wk = wave % WK;
    // ranges of one tile are consecutive workgroups
    const int split = blockIdx.x % p.split.splits, tile = blockIdx.x / p.split.splits;
    const int n0 = tile % p.tiles_n * BN, k0 = tile / p.tiles_n * BK;
    const int chunks = (p.M + MC - 1) / MC;
    const int c0 = split * p.split.per_split, c1 = min(c0 + p.split.per_split, chunks);
    const int y_row = (p.N * 2 + 15) / 16 * 16, kp = (p.K + 31) / 32 * 32;

    f32x16 acc[TN][TK];
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TK; ++j) acc[i][j] = f32x16{};

    const auto copy_y = [&](int c, uint8_t *st) {
        const int64_t m0 = (int64_t)c * MC;
        const int rows = (int)min((int64_t)MC, p.M - m0);
        const rsrc_t r = make_rsrc(p.Y + m0 * p.y_pitch + n0 * 2, (uint32_t)((rows - 1) * p.y_pitch + y_row - n0 * 2));
#pragma unroll
        for (int j = 0; j < YP; ++j) {
            const uint32_t P = j * NT + wave * 64 + lane, row = P / UY, u = (P % UY) ^ tr_swz<UY>(row);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)(st + (j * NT + wave * 64) * 16), 16,
                                                     (uint32_t)(row * p.y_pitch) + u * 16, 0, 0, 0);
        }
    };
    i32x4 xq[XU];
    uint32_t xe[XU];
    const auto load_x = [&](int c) {
        const int64_t m0 = (int64_t)c * MC;
        const int rows = (int)min((int64_t)MC, p.M - m0);
        const rsrc_t r = make_rsrc(p.Xq + m0 * p.q_pitch + k0, (uint32_t)((rows - 1) * p.q_pitch + kp - k0));
        const rsrc_t rs = make_rsrc(p.SX + (k0 / 128) * p.lds + m0, (uint32_t)(rows * 4));
#pragma unroll
        for (int j = 0; j < XU; ++j) {
            const uint32_t P = j * NT + tid, row = P / (BK / 16), u = P % (BK / 16);
            xq[j] = __builtin_amdgcn_raw_buffer_load_b128(r, (uint32_t)(row * p.q_pitch) + u * 16, 0, 0);
            xe[j] = __builtin_amdgcn_raw_buffer_load_b32(rs, row * 4, 0, 0) >> (8 * (u / 2));
        }
    };
    const auto put_x = [&](uint8_t *st) {
#pragma unroll
        for (int j = 0; j < XU; ++j) {
            const uint32_t P = j * NT + tid, row = P / (BK / 16), u = P % (BK / 16);
            i32x4 o[2];
            scaled16<DT, QT>(xq[j], xe[j] & 255u, o);
#pragma unroll
            for (int h = 0; h < 2; ++h)
                *reinterpret_cast<i32x4 *>(st + Y_BYTES + row * (BK * 2) + (((2 * u + h) ^ tr_swz<UX>(row)) << 4)) = o[h];
        }
    };

    if (c0 < c1) {
        copy_y(c0, smem);
        load_x(c0);
    }
    for (int c = c0; c < c1; ++c) {
        uint8_t *st = smem + ((c - c0) & 1) * STAGE;
        put_x(st);             // its last readers passed the barrier before this one
        wait_vm_lgkm0<0>();
        block_barrier();
        if (c + 1 < c1) {
            copy_y(c + 1, smem + ((c + 1 - c0) & 1) * STAGE);
            load_x(c + 1);
        }
#pragma unroll
        for (int s = 0; s < MC / 16; ++s) {
            i32x4 a[TN], b[TK];
#pragma unroll
            for (int i = 0; i < TN; ++i) a[i] = tr_frag<BN>(st, (wn * TN + i) * 32, s, lane);
#pragma unroll
            for (int j = 0; j < TK; ++j) b[j] = tr_frag<BK>(st + Y_BYTES, (wk * TK + j) * 32, s, lane);
#pragma unroll
            for (int i = 0; i < TN; ++i)
#pragma unroll
                for (int j = 0; j < TK; ++j) acc[i][j] = mma32<DT>(a[i], b[j], acc[i][j]);
        }
    }

    // ranges joined by the last to arrive, in range order (the partials at device scope, see the tiled GEMM)
    if (p.split.splits > 1) {
        constexpr int TILE_BYTES = BN * BK * 4;
        uint8_t *ws = p.split.partials + (int64_t)tile * p.split.splits * TILE_BYTES;
        const rsrc_t mine = make_rsrc(ws + (int64_t)split * TILE_BYTES, TILE_BYTES);
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int j = 0; j < TK; ++j)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const float e0 = acc[i][j][4 * g], e1 = acc[i][j][4 * g + 1], e2 = acc[i][j][4 * g + 2], e3 = acc[i][j][4 * g + 3];
                    const i32x4 v = {__builtin_bit_cast(int, e0), __builtin_bit_cast(int, e1), __builtin_bit_cast(int, e2),
                                     __builtin_bit_cast(int, e3)};
                    __builtin_amdgcn_raw_buffer_store_b128(v, mine, (uint32_t)((((i * TK + j) * 4 + g) * NT + tid) * 16), 0, kDeviceScope);
                }
        __builtin_amdgcn_s_waitcnt(0x0f70);   // vmcnt(0): the partial has reached device scope
        __syncthreads();
        uint32_t *arrived = reinterpret_cast<uint32_t *>(smem);
        if (tid == 0) {
            const uint32_t before = __hip_atomic_fetch_add(p.split.counters + tile, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            if (before == (uint32_t)p.split.splits - 1)
                __hip_atomic_store(p.split.counters + tile, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            *arrived = before;
        }
        __syncthreads();
        if (*arrived != (uint32_t)p.split.splits - 1) return;
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int j = 0; j < TK; ++j) {
                f32x16 sum = {};
                for (int r = 0; r < p.split.splits; ++r) {
                    const rsrc_t part = make_rsrc(ws + (int64_t)r * TILE_BYTES, TILE_BYTES);
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const i32x4 v = __builtin_amdgcn_raw_buffer_load_b128(
                            part, (uint32_t)((((i * TK + j) * 4 + g) * NT + tid) * 16), 0, kDeviceScope);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int w = v[e];
                            sum[4 * g + e] += __builtin_bit_cast(float, w);
                        }
                    }
                }
                acc[i][j] = sum;
            }
    }
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TK; ++j) {
            const int n = n0 + (wn * TN + i) * 32, k = k0 + (wk * TK + j) * 32 + (lane & 31);
            store_tile(p.out, n, p.N - n, k, k < p.K, acc[i][j]);
        }
}

template <int DT, int QT>
static hipError_t launch_as(const WgradParams &p, hipStream_t s) {
    const dim3 grid((unsigned)(p.tiles_n * p.tiles_k * p.split.splits)), block(256);
    switch (wgrad_rows(p.N)) {
    case 32: hipLaunchKernelGGL((gemm_mx8_wgrad_kernel<DT, QT, 32, 1, 4>), grid, block, 0, s, p); break;
    case 64: hipLaunchKernelGGL((gemm_mx8_wgrad_kernel<DT, QT, 64, 1, 4>), grid, block, 0, s, p); break;
    default: hipLaunchKernelGGL((gemm_mx8_wgrad_kernel<DT, QT, 128, 2, 2>), grid, block, 0, s, p); break;
    }
    return hipGetLastError();
}
template <int DT>
static hipError_t by_element(int q, const WgradParams &p, hipStream_t s) {
    switch (q) {
    case DT_E4M3: return launch_as<DT, DT_E4M3>(p, s);
    case DT_E5M2: return launch_as<DT, DT_E5M2>(p, s);
    case DT_I8: return launch_as<DT, DT_I8>(p, s);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_gemm_mx8_wgrad(int y, int q, const WgradParams &p, hipStream_t s) {
    if (y == DT_BF16) return by_element<DT_BF16>(q, p, s);
    if (y == DT_F16) return by_element<DT_F16>(q, p, s);
    return hipErrorInvalidValue;
}

}  // namespace mmac
