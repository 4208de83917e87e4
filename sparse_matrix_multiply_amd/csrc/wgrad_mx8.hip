// Weight gradient from an 8-bit input: D = alpha * dY^T * X + beta * C, dY M x N in 16
// bits, X M x K as 8-bit elements with a power-of-two scale per 32 along K.
//
// The sum runs over the rows m, so both operands are stored with the summed axis
// outermost, and X's scales change along it: they cannot be taken out of the sum
// and have to be applied to the elements.  An element has at most 8 significant
// bits and its scale is a power of two, so the product is exact in bf16 (in fp16
// within its range): X is brought to dY's type on its way from memory to LDS, and the
// sum itself runs on the 32 x 32 matrix instructions with fp32 accumulators.
// Inputs next to the end of dY's type may have been rounded up past it in their 8
// bits: finite elements saturate, as the dequantizer has them (the check for blocks where that
// can be takes 1 % of the widest tiles: 8190 x 4096 x 4096 306 -> 310 us).
//
// A workgroup owns a tile of D (32, 64 or 128 columns of dY by 128 of X, or 256 by 256)
// and walks a range of M in chunks of 64 rows.  dY's part of a chunk is copied
// straight into LDS; X's goes through registers, where its conversion costs one
// instruction per two elements, each element once per tile.  Both are loaded
// two to four chunks ahead.  Fragments are read with the transposing LDS reads,
// as the summed axis is outermost, a step ahead of their use.
//
// With few tiles M is cut into ranges; each writes its partial tile to the
// workspace, and the one that arrives last adds them in range order.
//
// Measured (bf16 x E4M3): 8190 x 4096 x 4096 with beta = 1 312 us (880 TFLOP/s), 8192^3 1069 us
// (1028 TFLOP/s); a bf16 product of a library with both operands transposed takes
// 286 us for the former.  128 x 128 tiles one chunk ahead took 383 and 1440 us.  For few
// columns of dY the time is that of streaming X: 8192 x 32 x 8192 26 us (2.7 TB/s),
// 8192 x 64 x 4096 26 us; what they lose against a copy is the join of the ranges.  In
// between the partial tiles weigh as much as the operands: 8192 x 256 x 4096 46 us, 64 tiles in 8
// ranges, 33.5 MB written and read back beside 43 MB of operands and result.
#include "gemm_tiled.h"
#include "lowbit.h"

namespace mmac {

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

// The first exponent at which an element of QT can pass DT's largest value: 256, 32768 or (int8) 128 times
// its power of two is 2^16 (fp16) or 2^128 (bf16).
template <int DT, int QT>
constexpr uint32_t kFirstPast = (DT == DT_F16 ? 127 + 16 : 127 + 128) - (QT == DT_E4M3 ? 8 : QT == DT_E5M2 ? 15 : 7);

// Sixteen elements of one block -> sixteen DT values (32 bytes), scaled: two elements per instruction for the fp8 types.
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
        } else if constexpr (DT == DT_BF16) {
            if constexpr (QT == DT_E4M3) {
                lo = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, scale, false));
                hi = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, scale, true));
            } else {
                lo = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(v, scale, false));
                hi = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(v, scale, true));
            }
        } else {
            if constexpr (QT == DT_E4M3) {
                lo = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v, scale, false));
                hi = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v, scale, true));
            } else {
                lo = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_bf8(v, scale, false));
                hi = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_bf8(v, scale, true));
            }
        }
        o[d >> 1][2 * (d & 1)] = lo;
        o[d >> 1][2 * (d & 1) + 1] = hi;
    }
    if (__any(e >= kFirstPast<DT, QT>)) {   // infinities that are not the element's own: the value before
        constexpr uint32_t kInf = DT == DT_F16 ? 0x7c00u : 0x7f80u;
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t element = (uint32_t)q[d] >> (8 * i), up = 16 * (i & 1);
                const uint32_t w = (uint32_t)o[d >> 1][2 * (d & 1) + i / 2];
                const bool own = QT == DT_E5M2 && (element & 0x7fu) == 0x7cu;
                if (((w >> up) & 0x7fffu) == kInf && !own) o[d >> 1][2 * (d & 1) + i / 2] = (int)(w - (1u << up));
            }
    }
}

// BN x BK tile, WN x WK waves, chunks loaded D ahead.
template <int DT, int QT, int BN, int BK, int WN, int WK, int D>
__global__ __launch_bounds__(WN * WK * 64) __attribute__((amdgpu_waves_per_eu(2)))
void gemm_mx8_wgrad_kernel(WgradParams p) {
    constexpr int MC = kWgradChunk, NT = WN * WK * 64;
    constexpr int TN = BN / WN / 32, TK = BK / WK / 32;
    constexpr bool SPLIT = BN < 256;                        // the widest tile is only taken where there are tiles enough
    constexpr int UY = BN / 8, UX = BK / 8;                 // 16-byte units per LDS row
    constexpr int YP = MC * UY / NT;                        // copy instructions of dY per chunk
    constexpr int XU = MC * BK / 16 / NT;                   // 16-element units of X per thread
    constexpr int LPT = YP + 2 * XU;                        // memory instructions per chunk
    constexpr int Y_BYTES = MC * BN * 2, X_BYTES = MC * BK * 2;
    constexpr int LDS_BYTES = (D + 1) * Y_BYTES + 2 * X_BYTES;
    static_assert(YP * NT == MC * UY && XU * NT * 16 == MC * BK, "whole copies");
    static_assert(LDS_BYTES <= 160 * 1024 && (D - 1) * LPT < 64, "LDS and counter range");
    __shared__ __attribute__((aligned(16))) uint8_t smem[LDS_BYTES];
    uint8_t *const smem_x = smem + (D + 1) * Y_BYTES;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave / WK, wk = wave % WK;
    // workgroup -> (tile, range): contiguous runs per XCD, so that the tiles an XCD has at once share their rows of
    // dY and columns of X in its L2; ranges of one tile are consecutive
    const int U = p.tiles_n * p.tiles_k * p.split.splits;
    const int xcd = blockIdx.x & 7, uq = U >> 3, ur = U & 7;
    const int unit = xcd * uq + (xcd < ur ? xcd : ur) + (blockIdx.x >> 3);
    const int split = unit % p.split.splits, tile = unit / p.split.splits;
    const int first = tile / (4 * p.tiles_k) * 4, gsz = min(p.tiles_n - first, 4), in = tile % (4 * p.tiles_k);
    const int n0 = (first + in % gsz) * BN, k0 = in / gsz * BK;
    const int chunks = (int)(((int64_t)p.M + MC - 1) / MC);
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
    i32x4 xq[D][XU];
    uint32_t xe[D][XU];
    const auto load_x = [&](int c, int d) {
        const int64_t m0 = (int64_t)c * MC;
        const int rows = (int)min((int64_t)MC, p.M - m0);
        const rsrc_t r = make_rsrc(p.Xq + m0 * p.q_pitch + k0, (uint32_t)((rows - 1) * p.q_pitch + kp - k0));
#pragma unroll
        for (int j = 0; j < XU; ++j) {
            const uint32_t P = j * NT + tid, row = P / (BK / 16), u = P % (BK / 16);
            // a tile of 256 columns has two strips of scale words; the second may lie past the last one
            const int strip = k0 / 128 + (int)(u / 8);
            const rsrc_t rs = make_rsrc(p.SX + (k0 / 128) * p.lds + m0, (uint32_t)(((p.K + 127) / 128 - k0 / 128 - 1) * p.lds * 4 + rows * 4));
            xq[d][j] = __builtin_amdgcn_raw_buffer_load_b128(r, (uint32_t)(row * p.q_pitch) + u * 16, 0, 0);
            xe[d][j] = __builtin_amdgcn_raw_buffer_load_b32(
                rs, (int)row < rows ? (uint32_t)(((strip - k0 / 128) * p.lds + row) * 4) : kOutOfRange, 0, 0);
        }
    };
    // the two halves of a unit in an order in which 16 lanes' writes meet 16 bank groups
    const auto put_x = [&](uint8_t *st, int d) {
#pragma unroll
        for (int j = 0; j < XU; ++j) {
            const uint32_t P = j * NT + tid, row = P / (BK / 16), u = P % (BK / 16);
            i32x4 o[2];
            scaled16<DT, QT>(xq[d][j], (xe[d][j] >> (8 * ((u / 2) & 3))) & 255u, o);
            const bool swap = lane & 8;
            const i32x4 w0 = swap ? o[1] : o[0], w1 = swap ? o[0] : o[1];
            uint8_t *at = st + row * (BK * 2);
            *reinterpret_cast<i32x4 *>(at + (((2 * u + (swap ? 1 : 0)) ^ tr_swz<UX>(row)) << 4)) = w0;
            *reinterpret_cast<i32x4 *>(at + (((2 * u + (swap ? 0 : 1)) ^ tr_swz<UX>(row)) << 4)) = w1;
        }
    };

#pragma unroll
    for (int d = 0; d < D; ++d)
        if (c0 + d < c1) {
            copy_y(c0 + d, smem + d * Y_BYTES);
            load_x(c0 + d, d);
        }
    int ys = 0;   // dY's stage of chunk c
    const auto chunk = [&](int c, int d) {
        uint8_t *sx = smem_x + ((c - c0) & 1) * X_BYTES;
        const uint8_t *sy = smem + ys * Y_BYTES;
        // dY's copy of chunk c has landed when at most the D - 1 chunks issued after it are outstanding (each is
        // exactly LPT memory instructions: its copies of dY, and an element and a scale load per unit of X)
        if (c + D <= c1) wait_vm_lgkm0<(D - 1) * LPT>();
        else wait_vm_lgkm0<0>();
        put_x(sx, d);          // its last readers passed the barrier before this one
        wait_lds();
        block_barrier();
        if (c + D < c1) {
            copy_y(c + D, smem + (ys == 0 ? D : ys - 1) * Y_BYTES);
            load_x(c + D, d);
        }
        i32x4 a[2][TN], b[2][TK];
        const auto read = [&](int s) {
#pragma unroll
            for (int i = 0; i < TN; ++i) a[s & 1][i] = tr_frag<BN>(sy, (wn * TN + i) * 32, s, lane);
#pragma unroll
            for (int j = 0; j < TK; ++j) b[s & 1][j] = tr_frag<BK>(sx, (wk * TK + j) * 32, s, lane);
        };
        read(0);
#pragma unroll
        for (int s = 0; s < MC / 16; ++s) {
            __builtin_amdgcn_sched_barrier(0);   // keeps a step's reads a step ahead of their use
            if (s + 1 < MC / 16) read(s + 1);
#pragma unroll
            for (int i = 0; i < TN; ++i)
#pragma unroll
                for (int j = 0; j < TK; ++j) acc[i][j] = mma32<DT>(a[s & 1][i], b[s & 1][j], acc[i][j]);
        }
        __builtin_amdgcn_sched_barrier(0);
        ys = ys == D ? 0 : ys + 1;
    };
    for (int c = c0; c < c1; c += D) {
#pragma unroll
        for (int d = 0; d < D; ++d)
            if (c + d < c1) chunk(c + d, d);
    }

    // ranges joined by the last to arrive, in range order (the partials at device scope, see the tiled GEMM)
    if (SPLIT && p.split.splits > 1) {
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
        constexpr int BATCH = TN * TK == 1 ? 4 : TN * TK == 2 ? 2 : 1;   // ranges whose loads are in flight together
        f32x16 sum[TN][TK];
        for (int r0 = 0; r0 < p.split.splits; r0 += BATCH) {
            i32x4 v[BATCH][TN][TK][4];
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                const bool real = r0 + b < p.split.splits;   // past the last range: offsets past the buffer, zeros
                const rsrc_t part = make_rsrc(ws + (int64_t)(real ? r0 + b : 0) * TILE_BYTES, TILE_BYTES);
#pragma unroll
                for (int i = 0; i < TN; ++i)
#pragma unroll
                    for (int j = 0; j < TK; ++j)
#pragma unroll
                        for (int g = 0; g < 4; ++g)
                            v[b][i][j][g] = __builtin_amdgcn_raw_buffer_load_b128(
                                part, real ? (uint32_t)((((i * TK + j) * 4 + g) * NT + tid) * 16) : kOutOfRange, 0, kDeviceScope);
            }
#pragma unroll
            for (int b = 0; b < BATCH; ++b)
#pragma unroll
                for (int i = 0; i < TN; ++i)
#pragma unroll
                    for (int j = 0; j < TK; ++j)
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int w = v[b][i][j][e / 4][e % 4];
                            const float f = __builtin_bit_cast(float, w);
                            sum[i][j][e] = r0 == 0 && b == 0 ? f : sum[i][j][e] + f;
                        }
        }
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int j = 0; j < TK; ++j) acc[i][j] = sum[i][j];
    }
    by_out_type(p.out.d_type, [&](auto type) {
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int j = 0; j < TK; ++j) {
                const int n = n0 + (wn * TN + i) * 32, k = k0 + (wk * TK + j) * 32 + (lane & 31);
                store_tile<decltype(type)::value>(p.out, n, p.N - n, k, k < p.K, acc[i][j]);
            }
    });
}

template <int DT, int QT>
static hipError_t launch_as(const WgradParams &p, hipStream_t s) {
    const dim3 grid((unsigned)(p.tiles_n * p.tiles_k * p.split.splits));
    switch (p.tile) {
    case WGRAD_32x128: hipLaunchKernelGGL((gemm_mx8_wgrad_kernel<DT, QT, 32, 128, 1, 4, 4>), grid, dim3(256), 0, s, p); break;
    case WGRAD_64x128: hipLaunchKernelGGL((gemm_mx8_wgrad_kernel<DT, QT, 64, 128, 1, 4, 3>), grid, dim3(256), 0, s, p); break;
    case WGRAD_128x128: hipLaunchKernelGGL((gemm_mx8_wgrad_kernel<DT, QT, 128, 128, 2, 2, 2>), grid, dim3(256), 0, s, p); break;
    default: hipLaunchKernelGGL((gemm_mx8_wgrad_kernel<DT, QT, 256, 256, 2, 4, 2>), grid, dim3(512), 0, s, p); break;
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
