// Products with 4-bit weights and group scales, many rows (prompts): D = A * W.
//
// The mathematics is that of the row kernel: per group of a weight row the sum of
// a * n runs on the matrix instructions with exact codes, and at the group's end
// s * (sum a*n - z * sum a) joins the fp32 total.  Here the zero point's term is one
// more instruction step of the same sum: with the group's sum of a row of A
// split into three bf16 terms (24 bits together) against -z in three operand
// slots, the accumulator receives - z * sum a.
//
// A workgroup of eight waves computes 128 x 256, 128 x 128 or 64 x 128 of D, a wave 32
// columns of 128, 64 or 32 rows, and walks K in chunks of 128.  A's chunk and each
// wave's own codes and scale words are copied straight into LDS, three or four
// stages; codes become operands in registers, so in the widest tile every code
// is converted once per workgroup.  While a chunk is multiplied, each wave sums
// the rows of A that it copied itself for the next one's zero points.
//
// A group's sums have to be scaled by vector instructions, 16 per instruction tile
// and group.  The work of a chunk is therefore cut into phases (one group of K
// for half of the wave's tiles) with two sets of sums: one phase's are scaled and
// added while the matrix instructions of the next run.
//
// Measured at 2048 x 8192 x 8192 (bf16, groups of 128): U4 312 us (880 TFLOP/s), E2M1 254
// us (1080), U4 in groups of 32 469 us; a bf16 product of a library at these sizes takes
// 210 us.  The widest U4 tile in groups of 128 needs all 256 registers and keeps three values
// in scratch, outside of its main loop.  The matrix instructions are busy 42 % of the cycles; stand-ins
// that leave a part out ran 17 % (the copies), 8 % (the row sums) and 5 % (the
// scaling) faster, one with operands that need no conversion no faster, and
// neither deeper prefetch of the fragments nor 64 x 64 wave tiles (half of
// the LDS reads, twice the conversions; 349 us against 337) nor one wave per SIMD with
// 128 x 64 (443 us) changed that.
#include "gemm_tiled.h"
#include "w4_operand.h"

namespace mmac {

// bf16 bits nearest to x, in the low half (finite x of moderate size; NaN stays NaN).
__device__ __forceinline__ uint32_t bf16_bits(float x) {
    return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x);
}

// x as three bf16 terms, 24 bits together: the first two in one word, the last in the other.
__device__ __forceinline__ u32x2 three_terms(float x) {
    const uint32_t hi = bf16_bits(x);
    const float r = x - __builtin_bit_cast(float, hi << 16);
    const uint32_t mid = bf16_bits(r);
    return u32x2{hi | (mid << 16), bf16_bits(r - __builtin_bit_cast(float, mid << 16))};
}

// Wave tiles of 32 TI rows x 32 columns, WM x WN waves.
template <int DT, int QT, int GROUP, int TI, int WM, int WN, int STAGES>
__global__ __launch_bounds__(WM * WN * 64) __attribute__((amdgpu_waves_per_eu(2, 2)))
void gemm_w4_tiled_kernel(W4Params p) {
    constexpr int BM = 32 * TI * WM, BN = 32 * WN, KC = kW4Chunk, NT = WM * WN * 64;
    constexpr int HT = TI > 1 ? TI / 2 : 1, NH = TI / HT;         // tiles of a phase, phases of a group
    constexpr bool PIPE = NH * (KC / GROUP) % 2 == 0;             // phases alternate between two sets of sums
    constexpr bool SPLIT = TI < 4;                                // the widest tile is only taken where there are tiles enough
    constexpr int GPC = KC / GROUP, SPG = GROUP / 16;             // groups of a chunk, steps of a group
    constexpr int AP = BM * KC * 2 / 16 / NT;                     // copy instructions of A per chunk: 4 rows each
    constexpr int SP = (32 * GPC + 63) / 64;                      // of scale words
    constexpr int LPT = AP + 2 + SP;                              // of a wave's chunk in all
    constexpr int LPR = 16 / AP, KL = KC / LPR;                   // lanes per row, elements per lane when rows are summed
    static_assert(LPR <= 8 && KL <= 32 && GROUP % KL == 0, "row sums: up to 8 lanes a row, each within a group");
    // a stage: A's rows, then each wave's codes and scale words
    constexpr int A_BYTES = BM * KC * 2, C_BYTES = 32 * KC / 2, W_BYTES = C_BYTES + SP * 256;
    constexpr int STAGE = A_BYTES + WM * WN * W_BYTES;
    // sums of A's rows: per row and group three bf16 terms (two, then the last), or with groups of 32, where LDS
    // is short of that, the fp32 sum, split where it is read
    constexpr bool TERMS = GROUP > 32;
    constexpr int EXT_BYTES = GPC * BM * (TERMS ? 6 : 4);
    constexpr int LDS_BYTES = STAGES * STAGE + 2 * EXT_BYTES;
    static_assert(NT == 512 && LDS_BYTES <= 160 * 1024, "eight waves, LDS of one workgroup per compute unit");
    __shared__ __attribute__((aligned(16))) uint8_t smem[LDS_BYTES];
    uint8_t *ext = smem + STAGES * STAGE;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g2 = lane >> 5, l32 = lane & 31, wm = wave / WN, wn = wave % WN;

    // workgroup -> (tile, range): contiguous runs per XCD, then groups of 4 tile rows column by column
    const int U = p.tiles_m * p.tiles_n * p.split.splits;
    const int x = blockIdx.x & 7, uq = U >> 3, ur = U & 7;
    const int unit = x * uq + (x < ur ? x : ur) + (blockIdx.x >> 3);
    const int tile = unit / p.split.splits, split = unit % p.split.splits;
    const int first = tile / (4 * p.tiles_n) * 4, gsz = min(p.tiles_m - first, 4), in = tile % (4 * p.tiles_n);
    const int row0 = (first + in % gsz) * BM, col0 = in / gsz * BN;

    const int rows = min(p.M - row0, BM), cols = min(p.N - col0, BN);
    const int row_bytes = (p.K + 31) / 32 * 16;
    const rsrc_t ra = make_rsrc(p.A + (int64_t)row0 * p.a_pitch, (uint32_t)(rows * p.a_pitch));
    const rsrc_t rw = make_rsrc(p.codes + (int64_t)col0 * p.pitch, (uint32_t)((cols - 1) * p.pitch + row_bytes));
    const rsrc_t rs = make_rsrc(p.words + col0, (uint32_t)(((p.groups - 1) * p.ldw + cols) * 4));
    const int nall = (p.K + KC - 1) / KC, nfull = p.K / KC;
    const int c0 = split * p.split.per_split, c1 = min(c0 + p.split.per_split, nall);

    // A's chunk c -> LDS rows of 256 bytes, unit u of row r at u ^ (r mod 16)
    const auto copy_a = [&](int c, uint8_t *st) {
        if (c < nfull) {
#pragma unroll
            for (int j = 0; j < AP; ++j) {
                const uint32_t P = j * NT + wave * 64 + lane, r = P >> 4, u = (P & 15) ^ (r & 15);
                __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void *)(st + (j * NT + wave * 64) * 16), 16,
                                                         r * (uint32_t)p.a_pitch + (uint32_t)c * (KC * 2) + u * 16, 0, 0, 0);
            }
        } else {   // K ends inside: through registers, zero past K
            for (int j = 0; j < AP; ++j) {
                const uint32_t P = j * NT + tid, r = P >> 4, u = (P & 15) ^ (r & 15);
                const int e0 = c * KC + (int)u * 8;
                *reinterpret_cast<i32x4 *>(st + P * 16) = masked_unit<2>(ra, r * (uint32_t)p.a_pitch + (uint32_t)e0 * 2, e0, p.K);
            }
        }
    };
    // this wave's columns wn * 32 + r of chunk c: 64 bytes of codes each, 16-byte unit u of column r
    // at u ^ ((r / 4) mod 4); then their scale words, [group][column]
    const auto copy_w = [&](int c, uint8_t *st) {
        uint8_t *to = st + A_BYTES + wave * W_BYTES;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t r = j * 16 + (lane >> 2), u = (lane & 3) ^ ((r >> 2) & 3);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void *)(to + j * 1024), 16,
                                                     (wn * 32 + r) * (uint32_t)p.pitch + (uint32_t)c * (KC / 2) + u * 16, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < SP; ++j) {
            const int d = j * 64 + lane, g = p.group == 0 ? 0 : c * GPC + d / 32, col = wn * 32 + d % 32;
            const uint32_t off = d < GPC * 32 && g < p.groups ? (uint32_t)((g * p.ldw + col) * 4) : kOutOfRange;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void *)(to + C_BYTES + j * 256), 4, off, 0, 0, 0);
        }
    };
    const auto load_w = [&](const uint8_t *st, i32x4 (&cd)[2], uint32_t (&sw)[GPC]) {
        const uint8_t *from = st + A_BYTES + wave * W_BYTES;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            cd[h] = *reinterpret_cast<const i32x4 *>(from + l32 * 64 + (((2 * h + g2) ^ ((l32 >> 2) & 3)) << 4));
#pragma unroll
        for (int g = 0; g < GPC; ++g) sw[g] = *reinterpret_cast<const uint32_t *>(from + C_BYTES + (g * 32 + l32) * 4);
    };
    // sums of A's rows over each group of the chunk in `st`, three bf16 terms each: a wave has the
    // rows it copied itself, LPR lanes a row
    const auto sum_rows = [&](const uint8_t *st, uint8_t *to) {
        const int r = lane / (64 / AP) * (NT / 16) + wave * 4 + lane / LPR % 4, part = lane % LPR;
        float sum = 0.0f;
#pragma unroll
        for (int u = 0; u < KL / 8; ++u) {
            const i32x4 v = *reinterpret_cast<const i32x4 *>(st + r * 256 + (((KL / 8 * part + u) ^ (r & 15)) << 4));
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const int w = v[d];
                if constexpr (DT == DT_BF16)
                    sum = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w), bf16x2{(__bf16)1.0f, (__bf16)1.0f}, sum, false);
                else
                    sum = __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, w), f16x2{(_Float16)1.0f, (_Float16)1.0f}, sum, false);
            }
        }
        const auto add = [](uint32_t a, uint32_t b) {
            return __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
        };
        uint32_t s = __builtin_bit_cast(uint32_t, sum);
        if constexpr (GROUP / KL >= 2) s = add(s, dpp<kDppXor1>(s));
        if constexpr (GROUP / KL >= 4) s = add(s, dpp<kDppXor2>(s));
        if constexpr (GROUP / KL >= 8) s = add(s, dpp<kDppMirror8>(s));
        sum = __builtin_bit_cast(float, s);
        if (part % (GROUP / KL) == 0) {
            const int at = part / (GROUP / KL) * BM + r;
            if constexpr (TERMS) {
                const u32x2 e = three_terms(sum);
                reinterpret_cast<uint32_t *>(to)[at] = e[0];
                reinterpret_cast<uint16_t *>(to + GPC * BM * 4)[at] = (uint16_t)e[1];
            } else {
                reinterpret_cast<float *>(to)[at] = sum;
            }
        }
    };

    f32x16 acc[TI];
#pragma unroll
    for (int i = 0; i < TI; ++i) acc[i] = f32x16{};

    // chunk c's copies have landed when at most those of the chunks issued after it are outstanding; the chunk K
    // ends inside goes partly through registers, then everything is waited for
    const int whole = min(c1, nfull);
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i)
        if (c0 + i < c1) {
            copy_a(c0 + i, smem + i * STAGE);
            copy_w(c0 + i, smem + i * STAGE);
        }
    const auto landed = [&](int c, int last) {   // last: the last chunk issued so far
        wait_copies<LPT, STAGES - 2>(last < whole ? last - c : 0);
    };
    if (c0 < c1) {
        landed(c0, min(c0 + STAGES - 2, c1 - 1));
        if constexpr (QT == DT_U4) sum_rows(smem, ext);
        wait_lds();
        block_barrier();
    }
    // The chunk's work in phases: one group of K for HT of the TI tiles.  A phase's sums are scaled and added
    // while the matrix instructions of the next phase run (the last phase's in the next chunk).
    f32x16 t[2][HT];
    float scale = 0.0f;   // of the phase whose sums wait in t[1] when a chunk begins
#pragma unroll
    for (int i = 0; i < HT; ++i) t[1][i] = f32x16{};
    const auto add_up = [&](int buf, int half, float s) {
#pragma unroll
        for (int i = 0; i < HT; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[half * HT + i][e] = fmaf(s, t[buf][i][e], acc[half * HT + i][e]);
    };
    int cur = 0;
    const auto chunk = [&](auto steady, int c) {
        constexpr bool STEADY = decltype(steady)::value;   // chunks c + 1 .. c + STAGES - 1 are there, and whole
        const uint8_t *st = smem + cur * STAGE;
        const int next = cur + 1 == STAGES ? 0 : cur + 1, freed = cur == 0 ? STAGES - 1 : cur - 1;
        const uint8_t *ex = ext + ((c - c0) & 1) * EXT_BYTES;
        uint8_t *ex1 = ext + ((c + 1 - c0) & 1) * EXT_BYTES;
        // this wave's copies of chunk c + 1 have landed; those of later chunks may be outstanding
        if (STEADY) {
            wait_vm_lgkm0<(STAGES - 3) * LPT>();
        } else if (c + 1 < c1) {
            const int last = min(c + STAGES - 2, c1 - 1);
            wait_copies<LPT, STAGES - 2>(last < whole ? last - c - 1 : 0);
        }
        if (STEADY || c + STAGES - 1 < c1) {
            copy_a(c + STAGES - 1, smem + freed * STAGE);
            copy_w(c + STAGES - 1, smem + freed * STAGE);
        }
        i32x4 cd[2];
        uint32_t sw[GPC];
        load_w(st, cd, sw);
        // operand order: GROUP >= 64, step 4 h + d is word d of the lane's unit 2 h + g2; GROUP 32: the lane halves
        // trade words so that every two steps are one unit
        if constexpr (GROUP == 32) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int d = 0; d < 2; ++d) {
                    const auto x = __builtin_amdgcn_permlane32_swap((uint32_t)cd[h][d], (uint32_t)cd[h][d + 2], false, false);
                    cd[h][d] = (int)x[0];
                    cd[h][d + 2] = (int)x[1];
                }
        }
        if constexpr (QT == DT_U4) {
            if (STEADY || c + 1 < c1) sum_rows(smem + next * STAGE, ex1);
        }
        // The steps of all phases in one row: step n of SPP is k = n % SPP of phase n / SPP (of group phase / NH and
        // half phase % NH); with U4 the last k of a phase is the zero points' term.  A's fragments are read AHEAD
        // steps before their use; the compiler would move the reads next to the uses, hence the scheduling barriers.
        constexpr int SPP = SPG + (QT == DT_U4 ? 1 : 0), STEPS = GPC * NH * SPP, AHEAD = 2;
        i32x4 a[AHEAD + 1][HT], b[SPG];
        const auto read = [&](int n) {
            const int k = n % SPP, phase = n / SPP, g = phase / NH, half = phase % NH;
#pragma unroll
            for (int i = 0; i < HT; ++i) {
                const int r = (wm * TI + half * HT + i) * 32 + l32;
                i32x4 &f = a[n % (AHEAD + 1)][i];
                if (k < SPG) {
                    const int s = g * SPG + k;
                    const int u = GROUP == 32 ? 4 * (s / 2) + 2 * g2 + s % 2 : 4 * (2 * (s / 4) + g2) + s % 4;
                    f = *reinterpret_cast<const i32x4 *>(st + r * 256 + ((u ^ (r & 15)) << 4));
                } else {
                    u32x2 e;
                    if constexpr (TERMS)
                        e = u32x2{reinterpret_cast<const uint32_t *>(ex)[g * BM + r],
                                  reinterpret_cast<const uint16_t *>(ex + GPC * BM * 4)[g * BM + r]};
                    else
                        e = three_terms(reinterpret_cast<const float *>(ex)[g * BM + r]);
                    f = i32x4{(int)e[0], (int)e[1], 0, 0};
                }
            }
        };
        const auto operand = [&](int n) {   // the weight's, shared by the halves of a group
            const int k = n % SPP, phase = n / SPP, s = phase / NH * SPG + k;
            if (phase % NH == 0 && k < SPG) b[k] = operand_of<DT, QT>((uint32_t)cd[s / 4][s % 4]);
        };
#pragma unroll
        for (int n = 0; n < AHEAD; ++n) read(n);
        operand(0);
#pragma unroll
        for (int n = 0; n < STEPS; ++n) {
            const int k = n % SPP, phase = n / SPP, g = phase / NH, half = phase % NH, buf = phase & 1;
            __builtin_amdgcn_sched_barrier(0);
            if (n + AHEAD < STEPS) read(n + AHEAD);
            const float s1 = __builtin_bit_cast(float, sw[g] & ~0xffu);
            if (k < SPG) {
#pragma unroll
                for (int i = 0; i < HT; ++i)
                    t[buf][i] = mma32<DT>(a[n % (AHEAD + 1)][i], b[k], k == 0 ? f32x16{} : t[buf][i]);
            } else {   // - z * sum a: only the lanes of the first half carry terms
                const int z = g2 ? 0 : (int)bf16_bits(-(float)(sw[g] & 0xffu));
#pragma unroll
                for (int i = 0; i < HT; ++i)
                    t[buf][i] = mma32<DT_BF16>(a[n % (AHEAD + 1)][i], i32x4{z | (z << 16), z, 0, 0}, t[buf][i]);
            }
            if (n + 1 < STEPS) operand(n + 1);
            // a share of the phase before this one
            if constexpr (PIPE) {
                constexpr int kShare = (16 * HT + SPP - 1) / SPP;
#pragma unroll
                for (int x = k * kShare; x < min((k + 1) * kShare, 16 * HT); ++x) {
                    const int i = x / 16, e = x % 16, h = half == 0 ? NH - 1 : half - 1;
                    const float sc = half == 0 ? scale : s1;
                    acc[h * HT + i][e] = fmaf(sc, t[buf ^ 1][i][e], acc[h * HT + i][e]);
                }
                if (k == SPP - 1 && half == NH - 1) scale = s1;
            } else if (k == SPP - 1) {
                add_up(buf, half, s1);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        wait_lds();
        block_barrier();
        cur = next;
    };
    int c = c0;
    for (; c + STAGES - 1 < whole; ++c) chunk(std::true_type{}, c);
    for (; c < c1; ++c) chunk(std::false_type{}, c);
    if constexpr (PIPE) add_up(1, NH - 1, scale);

    // ranges joined by the last to arrive, in range order (the partials at device scope, see the tiled GEMM)
    if (SPLIT && p.split.splits > 1) {
        constexpr int TILE_BYTES = BM * BN * 4;
        uint8_t *ws = p.split.partials + (int64_t)tile * p.split.splits * TILE_BYTES;
        const rsrc_t mine = make_rsrc(ws + (int64_t)split * TILE_BYTES, TILE_BYTES);
#pragma unroll
        for (int i = 0; i < TI; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const float e0 = acc[i][4 * g], e1 = acc[i][4 * g + 1], e2 = acc[i][4 * g + 2], e3 = acc[i][4 * g + 3];
                const i32x4 v = {__builtin_bit_cast(int, e0), __builtin_bit_cast(int, e1), __builtin_bit_cast(int, e2),
                                 __builtin_bit_cast(int, e3)};
                __builtin_amdgcn_raw_buffer_store_b128(v, mine, (uint32_t)(((i * 4 + g) * NT + tid) * 16), 0, kDeviceScope);
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
        constexpr int BATCH = 4;   // ranges whose loads are in flight together
        f32x16 sum[TI];
        for (int r0 = 0; r0 < p.split.splits; r0 += BATCH) {
            i32x4 v[BATCH][TI][4];
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                const bool real = r0 + b < p.split.splits;   // past the last range: offsets past the buffer, zeros
                const rsrc_t part = make_rsrc(ws + (int64_t)(real ? r0 + b : 0) * TILE_BYTES, TILE_BYTES);
#pragma unroll
                for (int i = 0; i < TI; ++i)
#pragma unroll
                    for (int g = 0; g < 4; ++g)
                        v[b][i][g] = __builtin_amdgcn_raw_buffer_load_b128(
                            part, real ? (uint32_t)(((i * 4 + g) * NT + tid) * 16) : kOutOfRange, 0, kDeviceScope);
            }
#pragma unroll
            for (int b = 0; b < BATCH; ++b)
#pragma unroll
                for (int i = 0; i < TI; ++i)
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int w = v[b][i][e / 4][e % 4];
                        const float f = __builtin_bit_cast(float, w);
                        sum[i][e] = r0 == 0 && b == 0 ? f : sum[i][e] + f;
                    }
        }
#pragma unroll
        for (int i = 0; i < TI; ++i) acc[i] = sum[i];
    }
#pragma unroll
    for (int i = 0; i < TI; ++i) {
        const int r = (wm * TI + i) * 32, col = wn * 32 + l32;
        by_out_type(p.out.d_type, [&](auto type) {
            store_tile<decltype(type)::value>(p.out, row0 + r, rows - r, col0 + col, col < cols, acc[i]);
        });
    }
}

template <int DT, int QT, int GROUP>
static hipError_t launch_tiles(const W4Params &p, hipStream_t s) {
    const dim3 grid((unsigned)(p.tiles_m * p.tiles_n * p.split.splits)), block(512);
    switch (p.tile) {
    case W4_128x256: hipLaunchKernelGGL((gemm_w4_tiled_kernel<DT, QT, GROUP, 4, 1, 8, 3>), grid, block, 0, s, p); break;
    case W4_128x128: hipLaunchKernelGGL((gemm_w4_tiled_kernel<DT, QT, GROUP, 2, 2, 4, 3>), grid, block, 0, s, p); break;
    default: hipLaunchKernelGGL((gemm_w4_tiled_kernel<DT, QT, GROUP, 1, 2, 4, 4>), grid, block, 0, s, p); break;
    }
    return hipGetLastError();
}
template <int DT, int QT>
static hipError_t by_group(const W4Params &p, hipStream_t s) {
    switch (p.group) {
    case 32: return launch_tiles<DT, QT, 32>(p, s);
    case 64: return launch_tiles<DT, QT, 64>(p, s);
    case 0:
    case 128: return launch_tiles<DT, QT, 128>(p, s);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_gemm_w4_tiled(int a, int q, const W4Params &p, hipStream_t s) {
    if (a == DT_BF16) return q == DT_FP4 ? by_group<DT_BF16, DT_FP4>(p, s) : by_group<DT_BF16, DT_U4>(p, s);
    if (a == DT_F16) return q == DT_FP4 ? by_group<DT_F16, DT_FP4>(p, s) : by_group<DT_F16, DT_U4>(p, s);
    return hipErrorInvalidValue;
}

}  // namespace mmac
