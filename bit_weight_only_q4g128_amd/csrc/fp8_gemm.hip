// Product in 8-bit floating point with a scale for each block of 128 (gfx950,
// v_mfma_f32_16x16x128_f8f6f4):
//     y[m, n] = RN_bf16(sum_g xs[m, g] * ws[n / 128, g] * P[m, n, g] (+ resid[m, n])),
//     P[m, n, g] = sum over the columns k of block g of x[m, k] * w[n, k],
// x and w e4m3, every block sum P and the sum over blocks in fp32, one
// rounding at the end.  (Inside P the matrix cores align each 8 consecutive
// columns' products to the largest and drop what lies below 2^-13 of it; the
// sums of those octets are fp32.  Against a bf16 output that is small, about
// 1e-4 of a typical |y| where bf16 rounds by 1.7e-3, and the 16-bit products
// that keep more run at half the rate.)  One MFMA spans exactly one 128-column block, so its
// result starts from zero and folds into the accumulator with one FMA per
// value: the scale of a lane's results is one number (all of a lane's batch
// row, all weight rows of one 128-row block).
//
// MFMA operands (16x16x128): lane l holds A row l % 16 (a weight row) and B
// column l % 16 (a batch row), 32 of the block's columns each; the order of
// the columns within a block is free as long as both operands share it.  D:
// lane l holds weight rows 4 (l / 16) + v, v = 0..3, of batch row l % 16.
#include "fp8.h"
#include "internal.h"

namespace q4 {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ u32x4 ld16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
}
__device__ __forceinline__ f32x4 mfma(const u32x4 (&a)[2], const u32x4 (&b)[2]) {
    const i32x8 av = {(int)a[0].x, (int)a[0].y, (int)a[0].z, (int)a[0].w, (int)a[1].x, (int)a[1].y, (int)a[1].z, (int)a[1].w};
    const i32x8 bv = {(int)b[0].x, (int)b[0].y, (int)b[0].z, (int)b[0].w, (int)b[1].x, (int)b[1].y, (int)b[1].z, (int)b[1].w};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

// Rows n .. n + 3 of batch row m: one rounding, the residual added before it.
// 8-byte accesses where every row start allows them.
__device__ __forceinline__ void store4(const f32x4& v, const uint16_t* resid, uint16_t* y, int N, int m, int n, bool vec, bool rvec) {
    const size_t at = (size_t)m * N + n;
    f32x4 o = v;
    if (resid) {
        if (rvec && n + 3 < N) {
            const uint2 r = *reinterpret_cast<const uint2*>(resid + at);
            o += f32x4{bf16lo(r.x), bf16hi(r.x), bf16lo(r.y), bf16hi(r.y)};
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n + i < N) o[i] += __builtin_bit_cast(float, (uint32_t)resid[at + i] << 16);
        }
    }
    if (vec && n + 3 < N) {
        *reinterpret_cast<uint2*>(y + at) = make_uint2((uint32_t)f32_to_bf16(o[0]) | ((uint32_t)f32_to_bf16(o[1]) << 16),
                                                       (uint32_t)f32_to_bf16(o[2]) | ((uint32_t)f32_to_bf16(o[3]) << 16));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + i < N) y[at + i] = f32_to_bf16(o[i]);
    }
}
__device__ __forceinline__ bool rows_aligned8(const uint16_t* p, int N) { return (N & 3) == 0 && (reinterpret_cast<uintptr_t>(p) & 7) == 0; }

struct Fp8Group {
    Fp8Args t[kFp8MaxTasks];
    int first[kFp8MaxTasks + 1];   // first row block of each task
    int count, M;
};

// A workgroup of eight waves owns 16 R weight rows and 16 MT batch rows; the
// waves share the 128-column blocks of K and meet in LDS.
constexpr int kWaves = 8;

template <int MT, int R>
__global__ __launch_bounds__(kWaves * 64) void fp8_rows_kernel(Fp8Group p) {
    __shared__ __attribute__((aligned(16))) f32x4 part[kWaves][R * MT][64];
    const int lane = threadIdx.x & 63, lr = lane & 15, lq = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int ti = 0;
    while (ti + 1 < p.count && (int)blockIdx.x >= p.first[ti + 1]) ++ti;
    const Fp8Args a = p.t[ti];
    const int n0 = ((int)blockIdx.x - p.first[ti]) * 16 * R, m0 = blockIdx.y * 16 * MT;
    const int K = a.K, G = (K + 127) >> 7;
    const int rows_n = a.N - n0 < 16 * R ? a.N - n0 : 16 * R, rows_m = p.M - m0 < 16 * MT ? p.M - m0 : 16 * MT;
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(a.w + (size_t)n0 * K, (uint32_t)rows_n * (uint32_t)K);
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x + (size_t)m0 * K, (uint32_t)rows_m * (uint32_t)K);
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(a.xs + (size_t)m0 * G, (uint32_t)rows_m * (uint32_t)G * 4u);
    const float* wsrow = a.ws + (size_t)(n0 >> 7) * G;      // (16 R divides 128: one scale row)

    f32x4 acc[R][MT];
#pragma unroll
    for (int t = 0; t < R; ++t)
#pragma unroll
        for (int u = 0; u < MT; ++u) acc[t][u] = f32x4{0.f, 0.f, 0.f, 0.f};

    const int per = (G + kWaves - 1) / kWaves;
    const int g0 = wave * per, g1 = g0 + per < G ? g0 + per : G;
    for (int g = g0; g < g1; ++g) {
        u32x4 wf[R][2], xf[MT][2];
        float f[MT];
        const uint32_t k = 128u * g + 32u * lq;
#pragma unroll
        for (int t = 0; t < R; ++t)
#pragma unroll
            for (int c = 0; c < 2; ++c)     // a row at or past N, or a column past K, reads as zero
                wf[t][c] = ld16(rw, k + 16 * c < (uint32_t)K ? (uint32_t)(16 * t + lr) * K + k + 16 * c : 0xFFFFFFF0u);
#pragma unroll
        for (int u = 0; u < MT; ++u) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
                xf[u][c] = ld16(rx, k + 16 * c < (uint32_t)K ? (uint32_t)(16 * u + lr) * K + k + 16 * c : 0xFFFFFFF0u);
            f[u] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, (int)(((16 * u + lr) * G + g) * 4), 0, 0));
        }
        const float s = wsrow[g];
#pragma unroll
        for (int u = 0; u < MT; ++u) {
            const float fs = f[u] * s;
#pragma unroll
            for (int t = 0; t < R; ++t) {
                const f32x4 d = mfma(wf[t], xf[u]);
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[t][u][v] = __builtin_fmaf(fs, d[v], acc[t][u][v]);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < R; ++t)
#pragma unroll
        for (int u = 0; u < MT; ++u) part[wave][t * MT + u][lane] = acc[t][u];
    __syncthreads();
    const bool vec = rows_aligned8(a.y, a.N), rvec = a.resid && rows_aligned8(a.resid, a.N);
    for (int q = wave; q < R * MT; q += kWaves) {
        f32x4 v = part[0][q][lane];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) v += part[w][q][lane];
        const int t = q / MT, u = q % MT;
        const int m = m0 + 16 * u + lr, n = n0 + 16 * t + 4 * lq;
        if (m < p.M && n < a.N) store4(v, a.resid, a.y, a.N, m, n, vec, rvec);
    }
}

template <int MT, int R>
hipError_t launch_rows(const Fp8Args* tasks, int count, int M, hipStream_t s) {
    Fp8Group p;
    p.count = count;
    p.M = M;
    p.first[0] = 0;
    for (int i = 0; i < count; ++i) {
        p.t[i] = tasks[i];
        p.first[i + 1] = p.first[i] + (tasks[i].N + 16 * R - 1) / (16 * R);
    }
    return launch_kernel(fp8_rows_kernel<MT, R>, dim3(p.first[count], (M + 16 * MT - 1) / (16 * MT)), dim3(kWaves * 64), 0, s, p);
}

// ---------------------------------------------------------------------------
// Many rows: workgroup tiles of BM batch rows x BN weight rows over all of K,
// WM x WN waves, each BM / WM x BN / WN.  Per 128-column block the tile's rows
// go straight from memory to LDS (16 bytes per lane, no registers), into one
// of two stages: while the waves compute a block, the next one is on its way;
// one barrier per block.
//
// LDS holds rows of 128 bytes; 16-byte chunk c of row r sits at chunk
// c ^ (r / 2 % 8), so that one chunk of 16 consecutive rows (a quarter of a
// fragment read) covers the 64 banks once: 4 cycles per read, where chunk
// c ^ (r % 8) takes 8.  The swizzle is on the memory side of the load: LDS is
// written in lane order.
// ---------------------------------------------------------------------------
typedef __attribute__((address_space(3))) void lds_void;
// read through the scalar cache (a vector load would join the queue of the
// loads to LDS, and its wait would wait for all of them)
typedef const __attribute__((address_space(4))) float const_float;

// Ends a phase of the tile kernel: nothing moves across, no wait is implied.
__device__ __forceinline__ void phase() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

template <int BM, int BN>
struct TileLds {
    static constexpr int kXStage = BM * 128, kWStage = BN * 128;
    static constexpr int kX = 0, kW = 2 * kXStage, kS = kW + 2 * kWStage;    // two stages of each
    static constexpr int kQuad = BM * 16, kBytes = kS + 2 * kQuad;           // scales of 4 blocks per row, two such
};

template <int BM, int BN, int WM, int WN>
__device__ __forceinline__ void tile(const Fp8Group& p, uint8_t* lds) {
    using L = TileLds<BM, BN>;
    constexpr int kW = WM * WN, TM = BM / WM / 16, TN = BN / WN / 16;
    constexpr int kXLoads = BM / 8 / kW, kWLoads = BN / 8 / kW;      // 1 KB loads per wave and block
    static_assert(BM % (8 * kW) == 0 && BN % (8 * kW) == 0 && BN / WN <= 128 && BM / 64 <= kW && kW % 2 == 0 && BM / 64 <= kW / 2, "tile");

    const int lane = threadIdx.x & 63, lr = lane & 15, lq = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave % WM, wn = wave / WM;

    // the tile: XCD-contiguous ranges of one task's tiles, walked in
    // super-rows of 8 batch blocks
    int ti = 0;
    while (ti + 1 < p.count && (int)blockIdx.x >= p.first[ti + 1]) ++ti;
    const Fp8Args a = p.t[ti];
    const int nM = (p.M + BM - 1) / BM, nN = (a.N + BN - 1) / BN;
    const int T = nM * nN, i = (int)blockIdx.x - p.first[ti], xcd = i & 7, q8 = T >> 3, r8 = T & 7;
    const int at_tile = xcd * q8 + (xcd < r8 ? xcd : r8) + (i >> 3);
    const int per_super = 8 * nN, sup = at_tile / per_super, within = at_tile - sup * per_super;
    const int rows_here = nM - sup * 8 < 8 ? nM - sup * 8 : 8;
    const int m0 = (sup * 8 + within % rows_here) * BM, n0 = within / rows_here * BN;

    const int K = a.K, G = (K + 127) >> 7;
    const int rows_m = p.M - m0 < BM ? p.M - m0 : BM, rows_n = a.N - n0 < BN ? a.N - n0 : BN;
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x + (size_t)m0 * K, (uint32_t)rows_m * (uint32_t)K);
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(a.w + (size_t)n0 * K, (uint32_t)rows_n * (uint32_t)K);
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(a.xs + (size_t)m0 * G, (uint32_t)rows_m * (uint32_t)G * 4u);
    const int nb = (n0 + wn * (BN / WN)) >> 7;
    const const_float* wsrow = (const const_float*)(uintptr_t)(a.ws + (size_t)(nb * 128 < a.N ? nb : 0) * G);

    // this lane's place in a 1 KB load: row lane / 8 of the 8, chunk lane % 8
    // of LDS = chunk (lane % 8) ^ (row / 2 % 8) of memory (kW is even, so the
    // wave's loads all lie in even or all in odd groups of 8 rows)
    const uint32_t chunk = (uint32_t)((lane & 7) ^ (lane >> 4) ^ ((wave & 1) << 2)) * 16u;
    const uint32_t off = (uint32_t)(8 * wave + (lane >> 3)) * (uint32_t)K + chunk;
    const uint32_t soff = (uint32_t)(64 * wave + lane) * (uint32_t)G * 4u;
    const bool tail = K & 127;
    constexpr int kLoads = kXLoads + kWLoads;
    // Load j of block g.  o = at(g): this lane's offset, or one past the matrix
    // for a column past K and for a block past the last; such loads, like rows
    // past the matrix, put zeros into LDS.
    auto at = [&](int g) { return g >= G || (tail && g == G - 1 && 128u * g + chunk >= (uint32_t)K) ? 0xFFFF0000u : off; };
    auto piece = [&](int g, uint32_t o, int j) {
        const int i = j < kXLoads ? j : j - kXLoads;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(j < kXLoads ? rx : rw,
                                                 (lds_void*)(lds + (j < kXLoads ? L::kX + (g & 1) * L::kXStage : L::kW + (g & 1) * L::kWStage) +
                                                             (wave + kW * i) * 1024),
                                                 16, (int)o, i * kW * 8 * K + g * 128, 0, 0);
    };
    // Scales of blocks 4 q .. 4 q + 3: a row's scales are adjacent, so four
    // cost the lines of one (every block alone: 20 % of the whole kernel).  The
    // last four end at G.
    auto quad_first = [&](int q) { return 4 * q + 4 <= G ? 4 * q : G - 4; };
    auto scales = [&](int g) {
        if ((g & 3) || g >= G || wave >= BM / 64) return;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(lds + L::kS + ((g >> 2) & 1) * L::kQuad + wave * 1024), 16, (int)soff,
                                                 quad_first(g >> 2) * 4, 0, 0);
    };
    auto load = [&](int g) {
        scales(g);
        const uint32_t o = at(g);
#pragma unroll
        for (int j = 0; j < kLoads; ++j) piece(g, o, j);
    };

    f32x4 acc[TN][TM];
#pragma unroll
    for (int t = 0; t < TN; ++t)
#pragma unroll
        for (int u = 0; u < TM; ++u) acc[t][u] = f32x4{0.f, 0.f, 0.f, 0.f};

    const int c0 = ((2 * lq) ^ (lr >> 1)) * 16, c1 = ((2 * lq + 1) ^ (lr >> 1)) * 16;
    uint32_t xat[2] = {(uint32_t)(L::kX + (wm * (BM / WM) + lr) * 128 + c0), (uint32_t)(L::kX + (wm * (BM / WM) + lr) * 128 + c1)};
    uint32_t wat[2] = {(uint32_t)(L::kW + (wn * (BN / WN) + lr) * 128 + c0), (uint32_t)(L::kW + (wn * (BN / WN) + lr) * 128 + c1)};
    // Two groups of waves take turns (one of each shares a SIMD): while one
    // multiplies, the other reads its next fragments.  Phase 2 g: group 0 reads
    // block g, group 1 multiplies block g - 1; phase 2 g + 1 the other way
    // round.  Block g + 1 goes on its way in phase 2 g, when the last reads of
    // its stage (block g - 1, group 1) are a barrier behind, and has arrived
    // (every wave's vmcnt) by the barrier that ends phase 2 g + 1.
    auto walk = [&](const bool kSecond) __attribute__((always_inline)) {
        u32x4 xf[TM][2], wf[TN][2];
        float f[TM];
        float next = wsrow[0];
        load(0);
        __builtin_amdgcn_s_waitcnt(0x0F70);      // vmcnt(0)
        phase();
        if (kSecond) {
            load(1);
            phase();
        }
        for (int g = 0; g < G; ++g) {
            const float s = next;
            if (g + 1 < G) next = wsrow[g + 1];
            const uint8_t* sc = lds + L::kS + ((g >> 2) & 1) * L::kQuad + (g - quad_first(g >> 2)) * 4;
#pragma unroll
            for (int u = 0; u < TM; ++u) {
#pragma unroll
                for (int h = 0; h < 2; ++h) xf[u][h] = *reinterpret_cast<const u32x4*>(lds + xat[h] + u * 2048);
                f[u] = *reinterpret_cast<const float*>(sc + (wm * (BM / WM) + 16 * u + lr) * 16);
            }
#pragma unroll
            for (int t = 0; t < TN; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h) wf[t][h] = *reinterpret_cast<const u32x4*>(lds + wat[h] + t * 2048);
            // the other stage
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                xat[h] ^= L::kXStage;
                wat[h] = L::kW + ((wat[h] - L::kW) ^ L::kWStage);
            }
            if (!kSecond) load(g + 1);
            const uint32_t o = at(g + 2);
#pragma unroll
            for (int u = 0; u < TM; ++u) f[u] *= s;
            if (kSecond) __builtin_amdgcn_s_waitcnt(0x0070);      // vmcnt(0), lgkmcnt(0)
            else __builtin_amdgcn_s_waitcnt(0xC07F);              // lgkmcnt(0)
            phase();
            __builtin_amdgcn_s_setprio(1);
            // result i folds while the matrix cores work on i + 1 .. i + kAhead
            constexpr int kAhead = 3, kN = TN * TM;
            f32x4 d[kAhead + 1];
#pragma unroll
            for (int i = 0; i < kN + kAhead; ++i) {
                if (i < kN) d[i % (kAhead + 1)] = mfma(wf[i / TM], xf[i % TM]);
                if (i >= kAhead) {
                    const int o = i - kAhead;
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        acc[o / TM][o % TM][v] = __builtin_fmaf(f[o % TM], d[o % (kAhead + 1)][v], acc[o / TM][o % TM][v]);
                }
                if (i < kN) __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                if (i >= kAhead) __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
                if (kSecond && i < kN && i % (kN / kLoads) == 0) {
                    piece(g + 2, o, i / (kN / kLoads));
                    __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
                }
            }
            // (the folds stay in this block: sunk into a later one they would cost the overlap)
#pragma unroll
            for (int t = 0; t < TN; ++t)
#pragma unroll
                for (int u = 0; u < TM; ++u) asm volatile("" : "+v"(acc[t][u]));
            __builtin_amdgcn_s_setprio(0);
            if (!kSecond) __builtin_amdgcn_s_waitcnt(0x0F70);     // vmcnt(0)
            if (!kSecond || g + 1 < G) phase();
        }
    };
    if (wave < kW / 2) walk(false);
    else walk(true);
    __builtin_amdgcn_s_waitcnt(0x0F70);      // no load to LDS outlives the workgroup

    const bool vec = rows_aligned8(a.y, a.N), rvec = a.resid && rows_aligned8(a.resid, a.N);
#pragma unroll
    for (int u = 0; u < TM; ++u) {
        const int m = m0 + wm * (BM / WM) + 16 * u + lr;
        if (m >= p.M) continue;
#pragma unroll
        for (int t = 0; t < TN; ++t) {
            const int n = n0 + wn * (BN / WN) + 16 * t + 4 * lq;
            if (n < a.N) store4(acc[t][u], a.resid, a.y, a.N, m, n, vec, rvec);
        }
    }
}

template <int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 2) void fp8_tile_kernel(Fp8Group p) {
    __shared__ __attribute__((aligned(16))) uint8_t lds[TileLds<BM, BN>::kBytes];
    tile<BM, BN, WM, WN>(p, lds);
}

template <int BM, int BN, int WM, int WN>
hipError_t launch_tile(const Fp8Args* tasks, int count, int M, hipStream_t s) {
    Fp8Group p;
    p.count = count;
    p.M = M;
    p.first[0] = 0;
    for (int i = 0; i < count; ++i) {
        p.t[i] = tasks[i];
        p.first[i + 1] = p.first[i] + ((M + BM - 1) / BM) * ((tasks[i].N + BN - 1) / BN);
    }
    return launch_kernel(fp8_tile_kernel<BM, BN, WM, WN>, dim3(p.first[count]), dim3(64 * WM * WN), 0, s, p);
}

}  // namespace

size_t fp8_gemm_ws_bytes(const Fp8Args*, int, int) { return 0; }

// Fewest 128-column blocks of any task (the tile kernel needs kTileMinBlocks).
static int min_blocks(const Fp8Args* tasks, int count) {
    int g = tasks[0].K;
    for (int i = 1; i < count; ++i) g = tasks[i].K < g ? tasks[i].K : g;
    return (g + 127) / 128;
}

hipError_t launch_fp8_gemm(const Fp8Args* tasks, int count, int M, void*, size_t, hipStream_t s) {
    if (M > 128 && min_blocks(tasks, count) >= 4) return launch_tile<256, 256, 4, 2>(tasks, count, M, s);
    return M <= 16 ? launch_rows<1, 1>(tasks, count, M, s) : launch_rows<4, 1>(tasks, count, M, s);
}

}  // namespace q4
