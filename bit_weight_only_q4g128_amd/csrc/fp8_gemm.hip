// Product in 8-bit floating point with a scale for each block of 128 (gfx950,
// v_mfma_f32_16x16x128_f8f6f4):
//     y[m, n] = RN_bf16(sum_g xs[m, g] * ws[n / 128, g] * P[m, n, g] (+ resid[m, n])),
//     P[m, n, g] = sum over the columns k of block g of x[m, k] * w[n, k],
// x and w e4m3, every block sum P and the sum over blocks in fp32, one
// rounding at the end.  (Inside P the matrix cores align each 8 consecutive
// columns' products to the largest and drop what lies below 2^-13 of it; the
// sums of those octets are fp32.  Against a bf16 output that is small, about
// 1e-4 of a typical |y| where bf16 rounds by 1.7e-3, and the 16-bit products
// that keep more run at half the rate.)  One MFMA spans exactly one 128-column
// block, so its result starts from zero and folds into the accumulator with one
// FMA per value: the scale of a lane's results is one number (all of a lane's
// batch row, all weight rows of one 128-row block).
//
// MFMA operands (16x16x128): lane l holds A row l % 16 (a weight row) and B
// column l % 16 (a batch row), 32 of the block's columns each; the order of
// the columns within a block is free as long as both operands share it.  D:
// lane l holds weight rows 4 (l / 16) + v, v = 0..3, of batch row l % 16.
#include <iterator>

#include "fp8.h"
#include "internal.h"
#include "topk.h"

namespace q4 {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void lds_void;
// the weights' scales, through the scalar cache (a vector load would join the
// queue of the loads to LDS, and its wait would wait for all of them)
typedef const __attribute__((address_space(4))) float const_float;

__device__ __forceinline__ u32x4 ld16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
}
// Loads straight to LDS, 16 or 4 bytes per lane in lane order from LDS address
// `to` on.  Assembly, because around the builtin the compiler waits for every
// such load before any read of LDS, also of another stage; the kernels below
// wait by themselves (vmcnt, then a barrier).  Nothing is written to registers;
// the compiler puts `to` into m0 (a wait state before its use).  There is no
// memory clobber, which would bring those waits back: that LDS is not read before
// the load has ended, nor written while it is read, rests on the s_waitcnt and
// phase() (a barrier across which nothing moves) around it.
// The descriptor's check covers the sum of a lane's and the scalar offset and
// does not wrap (measured with both past it): what lies behind gives zeros.
typedef int i32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ i32x4 rsrc_words(const void* base, uint32_t bytes) {
    const uint64_t b = reinterpret_cast<uintptr_t>(base);
    return i32x4{(int)(uint32_t)b, (int)(uint32_t)(b >> 32), (int)bytes, kBufferFlags};
}
__device__ __forceinline__ void to_lds16(i32x4 r, uint32_t off, uint32_t soff, uint32_t to) {
    asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds" ::"v"(off), "s"(r), "s"(soff), "{m0}"(to));
}
__device__ __forceinline__ uint32_t lds_address(const uint8_t* p) { return (uint32_t)(uintptr_t)(lds_void*)p; }

__device__ __forceinline__ f32x4 mfma(const u32x4 (&a)[2], const u32x4 (&b)[2]) {
    const i32x8 av = {(int)a[0].x, (int)a[0].y, (int)a[0].z, (int)a[0].w, (int)a[1].x, (int)a[1].y, (int)a[1].z, (int)a[1].w};
    const i32x8 bv = {(int)b[0].x, (int)b[0].y, (int)b[0].z, (int)b[0].w, (int)b[1].x, (int)b[1].y, (int)b[1].z, (int)b[1].w};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

// The residual is added before the one rounding.
__device__ __forceinline__ uint32_t pack2(float lo, float hi) { return (uint32_t)f32_to_bf16(lo) | ((uint32_t)f32_to_bf16(hi) << 16); }
__device__ __forceinline__ bool rows_aligned8(const uint16_t* p, int ld) { return (ld & 3) == 0 && (reinterpret_cast<uintptr_t>(p) & 7) == 0; }

// Columns n .. n + 3 of row m, where every row start is 8-byte aligned; rows are
// ld elements apart.
__device__ __forceinline__ void store4(f32x4 o, const uint16_t* resid, uint16_t* y, int ld, int m, int n) {
    const size_t at = (size_t)m * ld + n;
    if (resid) {
        const uint2 r = *reinterpret_cast<const uint2*>(resid + at);
        o += f32x4{bf16lo(r.x), bf16hi(r.x), bf16lo(r.y), bf16hi(r.y)};
    }
    *reinterpret_cast<uint2*>(y + at) = make_uint2(pack2(o[0], o[1]), pack2(o[2], o[3]));
}

// 16 rows x W columns from (m, n), in a wave's fragments, to rows at any even
// address: through LDS (buf: 16 rows of W + 4 floats, the wave's own), so that
// a store writes consecutive elements.  (Straight from the fragments a store
// touches 16 rows with 8 bytes each; M = 240, N = 16385, K = 2048: 26.8 us so,
// 23 us through LDS.)
template <int W>
struct RowOrder {
    static constexpr int kEach = 16 * W / 64;      // elements of a lane, consecutive ones in consecutive lanes
    static __device__ __forceinline__ int row(int i, int lane) { return W < 64 ? lane / W + 64 / W * i : i / (W / 64); }
    static __device__ __forceinline__ int col(int i, int lane) { return W < 64 ? lane % W : lane + 64 * (i % (W / 64)); }
};
// The residual's elements, all on their way together (one by one, between the
// stores: 3855 x 2311 x 256 48 us, so 26).
template <int W>
__device__ __forceinline__ void load_rows(const uint16_t* resid, int M, int N, int ld, int m, int n, int lane, uint16_t (&e)[RowOrder<W>::kEach]) {
#pragma unroll
    for (int i = 0; i < RowOrder<W>::kEach; ++i) {
        const int r = m + RowOrder<W>::row(i, lane), c = n + RowOrder<W>::col(i, lane);
        e[i] = resid[r < M && c < N ? (size_t)r * ld + c : 0];
    }
}
template <int W>
__device__ __forceinline__ void store_rows(const f32x4* v, int stride, float* buf, bool add, const uint16_t (&e)[RowOrder<W>::kEach],
                                           uint16_t* y, int M, int N, int ld, int m, int n, int lane) {
    constexpr int kPitch = W + 4;
    const int lr = lane & 15, lq = lane >> 4;
#pragma unroll
    for (int t = 0; t < W / 16; ++t) *reinterpret_cast<f32x4*>(buf + lr * kPitch + 16 * t + 4 * lq) = v[t * stride];
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < RowOrder<W>::kEach; ++i) {
        const int r = RowOrder<W>::row(i, lane), c = RowOrder<W>::col(i, lane);
        float o = buf[r * kPitch + c];
        if (add) o += __builtin_bit_cast(float, (uint32_t)e[i] << 16);
        if (m + r < M && n + c < N) y[(size_t)(m + r) * ld + n + c] = f32_to_bf16(o);
    }
    __builtin_amdgcn_wave_barrier();
}

// A wave's TM x TN fragments, rows from m and columns from n on.  lds: free
// for all waves.
template <int TM, int TN>
__device__ __forceinline__ void store_tile(const f32x4* v, uint8_t* lds, const uint16_t* resid, uint16_t* y, int M, int N, int ld, int m, int n,
                                           int wave, int lane) {
    // v[t * TM + u]: columns n + 16 t + 4 (lane / 16) .. + 3 of row m + 16 u + lane % 16
    const int lr = lane & 15, lq = lane >> 4;
    if (rows_aligned8(y, ld) && (!resid || rows_aligned8(resid, ld))) {
#pragma unroll
        for (int u = 0; u < TM; ++u)
#pragma unroll
            for (int t = 0; t < TN; ++t)
                if (m + 16 * u + lr < M && n + 16 * t + 4 * lq < N)
                    store4(v[t * TM + u], resid, y, ld, m + 16 * u + lr, n + 16 * t + 4 * lq);
    } else {
        constexpr int W = 16 * TN;
        float* buf = reinterpret_cast<float*>(lds) + wave * 16 * (W + 4);
        uint16_t e[2][RowOrder<W>::kEach];
        if (resid) load_rows<W>(resid, M, N, ld, m, n, lane, e[0]);
#pragma unroll
        for (int u = 0; u < TM; ++u) {
            if (resid && u + 1 < TM) load_rows<W>(resid, M, N, ld, m + 16 * (u + 1), n, lane, e[(u + 1) & 1]);
            if (m + 16 * u < M) store_rows<W>(v + u, TM, buf, resid != nullptr, e[u & 1], y, M, N, ld, m + 16 * u, n, lane);
        }
    }
}

struct Fp8Group {
    Fp8Args t[kFp8MaxTasks];
    int first[kFp8MaxTasks + 1];      // first workgroup of each task
    int ks[kFp8MaxTasks];             // slices of K of each task
    uint32_t tile0[kFp8MaxTasks];     // of the split tasks: first counter, and
    size_t part0[kFp8MaxTasks];       // byte offset of the first partial tile
    unsigned* cnt;
    uint8_t* part;
    int count, M;
};

// A workgroup's task, its tile within the task and its slice of K.  Workgroups
// go to the eight XCDs in turn; each XCD takes a contiguous range of the tiles,
// so that tiles which share operands share an L2.
struct Where {
    int task, tile, slice;
};
__device__ __forceinline__ Where where(const Fp8Group& p, int block) {
    int t = 0;
    while (t + 1 < p.count && block >= p.first[t + 1]) ++t;
    const int i = block - p.first[t], T = p.first[t + 1] - p.first[t], xcd = i & 7, q8 = T >> 3, r8 = T & 7;
    const int at = xcd * q8 + (xcd < r8 ? xcd : r8) + (i >> 3), ks = p.ks[t];
    return Where{t, at / ks, at % ks};
}

// Batch and weight block of a tile: super-rows of 8 batch blocks, weight block
// by weight block.
struct Block {
    int m, n;
};
__device__ __forceinline__ Block block_of(int tile, int nM, int nN) {
    const int per = 8 * nN, sup = tile / per, within = tile - sup * per;
    const int here = nM - sup * 8 < 8 ? nM - sup * 8 : 8;
    return Block{sup * 8 + within % here, within / here};
}

// Joins the slices of a tile: each of the first `waves` waves stores its NF
// fragments; in the workgroup that arrives last they become the sums over the
// slices, in slice order, and the result is true.
constexpr int kCoherent = 16;    // buffer cache policy sc1: device-coherent, not held in the per-XCD L2
template <int NF>
__device__ __forceinline__ bool join(f32x4 (&v)[NF], const Fp8Group& p, const Where& at, int waves, int wave, int lane, unsigned* s_prev) {
    const int ks = p.ks[at.task];
    const uint32_t slice_bytes = (uint32_t)waves * NF * 1024u;
    const __amdgpu_buffer_rsrc_t r = make_rsrc(p.part + p.part0[at.task] + (size_t)at.tile * ks * slice_bytes, (uint32_t)ks * slice_bytes);
    const uint32_t mine = (uint32_t)(wave * NF * 64 + lane) * 16u;
    if (wave < waves) {
#pragma unroll
        for (int i = 0; i < NF; ++i)
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v[i]), r, (int)(mine + i * 1024u),
                                                   at.slice * (int)slice_bytes, kCoherent);
    }
    if (!arrive_last(p.cnt + (size_t)(p.tile0[at.task] + at.tile) * kCtrWords, ks, threadIdx.x, s_prev)) return false;
#pragma unroll
    for (int i = 0; i < NF; ++i) v[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (wave >= waves) return true;
    for (int s = 0; s < ks; ++s) {
        u32x4 o[NF];
#pragma unroll
        for (int i = 0; i < NF; ++i)
            o[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)(mine + i * 1024u), s * (int)slice_bytes, kCoherent));
#pragma unroll
        for (int i = 0; i < NF; ++i) v[i] += __builtin_bit_cast(f32x4, o[i]);
    }
    return true;
}

// ---------------------------------------------------------------------------
// Few rows: a workgroup of eight waves owns 16 R weight rows and 16 batch rows
// over a slice of K; the waves share the slice's blocks, each loading its
// own fragments straight into registers, and meet in LDS.  Bound by the latency
// of a launch and of one round of loads: 1 x 2048 x 8192 (M x N x K) 7.7 us for
// 16.8 MB, 1 x 2048 x 2048 4.5 us; at 8 x 8192 x 8192 17 us, 3.9 TB/s.
// ---------------------------------------------------------------------------
constexpr int kWaves = 8;

template <int R>
__global__ __launch_bounds__(kWaves * 64) void fp8_rows_kernel(Fp8Group p) {
    constexpr int U = 4;     // blocks whose loads are in flight together
    __shared__ __attribute__((aligned(16))) f32x4 part[kWaves][R][64];
    __shared__ __attribute__((aligned(16))) float turn[kWaves][16 * 20];
    __shared__ unsigned s_prev;
    const int lane = threadIdx.x & 63, lr = lane & 15, lq = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Where at = where(p, blockIdx.x);
    const Fp8Args a = p.t[at.task];
    const Block blk = block_of(at.tile, (p.M + 15) / 16, (a.N + 16 * R - 1) / (16 * R));
    const int n0 = blk.n * 16 * R, m0 = blk.m * 16;
    const int K = a.K, G = (K + 127) >> 7;
    const int rows_n = a.N - n0 < 16 * R ? a.N - n0 : 16 * R, rows_m = p.M - m0 < 16 ? p.M - m0 : 16;
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(a.w + (size_t)n0 * K, (uint32_t)rows_n * (uint32_t)K);
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x + (size_t)m0 * K, (uint32_t)rows_m * (uint32_t)K);
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(a.xs + (size_t)m0 * G, (uint32_t)rows_m * (uint32_t)G * 4u);
    const const_float* wsrow = (const const_float*)(uintptr_t)(a.ws + (size_t)(n0 >> 7) * G);      // (16 R divides 128: one row)

    f32x4 acc[R];
#pragma unroll
    for (int t = 0; t < R; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};

    const int ks = p.ks[at.task];
    const int b0 = G * at.slice / ks, b1 = G * (at.slice + 1) / ks;
    const int g0 = b0 + (b1 - b0) * wave / kWaves, g1 = b0 + (b1 - b0) * (wave + 1) / kWaves;
    for (int gu = g0; gu < g1; gu += U) {
        u32x4 wf[U][R][2], xf[U][2];
        float f[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            // a row past the matrix, a column past K and a block past the
            // wave's last read as zero
            const int g = gu + j;
            const bool in = g < g1;
            const uint32_t k = 128u * g + 16u * lq;     // (chunks lq and 4 + lq: 64 consecutive bytes of a row per load)
#pragma unroll
            for (int t = 0; t < R; ++t)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    wf[j][t][c] = ld16(rw, in && k + 64 * c < (uint32_t)K ? (uint32_t)(16 * t + lr) * K + k + 64 * c : 0xFFFFFFF0u);
#pragma unroll
            for (int c = 0; c < 2; ++c)
                xf[j][c] = ld16(rx, in && k + 64 * c < (uint32_t)K ? (uint32_t)lr * K + k + 64 * c : 0xFFFFFFF0u);
            f[j] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, in ? (lr * G + g) * 4 : (int)0xFFFFFFF0u, 0, 0));
        }
        __builtin_amdgcn_sched_barrier(0);      // every load is on its way before the first wait
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const float sw = wsrow[gu + j < g1 ? gu + j : g1 - 1], fs = f[j] * (gu + j < g1 ? sw : 0.0f);      // (sw may be infinite)
#pragma unroll
            for (int t = 0; t < R; ++t) {
                const f32x4 d = mfma(wf[j][t], xf[j]);
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[t][v] = __builtin_fmaf(fs, d[v], acc[t][v]);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < R; ++t) part[wave][t][lane] = acc[t];
    __syncthreads();
    f32x4 v[1] = {part[0][wave < R ? wave : 0][lane]};
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v[0] += part[w][wave < R ? wave : 0][lane];
    if (ks > 1 && !join(v, p, at, R, wave, lane, &s_prev)) return;
    if (wave < R) store_tile<1, 1>(v, reinterpret_cast<uint8_t*>(turn), a.resid, a.y, p.M, a.N, a.ld, m0, n0 + 16 * wave, wave, lane);
}

// ---------------------------------------------------------------------------
// Many rows: workgroup tiles of BM batch rows x BN weight rows over all of K,
// WM x WN waves, each BM / WM x BN / WN.  Per 128-column block the tile's rows
// go straight from memory to LDS (16 bytes per lane, no registers), into one
// of two stages: while the waves compute a block, the next one is on its way.
// Bound by the matrix cores' power: 8192 x 8192 x 8192 456 us a call in a stream of
// calls, 2410 TFLOP/s (the
// card lowers its clock to about 1.95 GHz under it; the matrix cores are then
// busy for 60 to 65 % of the cycles, the rest being the folds and the reads of
// LDS that do not overlap them, and the last round's tail).
//
// LDS holds rows of 128 bytes; 16-byte chunk c of row r sits at chunk
// c ^ (r / 2 % 8), so that one chunk of 16 consecutive rows (a quarter of a
// fragment read) covers the 64 banks once: 4 cycles per read, where chunk
// c ^ (r % 8) takes 8.  The swizzle is on the memory side of the load: LDS is
// written in lane order.
// ---------------------------------------------------------------------------
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

    const Where where_ = where(p, blockIdx.x);
    const Fp8Args a = p.t[where_.task];
    const Block blk = block_of(where_.tile, (p.M + BM - 1) / BM, (a.N + BN - 1) / BN);
    const int m0 = blk.m * BM, n0 = blk.n * BN;
    const int K = a.K, G = (K + 127) >> 7;
    const int rows_m = p.M - m0 < BM ? p.M - m0 : BM, rows_n = a.N - n0 < BN ? a.N - n0 : BN;
    const i32x4 rx = rsrc_words(a.x + (size_t)m0 * K, (uint32_t)rows_m * (uint32_t)K);
    const i32x4 rw = rsrc_words(a.w + (size_t)n0 * K, (uint32_t)rows_n * (uint32_t)K);
    const i32x4 rs = rsrc_words(a.xs + (size_t)m0 * G, (uint32_t)rows_m * (uint32_t)G * 4u);
    const uint32_t base = lds_address(lds);
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
        to_lds16(j < kXLoads ? rx : rw, o, (uint32_t)(i * kW * 8 * K + g * 128),
                 base + (j < kXLoads ? L::kX + (g & 1) * L::kXStage : L::kW + (g & 1) * L::kWStage) + (wave + kW * i) * 1024);
    };
    // Scales of blocks 4 q .. 4 q + 3: a row's scales are adjacent, so four
    // cost the lines of one (every block alone: 20 % of the whole kernel).  The
    // last four end at G.
    auto quad_first = [&](int q) { return 4 * q + 4 <= G ? 4 * q : G - 4; };
    auto scales = [&](int g) {
        if ((g & 3) || g >= G || wave >= BM / 64) return;
        to_lds16(rs, soff, (uint32_t)quad_first(g >> 2) * 4, base + L::kS + ((g >> 2) & 1) * L::kQuad + wave * 1024);
    };
    auto load = [&](int g) {
        scales(g);
        const uint32_t o = at(g);
#pragma unroll
        for (int j = 0; j < kLoads; ++j) piece(g, o, j);
    };

    f32x4 acc[TN * TM];
#pragma unroll
    for (int i = 0; i < TN * TM; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};

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
                        acc[o][v] = __builtin_fmaf(f[o % TM], d[o % (kAhead + 1)][v], acc[o][v]);
                }
                if (i < kN) __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                if (i >= kAhead) __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
                if (kSecond && i < kN && i % (kN / kLoads) == 0) {
                    piece(g + 2, o, i / (kN / kLoads));
                }
            }
            // (the folds stay in this block: sunk into a later one they would cost the overlap)
#pragma unroll
            for (int i = 0; i < TN * TM; ++i) asm volatile("" : "+v"(acc[i]));
            __builtin_amdgcn_s_setprio(0);
            if (!kSecond) __builtin_amdgcn_s_waitcnt(0x0F70);     // vmcnt(0)
            if (!kSecond || g + 1 < G) phase();
        }
    };
    if (wave < kW / 2) walk(false);
    else walk(true);
    __builtin_amdgcn_s_waitcnt(0x0F70);      // no load to LDS outlives the workgroup

    phase();                                 // nor reaches LDS while the epilogue uses it
    store_tile<TM, TN>(acc, lds, a.resid, a.y, p.M, a.N, a.ld, m0 + wm * (BM / WM), n0 + wn * (BN / WN), wave, lane);
}

template <int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 2) void fp8_tile_kernel(Fp8Group p) {
    __shared__ __attribute__((aligned(16))) uint8_t lds[TileLds<BM, BN>::kBytes];
    tile<BM, BN, WM, WN>(p, lds);
}

// ---------------------------------------------------------------------------
// In between: tiles of BM x BN, S stages in LDS, one barrier per block: block
// g + S - 1 goes on its way when the waves have left block g - 1, whose stage
// it takes.  Several workgroups share a CU and fill each other's waits; K may
// be split over workgroups where the tiles alone are too few.  Bound by the
// weights' bytes and the fill of the stages: 48 x (2048, 512, 512, 8192, 8192) x
// 2048 12.8 us, 3.3 TB/s; 240 x 16385 x 2048 22 us; 240 x 2048 x 8192 14 us;
// 2048 x 2048 x 2048 16.5 us, 1040 TFLOP/s.
// ---------------------------------------------------------------------------
template <int BM, int BN, int S>
struct MidLds {
    static constexpr int kXStage = BM * 128, kWStage = BN * 128;
    static constexpr int kX = 0, kW = S * kXStage, kS = kW + S * kWStage;
    static constexpr int kScaleWaves = (BM + 63) / 64;
    static constexpr int kQuad = kScaleWaves * 1024, kQuads = (S + 2) / 4 + 1, kBytes = kS + kQuads * kQuad;    // scales of 4 blocks per row
};

// ANY: also takes tasks of fewer than four blocks, whose rows' scales do not
// fill a 16-byte load; they go to registers before the first block.
template <int BM, int BN, int WM, int WN, int S, bool ANY>
__device__ __forceinline__ void mid(const Fp8Group& p, uint8_t* lds, unsigned* s_prev) {
    using L = MidLds<BM, BN, S>;
    constexpr int kW = WM * WN, TM = BM / WM / 16, TN = BN / WN / 16;
    constexpr int kXLoads = BM / 8 / kW, kWLoads = BN / 8 / kW, kLoads = kXLoads + kWLoads;
    static_assert(BM % (8 * kW) == 0 && BN % (8 * kW) == 0 && 128 % (BN / WN) == 0 && L::kScaleWaves <= kW && kW % 2 == 0 &&
                      S >= 2,
                  "tile");
    const int lane = threadIdx.x & 63, lr = lane & 15, lq = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave % WM, wn = wave / WM;
    const Where at = where(p, blockIdx.x);
    const Fp8Args a = p.t[at.task];
    const Block blk = block_of(at.tile, (p.M + BM - 1) / BM, (a.N + BN - 1) / BN);
    const int m0 = blk.m * BM, n0 = blk.n * BN;
    const int K = a.K, G = (K + 127) >> 7;
    const int rows_m = p.M - m0 < BM ? p.M - m0 : BM, rows_n = a.N - n0 < BN ? a.N - n0 : BN;
    const i32x4 rx = rsrc_words(a.x + (size_t)m0 * K, (uint32_t)rows_m * (uint32_t)K);
    const i32x4 rw = rsrc_words(a.w + (size_t)n0 * K, (uint32_t)rows_n * (uint32_t)K);
    const i32x4 rs = rsrc_words(a.xs + (size_t)m0 * G, (uint32_t)rows_m * (uint32_t)G * 4u);
    const uint32_t base = lds_address(lds);
    const int nb = (n0 + wn * (BN / WN)) >> 7;
    const const_float* wsrow = (const const_float*)(uintptr_t)(a.ws + (size_t)(nb * 128 < a.N ? nb : 0) * G);

    // LDS layout, swizzle and zero fill as in the tile kernel
    const uint32_t chunk = (uint32_t)((lane & 7) ^ (lane >> 4) ^ ((wave & 1) << 2)) * 16u;
    const uint32_t off = (uint32_t)(8 * wave + (lane >> 3)) * (uint32_t)K + chunk;
    const uint32_t soff = (uint32_t)(64 * wave + lane) * (uint32_t)G * 4u;
    const bool tail = K & 127;
    const int ks = p.ks[at.task];
    const int g0 = G * at.slice / ks, g1 = G * (at.slice + 1) / ks;      // (a slice has at least four blocks)
    auto quad_first = [&](int q) { return 4 * q + 4 <= g1 - g0 ? g0 + 4 * q : g1 - 4; };
    const bool few = ANY && G < 4;
    float fs[3][TM];
    if (few) {
        const __amdgpu_buffer_rsrc_t r = make_rsrc(a.xs + (size_t)m0 * G, (uint32_t)rows_m * (uint32_t)G * 4u);
#pragma unroll
        for (int i = 0; i < 3; ++i)
#pragma unroll
            for (int u = 0; u < TM; ++u)
                fs[i][u] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                                                         r, i < G ? ((wm * (BM / WM) + 16 * u + lr) * G + i) * 4 : (int)0xFFFFFFF0u, 0, 0));
    }
    // block g0 + i into stage i % S; always kLoads loads, and those for the
    // scales before them, so that vmcnt counts blocks
    auto load = [&](int i, int stage) {
        const int g = g0 + i;
        if (!few && !(i & 3) && g < g1 && wave < L::kScaleWaves)
            to_lds16(rs, soff, (uint32_t)quad_first(i >> 2) * 4, base + L::kS + (i >> 2) % L::kQuads * L::kQuad + wave * 1024);
        const uint32_t o = g >= g1 || (tail && g == G - 1 && 128u * g + chunk >= (uint32_t)K) ? 0xFFFF0000u : off;
#pragma unroll
        for (int j = 0; j < kXLoads; ++j)
            to_lds16(rx, o, (uint32_t)(j * kW * 8 * K + g * 128), base + L::kX + stage * L::kXStage + (wave + kW * j) * 1024);
#pragma unroll
        for (int j = 0; j < kWLoads; ++j)
            to_lds16(rw, o, (uint32_t)(j * kW * 8 * K + g * 128), base + L::kW + stage * L::kWStage + (wave + kW * j) * 1024);
    };

    f32x4 acc[TN * TM];
#pragma unroll
    for (int i = 0; i < TN * TM; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int c0 = ((2 * lq) ^ (lr >> 1)) * 16, c1 = ((2 * lq + 1) ^ (lr >> 1)) * 16;
    const int xrow = L::kX + (wm * (BM / WM) + lr) * 128, wrow = L::kW + (wn * (BN / WN) + lr) * 128;
    const int srow = L::kS + (wm * (BM / WM) + lr) * 16;
#pragma unroll
    for (int i = 0; i < S - 1; ++i) load(i, i);
    float next = wsrow[g0];
    int stage = 0, ahead = S - 1;
    for (int i = 0; i < g1 - g0; ++i) {
        constexpr int kBehind = (S - 2) * kLoads;     // loads of the blocks behind block i
        __builtin_amdgcn_s_waitcnt(0x0F70 | (kBehind & 15) | ((kBehind >> 4) << 14));
        phase();
        const float s = next;
        if (g0 + i + 1 < g1) next = wsrow[g0 + i + 1];
        const uint8_t* sc = lds + srow + (i >> 2) % L::kQuads * L::kQuad + (few ? 0 : g0 + i - quad_first(i >> 2)) * 4;
        u32x4 xf[TM][2], wf[TN][2];
        float f[TM];
#pragma unroll
        for (int u = 0; u < TM; ++u) {
            xf[u][0] = *reinterpret_cast<const u32x4*>(lds + xrow + stage * L::kXStage + u * 2048 + c0);
            xf[u][1] = *reinterpret_cast<const u32x4*>(lds + xrow + stage * L::kXStage + u * 2048 + c1);
            f[u] = *reinterpret_cast<const float*>(sc + u * 256);
            if (few) f[u] = i == 0 ? fs[0][u] : i == 1 ? fs[1][u] : fs[2][u];
        }
#pragma unroll
        for (int t = 0; t < TN; ++t) {
            wf[t][0] = *reinterpret_cast<const u32x4*>(lds + wrow + stage * L::kWStage + t * 2048 + c0);
            wf[t][1] = *reinterpret_cast<const u32x4*>(lds + wrow + stage * L::kWStage + t * 2048 + c1);
        }
        __builtin_amdgcn_sched_barrier(0);      // the reads are asked for before the next loads
        load(i + S - 1, ahead);
        __builtin_amdgcn_sched_barrier(0);      // and none of these sinks behind the products
#pragma unroll
        for (int u = 0; u < TM; ++u) f[u] *= s;
#pragma unroll
        for (int t = 0; t < TN; ++t) {
            f32x4 d[TM];
#pragma unroll
            for (int u = 0; u < TM; ++u) d[u] = mfma(wf[t], xf[u]);
#pragma unroll
            for (int u = 0; u < TM; ++u)
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[t * TM + u][v] = __builtin_fmaf(f[u], d[u][v], acc[t * TM + u][v]);
        }
        stage = stage + 1 < S ? stage + 1 : 0;
        ahead = ahead + 1 < S ? ahead + 1 : 0;
        // this wave's reads of the stage are done before the next barrier lets
        // it be overwritten
        __builtin_amdgcn_s_waitcnt(0xC07F);
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);      // no load to LDS outlives the workgroup
    if (ks > 1 && !join(acc, p, at, kW, wave, lane, s_prev)) return;

    phase();
    store_tile<TM, TN>(acc, lds, a.resid, a.y, p.M, a.N, a.ld, m0 + wm * (BM / WM), n0 + wn * (BN / WN), wave, lane);
}

template <int BM, int BN, int WM, int WN, int S, bool ANY>
__global__ __launch_bounds__(64 * WM * WN, 2) void fp8_mid_kernel(Fp8Group p) {
    __shared__ __attribute__((aligned(16))) uint8_t lds[MidLds<BM, BN, S>::kBytes];
    __shared__ unsigned s_prev;
    mid<BM, BN, WM, WN, S, ANY>(p, lds, &s_prev);
}

// ---------------------------------------------------------------------------
// the plan: which tile, and how many slices of K
//
// The time of a launch is modelled as
//     fixed + rounds of resident workgroups, each steps x (time of one block)
// with the per-block times below, measured with 1, 2, ... workgroups on every
// CU (us; M = 512 .. 4096, K = 2048 and 8192), never less than the bytes at the
// rate such launches reach, plus the hand-over of a split.  Small tiles fill
// the CUs early, large ones move fewer bytes per product: at 240 x 8192 x 2048
// 64 x 64 takes 11.4 us and 256 x 128 21 us, at 4096 x 2048 x 8192 151 and 81.
// The model puts 240 x 16384 x 2048 at 16.6 us and 240 x 16385 x 2048 at 22.4, calls
// in a stream take 17.1 and 22.3; M = 512, N = 8249 at 58.9 us (K = 7904), measured 59.7.
// ---------------------------------------------------------------------------
constexpr int kMaxResident = 4;
struct Kind {
    int bm, bn;             // batch rows and weight rows of a workgroup
    int waves, frags;       // waves that hand fragments over when K is split, fragments of each
    int resident;           // workgroups that share a CU
    float fixed, block[kMaxResident];     // us; block[j]: with j + 1 workgroups on a CU
    int min_blocks;         // of a slice
    hipError_t (*launch)(const Fp8Group&, dim3, hipStream_t);
};

template <int R>
hipError_t go_rows(const Fp8Group& p, dim3 g, hipStream_t s) {
    return launch_kernel(fp8_rows_kernel<R>, g, dim3(kWaves * 64), 0, s, p);
}
template <int BM, int BN, int WM, int WN, int S, bool ANY>
hipError_t go_mid(const Fp8Group& p, dim3 g, hipStream_t s) {
    return launch_kernel(fp8_mid_kernel<BM, BN, WM, WN, S, ANY>, g, dim3(64 * WM * WN), 0, s, p);
}
template <int BM, int BN, int WM, int WN>
hipError_t go_tile(const Fp8Group& p, dim3 g, hipStream_t s) {
    return launch_kernel(fp8_tile_kernel<BM, BN, WM, WN>, g, dim3(64 * WM * WN), 0, s, p);
}
template <int BM, int BN, int WM, int WN, int S, bool ANY = false>
constexpr Kind mid_kind(int resident, float fixed, float b1, float b2 = 0, float b3 = 0, float b4 = 0) {
    return Kind{BM, BN, WM * WN, (BM / WM / 16) * (BN / WN / 16), resident, fixed, {b1, b2, b3, b4}, 4, go_mid<BM, BN, WM, WN, S, ANY>};
}

// few rows (no model: see plan_of)
const Kind kRows16 = {16, 16, 1, 1, 1, 0, {}, 1, go_rows<1>};
const Kind kRows32 = {16, 32, 2, 1, 1, 0, {}, 1, go_rows<2>};
const Kind kTiles[] = {
    mid_kind<32, 32, 2, 2, 4>(4, 3.5f, 0.20f, 0.30f, 0.42f, 0.55f),
    mid_kind<32, 64, 1, 4, 4>(3, 3.5f, 0.235f, 0.33f, 0.50f),
    mid_kind<64, 32, 2, 2, 4>(3, 3.5f, 0.25f, 0.335f, 0.52f),
    mid_kind<64, 64, 2, 2, 4>(2, 4.0f, 0.315f, 0.40f),
    mid_kind<64, 128, 2, 2, 3>(2, 4.0f, 0.48f, 0.79f),
    mid_kind<128, 64, 2, 2, 2>(3, 3.0f, 0.69f, 1.03f, 1.21f),
    mid_kind<128, 128, 2, 2, 2>(2, 3.0f, 1.106f, 1.243f),
    mid_kind<256, 128, 4, 2, 3>(1, 6.5f, 1.13f),
    {256, 256, 8, 0, 1, 14.0f, {1.604f}, 4, go_tile<256, 256, 4, 2>},
};
// where a task has fewer than four blocks (4096 x 4096 x 384: 21 us; loaded
// straight into registers, as few rows are, 106 us)
const Kind kShortTiles[] = {
    mid_kind<32, 64, 1, 4, 4, true>(3, 3.5f, 0.235f, 0.33f, 0.50f),
    mid_kind<64, 64, 2, 2, 4, true>(2, 4.0f, 0.315f, 0.40f),
    mid_kind<128, 128, 2, 2, 2, true>(2, 3.0f, 1.106f, 1.243f),
};
constexpr int kCUs = 256;
constexpr int kMostSlices = 16;

struct Plan {
    const Kind* kind;
    double time;            // modelled, us (0: not)
    int ks[kFp8MaxTasks];
    size_t ws;
};

int blocks_of(int K) { return (K + 127) / 128; }
long tiles_of(const Kind& k, int N, int M) { return (long)((N + k.bn - 1) / k.bn) * ((M + k.bm - 1) / k.bm); }

// Workspace bytes of a plan's splits (0: none), or SIZE_MAX where its tiles
// have too few counters.
size_t plan_ws(const Kind& k, const long* tiles, int count, const int* ks) {
    size_t part = 0, split = 0;
    for (int i = 0; i < count; ++i)
        if (ks[i] > 1) {
            part += (size_t)tiles[i] * ks[i] * k.waves * k.frags * 1024;
            split += tiles[i];
        }
    if (!part) return 0;
    return split * kCtrStride > kWsCounterBytes ? SIZE_MAX : kWsCounterBytes + part;
}

// Modelled time (us) of kind k with ks slices of K per task (G blocks each) and
// ws bytes of workspace; bytes: of all operands and outputs.
double plan_time(const Kind& k, const long* tiles, const int* G, int count, const int* ks, size_t ws, double bytes) {
    long groups = 0, steps = 0, work = 0;
    for (int i = 0; i < count; ++i) {
        const long s = (G[i] + ks[i] - 1) / ks[i], n = tiles[i] * ks[i];
        groups += n;
        work += n * s;
        steps = s > steps ? s : steps;
    }
    // whole rounds of resident workgroups, then the rest; workgroups of
    // unequal length even out
    const int r = k.resident;
    const double mean = (double)work / groups;
    const long full = groups / (kCUs * r), rest = groups - full * kCUs * r;
    double run = full * mean * k.block[r - 1];
    if (rest) run += (full ? mean : steps) * k.block[(rest + kCUs - 1) / kCUs - 1];
    // a further round fills its stages and stores its tiles anew
    run += (full + (rest > 0) - 1) * (r == 1 ? k.fixed - 3.5 : 2.0);
    const double memory = bytes / 4.6e6;
    const double join = ws ? 1.8 + 2.0 * (double)(ws - kWsCounterBytes) / 8e6 : 0.0;
    return k.fixed + (run > memory ? run : memory) + join;
}

Plan plan_of(const Fp8Args* t, int count, int M, size_t ws_bytes) {
    Plan p{};
    int G[kFp8MaxTasks], least = 1 << 30;
    long tiles[kFp8MaxTasks], n = 0;
    double bytes = 0;
    for (int i = 0; i < count; ++i) {
        p.ks[i] = 1;
        n += t[i].N;
        G[i] = blocks_of(t[i].K);
        least = G[i] < least ? G[i] : least;
        bytes += (double)t[i].N * t[i].K + (double)M * t[i].K + 2.0 * M * t[i].N;
    }
    // Up to one batch tile, and weights that give each CU no more than one such
    // workgroup (or long rows): the waves load for themselves, with no stages
    // to fill first (M = 1: N = K = 2048 4.5 us, in tiles 6.2; 8 x 8192 x 8192
    // 15.9 and 19.0; but N = 16385, K = 2048 11.0 and 9.0).
    if (M <= 16 && (n <= 32 * kCUs || least >= 32)) {
        p.kind = n <= 16 * kCUs || n > 32 * kCUs ? &kRows16 : &kRows32;
        if (n <= 8 * kCUs && least >= 32) {      // half the CUs: two slices (2048 x 8192: 7.2 us, unsplit 7.8)
            for (int i = 0; i < count; ++i) {
                p.ks[i] = 2;
                tiles[i] = tiles_of(*p.kind, t[i].N, M);
            }
            p.ws = plan_ws(*p.kind, tiles, count, p.ks);
            if (p.ws > ws_bytes) {
                for (int i = 0; i < count; ++i) p.ks[i] = 1;
                p.ws = 0;
            }
        }
        return p;
    }
    if (least < 4 && M <= 16) {
        p.kind = &kRows16;
        return p;
    }
    const Kind *kinds = least < 4 ? kShortTiles : kTiles, *end = least < 4 ? std::end(kShortTiles) : std::end(kTiles);
    double best = 0;
    for (; kinds != end; ++kinds) {
        const Kind& k = *kinds;
        int ks[kFp8MaxTasks];
        for (int i = 0; i < count; ++i) {
            ks[i] = 1;
            tiles[i] = tiles_of(k, t[i].N, M);
        }
        for (bool more = true; more;) {
            const size_t ws = plan_ws(k, tiles, count, ks);
            if (ws == SIZE_MAX) break;
            if (ws <= ws_bytes) {
                const double time = plan_time(k, tiles, G, count, ks, ws, bytes);
                if (!p.kind || time < best) {
                    p.time = best = time;
                    p.kind = &k;
                    p.ws = ws;
                    for (int i = 0; i < count; ++i) p.ks[i] = ks[i];
                }
            }
            // twice the slices, where a task's stay long enough
            more = false;
            for (int i = 0; k.frags && i < count; ++i)
                if (ks[i] <= kMostSlices / 2 && G[i] / (2 * ks[i]) >= k.min_blocks) {
                    ks[i] *= 2;
                    more = true;
                }
        }
    }
    return p;
}

constexpr int kCut = 256;      // weight rows of the largest tile
// A split's workspace is at most this (a plan that wants more is not made).
constexpr size_t kMostWs = 48u << 20;

// A grid holds fewer than 2^32 threads; eight tasks of few rows can have more
// (one has at most 2^20 workgroups of 512, and more rows have larger tiles:
// outputs of that many would not fit in memory).
bool one_grid(const Plan& p, const Fp8Args* t, int count, int M) {
    long groups = 0;
    for (int i = 0; i < count; ++i) groups += tiles_of(*p.kind, t[i].N, M) * p.ks[i];
    return count == 1 || groups < 1L << 23;
}

// Decides the launches of a call that may use ws_bytes of workspace and hands
// them to f(plan, tasks, count), in order, until one fails.  Everything that
// asks how a call runs (the launch, the workspace query) asks here.  A plan is
// the best of those whose splits fit, so any workspace of at least the largest
// plan.ws that kMostWs gives has the same launches as kMostWs.
template <typename F>
hipError_t each_launch(const Fp8Args* t, int count, int M, size_t ws_bytes, F&& f) {
    if (ws_bytes > kMostWs) ws_bytes = kMostWs;
    const Plan plan = plan_of(t, count, M, ws_bytes);
    // Weight rows behind the last whole 256 in a launch of their own, where the
    // model has both done sooner by more than a launch costs the host: a last
    // round that is nearly empty is left out (4096 x 4097 x 4096: 125 us in one,
    // 85 in two; 8192 x 8193 x 8192 511 and 460; but 4096 x 6000 x 4096 123 in
    // one).  Only where there are microseconds to plan in.
    if (count == 1 && plan.time > 40 && t->N > kCut && t->N % kCut) {
        Fp8Args whole = *t, rest = *t;
        whole.N = t->N - t->N % kCut;
        rest.N = t->N % kCut;
        rest.w += (size_t)whole.N * t->K;
        rest.ws += (size_t)(whole.N / kFp8Block) * blocks_of(t->K);
        if (rest.resid) rest.resid += whole.N;
        rest.y += whole.N;
        const Plan first = plan_of(&whole, 1, M, ws_bytes), second = plan_of(&rest, 1, M, ws_bytes);
        if (first.time + second.time + 3 < plan.time) {
            const hipError_t e = f(first, &whole, 1);
            return e == hipSuccess ? f(second, &rest, 1) : e;
        }
    }
    if (one_grid(plan, t, count, M)) return f(plan, t, count);
    for (int i = 0; i < count; ++i) {
        const hipError_t e = each_launch(t + i, 1, M, ws_bytes, f);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_plan(const Plan& plan, const Fp8Args* tasks, int count, int M, void* ws, hipStream_t s) {
    const Kind& k = *plan.kind;
    Fp8Group p{};
    p.count = count;
    p.M = M;
    p.cnt = static_cast<unsigned*>(plan.ws ? ws : nullptr);
    p.part = plan.ws ? static_cast<uint8_t*>(ws) + kWsCounterBytes : nullptr;
    uint32_t tile = 0;
    size_t part = 0;
    for (int i = 0; i < count; ++i) {
        const int tiles = (int)tiles_of(k, tasks[i].N, M);
        p.t[i] = tasks[i];
        p.ks[i] = plan.ks[i];
        p.first[i + 1] = p.first[i] + tiles * plan.ks[i];
        if (plan.ks[i] > 1) {
            p.tile0[i] = tile;
            p.part0[i] = part;
            tile += (uint32_t)tiles;
            part += (size_t)tiles * plan.ks[i] * k.waves * k.frags * 1024;
        }
    }
    return k.launch(p, dim3(p.first[count]), s);
}

}  // namespace

size_t fp8_gemm_ws_bytes(const Fp8Args* tasks, int count, int M) {
    size_t most = 0;
    (void)each_launch(tasks, count, M, kMostWs, [&](const Plan& p, const Fp8Args*, int) {
        most = p.ws > most ? p.ws : most;
        return hipSuccess;
    });
    return most;
}

hipError_t launch_fp8_gemm(const Fp8Args* tasks, int count, int M, void* ws, size_t ws_bytes, hipStream_t s) {
    return each_launch(tasks, count, M, ws ? ws_bytes : 0,
                       [&](const Plan& p, const Fp8Args* t, int n) { return launch_plan(p, t, n, M, ws, s); });
}

int fp8_gemm_launches(const Fp8Args* tasks, int count, int M, size_t ws_bytes, fp8b128_launch* out, int most) {
    int n = 0;
    (void)each_launch(tasks, count, M, ws_bytes, [&](const Plan& p, const Fp8Args* t, int c) {
        if (n < most) {
            fp8b128_launch& l = out[n];
            l = fp8b128_launch{};
            l.tile_m = p.kind->bm;
            l.tile_n = p.kind->bn;
            l.count = c;
            l.workspace_bytes = p.ws;
            for (int i = 0; i < c; ++i) {
                l.N[i] = t[i].N;
                l.slices[i] = p.ks[i];
            }
        }
        ++n;
        return hipSuccess;
    });
    return n;
}

}  // namespace q4
