// Attention of a sequence's new tokens over a paged cache.
//
//     y[b, i, head] = sum_j p_j v_j,  p = softmax over seen keys j of scale * q[b, i, head] . k_j
//
// Row i of a sequence's n new tokens sees keys j < length - n + i + 1, of
// those the last `window` (0: all), and of those the ones whose page is in the
// cache.  Rows that see nothing are 0.
//
// Bound by memory: every key and value is read once for all heads and rows
// that share it, 16 rows (heads of the group x new tokens) to a matrix
// instruction, whose other rows are idle where there are fewer; the matrix
// cores have ten times the rate that this needs, so nothing is gained by
// filling them.
//
// Nothing passes through LDS on the way: a wave takes 32 keys at a time
// straight into registers, as S^T = K Q^T and O^T = V^T P^T (16x16x32).
//   K, 16 bytes of a row per lane, is the first product's operand as it lies:
//     lane (g, c) = (lane / 16, lane % 16) holds key 8 (c / 4) + 4 t + c % 4 of
//     the 32, t the tile, and D / 4 of its columns in pieces;
//   its result leaves lane (g, c) with row c's scores of keys 8 g .. 8 g + 7,
//     which is how the second product wants P^T: the softmax needs two lane
//     moves for the maximum and none for P;
//   V: lane (g, c) loads D / 16 columns of keys 8 g .. 8 g + 7, which after a
//     transposition inside the lane (v_perm) is V^T's operand, the column
//     e + (D / 16) c being row c of tile e.
// A wave's next 32 keys are in flight while it works on the present ones (16
// KB a wave, 128 KB a CU), the page numbers one step ahead of them.
//
// The work is the list of all (sequence, key head, rows) in blocks of 128
// keys; every workgroup takes an equal, contiguous part of it, whatever the
// lengths are: they are only known on the device, and ragged ones are as
// balanced as equal ones.  A part of a sequence leaves its maxima, sums and
// fp32 outputs in the workspace, and the workgroup that arrives last joins
// them, in order, so that results do not depend on timing.
#include "attention.h"
#include "attn_common.h"
#include "internal.h"
#include "topk.h"

namespace q4 {

namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kTile = 32;                    // keys of a wave's step
constexpr int kBlock = kTile * kWaves;       // keys of a unit of work
constexpr int kMaxWgs = (int)(kWsCounterBytes / kCtrStride);
constexpr int kCoherent = 16;                // buffer cache policy sc1: device-coherent, not held in the per-XCD L2

struct DecodeParams {
    DecodeArgs a;
    Cache cache;
    float* part;
    unsigned* cnt;
    float c;             // scale * log2 e
    int G, R, Z, W;      // heads that share keys, rows of a key head, their chunks, workgroups
};

// keys that rows hold nothing for are read from here
__device__ u32x4 kNothing[128];

struct Span {
    int n, len, lo, hi, blocks;   // new tokens, keys; the keys [lo, hi) that rows see, lo at a block
};
__device__ __forceinline__ Span span_of(const DecodeParams& p, int b) {
    Span s;
    const int most = p.a.width << p.cache.shift;
    s.len = min(max(p.a.lengths[b], 0), most);
    s.n = p.a.n_new ? min(max(p.a.n_new[b], 0), p.a.T) : p.a.T;
    s.hi = s.n ? s.len : 0;
    s.lo = p.a.window ? max(0, s.len - s.n + 1 - p.a.window) & ~(kBlock - 1) : 0;
    s.blocks = max(1, (s.hi - s.lo + kBlock - 1) / kBlock);
    return s;
}

template <int SEL>
__device__ __forceinline__ uint32_t bf16x2_of_e4m3(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, SEL));
}
__device__ __forceinline__ bf16x8 operand(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __builtin_bit_cast(bf16x8, u32x4{a, b, c, d});
}

// Where this lane's rows of 32 keys lie.
struct Rows {
    int page, page_v;     // of keys 8 (c / 4) .. + 7, and 8 g .. + 7; -1: none
    int k0;
};

template <int D, bool kE4m3>
struct Keys {
    static constexpr int kRow = kE4m3 ? D : 2 * D;    // bytes of a row
    static constexpr int kLoads = kRow / 64;          // 16-byte loads per lane and row
    u32x4 k[2][kLoads];
    f32x4 scale[2];       // of keys 8 g + 4 t ..

    __device__ __forceinline__ void load(const DecodeParams& p, const Rows& at, int head, int lane) {
        const int g = lane >> 4, c = lane & 15, shift = p.cache.shift, in_page = (1 << shift) - 1;
        const long row = (((long)at.page * p.a.Hk + head) << shift) + ((at.k0 + 8 * (c >> 2)) & in_page);
        const uint8_t* from = (at.page >= 0 ? p.cache.k + row * kRow : reinterpret_cast<const uint8_t*>(kNothing)) + (c & 3) * kRow + 16 * g;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int s = 0; s < kLoads; ++s)
                k[t][s] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(from + 4 * t * kRow + 64 * s));
        if constexpr (kE4m3) {
            const long first = (((long)at.page_v * p.a.Hk + head) << shift) + ((at.k0 + 8 * g) & in_page);
            const f32x4* of = reinterpret_cast<const f32x4*>(at.page_v >= 0 ? p.cache.ks + first : reinterpret_cast<const float*>(kNothing));
            scale[0] = of[0], scale[1] = of[1];
        }
    }
};

template <int D, bool kE4m3>
struct Values {
    static constexpr int kRow = kE4m3 ? D : 2 * D;
    static constexpr int kWords = kRow / 64;          // dwords of a row per lane
    uint32_t v[8][kWords];
    f32x4 scale[2];

    __device__ __forceinline__ void load(const DecodeParams& p, const Rows& at, int head, int lane) {
        const int g = lane >> 4, c = lane & 15, shift = p.cache.shift, in_page = (1 << shift) - 1;
        const long row = (((long)at.page_v * p.a.Hk + head) << shift) + ((at.k0 + 8 * g) & in_page);
        const uint8_t* from = (at.page_v >= 0 ? p.cache.v + row * kRow : reinterpret_cast<const uint8_t*>(kNothing)) + c * (kRow / 16);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (kWords == 4) {
                const u32x4 w = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(from + j * kRow));
                v[j][0] = w.x, v[j][1] = w.y, v[j][2] = w.z, v[j][3] = w.w;
            } else if constexpr (kWords == 2) {
                const u32x2 w = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(from + j * kRow));
                v[j][0] = w.x, v[j][1] = w.y;
            } else {
                v[j][0] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(from + j * kRow));
            }
        }
        if constexpr (kE4m3) {
            const f32x4* of = reinterpret_cast<const f32x4*>(at.page_v >= 0 ? p.cache.vs + row : reinterpret_cast<const float*>(kNothing));
            scale[0] = of[0], scale[1] = of[1];
        }
    }

    __device__ __forceinline__ void widen(uint32_t (&w)[8][D / 32]) const {
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int x = 0; x < D / 32; ++x) {
                if constexpr (kE4m3) w[j][x] = (x & 1) ? bf16x2_of_e4m3<true>(v[j][x >> 1]) : bf16x2_of_e4m3<false>(v[j][x >> 1]);
                else w[j][x] = v[j][x];
            }
    }

    // P^T's operands; the scale of an 8-bit value is taken before the rounding to bf16
    template <int NT>
    __device__ __forceinline__ void operands(bf16x8 (&pr)[NT], const float (&z)[NT][8]) const {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                w[j] = z[n][j];
                if constexpr (kE4m3) w[j] = w[j] == 0.f ? 0.f : w[j] * scale[j >> 2][j & 3];
            }
            pr[n] = operand(pack_bf16(w[0], w[1]), pack_bf16(w[2], w[3]), pack_bf16(w[4], w[5]), pack_bf16(w[6], w[7]));
        }
    }
};

// What a wave holds of 16 * NT rows: lane (g, c) row c of each 16.
template <int D, int NT>
struct State {
    f32x4 o[NT][D / 16];      // D / 16 tiles e: columns (D / 16) (4 g + r) + e
    float m[NT], l[NT];       // largest score so far, this lane's share of the sum
    int end[NT], low[NT];     // the row sees keys [low, end)
};

// z: the lane's scores of keys 8 g + j, in units of log2
template <int D, bool kE4m3, int NT>
__device__ __forceinline__ void scores(float (&z)[NT][8], const Keys<D, kE4m3>& t, const bf16x8 (&q)[NT][D / 32], float unit) {
    using L = Keys<D, kE4m3>;
    f32x4 s[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) s[n][i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < L::kLoads; ++w)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const u32x4 k = t.k[i][w];
            if constexpr (kE4m3) {
                const bf16x8 lo = operand(bf16x2_of_e4m3<false>(k.x), bf16x2_of_e4m3<true>(k.x), bf16x2_of_e4m3<false>(k.y), bf16x2_of_e4m3<true>(k.y));
                const bf16x8 hi = operand(bf16x2_of_e4m3<false>(k.z), bf16x2_of_e4m3<true>(k.z), bf16x2_of_e4m3<false>(k.w), bf16x2_of_e4m3<true>(k.w));
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    s[n][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo, q[n][2 * w], s[n][i], 0, 0, 0);
                    s[n][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi, q[n][2 * w + 1], s[n][i], 0, 0, 0);
                }
            } else {
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    s[n][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, k), q[n][w], s[n][i], 0, 0, 0);
            }
        }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                z[n][4 * i + r] = s[n][i][r] * unit;
                if constexpr (kE4m3) z[n][4 * i + r] *= t.scale[i][r];
            }
}

// The softmax's next 32 keys: scores to weights (z in place), earlier outputs rescaled.
template <int D, int NT>
__device__ __forceinline__ void weights(State<D, NT>& st, float (&z)[NT][8]) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float top = fmaxf(fmaxf(fmaxf(z[n][0], z[n][1]), fmaxf(z[n][2], z[n][3])), fmaxf(fmaxf(z[n][4], z[n][5]), fmaxf(z[n][6], z[n][7])));
        top = max_xor16(max_xor32(top));
        if (__any(top > st.m[n])) {
            const float m = fmaxf(st.m[n], top);
            const float f = m == st.m[n] ? 1.0f : __builtin_amdgcn_exp2f(st.m[n] - m);
            st.m[n] = m;
            st.l[n] *= f;
#pragma unroll
            for (int e = 0; e < D / 16; ++e) st.o[n][e] *= f;
        }
        const float m = st.m[n] == -__builtin_inff() ? 0.f : st.m[n];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            z[n][j] = __builtin_amdgcn_exp2f(z[n][j] - m);
            st.l[n] += z[n][j];
        }
    }
}

// Scores of keys that a row does not see, of the lane's 8 from `key` on, take no part.
template <int D, int NT>
__device__ __forceinline__ void hide_scores(float (&z)[NT][8], const State<D, NT>& st, int key, bool held) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 8; ++j) z[n][j] = key + j >= st.low[n] && key + j < st.end[n] && held ? z[n][j] : -__builtin_inff();
}

// Values of keys that no row sees may be anything, and 0 * infinity is no 0:
// they become 0.  Whether one of the wave's others is not finite.
template <int E>
__device__ __forceinline__ bool hide_values(uint32_t (&v)[8][E / 2], int key, int lo, int hi) {
    bool odd = false;
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int w = 0; w < E / 2; ++w) {
            v[j][w] = key + j >= lo && key + j < hi ? v[j][w] : 0u;
            odd |= odd_halves(v[j][w]) != 0;
        }
    return __any(odd);
}

// V^T's operand of tile e from the lane's rows
template <int E>
__device__ __forceinline__ bf16x8 values_of(const uint32_t (&v)[8][E / 2], int e) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = (e & 1) ? halves_hi(v[2 * i + 1][e >> 1], v[2 * i][e >> 1]) : halves_lo(v[2 * i + 1][e >> 1], v[2 * i][e >> 1]);
    return operand(w[0], w[1], w[2], w[3]);
}

// Rare: some rows see these keys, others do not, and some of their values are
// infinities or NaNs.  Those values alone, key by key, into the rows that see them.
template <int D, int NT>
__device__ __forceinline__ void add_key_by_key(State<D, NT>& st, const uint32_t (&v)[8][D / 32], const bf16x8 (&pr)[NT], int k0, int g) {
#pragma unroll
    for (int e = 0; e < D / 16; ++e) {
        u32x4 vt = __builtin_bit_cast(u32x4, values_of<D / 16>(v, e));
#pragma unroll
        for (int i = 0; i < 4; ++i) vt[i] &= odd_halves(vt[i]);
#pragma unroll 1
        for (int j = 0; j < kTile; ++j) {
            const uint32_t keep = (j >> 3) == g ? ((j & 1) ? 0xFFFF0000u : 0x0000FFFFu) : 0u;
            const int at = (j & 7) >> 1, key = k0 + j;
            const u32x4 mask{at == 0 ? keep : 0u, at == 1 ? keep : 0u, at == 2 ? keep : 0u, at == 3 ? keep : 0u};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const bf16x8 one = __builtin_bit_cast(bf16x8, __builtin_bit_cast(u32x4, pr[n]) & mask);
                const f32x4 add = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, vt & mask), one, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
                const bool in = key >= st.low[n] && key < st.end[n];
#pragma unroll
                for (int r = 0; r < 4; ++r) st.o[n][e][r] += in ? add[r] : 0.f;
            }
        }
    }
}

template <int D, bool kE4m3, int NT>
__global__ __launch_bounds__(kThreads, 2) void attn_decode_kernel(const DecodeParams p) {
    constexpr int E = D / 16, kRows = 16 * NT, kStride = D + 4;     // a row of LDS and of a part: D outputs, then its maximum and sum
    __shared__ __align__(16) float s_o[kWaves * kRows * kStride];
    __shared__ float s_m[kWaves][kRows], s_l[kWaves][kRows];
    __shared__ unsigned s_prev;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, c = lane & 15;
    const int B = p.a.B, HZ = p.a.Hk * p.Z;

    auto count = [&](int b) -> uint32_t { return (uint32_t)span_of(p, b).blocks; };
    const Runs runs = count_runs(B, lane, count);
    const long total = (long)runs.total * HZ;
    const long W = total < p.W ? total : p.W;      // workgroups that have work
    const long w = blockIdx.x;
    if (w >= W) return;
    long pos = w * total / W;
    const long stop = (w + 1) * total / W;
    // a sequence's HZ units follow each other
    const Place place = find_place(runs, B, lane, (uint32_t)(pos / HZ), count);
    int b = place.seq;
    Span sp = span_of(p, b);
    const uint32_t inside = place.at * HZ + (uint32_t)(pos % HZ);      // blocks before pos in its sequence
    int hz = (int)(inside / sp.blocks), blk = (int)(inside % sp.blocks);
    const __amdgpu_buffer_rsrc_t parts = make_rsrc(p.part, 2u * kMaxWgs * kRows * kStride * 4u);

    while (pos < stop) {
        const int blocks = (int)min((long)(sp.blocks - blk), stop - pos);
        const int head = hz / p.Z, row0 = (hz - head * p.Z) * kRows;
        const int rows = min(kRows, p.R - row0);
        // this lane's rows
        State<D, NT> st;
        bf16x8 q[NT][D / 32];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = 16 * n + c, at = row0 + r, i = at / p.G, h = head * p.G + (at - i * p.G);
            st.end[n] = r < rows && i < sp.n ? sp.len - sp.n + i + 1 : 0;
            st.low[n] = p.a.window ? st.end[n] - p.a.window : 0;
            st.m[n] = -__builtin_inff();
            st.l[n] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) st.o[n][e] = f32x4{0.f, 0.f, 0.f, 0.f};
            const uint16_t* src = p.a.q + ((long)b * p.a.T + i) * p.a.qs + h * D;
#pragma unroll
            for (int s = 0; s < D / 32; ++s) {
                const int col = kE4m3 ? 64 * (s >> 1) + 16 * g + 8 * (s & 1) : 32 * s + 8 * g;
                q[n][s] = __builtin_bit_cast(bf16x8, r < rows ? *reinterpret_cast<const u32x4*>(src + col) : u32x4{0, 0, 0, 0});
            }
        }
        const int first_end = sp.len - sp.n + 1;                  // of row 0; the last row's is len
        const int seen_lo = p.a.window ? max(0, first_end - p.a.window) : 0, last_low = p.a.window ? sp.len - p.a.window : 0;
        const int hi = min(sp.hi, sp.lo + (blk + blocks) * kBlock);
        int k0 = sp.lo + blk * kBlock + wave * kTile;

        auto page_at = [&](int key0) -> int {
            const int key = key0 + 8 * (c >> 2);
            if (key >= hi) return -1;
            const int page = p.a.table[(long)b * p.a.width + (key >> p.cache.shift)];
            return (unsigned)page < (unsigned)p.cache.pages ? page : -1;
        };
        if (k0 < hi) {
            Keys<D, kE4m3> keys;
            Values<D, kE4m3> values;
            Rows at;
            int later = -1, later2 = -1;      // of a sequence's first or last keys
            at.k0 = k0;
            at.page = page_at(k0);
            int next = page_at(k0 + kBlock);
            at.page_v = __shfl(at.page, 4 * g);
            keys.load(p, at, head, lane);
            values.load(p, at, head, lane);
            while (true) {
                const bool held = at.page_v >= 0, more = k0 + kBlock < hi;
                const int after = page_at(k0 + 2 * kBlock);
                float z[NT][8];
                scores<D, kE4m3, NT>(z, keys, q, p.c);
                at.k0 = k0 + kBlock;
                at.page = next;
                at.page_v = __shfl(next, 4 * g);
                next = after;
                if (more) keys.load(p, at, head, lane);
                // the lane's values of keys 8 g + j as bf16: columns E c + 2 w, E c + 2 w + 1
                uint32_t v[8][E / 2];
                values.widen(v);
                if (k0 + kTile > first_end || k0 < last_low || k0 < seen_lo || __any(!held)) {
                    // (new tokens are at most 64, so that at most one step of a wave lies
                    // where the keys that rows see begin, and one where they end)
                    const bool partly = sp.n > 1 && (k0 + kTile > first_end || k0 < last_low);
                    const bool odd = hide_values<E>(v, k0 + 8 * g, seen_lo, sp.hi) && partly;
                    hide_scores<D, NT>(z, st, k0 + 8 * g, held);
                    if (odd) {
                        later2 = later;
                        later = k0;
#pragma unroll
                        for (int j = 0; j < 8; ++j)
#pragma unroll
                            for (int x = 0; x < E / 2; ++x) v[j][x] &= ~odd_halves(v[j][x]);
                    }
                }
                weights<D, NT>(st, z);
                bf16x8 pr[NT];
                values.template operands<NT>(pr, z);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const bf16x8 vt = values_of<E>(v, e);
#pragma unroll
                    for (int n = 0; n < NT; ++n) st.o[n][e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vt, pr[n], st.o[n][e], 0, 0, 0);
                }
                if (!more) break;
                values.load(p, at, head, lane);
                k0 += kBlock;
            }
            // rare: the (at most two) steps whose infinities and NaNs were left out above
#pragma unroll 1
            for (; later >= 0; later = later2, later2 = -1) {
                at.k0 = later;
                at.page = page_at(at.k0);
                at.page_v = __shfl(at.page, 4 * g);
                keys.load(p, at, head, lane);
                values.load(p, at, head, lane);
                float z[NT][8];
                scores<D, kE4m3, NT>(z, keys, q, p.c);
                hide_scores<D, NT>(z, st, at.k0 + 8 * g, at.page_v >= 0);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 8; ++j) z[n][j] = __builtin_amdgcn_exp2f(z[n][j] - (st.m[n] == -__builtin_inff() ? 0.f : st.m[n]));
                uint32_t v[8][E / 2];
                values.widen(v);
                hide_values<E>(v, at.k0 + 8 * g, seen_lo, sp.hi);
                bf16x8 pr[NT];
                values.template operands<NT>(pr, z);
                add_key_by_key<D, NT>(st, v, pr, at.k0, g);
            }
        }

        // the waves meet
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            st.l[n] = sum_xor16(sum_xor32(st.l[n]));
            if (g == 0) s_m[wave][16 * n + c] = st.m[n];
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float m = s_m[0][16 * n + c];
#pragma unroll
            for (int v = 1; v < kWaves; ++v) m = fmaxf(m, s_m[v][16 * n + c]);
            const float f = st.m[n] == m ? 1.0f : __builtin_amdgcn_exp2f(st.m[n] - m);
            if (g == 0) s_l[wave][16 * n + c] = st.l[n] * f;
            float* dst = s_o + (wave * kRows + 16 * n + c) * kStride;
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int e = 0; e < E; e += 4)
                    *reinterpret_cast<f32x4*>(dst + E * (4 * g + r) + e) =
                        f32x4{st.o[n][e][r] * f, st.o[n][e + 1][r] * f, st.o[n][e + 2][r] * f, st.o[n][e + 3][r] * f};
        }
        __syncthreads();
        const long unit = pos - blk;       // the place of this unit's first block
        const bool whole = blocks == sp.blocks;
        const int first = (int)(((unit + 1) * W - 1) / total), last = (int)(((unit + sp.blocks) * W - 1) / total);
        const int slot = 2 * (int)w + (pos == w * total / W ? 0 : 1);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = 16 * n + (tid >> 4), ch = tid & 15, at = row0 + r, i = at / p.G;
            if (r < rows) {
                float o[E], l = 0.f, m = s_m[0][r];
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll
                for (int v = 0; v < kWaves; ++v) {
                    m = fmaxf(m, s_m[v][r]);
                    l += s_l[v][r];
#pragma unroll
                    for (int e = 0; e < E; ++e) o[e] += s_o[(v * kRows + r) * kStride + E * ch + e];
                }
                if (i >= sp.n) {           // no token of its sequence: it saw keys of the rows beside it
                    m = -__builtin_inff();
                    l = 0.f;
#pragma unroll
                    for (int e = 0; e < E; ++e) o[e] = 0.f;
                }
                if (whole) {
                    const float f = l == 0.f ? 0.f : 1.0f / l;
                    uint16_t* y = p.a.out + (((long)b * p.a.T + i) * p.a.Hq + head * p.G + (at - i * p.G)) * D + E * ch;
#pragma unroll
                    for (int e = 0; e < E; e += 4) {
                        const bool none = l == 0.f;
                        *reinterpret_cast<u32x2*>(y + e) = u32x2{none ? 0u : pack_bf16(o[e] * f, o[e + 1] * f),
                                                                 none ? 0u : pack_bf16(o[e + 2] * f, o[e + 3] * f)};
                    }
                } else {
                    const uint32_t to = (uint32_t)((slot * kRows + r) * kStride) * 4u;
#pragma unroll
                    for (int e = 0; e < E; e += 4)
                        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, f32x4{o[e], o[e + 1], o[e + 2], o[e + 3]}), parts,
                                                               (int)(to + (E * ch + e) * 4u), 0, kCoherent);
                    if (ch == 0)
                        __builtin_amdgcn_raw_buffer_store_b64(u32x2{__builtin_bit_cast(uint32_t, m), __builtin_bit_cast(uint32_t, l)},
                                                              parts, (int)(to + D * 4u), 0, kCoherent);
                }
            }
        }
        if (!whole && arrive_last(p.cnt + (size_t)first * kCtrWords, last - first + 1, tid, &s_prev)) {
            // The parts of this unit, in order.  A row's D values take 16
            // threads; where 16 rows are more than there are, the threads left
            // over take every other part, and meet in LDS.
            int sets = 1;
            while (sets < 16 && rows <= 8 / sets) sets *= 2;
            const int width = 16 / sets;       // rows that the threads hold at a time
            const int set = (tid >> 4) / width;
#pragma unroll 1
            for (int r0 = 0; r0 < rows; r0 += width) {
                const int r = r0 + (tid >> 4) % width, ch = tid & 15;
                float o[E], l = 0.f, m = -__builtin_inff();
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] = 0.f;
                if (r < rows) {
                    constexpr int kAhead = 8;
                    for (int s0 = first + set; s0 <= last; s0 += kAhead * sets) {
                        f32x4 po[kAhead][E / 4];
                        u32x2 ml[kAhead];
#pragma unroll
                        for (int k = 0; k < kAhead; ++k) {
                            const int s = min(s0 + k * sets, last);
                            const int from = 2 * s + (s == first && (long)s * total / W < unit ? 1 : 0);
                            const uint32_t at = (uint32_t)((from * kRows + r) * kStride) * 4u;
                            ml[k] = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(parts, (int)(at + D * 4u), 0, kCoherent));
#pragma unroll
                            for (int e = 0; e < E / 4; ++e)
                                po[k][e] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(parts, (int)(at + (E * ch + 4 * e) * 4u), 0, kCoherent));
                        }
                        float top = m;
#pragma unroll
                        for (int k = 0; k < kAhead; ++k)
                            if (s0 + k * sets <= last) top = fmaxf(top, __builtin_bit_cast(float, (uint32_t)ml[k].x));
                        const float f = m == top ? 1.0f : __builtin_amdgcn_exp2f(m - top);
                        m = top;
                        l *= f;
#pragma unroll
                        for (int e = 0; e < E; ++e) o[e] *= f;
#pragma unroll
                        for (int k = 0; k < kAhead; ++k) {
                            if (s0 + k * sets > last) break;
                            const float pm = __builtin_bit_cast(float, (uint32_t)ml[k].x);
                            const float x = pm == m ? 1.0f : __builtin_amdgcn_exp2f(pm - m);
                            l = __builtin_fmaf(__builtin_bit_cast(float, (uint32_t)ml[k].y), x, l);
#pragma unroll
                            for (int e = 0; e < E; ++e) o[e] = __builtin_fmaf(po[k][e >> 2][e & 3], x, o[e]);
                        }
                    }
                }
                if (sets > 1) {
                    __syncthreads();
                    float* mine = s_o + (tid >> 4) * kStride;
#pragma unroll
                    for (int e = 0; e < E; ++e) mine[E * ch + e] = o[e];
                    if (ch == 0) mine[D] = m, mine[D + 1] = l;
                    __syncthreads();
                    if (set == 0) {
                        float top = m;
                        for (int k = 1; k < sets; ++k) top = fmaxf(top, s_o[((tid >> 4) + k * width) * kStride + D]);
                        const float f = m == top ? 1.0f : __builtin_amdgcn_exp2f(m - top);
                        l *= f;
#pragma unroll
                        for (int e = 0; e < E; ++e) o[e] *= f;
                        for (int k = 1; k < sets; ++k) {
                            const float* other = s_o + ((tid >> 4) + k * width) * kStride;
                            const float x = other[D] == top ? 1.0f : __builtin_amdgcn_exp2f(other[D] - top);
                            l = __builtin_fmaf(other[D + 1], x, l);
#pragma unroll
                            for (int e = 0; e < E; ++e) o[e] = __builtin_fmaf(other[E * ch + e], x, o[e]);
                        }
                    }
                }
                if (set == 0 && r < rows) {
                    const int at = row0 + r, i = at / p.G;
                    const bool none = l == 0.f;
                    const float f = 1.0f / l;
                    uint16_t* y = p.a.out + (((long)b * p.a.T + i) * p.a.Hq + head * p.G + (at - i * p.G)) * D + E * ch;
#pragma unroll
                    for (int e = 0; e < E; e += 4)
                        *reinterpret_cast<u32x2*>(y + e) = u32x2{none ? 0u : pack_bf16(o[e] * f, o[e + 1] * f),
                                                                 none ? 0u : pack_bf16(o[e + 2] * f, o[e + 3] * f)};
                }
            }
        }
        __syncthreads();       // LDS is free for the next unit
        pos += blocks;
        blk = 0;
        if (++hz == HZ && pos < stop) {
            hz = 0;
            sp = span_of(p, ++b);
        }
    }
}

template <int D, bool kE4m3>
hipError_t launch(DecodeParams p, hipStream_t s) {
    // 16 rows to a wave, or 32 where there are more: the cache is then read once
    // for both halves
    const bool two = p.R > 16;
    p.Z = (p.R + (two ? 31 : 15)) / (two ? 32 : 16);
    const long units = (long)p.a.B * p.a.Hk * p.Z * ((((long)p.a.width << p.cache.shift) + kBlock - 1) / kBlock);
    p.W = (int)(units < kMaxWgs ? units : kMaxWgs);
    const dim3 grid(p.W), block(kThreads);
    if (two) return launch_kernel(attn_decode_kernel<D, kE4m3, 2>, grid, block, 0, s, p);
    return launch_kernel(attn_decode_kernel<D, kE4m3, 1>, grid, block, 0, s, p);
}

}  // namespace

size_t attention_decode_ws_bytes(int T, int Hq, int Hk, int D) {
    const int rows = T * (Hq / Hk) > 16 ? 32 : 16;
    return kWsCounterBytes + 2 * (size_t)kMaxWgs * rows * (D + 4) * 4;
}

hipError_t launch_attention_decode(const DecodeArgs& a, const Cache& cache, void* ws, hipStream_t s) {
    DecodeParams p{a, cache, reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kWsCounterBytes), static_cast<unsigned*>(ws),
                   a.scale * kLog2e, a.Hq / a.Hk, a.T * (a.Hq / a.Hk), 1, 1};
    if (a.D == 128) return cache.ks ? launch<128, true>(p, s) : launch<128, false>(p, s);
    return cache.ks ? launch<64, true>(p, s) : launch<64, false>(p, s);
}

}  // namespace q4
