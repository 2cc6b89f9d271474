// Attention of a sequence's new tokens over a paged cache.
//
//     y[b, i, head] = sum_j p_j v_j,  p = softmax over seen keys j of scale * q[b, i, head] . k_j
//
// Row i of a sequence's n new tokens sees keys j < length - n + i + 1, of
// those the last `window` (0: all), and of those the ones whose page is in the
// cache.  Rows that see nothing are 0.
//
// Bound by memory: a key and value is read once for up to 32 of the rows (heads
// of the group x new tokens) that share it, and again for every 32 more; 16 rows
// are a matrix instruction's, whose other rows are idle where there are fewer:
// the matrix cores have ten times the rate that this needs, so nothing is gained
// by filling them.
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
// A wave's next 32 keys are in flight while it works on the present ones (16 KB
// a wave, 128 KB a CU; 64 keys of smaller rows are no faster).
// The pages of a workgroup's keys lie in LDS by then, a load apart from them
// and not in front of every step's.
//
// The work is the list of all units (sequence, key head, 32 rows) in tiles of
// 32 keys; every workgroup takes an equal, contiguous part of it, whatever the
// lengths are: they are only known on the device, and ragged ones are as
// balanced as equal ones.  A unit counts kOwn tiles more than it has, about
// what its heads, its pages and its join cost: without them the workgroups
// that hold many short ones end last.  A part of a unit leaves its maxima,
// sums and fp32 outputs in the workspace, and the workgroup that arrives last
// joins them, in order, so that results do not depend on timing.
//
// Measured (16 heads over 4, D = 128; us, and the bytes of q, y and the keys
// and values seen at that rate; the same cache again and again, and another one
// every time, 1.3 GB of them in turn):
//   one sequence, 2304 keys, bf16                    9.9         10.5
//   48 sequences up to 2304 keys, bf16                27   4.4    29
//   the same, e4m3                                    20   3.0    21
//   48 sequences up to 8192 keys, window 1024, bf16   24   4.0    26
//   48 sequences up to 2304, 5 rows each, bf16        33   3.6    36
//   48 sequences up to 4099, 5 rows each, e4m3        35   3.1    37
//   4 sequences up to 8192, 64 rows each, bf16        59   0.7    59   (keys read 8 times)
//   one sequence, 131071 keys, bf16                   49   5.5    63
//   32 sequences of 32768 keys, bf16                 326   6.6   360
// A copy of 2 GiB moves 4.9 TB/s, both directions counted.  The last is the
// memory's rate; before it stand the launch, the lengths, pages and heads one
// after the other, and behind it the join, some 9 us together, which is what
// the first has, and half of what 48 sequences in 8 bits take.  With several
// rows a unit's own instructions (heads, meeting, parts, joins) are half of all
// vector instructions; among them are the 49 to 56 scalars that the compiler
// keeps in lanes of vector registers.
#include "attention.h"
#include "attn_common.h"
#include "internal.h"
#include "topk.h"

namespace q4 {

namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kTile = 32;                    // keys of a wave's step
constexpr int kBlock = kTile * kWaves;       // keys of a workgroup's step
constexpr int kMaxWgs = (int)(kWsCounterBytes / kCtrStride);      // 512: two a CU
constexpr int kAhead = 4;                    // parts that a thread has in flight when it joins (8: up to 1 us more)
// A unit of more parts than kManyParts (for every set of threads) is joined in
// turns, by groups of up to kGroup (for every set), about as many as there are
// in a group.  One workgroup fetches parts at some 10 bytes a cycle: 128 parts of
// 32 rows took 128 us with the attention in one turn, 60 in groups of 16 and 8,
// 57 in groups of 4, 4 and 8; 128 parts of 4 rows 58 in one, 51.5 in two.  With 8
// parts (16 of 8 rows, 32 of 4) and less the second arrival costs more, 1 us.
constexpr int kManyParts = 8, kGroup = 4;
// parts of a group, as a power of two, where `left` parts are joined by `sets` sets of threads
__host__ __device__ constexpr int group_bits(int left, int sets) {
    int bits = 1;
    while ((1 << 2 * bits) < left && (1 << bits) < kGroup * sets) ++bits;
    return bits;
}
// Counters of a workgroup that a join of up to kMaxWgs parts reaches: the last
// turn's, and two of each turn before it (the first group's, whose workgroup
// may also be the last of the unit before, and another group's).
constexpr int join_counters() {
    int most = 1;
    for (int sets = 1; sets <= 16; sets *= 2)
        for (int parts = 1; parts <= kMaxWgs; ++parts) {
            int words = 1;
            for (int left = parts; left > kManyParts * sets; words += 2) {
                const int bits = group_bits(left, sets);
                left = (left + (1 << bits) - 1) >> bits;
            }
            most = words > most ? words : most;
        }
    return most;
}
static_assert(join_counters() == 7 && join_counters() <= kCtrWords, "a workgroup's counters are one line's");
// Tiles that a unit counts beside its own, us of (48 sequences up to 2304 keys
// bf16, the same in e4m3, 16 of a window of 1024 keys, 64 of 8192 keys e4m3,
// one of 8192): 0: 32.0 / 27.7 / 17.9 / 65 / 11.7; 4: 28.1 / 23.0 / 14.0 / 61.6 / 12.9;
// 8: 28.0 / 21.3 / 13.8 / 61.0 / 12.8; 12 (32 rows): as 8.
constexpr int kOwn = 8;
constexpr int kCoherent = 16;                // buffer cache policy sc1: device-coherent, not held in the per-XCD L2

struct DecodeParams {
    DecodeArgs a;
    Cache cache;
    float* part;
    unsigned* cnt;
    float c;             // scale * log2 e
    int G, R, Z, W;      // heads that share keys, rows of a key head, their chunks, workgroups
    int rows;            // of a part
    uint32_t by_G;       // 2^32 / G, rounded up: the high half of its product with a row (below 2^14) is row / G
};

struct Span {
    int n, len, lo, hi, tiles;    // new tokens, keys; the keys [lo, hi) that rows see, lo at a tile
};
__device__ __forceinline__ Span span_of(const DecodeParams& p, int b) {
    Span s;
    const int most = p.a.width << p.cache.shift;
    s.len = min(max(p.a.lengths[b], 0), most);
    s.n = p.a.n_new ? min(max(p.a.n_new[b], 0), p.a.T) : p.a.T;
    s.hi = s.n ? s.len : 0;
    s.lo = p.a.window ? max(0, s.len - s.n + 1 - p.a.window) & ~(kTile - 1) : 0;
    s.tiles = max(1, (s.hi - s.lo + kTile - 1) / kTile);
    return s;
}

template <int SEL>
__device__ __forceinline__ uint32_t bf16x2_of_e4m3(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, SEL));
}
__device__ __forceinline__ bf16x8 operand(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __builtin_bit_cast(bf16x8, u32x4{a, b, c, d});
}

// Lane (g, j) holds a value of key 8 g + j: those of the lane's 8 keys.
__device__ __forceinline__ void of_keys(float (&each)[8], float v) {
    each[0] = dpp<0x150>(v), each[1] = dpp<0x151>(v), each[2] = dpp<0x152>(v), each[3] = dpp<0x153>(v);      // row_newbcast
    each[4] = dpp<0x154>(v), each[5] = dpp<0x155>(v), each[6] = dpp<0x156>(v), each[7] = dpp<0x157>(v);
}

// Where this lane's rows of 32 keys lie: their numbers in the cache, of keys
// 8 (c / 4) + c % 4 (and 4 more) and of keys 8 g ..  Where nothing is held they
// are some row of the cache, read and not used.
struct Rows {
    uint32_t k, v;
    bool held;       // keys 8 g .. are there
};

template <int D, bool kE4m3>
struct Keys {
    static constexpr int kRow = kE4m3 ? D : 2 * D;    // bytes of a row
    static constexpr int kLoads = kRow / 64;          // 16-byte loads per lane and row
    u32x4 k[2][kLoads];
    float scale;          // of key 8 g + c % 8

    // (V's loads take whole rows and are marked as read once, K's take 64 bytes of
    // a row and are not: both marked cost 4 to 15 % where the cache is in reach of
    // the last level, 2 % where it is not; neither marked costs 4 to 12 % there)
    __device__ __forceinline__ void load(const DecodeParams& p, const Rows& at, int lane) {
        const uint8_t* from = p.cache.k + (uint64_t)at.k * kRow + 16 * (lane >> 4);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int s = 0; s < kLoads; ++s)
                k[t][s] = *reinterpret_cast<const u32x4*>(from + 4 * t * kRow + 64 * s);
        if constexpr (kE4m3) scale = p.cache.ks[(uint64_t)at.v + (lane & 7)];
    }
};

template <int D, bool kE4m3>
struct Values {
    static constexpr int kRow = kE4m3 ? D : 2 * D;
    static constexpr int kWords = kRow / 64;          // dwords of a row per lane
    uint32_t v[8][kWords];
    float scale;          // of key 8 g + c % 8

    __device__ __forceinline__ void load(const DecodeParams& p, const Rows& at, int lane) {
        const uint8_t* from = p.cache.v + (uint64_t)at.v * kRow + (lane & 15) * (kRow / 16);
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
        if constexpr (kE4m3) scale = p.cache.vs[(uint64_t)at.v + (lane & 7)];
    }

    // the lane's columns (D / 16) c + 2 x and the next of keys 8 g .. 8 g + 7, as bf16
    __device__ __forceinline__ void pairs(uint32_t (&w)[8], int x) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (kE4m3) w[j] = (x & 1) ? bf16x2_of_e4m3<true>(v[j][x >> 1]) : bf16x2_of_e4m3<false>(v[j][x >> 1]);
            else w[j] = v[j][x];
        }
    }

    // P^T's operands; the scale of an 8-bit value is taken before the rounding to
    // bf16 (edge: a key that a row does not see may have any scale)
    template <int NT>
    __device__ __forceinline__ void operands(bf16x8 (&pr)[NT], const float (&z)[NT][8], bool edge) const {
        float each[8];
        if constexpr (kE4m3) of_keys(each, scale);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                w[j] = z[n][j];
                if constexpr (kE4m3) w[j] = edge && w[j] == 0.f ? 0.f : w[j] * each[j];
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
    float each[8];
    if constexpr (kE4m3) of_keys(each, t.scale * unit);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 8; ++j) z[n][j] = s[n][j >> 2][j & 3] * (kE4m3 ? each[j] : unit);
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
        for (int j = 0; j < 8; ++j) z[n][j] = __builtin_amdgcn_exp2f(z[n][j] - m);
    }
}

// The sum of the weights.  They are rounded to bf16, the products' operands, and
// the sum is of the rounded ones, so that a row is a mean of its values: equal
// values are met exactly, where the sum of the others was off by up to 2^-8.  With
// 8-bit values, themselves up to 2^-4 off, a weight times its value's scale is
// rounded, and the sum is of the weights before: dividing each by its scale
// again would be two more operations a key and row.
template <int D, bool kE4m3, int NT>
__device__ __forceinline__ void add_up(State<D, NT>& st, const float (&z)[NT][8], const bf16x8 (&pr)[NT]) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        if constexpr (kE4m3) {
#pragma unroll
            for (int j = 0; j < 8; ++j) st.l[n] += z[n][j];
        } else {
            const u32x4 w = __builtin_bit_cast(u32x4, pr[n]);
#pragma unroll
            for (int j = 0; j < 4; ++j) st.l[n] = dot2(w[j], 0x3F803F80u, st.l[n]);
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

// Values that no row sees may be anything, and 0 * infinity is no 0: they become
// 0.  apart: infinities and NaNs do too; whether there were any.
__device__ __forceinline__ bool hide_values(uint32_t (&v)[8], int key, int lo, int hi, bool held, bool apart) {
    bool odd = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        v[j] = key + j >= lo && key + j < hi && held ? v[j] : 0u;
        const uint32_t bits = apart ? odd_halves(v[j]) : 0u;
        odd |= bits != 0;
        v[j] &= ~bits;
    }
    return odd;
}

// V^T's operand of tile 2 x (half = 0) or 2 x + 1 from the lane's columns
__device__ __forceinline__ u32x4 values_of(const uint32_t (&v)[8], int half) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = half ? halves_hi(v[2 * i + 1], v[2 * i]) : halves_lo(v[2 * i + 1], v[2 * i]);
    return w;
}

// Rare: some rows see these keys, others do not, and some of their values are
// infinities or NaNs.  Those values alone, key by key, into the rows that see
// them: v of tile e.
template <int D, int NT>
__device__ __forceinline__ void add_key_by_key(State<D, NT>& st, int e, u32x4 v, const bf16x8 (&pr)[NT], int k0, int g) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] &= odd_halves(v[i]);
#pragma unroll 1
    for (int j = 0; j < kTile; ++j) {
        const uint32_t keep = (j >> 3) == g ? ((j & 1) ? 0xFFFF0000u : 0x0000FFFFu) : 0u;
        const int at = (j & 7) >> 1, key = k0 + j;
        const u32x4 mask{at == 0 ? keep : 0u, at == 1 ? keep : 0u, at == 2 ? keep : 0u, at == 3 ? keep : 0u};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const bf16x8 one = __builtin_bit_cast(bf16x8, __builtin_bit_cast(u32x4, pr[n]) & mask);
            const f32x4 add = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, v & mask), one, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
            const bool in = key >= st.low[n] && key < st.end[n];
#pragma unroll
            for (int r = 0; r < 4; ++r) st.o[n][e][r] += in ? add[r] : 0.f;
        }
    }
}

template <int D, bool kE4m3, int NT>
__global__ __launch_bounds__(kThreads, 2) void attn_decode_kernel(const DecodeParams p) {
    constexpr int E = D / 16, kRows = 16 * NT, kStride = D + 4;     // a row of LDS and of a part: D outputs, then its maximum and sum
    __shared__ __align__(16) float s_o[kWaves * kRows * kStride];
    int32_t* s_table = reinterpret_cast<int32_t*>(s_o);      // the pages of the keys at hand, before the waves meet
    constexpr int kEntries = kWaves * kRows * kStride / (kBlock / 16) * (kBlock / 16);     // (whole steps, whatever the page size)
    __shared__ float s_m[kWaves][kRows], s_l[kWaves][kRows];
    __shared__ unsigned s_prev;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, c = lane & 15;
    const int B = p.a.B, HZ = p.a.Hk * p.Z;

    // up to 64 sequences: one to a lane, read once
    Span mine{0, 0, 0, 0, 0};
    Runs runs;
    auto count = [&](int b) -> uint32_t { return (uint32_t)(span_of(p, b).tiles + kOwn); };
    if (B <= 64) {
        if (lane < B) mine = span_of(p, lane);
        runs.run = 1;
        runs.upto = wave_scan(lane < B ? (uint32_t)(mine.tiles + kOwn) : 0u);
        runs.total = of_lane(runs.upto, 63);
    } else {
        runs = count_runs(B, lane, count);
    }
    auto span_at = [&](int b) -> Span {
        if (B > 64) return span_of(p, b);
        return Span{__builtin_amdgcn_readlane(mine.n, b), __builtin_amdgcn_readlane(mine.len, b), __builtin_amdgcn_readlane(mine.lo, b),
                    __builtin_amdgcn_readlane(mine.hi, b), __builtin_amdgcn_readlane(mine.tiles, b)};
    };
    const uint32_t total = runs.total * (uint32_t)HZ;                       // below 2^31
    const uint32_t share = max((total + (uint32_t)p.W - 1) / (uint32_t)p.W, (uint32_t)kWaves);     // tiles of a workgroup
    const uint32_t w = blockIdx.x, start = w * share;
    if (start >= total) return;
    const uint32_t stop = min(start + share, total);
    uint32_t pos = start;
    // a sequence's HZ units follow each other
    const uint32_t turn = pos / (uint32_t)HZ;
    const Place place = find_place(runs, B, lane, turn, count);
    int b = __builtin_amdgcn_readfirstlane(place.seq);
    Span sp = span_at(b);
    const uint32_t inside = place.at * (uint32_t)HZ + (pos - turn * (uint32_t)HZ);      // places before pos in its sequence
    int hz = (int)(inside / (uint32_t)(sp.tiles + kOwn)), place_in = (int)(inside - (uint32_t)hz * (uint32_t)(sp.tiles + kOwn));
    auto token_of = [&](int row) { return p.G == 1 ? row : (int)__umulhi((uint32_t)row, p.by_G); };     // row / G
    const __amdgpu_buffer_rsrc_t parts = make_rsrc(p.part, 2u * (uint32_t)p.W * (uint32_t)p.rows * kStride * 4u);

    while (pos < stop) {
        // (a part's own cost is the first kOwn places of its unit)
        const int at0 = max(place_in, kOwn), at1 = min(sp.tiles + kOwn, place_in + (int)(stop - pos)), tiles = at1 - at0, tile = at0 - kOwn;
        if (tiles <= 0) break;      // the range ends before the unit's first tile
        const int head = p.Z == 1 ? hz : hz / p.Z, row0 = (hz - head * p.Z) * kRows;
        const int rows = min(kRows, p.R - row0);
        // this lane's rows
        State<D, NT> st;
        bf16x8 q[NT][D / 32];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = 16 * n + c, at = row0 + r, i = token_of(at), h = head * p.G + (at - i * p.G);
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
        const int hi = min(sp.hi, sp.lo + (tile + tiles) * kTile);

        Keys<D, kE4m3> keys;
        Values<D, kE4m3> values;
        int later = -1, later2 = -1;      // of a sequence's first or last keys
        const int shift = p.cache.shift, in_page = (1 << shift) - 1;
        const int32_t* table = p.a.table + (long)b * p.a.width;
        // (as many pages at a time as LDS has room for)
        for (int part = sp.lo + tile * kTile, end; part < hi; part = end) {
            const int page0 = part >> shift;
            end = min(hi, (page0 + kEntries) << shift);
            if (page0 != (sp.lo + tile * kTile) >> shift) __syncthreads();      // (all are done with the pages before)
            for (int i = tid; i <= ((end - 1) >> shift) - page0; i += kThreads) {
                const int entry = table[page0 + i];
                s_table[i] = (unsigned)entry < (unsigned)p.cache.pages ? entry : -1;
            }
            __syncthreads();
            auto rows_at = [&](int key0) {
                const int key = key0 + 8 * (c >> 2), key_v = key0 + 8 * g;
                const int page = s_table[(min(key, end - 1) >> shift) - page0], page_v = s_table[(min(key_v, end - 1) >> shift) - page0];
                return Rows{(((uint32_t)max(page, 0) * (uint32_t)p.a.Hk + (uint32_t)head) << shift) + (uint32_t)((key & in_page) + (c & 3)),
                            (((uint32_t)max(page_v, 0) * (uint32_t)p.a.Hk + (uint32_t)head) << shift) + (uint32_t)(key_v & in_page),
                            key_v < end && page_v >= 0};
            };
            int k0 = part + wave * kTile;
            bool held = false;
            if (k0 < end) {
                const Rows at = rows_at(k0);
                held = at.held;
                keys.load(p, at, lane);
                values.load(p, at, lane);
            }
            for (; k0 < end; k0 += kBlock) {
                const bool here = held, more = k0 + kBlock < end;
                const Rows at = rows_at(k0 + kBlock);
                float z[NT][8];
                scores<D, kE4m3, NT>(z, keys, q, p.c);
                held = at.held;
                if (more) keys.load(p, at, lane);
                const bool edge = k0 + kTile > first_end || k0 < last_low || k0 < seen_lo || __any(!here);
                if (edge) hide_scores<D, NT>(z, st, k0 + 8 * g, here);
                weights<D, NT>(st, z);
                bf16x8 pr[NT];
                values.template operands<NT>(pr, z, edge);
                add_up<D, kE4m3, NT>(st, z, pr);
                // (new tokens are at most 64, so that at most one step of a wave lies
                // where the keys that rows see begin, and one where they end)
                const bool partly = sp.n > 1 && (k0 + kTile > first_end || k0 < last_low);
                bool odd = false;
#pragma unroll
                for (int x = 0; x < E / 2; ++x) {
                    uint32_t v[8];
                    values.pairs(v, x);
                    if (edge) odd |= hide_values(v, k0 + 8 * g, seen_lo, sp.hi, here, partly);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const bf16x8 vt = __builtin_bit_cast(bf16x8, values_of(v, h));
#pragma unroll
                        for (int n = 0; n < NT; ++n) st.o[n][2 * x + h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vt, pr[n], st.o[n][2 * x + h], 0, 0, 0);
                    }
                }
                if (edge && __any(odd)) {
                    later2 = later;
                    later = k0;
                }
                if (more) values.load(p, at, lane);
            }
            // rare: the (at most two) steps whose infinities and NaNs were left out above
#pragma unroll 1
            for (; later >= 0; later = later2, later2 = -1) {
                const Rows at = rows_at(later);
                keys.load(p, at, lane);
                values.load(p, at, lane);
                float z[NT][8];
                scores<D, kE4m3, NT>(z, keys, q, p.c);
                hide_scores<D, NT>(z, st, later + 8 * g, at.held);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 8; ++j) z[n][j] = __builtin_amdgcn_exp2f(z[n][j] - (st.m[n] == -__builtin_inff() ? 0.f : st.m[n]));
                bf16x8 pr[NT];
                values.template operands<NT>(pr, z, true);
#pragma unroll
                for (int x = 0; x < E / 2; ++x) {
                    uint32_t v[8];
                    values.pairs(v, x);
                    hide_values(v, later + 8 * g, seen_lo, sp.hi, at.held, false);
#pragma unroll
                    for (int h = 0; h < 2; ++h) add_key_by_key<D, NT>(st, 2 * x + h, values_of(v, h), pr, later, g);
                }
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
        const uint32_t unit = pos - (uint32_t)place_in + kOwn;       // the place of this unit's first tile
        const bool whole = tiles == sp.tiles;
        const int slot = 2 * (int)w + (unit + (uint32_t)tile <= start ? 0 : 1);
        // D / 16 columns of a row: its outputs, or its part
        auto give = [&](int r, int ch, const float (&o)[E], float l) {
            const int at = row0 + r, i = token_of(at);
            const bool none = l == 0.f;
            const float f = 1.0f / l;
            uint16_t* y = p.a.out + (((long)b * p.a.T + i) * p.a.Hq + head * p.G + (at - i * p.G)) * D + E * ch;
#pragma unroll
            for (int e = 0; e < E; e += 4)
                *reinterpret_cast<u32x2*>(y + e) = u32x2{none ? 0u : pack_bf16(o[e] * f, o[e + 1] * f),
                                                         none ? 0u : pack_bf16(o[e + 2] * f, o[e + 3] * f)};
        };
        auto keep = [&](int slot, int r, int ch, const float (&o)[E], float m, float l) {
            const uint32_t to = (uint32_t)((slot * p.rows + r) * kStride) * 4u;
#pragma unroll
            for (int e = 0; e < E; e += 4)
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, f32x4{o[e], o[e + 1], o[e + 2], o[e + 3]}), parts,
                                                       (int)(to + (E * ch + e) * 4u), 0, kCoherent);
            if (ch == 0)
                __builtin_amdgcn_raw_buffer_store_b64(u32x2{__builtin_bit_cast(uint32_t, m), __builtin_bit_cast(uint32_t, l)}, parts,
                                                      (int)(to + D * 4u), 0, kCoherent);
        };
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = 16 * n + (tid >> 4), ch = tid & 15, i = token_of(row0 + r);
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
                if (whole) give(r, ch, o, l);
                else keep(slot, r, ch, o, m, l);
            }
        }
        // The parts of a unit are joined in order by the workgroup that arrives
        // last; many of them, which are more than one workgroup fetches in good
        // time, first in groups, whose results take the place of their first parts.
        const int first = whole ? 0 : (int)(unit / share), last = whole ? 0 : (int)((unit + (uint32_t)sp.tiles - 1) / share);     // its workgroups
        // A row's D values take 16 threads; where 16 rows are more than there are,
        // the threads left over take every other part, and meet in LDS.
        int sets = 1;
        while (sets < 16 && rows <= 8 / sets) sets *= 2;
        int left = whole ? 0 : last - first + 1, part_at = (int)w - first, apart = 0;      // parts; this workgroup's; 2^apart workgroups from one to the next
#pragma unroll 1
        for (int turn = 1; left; turn += 2) {
            const bool all = left <= kManyParts * sets;
            const int bits = group_bits(left, sets);
            const int group = all ? 0 : part_at >> bits, n = all ? left : min(1 << bits, left - (group << bits));
            const int from = first + ((group << bits) << apart);
            // (a workgroup can be the last of one unit and the first of another)
            unsigned* const counter = p.cnt + (size_t)from * kCtrWords + (all ? 0 : group ? turn + 1 : turn);
            if (!arrive_last(counter, n, tid, &s_prev)) break;
            auto slot_of = [&](int k) { const int x = from + (k << apart); return 2 * x + (x == first && (uint32_t)x * share < unit ? 1 : 0); };
            const int width = 16 / sets;       // rows that the threads hold at a time
            const int set = (tid >> 4) / width;
#pragma unroll 1
            for (int r0 = 0; r0 < rows; r0 += width) {
                const int r = r0 + (tid >> 4) % width, ch = tid & 15;
                float o[E], l = 0.f, m = -__builtin_inff();
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] = 0.f;
                if (r < rows) {
                    for (int s0 = set; s0 < n; s0 += kAhead * sets) {
                        f32x4 po[kAhead][E / 4];
                        u32x2 ml[kAhead];
#pragma unroll
                        for (int k = 0; k < kAhead; ++k) {
                            const uint32_t at = (uint32_t)((slot_of(min(s0 + k * sets, n - 1)) * p.rows + r) * kStride) * 4u;
                            ml[k] = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(parts, (int)(at + D * 4u), 0, kCoherent));
#pragma unroll
                            for (int e = 0; e < E / 4; ++e)
                                po[k][e] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(parts, (int)(at + (E * ch + 4 * e) * 4u), 0, kCoherent));
                        }
                        float top = m;
#pragma unroll
                        for (int k = 0; k < kAhead; ++k)
                            if (s0 + k * sets < n) top = fmaxf(top, __builtin_bit_cast(float, (uint32_t)ml[k].x));
                        const float f = m == top ? 1.0f : __builtin_amdgcn_exp2f(m - top);
                        m = top;
                        l *= f;
#pragma unroll
                        for (int e = 0; e < E; ++e) o[e] *= f;
#pragma unroll
                        for (int k = 0; k < kAhead; ++k) {
                            if (s0 + k * sets >= n) break;
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
                        m = top;
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
                    if (all) give(r, ch, o, l);
                    else keep(slot_of(0), r, ch, o, m, l);
                }
            }
            part_at = group;
            apart += bits;
            left = all ? 0 : (left + (1 << bits) - 1) >> bits;
        }
        __syncthreads();       // LDS is free for the next unit
        pos = unit + (uint32_t)(tile + tiles);
        place_in = 0;
        if (++hz == HZ && pos < stop) {
            hz = 0;
            sp = span_at(++b);
        }
    }
}

template <int D, bool kE4m3>
hipError_t launch(DecodeParams p, hipStream_t s) {
    // 16 rows to a wave, or 32 where there are more: the cache is then read once
    // for both halves.  20 rows of 48 sequences up to 2304 keys, bf16: 32 us, in two
    // units of 16 each 45; up to 4099 keys, e4m3: 36 and 43.
    const bool two = p.R > 16;
    p.Z = (p.R + (two ? 31 : 15)) / (two ? 32 : 16);
    const long units = attention_decode_units(p.a, p.cache);
    p.rows = p.R < 32 ? p.R : 32;
    p.W = (int)(units < kMaxWgs * kWaves ? (units + kWaves - 1) / kWaves : kMaxWgs);
    p.by_G = p.G > 1 ? (uint32_t)((1ull << 32) / (unsigned)p.G) + 1 : 0;
    const dim3 grid(p.W), block(kThreads);
    if (two) return launch_kernel(attn_decode_kernel<D, kE4m3, 2>, grid, block, 0, s, p);
    return launch_kernel(attn_decode_kernel<D, kE4m3, 1>, grid, block, 0, s, p);
}

}  // namespace

long attention_decode_units(const DecodeArgs& a, const Cache& cache) {
    const int R = a.T * (a.Hq / a.Hk), Z = R > 16 ? (R + 31) / 32 : 1;
    return (long)a.B * a.Hk * Z * ((((long)a.width << cache.shift) + kTile - 1) / kTile + kOwn);
}

size_t attention_decode_ws_bytes(int T, int Hq, int Hk, int D) {
    const int R = T * (Hq / Hk), rows = R < 32 ? R : 32;
    return kWsCounterBytes + 2 * (size_t)kMaxWgs * rows * (D + 4) * 4;
}

hipError_t launch_attention_decode(const DecodeArgs& a, const Cache& cache, void* ws, hipStream_t s) {
    DecodeParams p{a, cache, reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kWsCounterBytes), static_cast<unsigned*>(ws),
                   a.scale * kLog2e, a.Hq / a.Hk, a.T * (a.Hq / a.Hk), 1, 1, 0, 0};
    if (a.D == 128) return cache.ks ? launch<128, true>(p, s) : launch<128, false>(p, s);
    return cache.ks ? launch<64, true>(p, s) : launch<64, false>(p, s);
}

}  // namespace q4
