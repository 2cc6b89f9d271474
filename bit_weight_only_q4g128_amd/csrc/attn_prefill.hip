// Causal attention over packed prompts.
//
//     y[t, head] = sum_j p_j v_j,  p = softmax over seen keys j of scale * q[t, head] . k_j
//
// Sequence b's tokens are rows starts[b] .. starts[b + 1] of q, its keys rows
// key_starts[b] .. key_starts[b + 1] of k and v; its last token sees its last
// key, each token before it one key less, and of those the last `window` (0:
// all).  Rows that see nothing are 0; rows of no sequence are left as they are.
//
// Bound by the matrix cores and, beside them, by the exponentials and LDS.
// The heads of a group are rows beside their tokens: row r of a sequence and
// key head is token r / G, head r % G, so that a workgroup's keys serve all of
// them and its rows end at nearly the same key.  A wave holds 32 rows and walks
// 64 keys at a time, as S^T = K Q^T and O^T = V^T P^T (32x32x16): the first
// product leaves a lane with one row's scores of 32 keys, which are the second
// product's operand as they are, so P stays in registers, the maximum needs one
// lane move and the sum none until the end.
//
// K and V go straight to LDS, once per workgroup and as they lie (16 bytes a
// lane, no registers), some steps ahead of their use.  A row's 16-byte chunks
// are exchanged on the way (the swizzle is on the memory side), so that the
// operands' reads touch every bank once: K by rows, V by the transposing reads
// that give a lane 4 keys of one column.
//
// Each wave computes a step's weights beside the matrix instructions of both
// products: those of this step's values, and the next step's scores.
//
// Measured (16 heads; us of a launch among others, and the products of the keys
// that rows see; on another card up to 3 % less):
//   one prompt of 77 tokens, D = 128 over 4                    7.7
//   48 prompts up to 2304 tokens, D = 128 over 4               468    790 TFLOP/s
//   5 prompts up to 1999 tokens behind 2048 keys, window
//   1024, D = 64 over 8                                         41    576 TFLOP/s
//   one prompt of 8192 tokens, D = 64 over 8                   168    819 TFLOP/s
//   one prompt of 16384 tokens, D = 128 over 4                1050   1048 TFLOP/s
// where the library's product of 8192 x 8192 x 8192 reaches 1605.  Neither unit
// is full: the matrix cores are busy for 56, 40 and 23 % of the cycles of the long
// prompt, the packed ones and the window, the vector unit for 47, 43 and 43 %, so
// that the one hardly works while the other does.  A wave has one block of rows,
// whose products wait for its weights; every step ends with a wait for all loads
// and a barrier; masked steps go over their values in LDS twice more; and some
// 6000 cycles of a workgroup pass before its first product.
#include "attention.h"
#include "attn_common.h"
#include "internal.h"
#include "lds_load.h"

#include <utility>

namespace q4 {

namespace {

constexpr int kKeys = 64;        // of a step
constexpr int kWaveRows = 32;
// Waves of a workgroup: 8 took 520 us for the packed prompts below where 4 took
// 507 (and 64 for the window where 4 took 49), 2 took 652.
constexpr int kWaves = 4;
// Workgroups that share a CU.  Registers set them; with heads of 64 columns a
// third one pays (window: 50 -> 43 us, long prompts of such heads 182 -> 171).
constexpr int workgroups(int D) { return D == 64 ? 3 : 2; }
// A score's exponent is z c - m c, rounded once, from m c rounded: off by half
// a step of m c, alike for all of a row's keys, which is 2^-13 below this size
// of m c and would be more than fp32's exponents hold from 2^31 on. From here on
// it is (z - m) c instead.
constexpr float kLarge = 0x1p12f;

struct PrefillParams {
    PrefillArgs a;
    float c;         // scale * log2 e
    int G;
};

struct Prompt {
    int q0, tokens, k0, keys;
};
__device__ __forceinline__ Prompt prompt_of(const PrefillArgs& a, int b) {
    Prompt s;
    s.q0 = min(max(a.starts[b], 0), a.T);
    s.tokens = min(max(a.starts[b + 1], s.q0), a.T) - s.q0;
    const int32_t* ks = a.key_starts ? a.key_starts : a.starts;
    s.k0 = min(max(ks[b], 0), a.S);
    s.keys = min(max(ks[b + 1], s.k0), a.S) - s.k0;
    return s;
}

// Where things lie in LDS and which of them a lane takes.  A stage holds 64
// rows of K, then of V, 2 D bytes each; 16-byte chunk c of row r of K sits at
// chunk c ^ (r % 16) (D = 64: c ^ (r / 2 % 8)), so that a chunk of 16 rows
// covers the banks once; of V at c ^ (r % 4 * 4) (D = 64: c ^ (r / 2 % 2 * 4)),
// so that 64 bytes of 4 rows do.
template <int D>
struct Tile {
    static constexpr int kRow = 2 * D, kBytes = kKeys * kRow, kStage = 2 * kBytes;
    static constexpr int kLoads = kBytes / 1024 / kWaves;            // 1 KB loads of a wave for 64 rows of K, or of V
    static constexpr int kLoadRows = 1024 / kRow;

    // (the chunk in LDS's place `lane` of the wave's loads, which are kWaves loads apart)
    static __device__ __forceinline__ uint32_t k_chunk(int lane, int wave) {
        return D == 128 ? (uint32_t)((lane & 15) ^ ((wave & 3) * 4 + (lane >> 4))) : (uint32_t)((lane & 7) ^ ((wave & 1) * 4 + (lane >> 4)));
    }
    static __device__ __forceinline__ uint32_t v_chunk(int lane) {
        return D == 128 ? (uint32_t)((lane & 15) ^ ((lane >> 4) * 4)) : (uint32_t)((lane & 7) ^ ((lane >> 4 & 1) * 4));
    }
    // the lane's address in K's rows of a tile of 32 keys, chunk `half`; chunk 2 j + half is at ^ 32 j
    static __device__ __forceinline__ uint32_t k_read(int lane) {
        const int row = lane & 31, half = lane >> 5;
        return (uint32_t)(row * kRow + ((half ^ (D == 128 ? row & 15 : row >> 1 & 7)) << 4));
    }
    // the lane's address in V's rows for columns 0 .. 31 of keys 4 half ..; columns 32 t are at ^ 64 t
    static __device__ __forceinline__ uint32_t v_read(int lane) {
        const int row = 4 * (lane >> 5) + (lane >> 2 & 3), turn = D == 128 ? row & 3 : row >> 1 & 1;
        return (uint32_t)(row * kRow + (turn << 6) + (((lane >> 4 & 1) * 2 + (lane >> 1 & 1)) << 4) + (lane & 1) * 8);
    }
};

// f(0) .. f(N - 1), each with its number as a constant
template <typename F, int... I>
__device__ __forceinline__ void each(F f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// V^T's operand of 16 keys and 32 columns: this lane's column of keys 4 half ..
// and 8 + 4 half .., at the rows' first address
template <int D>
__device__ __forceinline__ u32x4 columns(uint32_t at) {
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)at);
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)(at + 8 * 2 * D));
    const u32x2 x = __builtin_bit_cast(u32x2, a), y = __builtin_bit_cast(u32x2, b);
    return u32x4{x.x, x.y, y.x, y.y};
}

template <int D>
__global__ __launch_bounds__(64 * kWaves, workgroups(D)) void attn_prefill_kernel(const PrefillParams p) {
    using L = Tile<D>;
    constexpr int kRows = kWaveRows * kWaves, kTiles = D / 32;
    __shared__ __align__(2 * L::kStage) uint8_t lds[2 * L::kStage];
    __shared__ int s_odd;
    const PrefillArgs& a = p.a;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int half = lane >> 5, G = p.G;

    // The workgroup's rows.  Workgroups go to the XCDs in turn, so that with
    // the key head fastest a key head stays in one XCD's L2 (Hk dividing 8); a
    // prompt's last rows, which see most, come first.
    const int head = blockIdx.x % a.Hk;
    const uint32_t nth = blockIdx.x / a.Hk;
    auto tiles_of = [&](const Prompt& s) { return ((uint32_t)s.tokens * (uint32_t)G + kRows - 1) / kRows; };
    Prompt s{0, 0, 0, 0};
    Place place;
    if (a.B <= 64) {       // a prompt to a lane, read once
        if (lane < a.B) s = prompt_of(a, lane);
        const uint32_t upto = wave_scan(tiles_of(s)), total = of_lane(upto, 63);
        if (nth >= total) return;
        const uint32_t pos = total - 1 - nth;
        const int owner = __builtin_ctzll(__ballot(upto > pos));
        place = Place{owner, pos - (owner ? of_lane(upto, owner - 1) : 0u)};
        s = Prompt{__builtin_amdgcn_readlane(s.q0, owner), __builtin_amdgcn_readlane(s.tokens, owner), __builtin_amdgcn_readlane(s.k0, owner),
                   __builtin_amdgcn_readlane(s.keys, owner)};
    } else {
        auto count = [&](int b) -> uint32_t { return tiles_of(prompt_of(a, b)); };
        const Runs runs = count_runs(a.B, lane, count);
        if (nth >= runs.total) return;
        place = find_place(runs, a.B, lane, runs.total - 1 - nth, count);
        s = prompt_of(a, place.seq);
    }
    const int row0 = place.at * kRows, rows = min(kRows, s.tokens * G - row0);
    const int more = s.keys - s.tokens;                   // keys before the first token's own
    const int first = row0 / G, last = (row0 + rows - 1) / G;
    const int first_end = first + 1 + more, last_end = last + 1 + more;      // keys that the first and the last row see end here
    const int hi = max(0, last_end), lo = a.window ? max(0, first_end - a.window) : 0;
    const int begin = lo & ~(kKeys - 1), steps = hi > begin ? (hi - begin + kKeys - 1) / kKeys : 0;

    const int r = wave * kWaveRows + (lane & 31);
    const bool row_in = r < rows;
    const int token = (row0 + r) / G, q_head = head * G + (row0 + r - token * G);
    const int end = row_in ? token + 1 + more : 0, low = a.window ? end - a.window : 0;
    bf16x8 q[D / 16];
    {
        const uint16_t* src = a.q + (long)(s.q0 + token) * a.qs + q_head * D + 8 * half;
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
            q[i] = __builtin_bit_cast(bf16x8, row_in ? *reinterpret_cast<const u32x4*>(src + 16 * i) : u32x4{0, 0, 0, 0});
    }
    f32x16 o[kTiles];
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[t][i] = 0.f;
    float m = -__builtin_inff(), sum[4] = {0.f, 0.f, 0.f, 0.f};

    const uint16_t* kb = a.k + (long)s.k0 * a.ks + head * D;
    const uint16_t* vb = a.v + (long)s.k0 * a.vs + head * D;
    auto partly = [&](int i) {       // some rows see keys of step i that others do not
        const int key0 = begin + i * kKeys;
        return key0 + kKeys > first_end || (a.window && key0 < last_end - a.window);
    };

    const uint32_t base = lds_address(lds);
    const uint32_t k_off = (uint32_t)((wave * L::kLoadRows + lane / (D / 8)) * (int)a.ks) * 2u + L::k_chunk(lane, wave) * 16u;
    const uint32_t v_off = (uint32_t)((wave * L::kLoadRows + lane / (D / 8)) * (int)a.vs) * 2u + L::v_chunk(lane) * 16u;
    // Step i's keys (or values) on their way to an LDS stage; behind the last
    // key, and from the last step on, zeros.  A call takes the next step, into
    // the other stage than the one before it.
    struct Stream {
        const uint8_t* from;
        uint32_t row, to;      // bytes of a row
        int left;              // keys
    };
    auto source = [&](const Stream& f) {
        const int n = f.left;
        return rsrc_words(f.from, n >= kKeys ? (kKeys - 1) * f.row + 2 * D : n > 0 ? (uint32_t)(n - 1) * f.row + 2 * D : 0u);
    };
    auto load = [&](const Stream& f, i32x4 r, uint32_t off, int j) {
        to_lds16(r, off, (uint32_t)(j * kWaves * L::kLoadRows) * f.row, f.to + (uint32_t)((j * kWaves + wave) * 1024));
    };
    auto advance = [&](Stream& f) {
        if (f.left > 0) f.from += (uint64_t)kKeys * f.row;
        f.left -= kKeys;
        f.to ^= L::kStage;
    };
    auto fetch = [&](Stream& f, uint32_t off) {
        const i32x4 r = source(f);
#pragma unroll
        for (int j = 0; j < L::kLoads; ++j) load(f, r, off, j);
        advance(f);
    };
    // (stages lie kStage apart, a power of two at a multiple of twice its size)
    Stream ks{reinterpret_cast<const uint8_t*>(kb + begin * a.ks), (uint32_t)a.ks * 2u, base, hi - begin};
    Stream vs{reinterpret_cast<const uint8_t*>(vb + begin * a.vs), (uint32_t)a.vs * 2u, base + L::kBytes, hi - begin};
    auto fetch_k = [&] { fetch(ks, k_off); };
    auto fetch_v = [&] { fetch(vs, v_off); };
    // Values that no row sees may be anything, and 0 * infinity is no 0: where
    // rows see different keys, step i's values, there already, become 0 outside
    // [lo, hi), and infinities and NaNs are put off (s_odd).
    auto tame = [&](int i) {
        uint8_t* v = lds + (i & 1) * L::kStage + L::kBytes;
        bool odd = false;
        for (int at = tid; at < kKeys * D / 8; at += 64 * kWaves) {
            const int key = begin + i * kKeys + at / (D / 8);
            u32x4 w = *reinterpret_cast<const u32x4*>(v + at * 16);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const uint32_t bits = odd_halves(w[x]);
                const bool in = key >= lo && key < hi;
                odd |= in && bits;
                w[x] = in ? w[x] & ~bits : 0u;
            }
            *reinterpret_cast<u32x4*>(v + at * 16) = w;
        }
        if (odd) s_odd = 1;
    };

    const uint32_t k_read = L::k_read(lane), v_read = L::v_read(lane);
    auto scores = [&](f32x16 (&z)[2], int i) {
        const uint32_t at = base + (uint32_t)(i & 1) * L::kStage + k_read;
#pragma unroll
        for (int j = 0; j < 16; ++j) z[0][j] = z[1][j] = 0.f;
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const bf16x8 k = *(const __attribute__((address_space(3))) bf16x8*)(uintptr_t)((at ^ (32 * j)) + 32 * t * L::kRow);
                z[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k, q[j], z[t], 0, 0, 0);
            }
    };
    auto largest = [&](const f32x16 (&z)[2]) {
        float top = z[0][0];
#pragma unroll
        for (int j = 1; j < 32; ++j) top = fmaxf(top, z[j >> 4][j & 15]);
        return top;
    };
    // what a row's settled scores, times c, have subtracted (0 before its first key)
    auto taken = [&] {
        const float mc = m * p.c;
        return fabsf(mc) < kLarge ? mc : 0.f;
    };
    // A score of a row whose maximum is large: subtracted here.  Where the
    // maximum leaves fp32's range it is infinite: a row of infinity is NaN, and
    // of -infinity alone every weight is 0.
    auto reduced = [&](float x) {
        const float mc = m * p.c;
        if (fabsf(mc) < kLarge) return x;
        return mc == -__builtin_inff() ? x * p.c : x - (mc == __builtin_inff() ? __builtin_nanf("") : m);
    };
    // the scores' weights into the sums and outputs, with the values of step i
    auto outputs = [&](const f32x16 (&z)[2], int i) {
        const float mc = taken();
        const uint32_t at = base + (uint32_t)(i & 1) * L::kStage + L::kBytes + v_read;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            u32x4 w;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int e = 8 * (k & 1) + 2 * j;
                const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(z[k >> 1][e], p.c, -mc));
                const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(z[k >> 1][e + 1], p.c, -mc));
                w[j] = pack_bf16(x, y);
                sum[j] = dot2(w[j], 0x3F803F80u, sum[j]);
            }
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
                o[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, columns<D>((at ^ (64 * t)) + 16 * k * L::kRow)),
                                                               __builtin_bit_cast(bf16x8, w), o[t], 0, 0, 0);
        }
    };
    // step i's scores: what rows do not see taken out, and the maximum
    auto settle = [&](f32x16 (&z)[2], float top, int i) {
        if (partly(i)) {
            const int here = begin + i * kKeys + 4 * half, from = low - here, to = end - here;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int key = 32 * t + 8 * (j >> 2) + (j & 3);
                    z[t][j] = key >= from && key < to ? z[t][j] : -__builtin_inff();
                }
            top = max_xor32(largest(z));
        }
        // Weights may exceed 1: only a maximum that grew by more than 2^8
        // rescales what is there, which after the first steps is rare.  Each row
        // goes by its own: if the others of the wave moved it along, keys that it
        // does not see would change its roundings.
        const bool grown = (top - m) * p.c > 8.f;
        if (__any(grown)) {
            const float now = grown ? top : m;
            const float x = grown ? __builtin_amdgcn_exp2f((m - now) * p.c) : 1.0f;
            m = now;
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[j] *= x;
#pragma unroll
            for (int t = 0; t < kTiles; ++t) o[t] *= x;
        }
        if (__any(fabsf(m * p.c) >= kLarge && m > -__builtin_inff())) {
#pragma unroll
            for (int j = 0; j < 32; ++j) z[j >> 4][j & 15] = reduced(z[j >> 4][j & 15]);
        }
    };
    // One step: this step's weights and outputs beside the next one's scores,
    // in this order, which nothing changes: a matrix instruction, the fragment of
    // the fourth one after it, and a share of the arithmetic, which takes as
    // long as the matrix instruction.  A pair of weights begins (its scores
    // become exponentials) in one slot and ends (rounded, summed) in the next;
    // the next scores' maximum follows when they are there.
    auto step = [&](f32x16 (&z)[2], f32x16 (&next)[2], int i) {
        constexpr int kN = D / 8, kSpread = 2 * kN * 13 / 16;      // products of either kind; slots in which pairs begin
        constexpr int kAhead = D == 64 ? 2 : 4;      // fragments on their way (more registers with three workgroups a CU: 1 % slower)
        const uint32_t k_at = base + (uint32_t)((i + 1) & 1) * L::kStage + k_read;
        const uint32_t v_at = base + (uint32_t)(i & 1) * L::kStage + L::kBytes + v_read;
        const float mc = taken();
        u32x4 f[2 * kN], w[4];
        float e[16][2], top[2] = {-__builtin_inff(), -__builtin_inff()};
        auto read = [&](auto at) {
            constexpr int j = decltype(at)::value;
            if constexpr (j < kN) f[j] = *(const __attribute__((address_space(3))) u32x4*)(uintptr_t)((k_at ^ (32 * (j >> 1))) + 32 * (j & 1) * L::kRow);
            else if constexpr (j < 2 * kN) f[j] = columns<D>((v_at ^ (64 * ((j - kN) % kTiles))) + 16 * ((j - kN) / kTiles) * L::kRow);
        };
        each(read, std::make_integer_sequence<int, kAhead>());
        const i32x4 from_k = source(ks), from_v = source(vs);      // keys of step i + 2, values of step i + 1
#pragma unroll
        for (int j = 0; j < 16; ++j) next[0][j] = next[1][j] = 0.f;
        __builtin_amdgcn_sched_barrier(0);
        each([&](auto slot) {
            constexpr int j = decltype(slot)::value;
            const bf16x8 x = __builtin_bit_cast(bf16x8, f[j]);
            if constexpr (j < kN) next[j & 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, q[j >> 1], next[j & 1], 0, 0, 0);
            else o[(j - kN) % kTiles] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, __builtin_bit_cast(bf16x8, w[(j - kN) / kTiles]), o[(j - kN) % kTiles], 0, 0, 0);
            read(std::integral_constant<int, j + kAhead>{});
            if constexpr (j < 2 * L::kLoads) {      // (all of them ahead of the first: 1 to 6 % slower)
                if constexpr (j < L::kLoads) load(ks, from_k, k_off, j);
                else load(vs, from_v, v_off, j - L::kLoads);
            }
            each([&](auto pair) {
                constexpr int n = decltype(pair)::value;
                if constexpr (n * kSpread / 16 + 1 == j) {
                    w[n >> 2][n & 3] = pack_bf16(e[n][0], e[n][1]);
                    sum[n & 3] = dot2(w[n >> 2][n & 3], 0x3F803F80u, sum[n & 3]);
                    asm volatile("" : "+v"(sum[n & 3]));
                }
                if constexpr (n * kSpread / 16 == j) {
                    float a = z[n >> 3][2 * (n & 7)], b = z[n >> 3][2 * (n & 7) + 1];
                    asm volatile("" : "+v"(a), "+v"(b));
                    e[n][0] = __builtin_amdgcn_exp2f(__builtin_fmaf(a, p.c, -mc));
                    e[n][1] = __builtin_amdgcn_exp2f(__builtin_fmaf(b, p.c, -mc));
                    asm volatile("" : "+v"(e[n][0]), "+v"(e[n][1]));
                }
                if constexpr (kN + 2 + n * (kN - 2) / 16 == j) {
                    top[n & 1] = fmaxf(fmaxf(top[n & 1], next[n & 1][n & 14]), next[n & 1][(n & 14) + 1]);
                    asm volatile("" : "+v"(top[n & 1]));
                }
            }, std::make_integer_sequence<int, 16>());
            __builtin_amdgcn_sched_barrier(0);
        }, std::make_integer_sequence<int, 2 * kN>());
        advance(ks);
        advance(vs);
        settle(next, max_xor32(fmaxf(top[0], top[1])), i + 1);
        __builtin_amdgcn_s_waitcnt(0x0F70);      // vmcnt(0): this step's loads are there
        phase();
        if (partly(i + 1)) {
            tame(i + 1);
            __syncthreads();
        }
    };
    if (tid == 0) s_odd = 0;
    if (steps > 0) {
        fetch_k();
        fetch_v();
        fetch_k();
        __builtin_amdgcn_s_waitcnt(0x0F70);
        __syncthreads();
        if (partly(0)) tame(0);
        f32x16 z0[2], z1[2];
        scores(z0, 0);
        settle(z0, max_xor32(largest(z0)), 0);
        __syncthreads();       // K's first stage is free
        int i = 0;
        for (; i + 2 < steps; i += 2) {
            step(z0, z1, i);
            step(z1, z0, i + 1);
        }
        if (i + 1 < steps) {
            step(z0, z1, i);
            outputs(z1, i + 1);
        } else {
            outputs(z0, i);
        }
        __builtin_amdgcn_s_waitcnt(0x0F70);      // nothing is on its way to LDS
    }
    float l = (sum[0] + sum[1]) + (sum[2] + sum[3]);
    __syncthreads();
    if (s_odd) {
        // Rare: where some rows see keys that others do not, some values are
        // infinities or NaNs.  Those values alone, which were left out above,
        // key by key into the rows that see them.
        const float mc = taken();
#pragma unroll 1
        for (int i = 0; i < steps; ++i) {
            if (!partly(i)) continue;
            const int key0 = begin + i * kKeys;
            Stream k1{reinterpret_cast<const uint8_t*>(kb + key0 * a.ks), (uint32_t)a.ks * 2u, base, hi - key0};
            Stream v1{reinterpret_cast<const uint8_t*>(vb + key0 * a.vs), (uint32_t)a.vs * 2u, base + L::kBytes, hi - key0};
            fetch(k1, k_off);
            fetch(v1, v_off);
            __builtin_amdgcn_s_waitcnt(0x0F70);
            __syncthreads();
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
                f32x16 z;
#pragma unroll
                for (int j = 0; j < 16; ++j) z[j] = 0.f;
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    const bf16x8 x = *(const __attribute__((address_space(3))) bf16x8*)(uintptr_t)(((base + k_read) ^ (32 * j)) + 32 * (k >> 1) * L::kRow);
                    z = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, q[j], z, 0, 0, 0);
                }
                float w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(reduced((k & 1) ? z[8 + j] : z[j]), p.c, -mc));
                const u32x4 pk{pack_bf16(w[0], w[1]), pack_bf16(w[2], w[3]), pack_bf16(w[4], w[5]), pack_bf16(w[6], w[7])};
#pragma unroll 1
                for (int j = 0; j < 16; ++j) {
                    const uint32_t keep = (j >> 3) == half ? ((j & 1) ? 0xFFFF0000u : 0x0000FFFFu) : 0u;
                    const int at = (j & 7) >> 1, key = begin + i * kKeys + 16 * k + 8 * ((j >> 2) & 1) + 4 * (j >> 3) + (j & 3);
                    const u32x4 mask{at == 0 ? keep : 0u, at == 1 ? keep : 0u, at == 2 ? keep : 0u, at == 3 ? keep : 0u};
                    const bool in = key >= low && key < end;
#pragma unroll
                    for (int t = 0; t < kTiles; ++t) {
                        u32x4 v = columns<D>(((base + L::kBytes + v_read) ^ (64 * t)) + 16 * k * L::kRow);
#pragma unroll
                        for (int x = 0; x < 4; ++x) v[x] &= odd_halves(v[x]) & mask[x];
                        f32x16 none;
#pragma unroll
                        for (int x = 0; x < 16; ++x) none[x] = 0.f;
                        const f32x16 add = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, v), __builtin_bit_cast(bf16x8, pk & mask), none, 0, 0, 0);
#pragma unroll
                        for (int x = 0; x < 16; ++x) o[t][x] += in ? add[x] : 0.f;
                    }
                }
            }
            __syncthreads();
        }
    }
    l = sum_xor32(l);
    const bool none = l == 0.f;
    const float f0 = 1.0f / l;
    uint16_t* y = a.out + ((long)(s.q0 + token) * a.Hq + q_head) * D;
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int x = 0; x < 4; x += 2) {
            // columns 32 t + 8 x + 4 half .. and 8 more: of both halves' for one
            // half, the 8 more for the other, 16 bytes a store
            const auto lo = __builtin_amdgcn_permlane32_swap(pack_bf16(o[t][4 * x] * f0, o[t][4 * x + 1] * f0),
                                                             pack_bf16(o[t][4 * x + 4] * f0, o[t][4 * x + 5] * f0), false, false);
            const auto hi = __builtin_amdgcn_permlane32_swap(pack_bf16(o[t][4 * x + 2] * f0, o[t][4 * x + 3] * f0),
                                                             pack_bf16(o[t][4 * x + 6] * f0, o[t][4 * x + 7] * f0), false, false);
            if (row_in) *reinterpret_cast<u32x4*>(y + 32 * t + 8 * (x + half)) = none ? u32x4{0, 0, 0, 0} : u32x4{lo[0], hi[0], lo[1], hi[1]};
        }
}

template <int D>
hipError_t launch(const PrefillParams& p, hipStream_t s) {
    const long rows = kWaveRows * kWaves;
    const long tiles = ((long)p.a.T * p.G + rows - 1) / rows + p.a.B;     // at least the sum of the prompts' own
    return launch_kernel(attn_prefill_kernel<D>, dim3((unsigned)(tiles * p.a.Hk)), dim3(64 * kWaves), 0, s, p);
}

}  // namespace

hipError_t launch_attention_prefill(const PrefillArgs& a, hipStream_t s) {
    const PrefillParams p{a, a.scale * kLog2e, a.Hq / a.Hk};
    return a.D == 128 ? launch<128>(p, s) : launch<64>(p, s);
}

}  // namespace q4
