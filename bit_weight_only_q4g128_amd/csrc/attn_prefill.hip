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
// K and V pass through LDS once per workgroup, in the order in which the
// operands read them (16 bytes a lane, consecutive): K in columns of 8 elements
// (a column of 64 keys and 16 bytes more, so that a row's store touches every
// bank once); V transposed, in units of 4 keys by 4 columns that a thread turns
// in registers.  Two stages: the next 64 keys are stored while these are used,
// and the ones after them are in flight in registers.
#include "attention.h"
#include "attn_common.h"
#include "internal.h"

namespace q4 {

namespace {

constexpr int kKeys = 64;        // of a step
constexpr int kWaveRows = 32;

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

template <int D>
constexpr int kColumn = kKeys * 16 + 16;                   // bytes of 8 elements' column of K
template <int D>
constexpr int kKBytes = (D / 8) * kColumn<D>;
template <int D>
constexpr int kStage = kKBytes<D> + kKeys * D * 2;         // bytes of a stage

// A workgroup's share of 64 keys on the way to LDS.  A piece's place is a
// uniform part (step, row of the piece) and one 32-bit offset of the thread.
template <int D, int NW>
struct Fetch {
    static constexpr int kThreads = 64 * NW;
    static constexpr int kK = kKeys * (D / 8) / kThreads;                // 16-byte pieces of K per thread
    static constexpr int kKRows = kThreads / (D / 8);                    // keys between them
    static constexpr int kUnits = (kKeys / 4) * (D / 4);                 // units of V: 4 keys by 4 columns
    static constexpr int kV = (kUnits + kThreads - 1) / kThreads;
    static constexpr int kVRows = 8 * kThreads / (D / 2);                // keys between them
    u32x4 k[kK];
    u32x2 v[kV][4];

    // the thread's first piece of K, and first key of its first unit of V
    static __device__ __forceinline__ int k_row(int tid) { return tid / (D / 8); }
    static __device__ __forceinline__ int v_row(int tid) {
        const int hs = tid / (D / 2);
        return 16 * (hs >> 1) + 8 * (tid & 1) + 4 * (hs & 1);
    }
    static __device__ __forceinline__ int v_column(int tid) { return 4 * ((tid >> 1) & (D / 4 - 1)); }
    static __device__ __forceinline__ bool has_v(int tid) { return kUnits >= kThreads || tid < kUnits; }

    __device__ __forceinline__ void load(const PrefillArgs& a, const uint16_t* kb, const uint16_t* vb, int key0, int lo, int hi, int tid) {
        const uint8_t* k0 = reinterpret_cast<const uint8_t*>(kb + key0 * a.ks);
        const uint8_t* v0 = reinterpret_cast<const uint8_t*>(vb + key0 * a.vs);
        if (key0 >= lo && key0 + kKeys <= hi) {
            const uint32_t k_at = (uint32_t)(k_row(tid) * (int)a.ks + 8 * (tid & (D / 8 - 1))) * 2u;
            const uint32_t v_at = has_v(tid) ? (uint32_t)(v_row(tid) * (int)a.vs + v_column(tid)) * 2u : 0u;
#pragma unroll
            for (int i = 0; i < kK; ++i) k[i] = *reinterpret_cast<const u32x4*>(k0 + 2 * i * kKRows * a.ks + k_at);
#pragma unroll
            for (int i = 0; i < kV; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) v[i][r] = *reinterpret_cast<const u32x2*>(v0 + 2 * (i * kVRows + r) * a.vs + v_at);
            return;
        }
        // the first or last keys: none is read behind them, and values that no
        // row sees may be anything, and 0 * infinity is no 0
#pragma unroll
        for (int i = 0; i < kK; ++i) {
            const int row = min(k_row(tid) + i * kKRows, hi - 1 - key0);
            k[i] = *reinterpret_cast<const u32x4*>(k0 + ((long)row * a.ks + 8 * (tid & (D / 8 - 1))) * 2);
        }
#pragma unroll
        for (int i = 0; i < kV; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = v_row(tid) + i * kVRows + r;
                const bool in = key0 + row >= lo && key0 + row < hi && has_v(tid);
                v[i][r] = *reinterpret_cast<const u32x2*>(v0 + (in ? ((long)row * a.vs + v_column(tid)) * 2 : (lo - key0) * a.vs * 2));
                if (!in) v[i][r] = u32x2{0, 0};
            }
    }
    // takes infinities and NaNs out of V: whether there were any
    __device__ __forceinline__ bool tame() {
        bool odd = false;
#pragma unroll
        for (int i = 0; i < kV; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint32_t bits = odd_halves(v[i][r][x]);
                    odd |= bits != 0;
                    v[i][r][x] &= ~bits;
                }
        return odd;
    }
    __device__ __forceinline__ void store(uint8_t* stage, int tid) const {
        uint8_t* kt = stage + (tid & (D / 8 - 1)) * kColumn<D> + k_row(tid) * 16;
#pragma unroll
        for (int i = 0; i < kK; ++i) *reinterpret_cast<u32x4*>(kt + i * kKRows * 16) = k[i];
        if (!has_v(tid)) return;
        const int u = (tid >> 1) & (D / 4 - 1), hs = tid / (D / 2);
        // tile d % (D / 32), row d / (D / 32) of it for column d = 4 u + e
        constexpr int kTiles = D / 32;
        uint8_t* vt = stage + kKBytes<D> + ((hs >> 1) * kTiles * 2 + (hs & 1)) * 512 + (kTiles == 4 ? u : 2 * u) * 16 + (tid & 1) * 8;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const u32x2 t[4] = {u32x2{halves_lo(v[i][1].x, v[i][0].x), halves_lo(v[i][3].x, v[i][2].x)},
                                u32x2{halves_hi(v[i][1].x, v[i][0].x), halves_hi(v[i][3].x, v[i][2].x)},
                                u32x2{halves_lo(v[i][1].y, v[i][0].y), halves_lo(v[i][3].y, v[i][2].y)},
                                u32x2{halves_hi(v[i][1].y, v[i][0].y), halves_hi(v[i][3].y, v[i][2].y)}};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                *reinterpret_cast<u32x2*>(vt + i * (kVRows / 16) * kTiles * 1024 + (e & (kTiles - 1)) * 1024 + (kTiles == 4 ? 0 : (e >> 1) * 16)) = t[e];
        }
    }
};

template <int D, int NW>
__global__ __launch_bounds__(64 * NW, 2) void attn_prefill_kernel(const PrefillParams p) {
    constexpr int kRows = kWaveRows * NW, kTiles = D / 32;
    __shared__ __align__(16) uint8_t lds[2 * kStage<D>];
    __shared__ int s_odd;
    const PrefillArgs& a = p.a;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int half = lane >> 5, G = p.G;

    // The workgroup's rows.  Workgroups go to the XCDs in turn, so that with
    // the key head fastest a key head stays in one XCD's L2 (Hk dividing 8); a
    // prompt's last rows, which see most, come first.
    auto count = [&](int b) -> long { return ((long)prompt_of(a, b).tokens * G + kRows - 1) / kRows; };
    const int head = blockIdx.x % a.Hk;
    long upto;
    int run;
    const long total = count_all(a.B, lane, count, upto, run);
    const Place place = find_place(a.B, lane, total, upto, run, total - 1 - blockIdx.x / a.Hk, count);
    if (place.seq < 0) return;
    const Prompt s = prompt_of(a, place.seq);
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
    float m = -__builtin_inff(), l = 0.f;

    const uint16_t* kb = a.k + (long)s.k0 * a.ks + head * D;
    const uint16_t* vb = a.v + (long)s.k0 * a.vs + head * D;
    Fetch<D, NW> f;
    auto partly = [&](int key0) { return key0 + kKeys > first_end || (a.window && key0 < last_end - a.window); };
    auto put = [&](int i) {       // the fetched keys into their stage
        if (partly(begin + i * kKeys) && f.tame()) s_odd = 1;
        f.store(lds + (i & 1) * kStage<D>, tid);
    };
    if (tid == 0) s_odd = 0;
    __syncthreads();
    if (steps > 0) {
        f.load(a, kb, vb, begin, lo, hi, tid);
        put(0);
        if (steps > 1) f.load(a, kb, vb, begin + kKeys, lo, hi, tid);
    }
    for (int i = 0; i < steps; ++i) {
        __syncthreads();
        if (i + 1 < steps) put(i + 1);
        if (i + 2 < steps) f.load(a, kb, vb, begin + (i + 2) * kKeys, lo, hi, tid);
        const uint8_t* kt = lds + (i & 1) * kStage<D>;
        const uint8_t* vt = kt + kKBytes<D>;
        const int key0 = begin + i * kKeys;
        f32x16 z[2];
#pragma unroll
        for (int j = 0; j < 16; ++j) z[0][j] = z[1][j] = 0.f;
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const bf16x8 k = *reinterpret_cast<const bf16x8*>(kt + (2 * j + half) * kColumn<D> + (32 * t + (lane & 31)) * 16);
                z[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k, q[j], z[t], 0, 0, 0);
            }
        const bool edge = partly(key0);
        if (edge) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int key = key0 + 32 * t + 8 * (j >> 2) + 4 * half + (j & 3);
                    z[t][j] = key >= low && key < end ? z[t][j] : -__builtin_inff();
                }
        }
        float top = z[0][0];
#pragma unroll
        for (int j = 1; j < 32; ++j) top = fmaxf(top, z[j >> 4][j & 15]);
        top = max_xor32(top);
        // Weights may exceed 1: only a maximum that grew by more than 2^8
        // rescales what is there, which after the first steps is rare.
        if (__any((top - m) * p.c > 8.f)) {
            const float now = fmaxf(m, top);
            const float x = now == m ? 1.0f : __builtin_amdgcn_exp2f((m - now) * p.c);
            m = now;
            l *= x;
#pragma unroll
            for (int t = 0; t < kTiles; ++t) o[t] *= x;
        }
        const float mc = m == -__builtin_inff() ? 0.f : m * p.c;
        u32x4 pw[4];
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
            const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(z[j >> 4][j & 15], p.c, -mc));
            const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(z[j >> 4][(j & 15) + 1], p.c, -mc));
            sum[(j >> 1) & 3] += x + y;
            pw[j >> 3][(j & 7) >> 1] = pack_bf16(x, y);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
                const bf16x8 v = *reinterpret_cast<const bf16x8*>(vt + ((k * kTiles + t) * 2 + half) * 512 + (lane & 31) * 16);
                o[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, __builtin_bit_cast(bf16x8, pw[k]), o[t], 0, 0, 0);
            }
    }
    __syncthreads();
    if (s_odd) {
        // Rare: where some rows see keys that others do not, some values are
        // infinities or NaNs.  Those values alone, which were left out above,
        // key by key into the rows that see them.
#pragma unroll 1
        for (int key0 = begin; key0 < hi; key0 += kKeys) {
            if (!partly(key0)) continue;
            f.load(a, kb, vb, key0, lo, hi, tid);
            f.store(lds, tid);
            __syncthreads();
            const float mc = m == -__builtin_inff() ? 0.f : m * p.c;
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
                f32x16 z;
#pragma unroll
                for (int j = 0; j < 16; ++j) z[j] = 0.f;
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    const bf16x8 x = *reinterpret_cast<const bf16x8*>(lds + (2 * j + half) * kColumn<D> + (32 * (k >> 1) + (lane & 31)) * 16);
                    z = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, q[j], z, 0, 0, 0);
                }
                float w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = __builtin_amdgcn_exp2f(__builtin_fmaf((k & 1) ? z[8 + j] : z[j], p.c, -mc));
                const u32x4 pk{pack_bf16(w[0], w[1]), pack_bf16(w[2], w[3]), pack_bf16(w[4], w[5]), pack_bf16(w[6], w[7])};
#pragma unroll 1
                for (int j = 0; j < 16; ++j) {
                    const uint32_t keep = (j >> 3) == half ? ((j & 1) ? 0xFFFF0000u : 0x0000FFFFu) : 0u;
                    const int at = (j & 7) >> 1, key = key0 + 16 * k + 8 * ((j >> 2) & 1) + 4 * (j >> 3) + (j & 3);
                    const u32x4 mask{at == 0 ? keep : 0u, at == 1 ? keep : 0u, at == 2 ? keep : 0u, at == 3 ? keep : 0u};
                    const bool in = key >= low && key < end;
#pragma unroll
                    for (int t = 0; t < kTiles; ++t) {
                        u32x4 v = *reinterpret_cast<const u32x4*>(lds + kKBytes<D> + ((k * kTiles + t) * 2 + half) * 512 + (lane & 31) * 16);
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
    if (!row_in) return;
    const bool none = l == 0.f;
    const float f0 = 1.0f / l;
    uint16_t* y = a.out + ((long)(s.q0 + token) * a.Hq + q_head) * D;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        // columns (D / 32) (8 x + 4 half + b) + tile, b = 0 .. 3
        constexpr int kRun = D / 8;
        uint32_t w[kRun / 2];
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int t = 0; t < kTiles; t += 2)
                w[(b * kTiles + t) >> 1] = none ? 0u : pack_bf16(o[t][4 * x + b] * f0, o[t + 1][4 * x + b] * f0);
#pragma unroll
        for (int i = 0; i < kRun / 8; ++i)
            *reinterpret_cast<u32x4*>(y + 2 * kRun * x + kRun * half + 8 * i) = u32x4{w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
    }
}

template <int D, int NW>
hipError_t launch(const PrefillParams& p, hipStream_t s) {
    const long rows = kWaveRows * NW;
    const long tiles = ((long)p.a.T * p.G + rows - 1) / rows + p.a.B;     // at least the sum of the prompts' own
    return launch_kernel(attn_prefill_kernel<D, NW>, dim3((unsigned)(tiles * p.a.Hk)), dim3(64 * NW), 0, s, p);
}

}  // namespace

hipError_t launch_attention_prefill(const PrefillArgs& a, hipStream_t s) {
    const PrefillParams p{a, a.scale * kLog2e, a.Hq / a.Hk};
    const bool wide = (long)a.T * a.Hq >= 256l * 256;
    if (a.D == 128) return wide ? launch<128, 8>(p, s) : launch<128, 4>(p, s);
    return wide ? launch<64, 8>(p, s) : launch<64, 4>(p, s);
}

}  // namespace q4
