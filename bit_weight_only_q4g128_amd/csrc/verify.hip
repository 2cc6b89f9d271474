// Verification of drafted tokens against the target's distributions, from
// given uniform numbers (rejection sampling).  Sequence b has n drafted tokens
// d_0 .. d_{n-1}; row i of its logits is the target's distribution p_i after i
// of them, q_i the distribution the draft drew d_i from:
//   * d_i stands while u_i q_i(d_i) < p_i(d_i), that is with probability
//     min(1, p_i(d_i) / q_i(d_i)); a = how many stand from the first on;
//   * a < n: the next token is drawn from max(p_a - q_a, 0) (from p_a where
//     that is zero everywhere); a = n: from p_n.  The draw is the first entry,
//     in the distribution's order, whose running sum exceeds u_D times the
//     total.
// The tokens that come out are distributed as the target's own samples.
//
// Two forms of p and q: the top k of a row (the sampler's distribution:
// entries by larger logit, then lower index; the draft's as a list of indices
// and probabilities), and the softmax of a whole row in index order (the
// draft's as logits).  Both at temperature T.  A NaN logit counts as -inf
// (probability 0); a row whose largest logit is not finite has no
// distribution: p = 0 everywhere, the token drawn from it is -1.
//
// Whole numbers come out, so every quantity that decides one (exponentials,
// masses, running sums) is held in fp64, whose vector rate on this machine is
// that of unpacked fp32.  A probability is within about 5e-15 of its value, a
// boundary of the acceptance or of a draw from p within 1e-14 of its place.  For
// a draw from max(p - q, 0), whose total R shrinks as the draft nears the target,
// that is 1e-14 / R.
#include "internal.h"
#include "topk.h"
#include "verify.h"

namespace q4 {

namespace {

constexpr int kThreads = 256;

// 2^y for y >= -1000 (below, and for NaN: 2^-1000): y = n + f, |f| <= 1/2,
// with n from the low word of y + 1.5 * 2^52, and 2^f by a polynomial of degree
// 11 whose constant term is 1 (interpolated at Chebyshev nodes of the interval;
// it is off by 2e-17, its fp64 evaluation by 1.3e-16, so that differences of
// close probabilities keep what fp64 holds of them, and 2^0 is 1).  Conversions
// to integer and ldexp, which run at a fraction of the fp64 rate, are not needed.
__device__ __forceinline__ double exp2_raw(double y) {
    constexpr double kShift = 6755399441055744.0;
    y = __builtin_fmax(y, -1000.0);
    const double k = y + kShift, f = y - (k - kShift);
    double p = 4.4549605981865186e-10;
    p = __builtin_fma(p, f, 7.0725859492692234e-09);
    p = __builtin_fma(p, f, 1.0178062445845774e-07);
    p = __builtin_fma(p, f, 1.3215442587921689e-06);
    p = __builtin_fma(p, f, 1.5252733829836119e-05);
    p = __builtin_fma(p, f, 1.5403530441736050e-04);
    p = __builtin_fma(p, f, 1.3333558146416936e-03);
    p = __builtin_fma(p, f, 9.6181291076068882e-03);
    p = __builtin_fma(p, f, 5.5504108664821597e-02);
    p = __builtin_fma(p, f, 2.4022650695910097e-01);
    p = __builtin_fma(p, f, 6.9314718055994529e-01);
    p = __builtin_fma(p, f, 1.0);
    // (in assembly: the compiler makes five instructions of this addition)
    uint2 w = __builtin_bit_cast(uint2, p);
    asm("v_lshl_add_u32 %0, %1, 20, %0" : "+v"(w.y) : "v"(__builtin_bit_cast(uint2, k).x));
    return __builtin_bit_cast(double, w);
}
// The same with 0 below.
__device__ __forceinline__ double exp2_64(double y) {
    const double v = exp2_raw(y);
    return y > -1000.0 ? v : 0.0;
}

// Inclusive prefix sum over the 64 lanes, and the sum (lane 63's), by DPP
// moves: a shuffle through LDS costs several times their latency, and the
// verification of one sequence is little but such chains.
template <int CTRL, int ROW_MASK = 0xF>
__device__ __forceinline__ double dpp64(double v) {
    uint2 w = __builtin_bit_cast(uint2, v);
    w.x = (uint32_t)dpp_i<CTRL, ROW_MASK>((int)w.x);
    w.y = (uint32_t)dpp_i<CTRL, ROW_MASK>((int)w.y);
    return __builtin_bit_cast(double, w);
}
__device__ __forceinline__ double wave_scan(double v) {
    v += dpp64<0x111>(v);        // row_shr:1
    v += dpp64<0x112>(v);        // row_shr:2
    v += dpp64<0x114>(v);        // row_shr:4
    v += dpp64<0x118>(v);        // row_shr:8
    v += dpp64<0x142, 0xA>(v);   // row_bcast:15 into rows 1, 3
    v += dpp64<0x143, 0xC>(v);   // row_bcast:31 into rows 2, 3
    return v;
}
__device__ __forceinline__ double lane_value(double v, int lane) {      // lane: the same in every lane
    uint2 w = __builtin_bit_cast(uint2, v);
    w.x = (uint32_t)__builtin_amdgcn_readlane((int)w.x, lane);
    w.y = (uint32_t)__builtin_amdgcn_readlane((int)w.y, lane);
    return __builtin_bit_cast(double, w);
}
template <int CTRL, int ROW_MASK = 0xF>
__device__ __forceinline__ float dpp_max(float v) {
    const int b = __builtin_bit_cast(int, v);
    return fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(b, b, CTRL, ROW_MASK, 0xF, false)));
}
__device__ __forceinline__ float wave_max(float v) {
    v = dpp_max<0x111>(v);
    v = dpp_max<0x112>(v);
    v = dpp_max<0x114>(v);
    v = dpp_max<0x118>(v);
    v = dpp_max<0x142, 0xA>(v);
    v = dpp_max<0x143, 0xC>(v);
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}
__device__ __forceinline__ double wave_sum(double v) { return lane_value(wave_scan(v), 63); }

// Values that another workgroup of the same launch reads: device-coherent
// accesses, ordered by arrive_last().
template <typename T>
__device__ __forceinline__ void put(T* p, T v) { __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
template <typename T>
__device__ __forceinline__ T get(T* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

__device__ __forceinline__ int drafted(const VerifyArgs& a, int b) {
    if (!a.n_draft) return a.D;
    const int n = a.n_draft[b];
    return n < 0 ? 0 : n > a.D ? a.D : n;
}

__device__ __forceinline__ float accept_ratio(double p, double q) {
    return q > 0.0 ? (p < q ? (float)(p / q) : 1.0f) : (p > 0.0 ? 1.0f : 0.0f);
}

// ---------------------------------------------------------------------------
// top-k form.  Rows of at most kDirectVocab logits: one launch, a workgroup
// per sequence, one or two waves per row.  Longer rows: a first launch takes the
// top k of every block of 1024 or 4096, and the second merges a row's
// candidates.  Nothing is handed over inside a launch.
//
// Bound by latency and, for many rows, by the selection's instructions (about
// 550 per wave and block, half of them two sorts of 64), not by the 2 bytes per
// logit: one sequence with 4 drafted tokens, V = 2049, k = 30: 7.8 us, of which a
// launch is 1.5 and the logits' round trip about 2; 48 sequences, V = 16385: 9.0
// and 5.3 us.  Two waves share a row above 512 logits or candidates: V = 2049 in
// a graph 9.3 us, one wave with 40 logits per lane 12.5; V = 300 5.2 us in one.
// ---------------------------------------------------------------------------
constexpr int kRowsAtOnce = 8;                      // of a workgroup of the last launch
constexpr int kPairE = 20;                          // entries per lane of two waves that share a row
constexpr int kDirectVocab = 2 * 64 * kPairE;
constexpr int kBlockE = 4, kLongBlockE = 16;        // logits per thread of a block of the first launch

// NaN counts as -inf
__device__ __forceinline__ uint32_t entry_of(uint32_t bits, int col) {
    return topk_entry((bits & 0x7FFFu) > 0x7F80u ? 0xFF80u : bits, col);
}

template <int E>
__global__ __launch_bounds__(kThreads) void block_topk_kernel(VerifyArgs a, int nb, uint32_t* cand) {
    constexpr int kLogits = kThreads * E;
    __shared__ uint32_t lists[4 * 64];
    __shared__ uint32_t scratch[4 * 64 * E];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int row = blockIdx.x / nb, j = blockIdx.x - row * nb;
    const int b = row / (a.D + 1), r = row - b * (a.D + 1);
    if (r > drafted(a, b)) return;                        // no drafted token leads here
    const uint16_t* lg = a.logits + (size_t)row * a.V;
    uint32_t v[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int col = j * kLogits + tid + 256 * i;
        v[i] = lg[col < a.V ? col : 0];
    }
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int col = j * kLogits + tid + 256 * i;
        v[i] = col < a.V ? entry_of(v[i], col) : 0u;
    }
    const uint32_t top = wg_topk<E>(v, a.top_k, lists, scratch, wave, lane);
    if (wave == 0 && lane < a.top_k) cand[((size_t)row * nb + j) * a.top_k + lane] = top;
}

// One row's distribution over its k sorted entries, one entry per lane.
__device__ __forceinline__ double topk_prob64(uint32_t entry, int k, double c, int lane) {
    const float v = key_value(entry >> 16);
    const float top = __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, v)));
    const bool some = top > -__builtin_huge_valf() && top < __builtin_huge_valf();
    const double e = lane < k && some ? exp2_64(((double)v - (double)top) * c) : 0.0;
    const double s = wave_sum(e);
    return s > 0.0 ? e / s : 0.0;
}

// One workgroup per sequence, W waves per row.  cand null: rows are read as they
// are.  A wave whose drafted token is refused draws the token that comes out if
// all before it stand, so that nothing but tokens meets at the end.
template <int E, int W>
__global__ __launch_bounds__(kRowsAtOnce * W * 64) void verify_topk_kernel(VerifyArgs a, int nc, double c, const uint32_t* cand) {
    __shared__ uint32_t scratch[kRowsAtOnce * W][64 * E];
    __shared__ uint32_t s_list[W == 2 ? kRowsAtOnce * 64 : 1];
    __shared__ int s_token[kMaxDraft + 1];              // drawn at row i, or kStands
    constexpr int kStands = -2;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int b = blockIdx.x, n = drafted(a, b), k = a.top_k, D = a.D;
    const int slot = wave / W, part = wave % W;

    for (int i0 = 0; i0 <= n; i0 += kRowsAtOnce) {
        const int i = i0 + slot;
        if (i > n) {
            if constexpr (W == 2) {
                __syncthreads();
                __syncthreads();
            }
            break;
        }
        const size_t row = (size_t)b * (D + 1) + i;
        uint32_t v[E];
        auto at = [&](int j) { return lane + 64 * (W * j + part); };
        if (cand) {
            const auto cr = make_rsrc(cand + row * nc, (uint32_t)nc * 4);
#pragma unroll
            for (int j = 0; j < E; ++j) v[j] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(cr, 4 * at(j), 0, 0);      // (0 behind the end)
        } else {
            const auto lg = make_rsrc(a.logits + row * a.V, (uint32_t)a.V * 2);
#pragma unroll
            for (int j = 0; j < E; ++j) v[j] = buf_load2(lg, (uint32_t)(2 * at(j)), 0);
        }
        // the draft's side, asked for before the selection
        int d = -1, qi = -1;
        float qp = 0.f, ui = 0.f;
        const float ud = a.u[(size_t)b * (D + 1) + D];
        if (i < n) {
            d = a.draft[(size_t)b * D + i];
            ui = a.u[row];
            if (a.draft_index && lane < a.draft_k) {
                const size_t l = ((size_t)b * D + i) * a.draft_k + lane;
                qi = a.draft_index[l];
                qp = a.draft_prob[l];
            }
        }
        if (!cand) {
#pragma unroll
            for (int j = 0; j < E; ++j) v[j] = at(j) < a.V ? entry_of(v[j], at(j)) : 0u;
        }
        uint32_t e;
        if constexpr (W == 1) {
            e = wave_topk_sorted<E, true>(v, k, scratch[wave], lane);
        } else {
            __syncthreads();
            if (part) s_list[64 * slot + lane] = wave_topk_sorted<E, false>(v, k, scratch[wave], lane);
            else e = wave_topk_sorted<E, true>(v, k, scratch[wave], lane);
            __syncthreads();
            if (part) continue;
            e = merge_top64<true>(e, s_list[64 * slot + lane], lane);
        }
        const int index = (int)(0xFFFFu - (e & 0xFFFFu));
        double g = topk_prob64(e, k, c, lane);
        bool stands = false;
        if (i < n) {
            const double pd = wave_sum(index == d ? g : 0.0), qd = a.draft_index ? wave_sum(qi == d ? (double)qp : 0.0) : 1.0;
            stands = (double)ui * qd < pd;
            if (a.accept_prob && lane == 0) a.accept_prob[(size_t)b * D + i] = accept_ratio(pd, qd);
            if (!stands) {
                double q = 0.0;
                if (a.draft_index) {
#pragma unroll 4
                    for (int l = 0; l < a.draft_k; ++l) {
                        const float ql = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, qp), l));
                        q += __builtin_amdgcn_readlane(qi, l) == index ? (double)ql : 0.0;
                    }
                } else {
                    q = index == d ? 1.0 : 0.0;
                }
                const double rest = __builtin_fmax(g - q, 0.0);
                if (__any(rest > 0.0)) g = rest;
            }
        }
        int token = kStands;
        if (!stands) {
            const double run = wave_scan(g), x = (double)ud * lane_value(run, 63);
            const unsigned long long over = __ballot(run > x && g > 0.0), any = __ballot(g > 0.0);
            const int pick = over ? (int)__builtin_ctzll(over) : any ? 63 - (int)__builtin_clzll(any) : 0;
            token = any ? __builtin_amdgcn_readlane(index, pick) : -1;
        }
        if (lane == 0) s_token[i] = token;
    }
    if (a.accept_prob && tid >= n && tid < D) a.accept_prob[(size_t)b * D + tid] = 0.f;
    __syncthreads();
    if (wave == 0) {
        const int mine = s_token[lane <= n ? lane : n];
        const int stand = (int)__builtin_ctzll(__ballot(mine != kStands));
        if (lane <= D) a.token[(size_t)b * (D + 1) + lane] = lane < stand ? a.draft[(size_t)b * D + lane] : lane == stand ? mine : -1;
        if (lane == 0) a.count[b] = stand;
    }
}

// ---------------------------------------------------------------------------
// whole form.  First launch: the masses of all rows, in chunks; the workgroup
// that ends a sequence's last chunk verifies its drafted tokens.  Second
// launch: the sums of max(p - q, 0) and of p over the chunks of each sequence's
// stop row; the last one finds the chunk, then the entry, that the draw hits.
//
// Few sequences are bound by latency: one with 4 drafted tokens, V = 16385: 6.5
// and 7.3 us, each a launch, one round of loads, the arrival (about 2 us) and
// what the last workgroup does alone.  Many are bound by memory, and that at the
// ends: 32 with 7, V = 131072: 34.6 us for 101 to 126 MB, then 18.6 us, of which the
// stop rows' 15 MB are about 5 and the exponentials' arithmetic about half.
//
// A row starts at any even address.  It is read as the 16-byte aligned groups
// of 8 logits that touch it; the first and the last, where the row ends inside
// them, value by value.
// ---------------------------------------------------------------------------
constexpr int kSequences = (int)(kWsCounterBytes / kCtrStride);      // sequences of one pair of launches

struct Row {
    const uint16_t* p;     // first logit
    int off, groups;       // logits of the first group that lie before it; groups that touch the row
};
__device__ __forceinline__ Row row_of(const uint16_t* p, int V) {
    const int off = (int)((reinterpret_cast<uintptr_t>(p) & 15) >> 1);
    return Row{p, off, (off + V + 7) >> 3};
}
// Most groups of any row: rows that all start on 16 bytes touch none twice.
size_t row_groups(int V, bool aligned) { return aligned ? (size_t)V >> 3 : ((size_t)V + 14) >> 3; }

// Groups g[0 .. NJ) as bf16 pairs, -inf outside the row.  The loads of groups
// that lie in the row whole (the others take such a one's address) are all on
// their way before the few lanes with a row's end in a group read it value by
// value.
template <int NJ>
__device__ __forceinline__ void load_groups(const Row& r, int V, const int (&g)[NJ], u32x4 (&v)[NJ]) {
    constexpr uint32_t kNone = 0xFF80FF80u;
    const int lo = r.off ? 1 : 0, hi = (r.off + V) >> 3;      // whole groups: lo .. hi - 1
    bool edge = false;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const int at = g[j] < lo ? lo : g[j] >= hi ? hi - 1 : g[j];
        edge = edge || at != g[j];
        v[j] = hi > lo ? *reinterpret_cast<const u32x4*>(r.p + 8 * at - r.off) : u32x4{kNone, kNone, kNone, kNone};
    }
    if (!edge) return;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        if (g[j] >= lo && g[j] < hi) continue;
        const int i0 = 8 * g[j] - r.off;
        v[j] = u32x4{kNone, kNone, kNone, kNone};
        if (i0 <= -8 || i0 >= V) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = i0 + 2 * e, ia = i < 0 ? 0 : i < V ? i : V - 1, ib = i + 1 < 0 ? 0 : i + 1 < V ? i + 1 : V - 1;
            const uint32_t ra = r.p[ia], rb = r.p[ib];      // (inside the row, so that all are in flight together)
            const uint32_t a = ia == i ? ra : 0xFF80u, b = ib == i + 1 ? rb : 0xFF80u;
            v[j][e] = a | (b << 16);
        }
    }
}
__device__ __forceinline__ float half_of(const u32x4& v, int e) { return e & 1 ? bf16hi(v[e >> 1]) : bf16lo(v[e >> 1]); }

struct Mass {       // sum of 2^((z - top) c) and top of a part of a row
    double sum;
    double top;
};

// The mass of a whole row from its parts, by 16 adjacent lanes (all of them
// get it); sum 0 for a row without a distribution.
__device__ __forceinline__ Mass row_mass(Mass* part, int chunks, double c, int lane) {
    double sum = 0.0;
    float top = -__builtin_huge_valf();
    for (int i0 = 0; i0 < chunks; i0 += 64) {          // 4 parts per lane at a time
        double s[4];
        float t[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = i0 + 16 * j + (lane & 15);
            s[j] = i < chunks ? get(&part[i].sum) : 0.0;
            t[j] = i < chunks ? (float)get(&part[i].top) : -__builtin_huge_valf();       // (bf16 values)
        }
        float m = top;
#pragma unroll
        for (int j = 0; j < 4; ++j) m = fmaxf(m, t[j]);
#pragma unroll
        for (int k = 1; k < 16; k *= 2) m = fmaxf(m, __shfl_xor(m, k));
        sum *= exp2_64(((double)top - (double)m) * c);      // (0 * 0 at first)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum += s[j] * exp2_64(((double)t[j] - (double)m) * c);
        top = m;
    }
#pragma unroll
    for (int k = 1; k < 16; k *= 2) sum += __shfl_xor(sum, k);
    const bool some = top > -__builtin_huge_valf() && top < __builtin_huge_valf();
    return some ? Mass{sum, (double)top} : Mass{0.0, 0.0};
}

// p = 2^((z - top) c) inv; inv = 1 / sum, or 0 for a row without a distribution
__device__ __forceinline__ double inverse(const Mass& m) { return m.sum > 0.0 ? 1.0 / m.sum : 0.0; }
__device__ __forceinline__ double prob(float z, double top, double inv, double c) { return exp2_64(((double)z - top) * c) * inv; }

// Where a sequence stops, and the distributions there.
struct Stop {
    double p_top, p_inv, q_top, q_inv;
    int stand, has_q, qtoken;      // has_q: the draft's logits give q; else q = 1 at qtoken (-1: nowhere)
    int pad;
};

// Sequence b: accepts, writes everything but the drawn token.
__device__ __forceinline__ void accept(const VerifyArgs& a, int b, int n, int chunks, double c, Mass* mass, Stop* stop, int tid) {
    __shared__ Mass s_mass[2 * kMaxDraft + 1];
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), D = a.D, V = a.V;
    // lane i of wave 0: drafted token i, its logits asked for first
    int d = -1;
    uint32_t zd = 0, yd = 0;
    float ui = 0.f;
    if (wave == 0 && lane < n) {
        d = a.draft[(size_t)b * D + lane];
        ui = a.u[(size_t)b * (D + 1) + lane];
        if (d >= 0 && d < V) {
            zd = a.logits[((size_t)b * (D + 1) + lane) * V + d];
            if (a.draft_logits) yd = a.draft_logits[((size_t)b * D + lane) * V + d];
        }
    }
    // target rows 0 .. n, draft rows 0 .. n - 1, in the order of their masses
    const int rows = n + 1 + (a.draft_logits ? n : 0);
    for (int i0 = 4 * wave; i0 < rows; i0 += 16) {
        const int i = i0 + (lane >> 4) < rows ? i0 + (lane >> 4) : rows - 1;
        const Mass m = row_mass(mass + (size_t)(i <= n ? i : D + 1 + (i - n - 1)) * chunks, chunks, c, lane);
        if ((lane & 15) == 0) s_mass[i] = m;
    }
    __syncthreads();
    if (wave == 0) {
        bool ok = false;
        if (lane < n) {
            const bool in = d >= 0 && d < V;
            double pd = 0.0, qd = in ? 1.0 : 0.0;
            if (in) {
                pd = prob(__builtin_bit_cast(float, zd << 16), s_mass[lane].top, inverse(s_mass[lane]), c);
                if (a.draft_logits)
                    qd = prob(__builtin_bit_cast(float, yd << 16), s_mass[n + 1 + lane].top, inverse(s_mass[n + 1 + lane]), c);
            }
            ok = (double)ui * qd < pd;
            if (a.accept_prob) a.accept_prob[(size_t)b * D + lane] = accept_ratio(pd, qd);
        } else if (lane < D && a.accept_prob) {
            a.accept_prob[(size_t)b * D + lane] = 0.f;
        }
        const int stand = (int)__builtin_ctzll(~__ballot(ok));          // (lanes n .. 63 are never ok, and n <= 63)
        const bool refused = stand < n, has_q = refused && a.draft_logits;
        const int at = __shfl(d, stand);
        if (lane == 0) {
            const Mass pm = s_mass[stand], qm = has_q ? s_mass[n + 1 + stand] : Mass{0.0, 0.0};
            *stop = Stop{pm.top, inverse(pm), qm.top, inverse(qm), stand, has_q, refused && !has_q ? at : -1, 0};
            a.count[b] = stand;
        }
        if (lane <= D && lane != stand) a.token[(size_t)b * (D + 1) + lane] = lane < stand ? d : -1;
    }
}

// Block (sequence, row, chunk); a sequence's rows are the target's D + 1, then
// the draft's D.
struct MassBlock {
    int b, n, rest, chunk;      // sequence, its drafted tokens, row and chunk in one, chunk
    Row row;
    bool live;                  // a drafted token leads here
};
__device__ __forceinline__ MassBlock mass_block(const VerifyArgs& a, int rows, int chunks) {
    MassBlock m;
    m.b = blockIdx.x / (rows * chunks);
    m.rest = blockIdx.x - m.b * rows * chunks;
    const int i = m.rest / chunks;
    m.chunk = m.rest - i * chunks;
    m.n = drafted(a, m.b);
    const bool target = i <= a.D;
    m.live = target ? i <= m.n : i - a.D - 1 < m.n;
    m.row = row_of(target ? a.logits + ((size_t)m.b * (a.D + 1) + i) * a.V : a.draft_logits + ((size_t)m.b * a.D + (i - a.D - 1)) * a.V,
                   a.V);
    return m;
}
// The workgroup's mass from its threads' (top, sum); the workgroup that ends
// the sequence's last chunk accepts.
__device__ __forceinline__ void mass_end(const VerifyArgs& a, const MassBlock& mb, float top, double sum, int rows, int chunks, double c,
                                         Mass* mass, unsigned* cnt, Stop* stop) {
    __shared__ float s_top[4];
    __shared__ double s_sum[4];
    __shared__ unsigned s_prev;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    float m = wave_max(top);
    if (lane == 0) s_top[wave] = m;
    __syncthreads();
    m = fmaxf(fmaxf(s_top[0], s_top[1]), fmaxf(s_top[2], s_top[3]));
    sum = wave_sum(sum * exp2_64(((double)top - (double)m) * c));
    if (lane == 0) s_sum[wave] = sum;
    __syncthreads();
    Mass* mine = mass + (size_t)mb.b * rows * chunks;
    if (tid == 0) {
        put(&mine[mb.rest].sum, s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3]);
        put(&mine[mb.rest].top, (double)m);
    }
    const int active = mb.n + 1 + (a.draft_logits ? mb.n : 0);
    if (!arrive_last(cnt + (size_t)mb.b * kCtrWords, active * chunks, tid, &s_prev)) return;
    accept(a, mb.b, mb.n, chunks, c, mine, stop + mb.b, tid);
}

// Short rows: J groups per thread, one exponential per logit.  (z - top first:
// with z c and top c apart, rows that hold a mask's far value alone would keep
// the products' rounding, up to 2^75.)
template <int J>
__global__ __launch_bounds__(kThreads) void row_mass_kernel(VerifyArgs a, int rows, int chunks, double c, Mass* mass, unsigned* cnt,
                                                            Stop* stop) {
    const MassBlock mb = mass_block(a, rows, chunks);
    if (!mb.live) return;
    u32x4 v[J];
    int at[J];
#pragma unroll
    for (int j = 0; j < J; ++j) at[j] = (mb.chunk * J + j) * kThreads + (int)threadIdx.x;
    load_groups<J>(mb.row, a.V, at, v);
    float top = -__builtin_huge_valf();
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, half_of(v[j], e));
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += exp2_raw(((double)half_of(v[j], e) - (double)top) * c);
    mass_end(a, mb, top, sum, rows, chunks, c, mass, cnt, stop);
}

// Long rows of many sequences: a row's part holds few distinct bf16 values, so
// they are counted in LDS, one bin per value of 2^-12 <= |z| < 2^6, and each bin
// takes one exponential (18 per thread instead of up to 256; counts are exact,
// and the sum does not depend on the order of the additions to them).  Other
// values, rare in logits, are added one by one; -inf and NaN not at all.
// An exponential per logit is bound by the fp64 arithmetic: 32 sequences with 7
// drafted tokens and V = 131072, both launches, 79 us against 55 us, 128 with 4
// and V = 32768 55 against 51.  It stays the better one below that (128 with 4,
// V = 8192: 22 against 26 us), and for rows of other logits: nearly all of them
// the type's lowest value 74 against 103 us, all the same value 65 against 244
// (the bin's additions wait for each other).
constexpr int kHistJ = 32;                              // most groups per thread
constexpr int kHistStep = 4;                            // of them at a time
constexpr uint32_t kBinLow = 0x3980, kBins = 18 * 128;  // bits of 2^-12; bins of one sign
constexpr uint32_t kBinSign = 4096;                     // first bin of the negative values
constexpr int kBinWords = (int)(kBinSign + kBins + 64); // (behind either sign's: the other values, a bin per lane, not read)

__global__ __launch_bounds__(kThreads) void row_mass_hist_kernel(VerifyArgs a, int rows, int chunks, int steps, double c, Mass* mass,
                                                                 unsigned* cnt, Stop* stop) {
    __shared__ __attribute__((aligned(16))) uint32_t bins[(kBinWords + 3) & ~3];
    const MassBlock mb = mass_block(a, rows, chunks);
    if (!mb.live) return;
    const int tid = threadIdx.x;
    for (int i = tid; i < (kBinWords + 3) / 4; i += kThreads) reinterpret_cast<u32x4*>(bins)[i] = u32x4{0, 0, 0, 0};
    constexpr int J = kHistStep;
    u32x4 v[J];
    auto load = [&](int s) {
        int at[J];
#pragma unroll
        for (int j = 0; j < J; ++j) at[j] = ((mb.chunk * steps + s) * J + j) * kThreads + tid;
        load_groups<J>(mb.row, a.V, at, v);
    };
    load(0);
    __syncthreads();
    const unsigned short most = (unsigned short)(kBins + (tid & 63));
    float top = -__builtin_huge_valf();
    double sum = 0.0;
    const int inside = ((mb.row.off + a.V + 7) / 8 - mb.chunk * steps * J * kThreads + J * kThreads - 1) / (J * kThreads);
    const int end = inside < steps ? inside : steps;
#pragma unroll 1
    for (int s = 0; s < end; ++s) {
        // bin numbers in pairs of 16 bits: |z|'s bits less kBinLow (smaller ones
        // wrap), at most kBins + lane, plus the sign's 4096
        uint32_t t[J][4];
        bool other = false;
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
                const uint32_t pair = v[j][e];      // (a bit_cast of the vector's element itself reads element 0)
                const u16x2 b = __builtin_bit_cast(u16x2, pair);
                u16x2 m = (u16x2)(b & (unsigned short)0x7FFF) - (unsigned short)kBinLow;
                m = __builtin_elementwise_min(m, u16x2{most, most});
                other = other || m.x >= kBins || m.y >= kBins;
                m += (u16x2)((b >> 15) << 12);
                t[j][e] = __builtin_bit_cast(uint32_t, m);
            }
        if (__any(other)) {
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float z = half_of(v[j], e);
                    const bool mine = ((t[j][e >> 1] >> (e & 1 ? 16 : 0)) & (kBinSign - 1)) >= kBins && z > -__builtin_huge_valf();
                    if (!__any(mine)) continue;
                    // many of them are alike: zeros, masks of the type's lowest value
                    double r = 1.0;
                    if (__any(mine && z != top)) r = z == top ? 1.0 : exp2_64(-fabs((double)z - (double)top) * c);
                    const double more = z > top ? sum * r + 1.0 : sum + r;
                    sum = mine ? more : sum;
                    top = mine ? fmaxf(top, z) : top;
                }
        }
        if (s + 1 < end) load(s + 1);
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                atomicAdd(&bins[t[j][e] & 0xFFFFu], 1u);
                atomicAdd(&bins[t[j][e] >> 16], 1u);
            }
    }
    __syncthreads();
    // one exponential per bin in use
    constexpr int kPer = (int)(2 * kBins) / kThreads;
    static_assert(2 * kBins % kThreads == 0, "bins");
    float m = top;
    uint32_t n[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const uint32_t i = k * kThreads + tid, sign = i >= kBins, bin = i - (sign ? kBins : 0u);
        n[k] = bins[bin + sign * kBinSign];
        const float z = __builtin_bit_cast(float, (bin + kBinLow + (sign << 15)) << 16);
        m = n[k] ? fmaxf(m, z) : m;
    }
    sum *= exp2_64(((double)top - (double)m) * c);
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const uint32_t i = k * kThreads + tid, sign = i >= kBins, bin = i - (sign ? kBins : 0u);
        const float z = __builtin_bit_cast(float, (bin + kBinLow + (sign << 15)) << 16);
        if (n[k]) sum += (double)n[k] * exp2_64(((double)z - (double)m) * c);
    }
    mass_end(a, mb, m, sum, rows, chunks, c, mass, cnt, stop);
}

struct Part {
    double rest, all;    // sums of max(p - q, 0) and of p over a chunk
};

// The stop row's values of group g.
struct Values {
    double rest[8], all[8];
};
__device__ __forceinline__ void stop_values(const VerifyArgs& a, const Row& tr, const Row& dr, const Stop& st, double c, int g, Values& o) {
    u32x4 z[1], y[1];
    const int at[1] = {g};
    load_groups<1>(tr, a.V, at, z);
    if (st.has_q) {
        if (dr.off == tr.off) {
            load_groups<1>(dr, a.V, at, y);
        } else {        // the draft's row starts at another place of its group
            uint32_t h[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = 8 * g - tr.off + e;
                h[e] = dr.p[i < 0 ? 0 : i < a.V ? i : a.V - 1];       // (outside the row p is 0, whatever q)
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) y[0][e] = h[2 * e] | (h[2 * e + 1] << 16);
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const double p = prob(half_of(z[0], e), st.p_top, st.p_inv, c);
        o.all[e] = p;
        if (st.has_q) o.rest[e] = __builtin_fmax(p - prob(half_of(y[0], e), st.q_top, st.q_inv, c), 0.0);
        else o.rest[e] = 8 * g - tr.off + e == st.qtoken ? 0.0 : p;
    }
}

// Block (b, chunk); a chunk is a group per thread (two and four were no faster
// anywhere: 32 sequences with V = 131072, with the first launch and an exponential
// of three terms less, 51 us, 53 and 54).
__global__ __launch_bounds__(kThreads) void stop_draw_kernel(VerifyArgs a, int chunks, double c, const Stop* stop, unsigned* cnt, Part* parts) {
    __shared__ double s_wave[2][4];
    __shared__ unsigned s_prev;
    __shared__ int s_rest, s_chunk, s_first[4], s_last[4];
    __shared__ double s_before, s_x;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int b = blockIdx.x / chunks, chunk = blockIdx.x - b * chunks;
    const int D = a.D, V = a.V;
    const Stop st = stop[b];
    const Row tr = row_of(a.logits + ((size_t)b * (D + 1) + st.stand) * V, V);
    const Row dr = st.has_q ? row_of(a.draft_logits + ((size_t)b * D + st.stand) * V, V) : tr;

    Values v;
    stop_values(a, tr, dr, st, c, chunk * kThreads + tid, v);
    double rest = 0.0, all = 0.0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        rest += v.rest[e];
        all += v.all[e];
    }
    rest = wave_sum(rest);
    all = wave_sum(all);
    if (lane == 0) {
        s_wave[0][wave] = rest;
        s_wave[1][wave] = all;
    }
    __syncthreads();
    Part* mine = parts + (size_t)b * chunks;
    if (tid < 2) put(tid ? &mine[chunk].all : &mine[chunk].rest, s_wave[tid][0] + s_wave[tid][1] + s_wave[tid][2] + s_wave[tid][3]);
    if (!arrive_last(cnt + (size_t)b * kCtrWords, chunks, tid, &s_prev)) return;

    // the chunk where the running sum crosses u_D times the total
    if (wave == 0) {
        const int per = (chunks + 63) >> 6;
        double rs = 0.0, as = 0.0, ru = a.u[(size_t)b * (D + 1) + D];
        for (int i = lane * per; i < (lane + 1) * per && i < chunks; ++i) {
            rs += get(&mine[i].rest);
            as += get(&mine[i].all);
        }
        const bool use_rest = __ballot(rs > 0.0) != 0;
        const double own = use_rest ? rs : as;
        const double run = wave_scan(own), total = lane_value(run, 63);
        const double x = ru * total;
        // (own > 0: the lanes' prefix sums are rounded in different orders, so
        // that of a lane without mass can exceed its neighbour's by a bit)
        const unsigned long long over = __ballot(run > x && own > 0.0), any = __ballot(own > 0.0);
        const int l = over ? (int)__builtin_ctzll(over) : any ? 63 - (int)__builtin_clzll(any) : -1;
        if (l < 0) {
            if (lane == 0) s_chunk = -1;
        } else if (lane == l) {
            double before = run - own;
            int at = per == 1 ? lane : -1;
            s_before = before;
            for (int i = lane * per; per > 1 && i < (lane + 1) * per && i < chunks; ++i) {
                const double w = use_rest ? get(&mine[i].rest) : get(&mine[i].all);
                if (w > 0.0) {
                    at = i;
                    s_before = before;
                    if (before + w > x) break;
                }
                before += w;
            }
            s_chunk = at;
            s_x = x;
            s_rest = use_rest;
        }
    }
    __syncthreads();
    const int hit = s_chunk;
    int32_t* token = a.token + (size_t)b * (D + 1) + st.stand;
    if (hit < 0) {
        if (tid == 0) *token = -1;
        return;
    }
    if (hit != chunk) stop_values(a, tr, dr, st, c, hit * kThreads + tid, v);
    double own = 0.0;
    const bool use_rest = s_rest != 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (!use_rest) v.rest[e] = v.all[e];
        own += v.rest[e];
    }
    const double run = wave_scan(own), x = s_x;
    if (lane == 63) s_wave[0][wave] = run;
    __syncthreads();
    double before = s_before;
    for (int w = 0; w < wave; ++w) before += s_wave[0][w];
    before += run - own;
    // the first value whose running sum exceeds x; where rounding leaves none,
    // the chunk's last value above zero
    int first = 0x7FFFFFFF, last = -1;
    const int i0 = 8 * (hit * kThreads + tid) - tr.off;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        before += v.rest[e];
        if (v.rest[e] > 0.0) {
            if (before > x && first == 0x7FFFFFFF) first = i0 + e;
            last = i0 + e;
        }
    }
    const unsigned long long have = __ballot(first != 0x7FFFFFFF), some = __ballot(last >= 0);
    const int f = __shfl(first, have ? (int)__builtin_ctzll(have) : 0), g = __shfl(last, some ? 63 - (int)__builtin_clzll(some) : 0);
    if (lane == 0) {
        s_first[wave] = f;
        s_last[wave] = g;
    }
    __syncthreads();
    if (tid == 0) {
        const int lo = min(min(s_first[0], s_first[1]), min(s_first[2], s_first[3]));
        const int hi = max(max(s_last[0], s_last[1]), max(s_last[2], s_last[3]));
        *token = lo != 0x7FFFFFFF ? lo : hi;
    }
}

double log2e_over(float temperature) { return 1.4426950408889634 / (double)temperature; }
constexpr size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace

namespace {
int topk_blocks(int V, int e) { return (V + kThreads * e - 1) / (kThreads * e); }
// Long blocks share the two sorts of a wave between more logits: 48 sequences
// with 4 drafted tokens, V = 16385, k = 30: 16.8, 14.2 and 13.4 us (both
// launches) at 4, 8 and 16 logits per thread.  Too few workgroups to fill the
// card take short ones: one sequence 8.6, 9.0 and 10.0 us.
int topk_block_e(int B, int D, int V) {
    return (size_t)B * (D + 1) * topk_blocks(V, kLongBlockE) >= 512 ? kLongBlockE : kBlockE;
}
}  // namespace

// The workspace's first kWsCounterBytes are arrival counters (zero before and
// after every call), everything after them is scratch.  Sizes grow with every
// argument (here: as if all blocks were short), so that one made for the largest
// batch serves every smaller one.
size_t verify_topk_ws_bytes(int B, int D, int V, int top_k) {
    if (V <= kDirectVocab) return 0;
    return kWsCounterBytes + (size_t)B * (D + 1) * topk_blocks(V, kBlockE) * top_k * 4;
}

hipError_t launch_verify_topk(const VerifyArgs& a, void* ws, hipStream_t s) {
    const double c = log2e_over(a.temperature);
    const dim3 grid(a.B), block(kRowsAtOnce * 64), pairs(kRowsAtOnce * 2 * 64);
    if (a.V <= kDirectVocab) {
        const uint32_t* none = nullptr;
        if (a.V <= 512) return launch_kernel(verify_topk_kernel<8, 1>, grid, block, 0, s, a, 0, c, none);
        return launch_kernel(verify_topk_kernel<kPairE, 2>, grid, pairs, 0, s, a, 0, c, none);
    }
    const int be = topk_block_e(a.B, a.D, a.V), nb = topk_blocks(a.V, be), nc = nb * a.top_k;
    uint32_t* cand = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(ws) + kWsCounterBytes);
    const dim3 first((unsigned)(a.B * (a.D + 1) * nb)), threads(kThreads);
    hipError_t e = be == kBlockE ? launch_kernel(block_topk_kernel<kBlockE>, first, threads, 0, s, a, nb, cand)
                                 : launch_kernel(block_topk_kernel<kLongBlockE>, first, threads, 0, s, a, nb, cand);
    if (e != hipSuccess) return e;
    const uint32_t* in = cand;
    if (nc <= 512) return launch_kernel(verify_topk_kernel<8, 1>, grid, block, 0, s, a, nc, c, in);
    return launch_kernel(verify_topk_kernel<kPairE, 2>, grid, pairs, 0, s, a, nc, c, in);     // nc <= 30 * 64
}

namespace {
struct FullPlan {
    int rows, mass_steps, mass_j;     // steps of the counting kernel (0: the other, groups per thread)
    size_t mass_chunks, draw_chunks, stop_bytes, mass_bytes;
};
// Chunks of 256 J groups: as many groups per thread as leave the launch two
// workgroups per CU.  A batch of 32 with 131072 logits and 7 drafted tokens runs
// on parts of 8 steps of the counting kernel, one sequence with 16385 on one
// group per thread.
FullPlan full_plan(int B, int D, int V, bool drafts, bool aligned) {
    FullPlan p;
    const size_t g = row_groups(V, aligned);
    const int b = B < kSequences ? B : kSequences;
    auto chunks = [&](int j) { return (g + (size_t)kThreads * j - 1) / ((size_t)kThreads * j); };
    p.rows = D + 1 + (drafts ? D : 0);
    const size_t wanted = 512 / (size_t)b / p.rows + 1;
    p.mass_steps = 0;
    p.mass_j = chunks(4) >= wanted ? 4 : 1;
    p.mass_chunks = chunks(p.mass_j);
    if (chunks(kHistJ) >= wanted && g >= 16 * kThreads) {       // both sides measured at row_mass_hist_kernel
        p.mass_chunks = chunks(kHistJ);
        p.mass_steps = (int)((g + kThreads * kHistStep * p.mass_chunks - 1) / (kThreads * kHistStep * p.mass_chunks));
        p.mass_chunks = chunks(p.mass_steps * kHistStep);
    }
    p.draw_chunks = chunks(1);
    p.stop_bytes = up256((size_t)b * sizeof(Stop));
    p.mass_bytes = up256((size_t)b * p.rows * p.mass_chunks * sizeof(Mass));
    return p;
}
}  // namespace

// Stops, masses by chunk, partial sums by chunk.  The masses are at most
//   2048 with one group per thread (4 x 512, as the next size leaves fewer than
//        512 workgroups),
//   4096 or 4 per row with four (8 x 512, or a row of under 4096 groups),
//   a chunk of kHistJ groups each with the counting kernel.
size_t verify_full_ws_bytes(int B, int D, int V) {
    const size_t b = B < kSequences ? B : kSequences, rows = b * (2 * D + 1), g = row_groups(V, false);
    auto chunks = [&](int j) { return (g + (size_t)kThreads * j - 1) / ((size_t)kThreads * j); };
    const size_t few = chunks(4) < 4 ? chunks(4) : 4, each = few > chunks(kHistJ) ? few : chunks(kHistJ);
    const size_t masses = rows * each > 4096 ? rows * each : 4096;
    return kWsCounterBytes + up256(b * sizeof(Stop)) + up256(masses * sizeof(Mass)) + b * chunks(1) * sizeof(Part);
}

hipError_t launch_verify_full(const VerifyArgs& args, void* ws, hipStream_t s) {
    const bool aligned =
        args.V % 8 == 0 && ((reinterpret_cast<uintptr_t>(args.logits) | reinterpret_cast<uintptr_t>(args.draft_logits)) & 15) == 0;
    const FullPlan p = full_plan(args.B, args.D, args.V, args.draft_logits != nullptr, aligned);
    unsigned* cnt = static_cast<unsigned*>(ws);
    Stop* stop = reinterpret_cast<Stop*>(static_cast<uint8_t*>(ws) + kWsCounterBytes);
    Mass* mass = reinterpret_cast<Mass*>(reinterpret_cast<uint8_t*>(stop) + p.stop_bytes);
    Part* parts = reinterpret_cast<Part*>(reinterpret_cast<uint8_t*>(mass) + p.mass_bytes);
    const double c = log2e_over(args.temperature);
    for (int b0 = 0; b0 < args.B; b0 += kSequences) {
        VerifyArgs a = args;
        const size_t t0 = (size_t)b0 * (a.D + 1), d0 = (size_t)b0 * a.D;
        a.B = args.B - b0 < kSequences ? args.B - b0 : kSequences;
        a.logits += t0 * a.V;
        if (a.draft_logits) a.draft_logits += d0 * a.V;
        a.draft += d0;
        if (a.n_draft) a.n_draft += b0;
        a.u += t0;
        a.token += t0;
        a.count += b0;
        if (a.accept_prob) a.accept_prob += d0;
        const dim3 first((unsigned)((size_t)a.B * p.rows * p.mass_chunks)), second((unsigned)((size_t)a.B * p.draw_chunks)), block(kThreads);
        const int mc = (int)p.mass_chunks, dc = (int)p.draw_chunks;
        hipError_t e = p.mass_steps    ? launch_kernel(row_mass_hist_kernel, first, block, 0, s, a, p.rows, mc, p.mass_steps, c, mass, cnt, stop)
                       : p.mass_j == 4 ? launch_kernel(row_mass_kernel<4>, first, block, 0, s, a, p.rows, mc, c, mass, cnt, stop)
                                       : launch_kernel(row_mass_kernel<1>, first, block, 0, s, a, p.rows, mc, c, mass, cnt, stop);
        if (e != hipSuccess) return e;
        const Stop* st = stop;
        e = launch_kernel(stop_draw_kernel, second, block, 0, s, a, dc, c, st, cnt, parts);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace q4
