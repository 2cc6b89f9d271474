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
// that of unpacked fp32; a token can differ from exact arithmetic only where a
// uniform lies within about 1e-11 of a boundary.
#include "internal.h"
#include "topk.h"
#include "verify.h"

namespace q4 {

namespace {

constexpr int kThreads = 256;

// 2^y by the Taylor series of 2^f on |f| <= 1/2 (relative error 7e-12); y
// below -1100, and NaN, give 0.
__device__ __forceinline__ double exp2_64(double y) {
    y = __builtin_fmax(y, -1100.0);
    const double n = __builtin_rint(y), f = y - n;
    double p = 1.0178086009239699e-07;                       // (ln 2)^9 / 9!
    p = __builtin_fma(p, f, 1.3215486790144307e-06);
    p = __builtin_fma(p, f, 1.5252733804059841e-05);
    p = __builtin_fma(p, f, 1.5403530393381608e-04);
    p = __builtin_fma(p, f, 1.3333558146428443e-03);
    p = __builtin_fma(p, f, 9.6181291076284770e-03);
    p = __builtin_fma(p, f, 5.5504108664821580e-02);
    p = __builtin_fma(p, f, 2.4022650695910072e-01);
    p = __builtin_fma(p, f, 6.9314718055994531e-01);
    p = __builtin_fma(p, f, 1.0);
    return __builtin_amdgcn_ldexp(p, (int)n);
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int s = 1; s < 64; s *= 2) v += __shfl_xor(v, s);
    return v;
}
__device__ __forceinline__ double wave_scan(double v, int lane) {      // inclusive
#pragma unroll
    for (int s = 1; s < 64; s *= 2) {
        const double o = __shfl_up(v, s);
        v += lane >= s ? o : 0.0;
    }
    return v;
}
__device__ __forceinline__ double lane_value(double v, int lane) { return __shfl(v, lane); }

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

// The outputs of sequence b: the tokens that stand, the new one, -1 behind it.
__device__ __forceinline__ void write_tokens(const VerifyArgs& a, int b, int stand, int token, int tid) {
    if (tid <= a.D) a.token[(size_t)b * (a.D + 1) + tid] = tid < stand ? a.draft[(size_t)b * a.D + tid] : tid == stand ? token : -1;
    if (tid == 0) a.count[b] = stand;
}

// ---------------------------------------------------------------------------
// top-k form.  Rows of at most kDirectVocab logits: one launch, a workgroup
// per sequence, a wave per row.  Longer rows: a first launch takes the top k
// of every block of 1024 logits, and the waves of the second merge a row's
// candidates.  Nothing is handed over inside a launch.
// ---------------------------------------------------------------------------
constexpr int kTopkWaves = 8;
constexpr int kDirectE = 40;                        // logits per lane of the one-launch form
constexpr int kDirectVocab = 64 * kDirectE;

// NaN counts as -inf
__device__ __forceinline__ uint32_t entry_of(uint32_t bits, int col) {
    return topk_entry((bits & 0x7FFFu) > 0x7F80u ? 0xFF80u : bits, col);
}

__global__ __launch_bounds__(kThreads) void block_topk_kernel(VerifyArgs a, int nb, uint32_t* cand) {
    __shared__ uint32_t lists[4 * 64];
    __shared__ uint32_t scratch[4 * 64 * 4];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int row = blockIdx.x / nb, j = blockIdx.x - row * nb;
    const int b = row / (a.D + 1), r = row - b * (a.D + 1);
    if (r > drafted(a, b)) return;                        // no drafted token leads here
    const uint16_t* lg = a.logits + (size_t)row * a.V;
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int col = j * kSplitBlock + tid + 256 * i;
        v[i] = lg[col < a.V ? col : 0];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int col = j * kSplitBlock + tid + 256 * i;
        v[i] = col < a.V ? entry_of(v[i], col) : 0u;
    }
    const uint32_t top = wg_topk<4>(v, a.top_k, lists, scratch, wave, lane);
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

// One workgroup per sequence.  cand null: rows are read as they are.
template <int E>
__global__ __launch_bounds__(kTopkWaves * 64) void verify_topk_kernel(VerifyArgs a, int nc, double c, const uint32_t* cand) {
    __shared__ uint32_t scratch[kTopkWaves][64 * E];
    __shared__ double s_p[kMaxDraft + 1][64];
    __shared__ int s_index[kMaxDraft + 1][64];
    __shared__ int s_ok[kMaxDraft + 1];
    __shared__ int s_token;
    __shared__ int s_qi[64];
    __shared__ float s_qp[64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int b = blockIdx.x, n = drafted(a, b), k = a.top_k;

    for (int i = wave; i <= n; i += kTopkWaves) {
        const size_t row = (size_t)b * (a.D + 1) + i;
        uint32_t v[E];
        if (cand) {
            const uint32_t* cr = cand + row * nc;
#pragma unroll
            for (int j = 0; j < E; ++j) v[j] = cr[lane + 64 * j < nc ? lane + 64 * j : 0];
#pragma unroll
            for (int j = 0; j < E; ++j) v[j] = lane + 64 * j < nc ? v[j] : 0u;
        } else {
            const uint16_t* lg = a.logits + row * a.V;
#pragma unroll
            for (int j = 0; j < E; ++j) v[j] = lg[lane + 64 * j < a.V ? lane + 64 * j : 0];
#pragma unroll
            for (int j = 0; j < E; ++j) v[j] = lane + 64 * j < a.V ? entry_of(v[j], lane + 64 * j) : 0u;
        }
        const uint32_t e = wave_topk_sorted<E, true>(v, k, scratch[wave], lane);
        const int index = (int)(0xFFFFu - (e & 0xFFFFu));
        const double p = topk_prob64(e, k, c, lane);
        s_p[i][lane] = p;
        s_index[i][lane] = index;
        if (i == n) continue;
        const int d = a.draft[(size_t)b * a.D + i];
        const double pd = wave_sum(index == d ? p : 0.0);
        double qd = 1.0;
        if (a.draft_index) {
            const size_t at = ((size_t)b * a.D + i) * a.draft_k;
            qd = wave_sum(lane < a.draft_k && a.draft_index[at + lane] == d ? (double)a.draft_prob[at + lane] : 0.0);
        }
        if (lane == 0) {
            s_ok[i] = (double)a.u[(size_t)b * (a.D + 1) + i] * qd < pd;
            if (a.accept_prob) a.accept_prob[(size_t)b * a.D + i] = accept_ratio(pd, qd);
        }
    }
    if (a.accept_prob && tid >= n && tid < a.D) a.accept_prob[(size_t)b * a.D + tid] = 0.f;
    __syncthreads();
    int stand = 0;
    while (stand < n && s_ok[stand]) ++stand;
    if (wave == 0) {
        const int index = s_index[stand][lane];
        const double p = s_p[stand][lane];
        double q = 0.0;
        if (stand < n) {
            if (a.draft_index) {
                const size_t at = ((size_t)b * a.D + stand) * a.draft_k;
                if (lane < a.draft_k) {
                    s_qi[lane] = a.draft_index[at + lane];
                    s_qp[lane] = a.draft_prob[at + lane];
                }
                __builtin_amdgcn_wave_barrier();
                for (int i = 0; i < a.draft_k; ++i) q += s_qi[i] == index ? (double)s_qp[i] : 0.0;
            } else {
                q = index == a.draft[(size_t)b * a.D + stand] ? 1.0 : 0.0;
            }
        }
        double g = __builtin_fmax(p - q, 0.0);
        if (!(wave_sum(g) > 0.0)) g = p;
        const double run = wave_scan(g, lane), total = lane_value(run, 63);
        const double x = (double)a.u[(size_t)b * (a.D + 1) + a.D] * total;
        const unsigned long long over = __ballot(run > x && g > 0.0), any = __ballot(g > 0.0);
        const int pick = over ? (int)__builtin_ctzll(over) : any ? 63 - (int)__builtin_clzll(any) : -1;
        const int token = pick < 0 ? -1 : __shfl(index, pick);
        if (lane == 0) s_token = token;
    }
    __syncthreads();
    write_tokens(a, b, stand, s_token, tid);
}

// ---------------------------------------------------------------------------
// whole form: a launch for the masses of all rows, one for the acceptance and
// the draw.
//
// A row starts at any even address.  It is read as the 16-byte aligned groups
// of 8 logits that touch it; the first and the last, where the row ends inside
// them, value by value.
// ---------------------------------------------------------------------------
constexpr int kMassGroups = 1024;      // groups of 8 logits per workgroup of the first launch
constexpr int kDrawGroups = 512;       // of the second: 2 adjacent groups per thread

struct Row {
    const uint16_t* p;     // first logit
    int off, groups;       // logits of the first group that lie before it; groups that touch the row
};
__device__ __forceinline__ Row row_of(const uint16_t* p, int V) {
    const int off = (int)((reinterpret_cast<uintptr_t>(p) & 15) >> 1);
    return Row{p, off, (off + V + 7) >> 3};
}
__host__ __device__ constexpr int row_groups_most(int V) { return (V + 14) >> 3; }

// The 8 logits of group g as fp32, -inf where the group lies outside the row.
__device__ __forceinline__ void load_group(const Row& r, int V, int g, float (&z)[8]) {
    const int i0 = 8 * g - r.off;
    if (i0 >= 0 && i0 + 8 <= V) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(r.p + i0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            z[2 * i] = bf16lo(v[i]);
            z[2 * i + 1] = bf16hi(v[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool in = i0 + i >= 0 && i0 + i < V;
            z[i] = in ? __builtin_bit_cast(float, (uint32_t)r.p[in ? i0 + i : 0] << 16) : -__builtin_huge_valf();
        }
    }
}

struct Mass {       // sum of 2^((z - top) c) and top of a part of a row
    double sum;
    double top;
};

// Block (row, chunk): rows are the target's B (D + 1), then the draft's B D.
// The first block of a sequence clears the counter of the second launch.
__global__ __launch_bounds__(kThreads) void row_mass_kernel(VerifyArgs a, int chunks, double c, Mass* mass, unsigned* cnt) {
    __shared__ float s_top[4];
    __shared__ double s_sum[4];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int row = blockIdx.x / chunks, chunk = blockIdx.x - row * chunks;
    const int targets = a.B * (a.D + 1);
    const bool target = row < targets;
    const int per = target ? a.D + 1 : a.D, at = target ? row : row - targets;
    const int b = at / per, i = at - b * per;
    if (target && i == 0 && chunk == 0 && tid == 0) cnt[(size_t)b * kCtrWords] = 0;
    if (i >= drafted(a, b) + (target ? 1 : 0)) return;
    const Row r = row_of((target ? a.logits : a.draft_logits) + (size_t)at * a.V, a.V);
    float z[4][8];
    float top = -__builtin_huge_valf();
#pragma unroll
    for (int j = 0; j < 4; ++j) load_group(r, a.V, chunk * kMassGroups + j * kThreads + tid, z[j]);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, z[j][e]);
#pragma unroll
    for (int s = 1; s < 64; s *= 2) top = fmaxf(top, __shfl_xor(top, s));
    if (lane == 0) s_top[wave] = top;
    __syncthreads();
    top = fmaxf(fmaxf(s_top[0], s_top[1]), fmaxf(s_top[2], s_top[3]));
    double sum = 0.0;
    const double base = -(double)top * c;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += exp2_64(__builtin_fma((double)z[j][e], c, base));
    sum = wave_sum(sum);
    if (lane == 0) s_sum[wave] = sum;
    __syncthreads();
    if (tid == 0) mass[(size_t)row * chunks + chunk] = Mass{s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3], (double)top};
}

// The mass of a whole row from its parts (a wave); sum 0 for a row without a
// distribution.
__device__ __forceinline__ Mass row_mass(const Mass* part, int chunks, double c, int lane) {
    double top = -__builtin_huge_val();
    for (int i = lane; i < chunks; i += 64) top = __builtin_fmax(top, part[i].top);
#pragma unroll
    for (int s = 1; s < 64; s *= 2) top = __builtin_fmax(top, __shfl_xor(top, s));
    if (!(top > -__builtin_huge_val() && top < __builtin_huge_val())) return Mass{0.0, 0.0};
    double sum = 0.0;
    for (int i = lane; i < chunks; i += 64) sum += part[i].sum * exp2_64((part[i].top - top) * c);
    return Mass{wave_sum(sum), top};
}

__device__ __forceinline__ double prob(float z, const Mass& m, double inv, double c) {
    return exp2_64(((double)z - m.top) * c) * inv;      // inv = 1 / sum, or 0 for a row without a distribution
}

struct Part {
    double rest, all;    // sums of max(p - q, 0) and of p over a chunk
};

// The stop row's values of a thread's 16 adjacent logits.
struct Values {
    double rest[16], all[16];
};
__device__ __forceinline__ void stop_values(const VerifyArgs& a, const Row& tr, const Row& dr, bool has_q, int qtoken, const Mass& pm,
                                            double pinv, const Mass& qm, double qinv, double c, int g0, Values& o) {
    float z[8], y[8];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        load_group(tr, a.V, g0 + j, z);
        const int i0 = 8 * (g0 + j) - tr.off;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const double p = prob(z[e], pm, pinv, c);
            o.all[8 * j + e] = p;
            o.rest[8 * j + e] = i0 + e == qtoken ? 0.0 : p;
        }
        if (has_q) {
            if (dr.off == tr.off) {
                load_group(dr, a.V, g0 + j, y);
            } else {        // the draft's row starts at another place of its group
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int i = i0 + e;
                    const bool in = i >= 0 && i < a.V;
                    y[e] = in ? __builtin_bit_cast(float, (uint32_t)dr.p[in ? i : 0] << 16) : -__builtin_huge_valf();
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) o.rest[8 * j + e] = __builtin_fmax(o.all[8 * j + e] - prob(y[e], qm, qinv, c), 0.0);
        }
    }
}

// Block (b, chunk).
__global__ __launch_bounds__(kThreads) void verify_full_kernel(VerifyArgs a, int mass_chunks, int chunks, double c, const Mass* mass,
                                                               unsigned* cnt, Part* parts) {
    __shared__ Mass s_mass[2 * kMaxDraft + 1];
    __shared__ double s_wave[2][4];
    __shared__ unsigned s_prev;
    __shared__ int s_stand, s_token, s_chunk;
    __shared__ double s_before, s_x;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int b = blockIdx.x / chunks, chunk = blockIdx.x - b * chunks;
    const int n = drafted(a, b), D = a.D, V = a.V;
    const int targets = a.B * (D + 1);

    // the masses of the sequence's rows: target 0 .. n, draft 0 .. n - 1
    const int rows = n + 1 + (a.draft_logits ? n : 0);
    for (int i = wave; i < rows; i += 4) {
        const size_t row = i <= n ? (size_t)b * (D + 1) + i : (size_t)targets + (size_t)b * D + (i - n - 1);
        const Mass m = row_mass(mass + row * mass_chunks, mass_chunks, c, lane);
        if (lane == 0) s_mass[i] = m;
    }
    __syncthreads();
    if (wave == 0) {        // lane i: drafted token i
        bool ok = false;
        if (lane < n) {
            const int d = a.draft[(size_t)b * D + lane];
            const bool in = d >= 0 && d < V;
            double pd = 0.0, qd = in ? 1.0 : 0.0;
            if (in) {
                const Mass m = s_mass[lane];
                const uint32_t z = a.logits[((size_t)b * (D + 1) + lane) * V + d];
                pd = prob(__builtin_bit_cast(float, z << 16), m, m.sum > 0.0 ? 1.0 / m.sum : 0.0, c);
                if (a.draft_logits) {
                    const Mass w = s_mass[n + 1 + lane];
                    const uint32_t y = a.draft_logits[((size_t)b * D + lane) * V + d];
                    qd = prob(__builtin_bit_cast(float, y << 16), w, w.sum > 0.0 ? 1.0 / w.sum : 0.0, c);
                }
            }
            ok = (double)a.u[(size_t)b * (D + 1) + lane] * qd < pd;
            if (a.accept_prob && chunk == 0) a.accept_prob[(size_t)b * D + lane] = accept_ratio(pd, qd);
        } else if (lane < D && a.accept_prob && chunk == 0) {
            a.accept_prob[(size_t)b * D + lane] = 0.f;
        }
        const unsigned long long no = ~__ballot(ok);          // (lanes n .. 63 are never ok, and n <= 63)
        if (lane == 0) s_stand = (int)__builtin_ctzll(no);
    }
    __syncthreads();
    const int stand = s_stand;
    const bool refused = stand < n, has_q = refused && a.draft_logits;
    const int qtoken = refused && !a.draft_logits ? a.draft[(size_t)b * D + stand] : -1;
    const Row tr = row_of(a.logits + ((size_t)b * (D + 1) + stand) * V, V);
    const Row dr = has_q ? row_of(a.draft_logits + ((size_t)b * D + stand) * V, V) : tr;
    const Mass pm = s_mass[stand], qm = has_q ? s_mass[n + 1 + stand] : Mass{0.0, 0.0};
    const double pinv = pm.sum > 0.0 ? 1.0 / pm.sum : 0.0, qinv = qm.sum > 0.0 ? 1.0 / qm.sum : 0.0;

    Values v;
    stop_values(a, tr, dr, has_q, qtoken, pm, pinv, qm, qinv, c, chunk * kDrawGroups + 2 * tid, v);
    double rest = 0.0, all = 0.0;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
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
    if (tid == 0) {
        put(&mine[chunk].rest, s_wave[0][0] + s_wave[0][1] + s_wave[0][2] + s_wave[0][3]);
        put(&mine[chunk].all, s_wave[1][0] + s_wave[1][1] + s_wave[1][2] + s_wave[1][3]);
    }
    if (!arrive_last(cnt + (size_t)b * kCtrWords, chunks, tid, &s_prev)) return;

    // the chunk where the running sum crosses u_D times the total
    if (wave == 0) {
        const int per = (chunks + 63) >> 6;
        double rs = 0.0, as = 0.0;
        for (int i = lane * per; i < (lane + 1) * per && i < chunks; ++i) {
            rs += get(&mine[i].rest);
            as += get(&mine[i].all);
        }
        const bool use_rest = wave_sum(rs) > 0.0;
        const double own = use_rest ? rs : as;
        const double run = wave_scan(own, lane), total = lane_value(run, 63);
        const double x = (double)a.u[(size_t)b * (D + 1) + D] * total;
        const unsigned long long over = __ballot(run > x), any = __ballot(own > 0.0);
        const int l = over ? (int)__builtin_ctzll(over) : any ? 63 - (int)__builtin_clzll(any) : -1;
        if (l < 0) {
            if (lane == 0) s_chunk = -1;
        } else if (lane == l) {
            double before = run - own;
            int at = -1;
            for (int i = lane * per; i < (lane + 1) * per && i < chunks; ++i) {
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
            s_stand = use_rest ? 1 : 0;
        }
    }
    if (tid == 0) s_token = -1;
    __syncthreads();
    const int hit = s_chunk;
    if (hit >= 0) {
        const bool use_rest = s_stand != 0;
        const double x = s_x;
        stop_values(a, tr, dr, has_q, qtoken, pm, pinv, qm, qinv, c, hit * kDrawGroups + 2 * tid, v);
        double own = 0.0;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            if (!use_rest) v.rest[e] = v.all[e];
            own += v.rest[e];
        }
        const double run = wave_scan(own, lane);
        __syncthreads();
        if (lane == 63) s_wave[0][wave] = run;
        __syncthreads();
        double before = s_before;
        for (int w = 0; w < wave; ++w) before += s_wave[0][w];
        before += run - own;
        // the first value whose running sum exceeds x; where rounding leaves
        // none, the chunk's last value above zero
        int first = 0x7FFFFFFF, last = -1;
        const int i0 = 8 * (hit * kDrawGroups + 2 * tid) - tr.off;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            before += v.rest[e];
            if (v.rest[e] > 0.0) {
                if (before > x && first == 0x7FFFFFFF) first = i0 + e;
                last = i0 + e;
            }
        }
#pragma unroll
        for (int s = 1; s < 64; s *= 2) {
            first = min(first, __shfl_xor(first, s));
            last = max(last, __shfl_xor(last, s));
        }
        __shared__ int s_first[4], s_last[4];
        if (lane == 0) {
            s_first[wave] = first;
            s_last[wave] = last;
        }
        __syncthreads();
        if (tid == 0) {
            const int f = min(min(s_first[0], s_first[1]), min(s_first[2], s_first[3]));
            const int l = max(max(s_last[0], s_last[1]), max(s_last[2], s_last[3]));
            s_token = f != 0x7FFFFFFF ? f : l;
        }
        __syncthreads();
    }
    write_tokens(a, b, stand, s_token, tid);
}

double log2e_over(float temperature) { return 1.4426950408889634 / (double)temperature; }
constexpr size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace

// The workspace's first kWsCounterBytes stay as they are (other calls' arrival
// counters); everything after them is scratch that needs no clearing.
size_t verify_topk_ws_bytes(int B, int D, int V, int top_k) {
    if (V <= kDirectVocab) return 0;
    const size_t nb = (V + kSplitBlock - 1) / kSplitBlock;
    return kWsCounterBytes + (size_t)B * (D + 1) * nb * top_k * 4;
}

hipError_t launch_verify_topk(const VerifyArgs& a, void* ws, hipStream_t s) {
    const double c = log2e_over(a.temperature);
    const dim3 grid(a.B), block(kTopkWaves * 64);
    if (a.V <= kDirectVocab) {
        const uint32_t* none = nullptr;
        if (a.V <= 512) return launch_kernel(verify_topk_kernel<8>, grid, block, 0, s, a, 0, c, none);
        return launch_kernel(verify_topk_kernel<kDirectE>, grid, block, 0, s, a, 0, c, none);
    }
    const int nb = (a.V + kSplitBlock - 1) / kSplitBlock, nc = nb * a.top_k;
    uint32_t* cand = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(ws) + kWsCounterBytes);
    hipError_t e = launch_kernel(block_topk_kernel, dim3((unsigned)(a.B * (a.D + 1) * nb)), dim3(kThreads), 0, s, a, nb, cand);
    if (e != hipSuccess) return e;
    const uint32_t* in = cand;
    if (nc <= 512) return launch_kernel(verify_topk_kernel<8>, grid, block, 0, s, a, nc, c, in);
    return launch_kernel(verify_topk_kernel<32>, grid, block, 0, s, a, nc, c, in);     // nc <= 30 * 64
}

// Sequence counters (cleared by the first launch), the rows' masses by chunk,
// the sequences' partial sums by chunk.
size_t verify_full_ws_bytes(int B, int D, int V) {
    const size_t rows = (size_t)B * (2 * D + 1), g = row_groups_most(V);
    const size_t mc = (g + kMassGroups - 1) / kMassGroups, dc = (g + kDrawGroups - 1) / kDrawGroups;
    return kWsCounterBytes + up256((size_t)B * kCtrStride) + up256(rows * mc * sizeof(Mass)) + (size_t)B * dc * sizeof(Part);
}

hipError_t launch_verify_full(const VerifyArgs& a, void* ws, hipStream_t s) {
    const size_t rows = (size_t)a.B * (2 * a.D + 1), g = row_groups_most(a.V);
    const int mc = (int)((g + kMassGroups - 1) / kMassGroups), dc = (int)((g + kDrawGroups - 1) / kDrawGroups);
    uint8_t* p = static_cast<uint8_t*>(ws) + kWsCounterBytes;
    unsigned* cnt = reinterpret_cast<unsigned*>(p);
    Mass* mass = reinterpret_cast<Mass*>(p + up256((size_t)a.B * kCtrStride));
    Part* parts = reinterpret_cast<Part*>(reinterpret_cast<uint8_t*>(mass) + up256(rows * mc * sizeof(Mass)));
    const double c = log2e_over(a.temperature);
    const size_t run = a.draft_logits ? rows : (size_t)a.B * (a.D + 1);
    hipError_t e = launch_kernel(row_mass_kernel, dim3((unsigned)(run * mc)), dim3(kThreads), 0, s, a, mc, c, mass, cnt);
    if (e != hipSuccess) return e;
    return launch_kernel(verify_full_kernel, dim3((unsigned)(a.B * dc)), dim3(kThreads), 0, s, a, mc, dc, c, (const Mass*)mass, cnt,
                         parts);
}

}  // namespace q4
