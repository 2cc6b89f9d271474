// Heads normalised, rotated to their positions and appended to a paged cache.
//
// Per token t and head of q and k, x the head's D values:
//     h = x * w / sqrt(mean(x^2) + eps)                 (w null: h = x)
//     (a, b) -> (a cos f - b sin f, b cos f + a sin f),  f = pos[t] * inv_freq[i]
// for the rot / 2 pairs, which are elements (i, i + rot / 2), or (2i, 2i + 1)
// interleaved; the remaining elements stay h.  All in fp32, rounded to bf16
// once.  k, and v as it is, go to slot[t] of the cache: bf16, or e4m3 codes
// with one fp32 scale per token and head (fp8_codes.h), from the unrounded h.
//
// The angle is what fp32 cannot hold (position 10^6 at frequency 1 is off by
// 0.03 rad): pos * inv_freq / 2 pi is taken in fp64, whose fraction of a turn
// is exact to 2^-52 of the number of turns, and only that goes to fp32.  A
// table of angles would be read at 2 KB a token beside the 6 KB of its heads;
// here a thread computes one of the workgroup's angles, once for all heads of
// its token.
//
// Bound by memory, or for few tokens by the launch and one chain of loads,
// angles and a barrier.  A head is held by D / 8 lanes (16 bytes each), so a
// wave's load is whole rows; the norm's sum and a group's largest value meet in
// DPP steps, the halves of a pair by one lane move per element.
//
// Measured (16 heads over 4, D = 128, both norms; us of a launch among others):
// one token 4.5; 240 tokens into an e4m3 cache 5.0; 16385 tokens 37.5 into a bf16
// cache (218 MB read and written) and 36.2 into an e4m3 one (186 MB), the same
// again and again, of which the last level's cache holds a part; other tokens and
// caches every time 49 and 46, 4.4 and 4.0 TB/s (a copy of 2 GiB moves 4.9, both
// directions counted).
#include "attention.h"
#include "attn_common.h"
#include "fp8_codes.h"
#include "internal.h"

namespace q4 {

namespace {

constexpr int kThreads = 256;
constexpr int kAngles = 256;     // angles of a workgroup's tokens

struct RopeParams {
    RopeArgs a;
    Cache cache;
    int rows;        // heads of a token that are handled: q, k, and v where there is a cache
    long slots;      // of the cache
};

template <int D, bool kCache, bool kE4m3>
__global__ __launch_bounds__(kThreads) void rope_cache_kernel(const RopeParams p, const int tokens) {
    constexpr int kLanes = D / 8, kGroups = kThreads / kLanes;
    const RopeArgs& a = p.a;
    __shared__ float2 angles[kAngles];
    const int tid = threadIdx.x, lane = tid & 63;
    const int half = a.rot >> 1;
    const int t0 = blockIdx.x * tokens;
    if (half && tid < tokens * half) {
        const int ti = tid / half, i = tid - ti * half;
        if (t0 + ti < a.T) {
            constexpr double kTurn = 0.15915494309189533577;     // 1 / 2 pi
            const double turns = (double)a.pos[t0 + ti] * (double)a.inv_freq[i] * kTurn;
            float s, c;
            sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
            angles[tid] = make_float2(c, s);
        }
    }
    __syncthreads();
    const int group = tid / kLanes, c = tid & (kLanes - 1);
    const int ti = group & (tokens - 1), step = kGroups / tokens;     // tokens is a power of two
    const int t = t0 + ti;
    if (t >= a.T) return;
    // this lane's part of its token's rotation
    const int reach = half >> 3;      // lanes between the halves of a pair (not interleaved)
    const bool turned = 8 * c < a.rot;
    float cs[8], sn[8];
    if (half) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            int i = a.interleaved ? 4 * c + (j >> 1) : 8 * c + j;
            if (!a.interleaved && i >= half) i -= half;
            const float2 f = turned ? angles[ti * half + i] : make_float2(1.0f, 0.0f);
            cs[j] = f.x;
            // the partner's share of the first element of a pair is negative
            sn[j] = (a.interleaved ? (j & 1) == 0 : 8 * c < half) ? -f.y : f.y;
        }
    }
    const int partner = a.interleaved || !turned ? lane : 8 * c < half ? lane + reach : lane - reach;
    float wq[8], wk[8];
    const u32x4 one = u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
    const u32x4 q_w = a.q_norm ? *reinterpret_cast<const u32x4*>(a.q_norm + 8 * c) : one;
    const u32x4 k_w = a.k_norm ? *reinterpret_cast<const u32x4*>(a.k_norm + 8 * c) : one;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        wq[2 * j] = bf16lo(q_w[j]), wq[2 * j + 1] = bf16hi(q_w[j]);
        wk[2 * j] = bf16lo(k_w[j]), wk[2 * j + 1] = bf16hi(k_w[j]);
    }
    long row = -1;      // of the cache, head 0
    if (kCache) {
        const int64_t slot = a.slots[t];
        if (slot >= 0 && slot < p.slots) row = (((slot >> p.cache.shift) * a.Hk) << p.cache.shift) + (slot & ((1 << p.cache.shift) - 1));
    }
    for (int r = group / tokens; r < p.rows; r += step) {
        const bool is_q = r < a.Hq, is_v = r >= a.Hq + a.Hk;
        const int head = is_q ? r : is_v ? r - a.Hq - a.Hk : r - a.Hq;
        const uint16_t* src = is_q ? a.q + t * a.qs : is_v ? a.v + t * a.vs : a.k + t * a.ks;
        const u32x4 x = *reinterpret_cast<const u32x4*>(src + head * D + 8 * c);
        float h[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) h[2 * j] = bf16lo(x[j]), h[2 * j + 1] = bf16hi(x[j]);
        if (!is_v) {
            if (is_q ? a.q_norm != nullptr : a.k_norm != nullptr) {
                float ss = 0.f, eps = a.eps;
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(h[j], h[j], ss);
                ss = group_sum(ss, kLanes);
                const float mean = __builtin_fmaf(ss, 1.0f / D, eps);
                // rare: a mean near the ends of fp32's range, whose squares may have left it or
                // lost bits; head and eps are scaled, which the quotient does not see
                if (!(mean < 0x1p120f) || mean < 0x1p-80f) {
                    const float f = mean < 0x1p-80f ? 0x1p70f : 0x1p-70f;
                    ss = 0.f, eps = eps * f * f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) h[j] *= f, ss = __builtin_fmaf(h[j], h[j], ss);
                    ss = group_sum(ss, kLanes);
                }
                const float inv = rsqrtf(__builtin_fmaf(ss, 1.0f / D, eps));
#pragma unroll
                for (int j = 0; j < 8; ++j) h[j] = h[j] * inv * (is_q ? wq[j] : wk[j]);
            }
            if (half) {
                float o[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = a.interleaved ? h[j ^ 1] : __shfl(h[j], partner);
#pragma unroll
                for (int j = 0; j < 8; ++j) h[j] = turned ? __builtin_fmaf(o[j], sn[j], h[j] * cs[j]) : h[j];
            }
        }
        u32x4 y;
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = pack_bf16(h[2 * j], h[2 * j + 1]);
        if (is_q) {
            *reinterpret_cast<u32x4*>(a.q_out + t * a.qos + head * D + 8 * c) = y;
            continue;
        }
        if (!is_v && a.k_out) *reinterpret_cast<u32x4*>(a.k_out + t * a.kos + head * D + 8 * c) = y;
        if (kCache && row >= 0) {
            const long at = row + ((long)head << p.cache.shift);
            uint8_t* dst = is_v ? p.cache.v : p.cache.k;
            if (kE4m3) {
                uint32_t top = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float v = h[j];
                    const uint32_t b = __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu;
                    top = b > top ? b : top;
                }
                const Codes8 e = e4m3_codes<kLanes>(h, lanes_max<kLanes>(top));
                *reinterpret_cast<uint2*>(dst + at * D + 8 * c) = e.codes;
                if (c == 0) (is_v ? p.cache.vs : p.cache.ks)[at] = e.scale;
            } else {
                *reinterpret_cast<u32x4*>(dst + at * (2 * D) + 16 * c) = y;
            }
        }
    }
}

template <int D>
hipError_t launch(const RopeParams& p, bool cache, hipStream_t s) {
    // Few tokens: one to a workgroup, its heads side by side.  Many: as many as
    // the workgroup has angles for, so that each thread computes one.  us, 16 heads
    // over 4 of 128 (and 64) values: 240 tokens 4.4 (3.8) and 6.7 (6.5); 2048: 8.4
    // (6.6) and 8.7 (7.3); 4096: 13.9 (10.7) and 11.9 (8.5); 16385: 40.7 (32.4) and
    // 34.9 (21.2).
    const int tokens = p.a.T >= 2560 ? kAngles * 2 / D : 1;
    const dim3 grid((p.a.T + tokens - 1) / tokens), block(kThreads);
    if (!cache) return launch_kernel(rope_cache_kernel<D, false, false>, grid, block, 0, s, p, tokens);
    if (!p.cache.ks) return launch_kernel(rope_cache_kernel<D, true, false>, grid, block, 0, s, p, tokens);
    return launch_kernel(rope_cache_kernel<D, true, true>, grid, block, 0, s, p, tokens);
}

}  // namespace

hipError_t launch_rope_cache(const RopeArgs& a, const Cache* cache, hipStream_t s) {
    RopeParams p{a, cache ? *cache : Cache{}, a.Hq + a.Hk + (cache ? a.Hk : 0), 0};
    if (cache) p.slots = (long)cache->pages << cache->shift;
    return a.D == 128 ? launch<128>(p, cache != nullptr, s) : launch<64>(p, cache != nullptr, s);
}

}  // namespace q4
