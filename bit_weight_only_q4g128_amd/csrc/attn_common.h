// Device helpers shared by the attention kernels.
#pragma once

#include "common.h"

namespace q4 {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.44269504088896341f;

// the 16-bit halves of two dwords: (low of b, low of a), (high of b, high of a)
__device__ __forceinline__ uint32_t halves_lo(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(a, b, 0x05040100u); }
__device__ __forceinline__ uint32_t halves_hi(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(a, b, 0x07060302u); }

// two fp32 to bf16, rounded to nearest even (one v_cvt_pk_bf16_f32)
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

// Which of a dword's two bf16 values are infinities or NaNs: their bits set.
__device__ __forceinline__ uint32_t odd_halves(uint32_t w) {
    return ((w & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u) | ((w & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u);
}

// v of the lane and of lane ^ 32, lane ^ 16, met (the swapped words are copied
// out before their bits are taken as floats: a cast of a vector's element
// reads its first)
struct Pair {
    float a, b;
};
__device__ __forceinline__ Pair pair_xor32(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
    const uint32_t a = r[0], b = r[1];
    return Pair{__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)};
}
__device__ __forceinline__ Pair pair_xor16(float v) {
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
    const uint32_t a = r[0], b = r[1];
    return Pair{__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)};
}
__device__ __forceinline__ float max_xor32(float v) {
    const Pair p = pair_xor32(v);
    return fmaxf(p.a, p.b);
}
__device__ __forceinline__ float max_xor16(float v) {
    const Pair p = pair_xor16(v);
    return fmaxf(p.a, p.b);
}
__device__ __forceinline__ float sum_xor32(float v) {
    const Pair p = pair_xor32(v);
    return p.a + p.b;
}
__device__ __forceinline__ float sum_xor16(float v) {
    const Pair p = pair_xor16(v);
    return p.a + p.b;
}

// Where a running position falls among B sequences of count(b) units each:
// the sequence, the units before the position inside it, and the units of all
// sequences (seq is -1 where the position lies behind the last).  Every wave
// works it out for itself: each lane counts a run of ceil(B / 64) <= 64
// sequences, the wave sums the runs up to each lane, and the run that holds
// the position is then spread over the lanes the same way.
struct Place {
    int seq;
    int at;
    long total;
};
__device__ __forceinline__ long wave_scan(long v, int lane) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int lo = __shfl_up((int)(uint32_t)v, d), hi = __shfl_up((int)(v >> 32), d);
        if (lane >= d) v += ((long)hi << 32) | (uint32_t)lo;
    }
    return v;
}
__device__ __forceinline__ long wave_pick(long v, int lane) {
    return ((long)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32) | (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
}
template <typename Count>
__device__ __forceinline__ long count_all(int B, int lane, Count count, long& upto, int& run) {
    run = (B + 63) >> 6;
    long mine = 0;
    for (int i = 0; i < run; ++i) {
        const int b = lane * run + i;
        if (b < B) mine += count(b);
    }
    upto = wave_scan(mine, lane);
    return wave_pick(upto, 63);
}
template <typename Count>
__device__ __forceinline__ Place find_place(int B, int lane, long total, long upto, int run, long pos, Count count) {
    if (pos < 0 || pos >= total) return Place{-1, 0, total};
    int owner = __builtin_ctzll(__ballot(upto > pos));
    long before = owner ? wave_pick(upto, owner - 1) : 0;
    int b0 = owner * run;
    if (run > 1) {
        const int b = b0 + lane;
        const long up = wave_scan(lane < run && b < B ? count(b) : 0, lane);
        const int o = __builtin_ctzll(__ballot(up > pos - before));
        if (o) before += wave_pick(up, o - 1);
        b0 += o;
    }
    return Place{b0, (int)(pos - before), total};
}

}  // namespace q4
