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

// ---------------------------------------------------------------------------
// Where a workgroup's part of the work lies among B <= 4096 sequences of some
// units each, which only the device knows.  Every wave works it out for itself:
// a lane counts a run of ceil(B / 64) <= 64 sequences, the wave sums the runs up
// to each lane, and the run that holds a position is then spread over the
// lanes the same way.
// All of this needs the whole wave: a scan reads its neighbours' registers, and
// a lane that is switched off (a branch or the right side of && that only some
// lanes reach) is read as it last was, or not at all, so that the place found
// can lie outside the work.  Lanes without a sequence count 0.
// ---------------------------------------------------------------------------
template <int CTRL, int ROW_MASK = 0xF>
__device__ __forceinline__ uint32_t dpp_add(uint32_t v) {
    return v + (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROW_MASK, 0xF, false);
}
// Inclusive prefix sum over the 64 lanes, all of them active (shifts within rows
// of 16, then the row totals broadcast forward).
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
    v = dpp_add<0x111>(v);
    v = dpp_add<0x112>(v);
    v = dpp_add<0x114>(v);
    v = dpp_add<0x118>(v);
    v = dpp_add<0x142, 0xA>(v);
    return dpp_add<0x143, 0xC>(v);
}
__device__ __forceinline__ uint32_t of_lane(uint32_t v, int lane) { return (uint32_t)__builtin_amdgcn_readlane((int)v, lane); }

struct Runs {
    int run;            // sequences of a lane
    uint32_t upto;      // units up to this lane's run and with it
    uint32_t total;     // of all
};
// (the whole wave)
template <typename Count>
__device__ __forceinline__ Runs count_runs(int B, int lane, Count count) {
    Runs r{(B + 63) >> 6, 0, 0};
    uint32_t mine = 0;
    for (int i = 0; i < r.run; ++i) {
        const int b = lane * r.run + i;
        if (b < B) mine += count(b);
    }
    r.upto = wave_scan(mine);
    r.total = of_lane(r.upto, 63);
    return r;
}

struct Place {
    int seq;         // the sequence that holds a position
    uint32_t at;     // units before the position inside it
};
// pos < r.total, the same in all lanes (the whole wave)
template <typename Count>
__device__ __forceinline__ Place find_place(const Runs& r, int B, int lane, uint32_t pos, Count count) {
    const int owner = __builtin_ctzll(__ballot(r.upto > pos));
    uint32_t before = owner ? of_lane(r.upto, owner - 1) : 0;
    int b0 = owner * r.run;
    if (r.run > 1) {
        const int b = b0 + lane;
        const uint32_t up = wave_scan(lane < r.run && b < B ? count(b) : 0);
        const int o = __builtin_ctzll(__ballot(up > pos - before));
        if (o) before += of_lane(up, o - 1);
        b0 += o;
    }
    return Place{b0, pos - before};
}

}  // namespace q4
