// e4m3 codes and the scale of a group of values held 8 to a lane: the rounding
// shared by the quantisation of activations (fp8_quant.hip) and the 8-bit
// cache (rope_cache.hip).
//
// With a the largest |h| of the group's finite values:
//     scale = RN_fp32(a / 448),    code = RN_e4m3(h * 448 / a).
// 448 is the largest e4m3 value, so nothing saturates.  A group of zeros has
// scale 0 and codes 0; a value that is not finite gets the NaN code.
//
// The quotient h * 448 / a must round once: for bf16 h it often is an exact
// tie of e4m3, which a quotient off by one fp32 ulp would break.  With
// c = 448 / a held as c_hi (16 significant bits) + c_lo, h * c_hi is exact in
// fp32 for a bf16 h and fma(h, c_lo, h * c_hi) is the quotient times
// 1 + 2^-38, rounded once: an exact tie stays exact, and quotients that are no
// tie differ from one by at least 2^-13 of their value (an 11-bit by an 8-bit
// integer).
#pragma once

#include "common.h"

namespace q4 {

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
    return v > o ? v : o;
}
// largest of aligned groups of LANES = 8 or 16 lanes (a DPP row), in all of them
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
    static_assert(LANES == 8 || LANES == 16, "");
    v = dpp_max<0x141>(dpp_max<0x4E>(dpp_max<0xB1>(v)));
    return LANES == 16 ? dpp_max<0x140>(v) : v;
}

struct Codes8 {
    uint2 codes;   // of the lane's 8 values, in order
    float scale;   // of the group, in every lane
};

// top: the bits of the largest |h| of the lanes' values (integers order as the
// values; infinities and NaNs are above every finite value), already met over
// the group's lanes.
template <int LANES>
__device__ __forceinline__ Codes8 e4m3_codes(float h[8], uint32_t top) {
    float a = __builtin_bit_cast(float, top);
    float s = a;
    // rare: a value that is not finite, or a block so small or large that
    // 1 / a leaves the normal range (scaled by 2^64 or 2^-64, exactly)
    if (__any(!(a < 0x1p100f) || (a < 0x1p-100f && top != 0))) {
        top = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float v = h[k];
            const uint32_t b = __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu;
            if (b >= 0x7F800000u) h[k] = __builtin_nanf("");
            else top = b > top ? b : top;
        }
        top = lanes_max<LANES>(top);
        s = __builtin_bit_cast(float, top);
        const float f = s < 0x1p-100f ? 0x1p64f : s > 0x1p100f ? 0x1p-64f : 1.0f;
        a = s * f;
#pragma unroll
        for (int k = 0; k < 8; ++k) h[k] *= f;
    }
    const float r = __builtin_amdgcn_rcpf(a);
    float hi = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, 448.0f * r) & 0xFFFFFF00u);
    float lo = __builtin_fmaf(-hi, a, 448.0f) * r;
    if (top == 0) hi = lo = 0.0f;
    float c[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) c[k] = __builtin_fmaf(h[k], lo, h[k] * hi);
    int w0 = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], 0, false);
    w0 = __builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], w0, true);
    int w1 = __builtin_amdgcn_cvt_pk_fp8_f32(c[4], c[5], 0, false);
    w1 = __builtin_amdgcn_cvt_pk_fp8_f32(c[6], c[7], w1, true);
    return Codes8{make_uint2((uint32_t)w0, (uint32_t)w1), s / 448.0f};
}

}  // namespace q4
