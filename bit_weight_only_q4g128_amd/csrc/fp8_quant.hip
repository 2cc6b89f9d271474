// Quantisation of activations to 8-bit floating point with one scale for each
// 128 columns of a row: the operand form of the block-scaled product
// (fp8_gemm.hip).
//
// Per row m and block g of 128 columns, with h = x, or h = silu(x) * up (the
// gated MLP's activation) in fp32, and a = the largest |h| of the block's
// finite values:
//     scale[m, g] = RN_fp32(a / 448),    code = RN_e4m3(h * 448 / a).
// 448 is the largest e4m3 value, so nothing saturates.  A block of zeros has
// scale 0 and codes 0; a value that is not finite (x, or x * up in fp32) gets
// the NaN code.
//
// The rounding is fp8_codes.h's: the quotient rounds once where h is a bf16
// value.  A gated h is an fp32 number a few ulps from silu(x) up, and its quotient rounds twice:
// about one code in 10^6, whose quotient lies at a tie, is the other neighbour
// than exact arithmetic's (8192 x 8192: 74 to 94 codes of 67 million; the formula in
// fp32 operations 78 to 93, so the fp32 h is the limit).
//
// Bound by memory: 3 bytes per value and 4 per block (5 per value gated).
// Sixteen lanes hold one block (8 columns each, one 16-byte load), a wave four
// blocks of a row; the largest value meets in four DPP steps, so that a value is
// read once and nothing passes through LDS.  Waves are short and many: enough
// loads are in flight without more than one unit per wave.  8192 x 8192 gated:
// 64 us, 5.3 TB/s (a large copy reaches 5.1 TB/s); 4099 x 2000: 6.1 us, 4.1 TB/s,
// from the cache behind L2; 240 x 8192 gated 4.2 us and one row of 2048 1.6 us,
// a launch's own time.
#include "fp8.h"
#include "fp8_codes.h"
#include "internal.h"

namespace q4 {

namespace {

constexpr int kThreads = 256;
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pk_abs_max(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a & 0x7FFF7FFFu),
                                                                  __builtin_bit_cast(u16x2, b & 0x7FFF7FFFu)));
}

// silu(g) * u = g u / (1 + e^-g) in fp32 for bf16 g and u.  g u is exact.
// e^-g = 2^(-g kHi) * e^(-g (1 - kHi ln 2)): kHi holds 16 bits of log2 e, so
// g kHi is exact, the hardware exp2 gives the first factor and 1 - g kLo the
// second (its square term is below 2^-23 for |g| < 87).  The quotient is
// corrected once.  Gates below -87.3, where e^-g nears the largest fp32 value, give 0
// (silu is then under 2^-119).
__device__ __forceinline__ float gated(float g, float u) {
    constexpr float kHi = 1.44268798828125f;    // log2 e to 16 bits
    constexpr float kLo = 4.8884952e-6f;        // (log2 e - kHi) * ln 2
    constexpr float kFar = -87.3f;
    const float gc = fmaxf(g, kFar);
    const float e0 = __builtin_amdgcn_exp2f(-gc * kHi);
    const float d = 1.0f + __builtin_fmaf(e0, -gc * kLo, e0);
    const float n = g * u;
    const float r = g > kFar ? __builtin_amdgcn_rcpf(d) : 0.0f;
    const float q = n * r;
    return __builtin_fmaf(__builtin_fmaf(-q, d, n), r, q);
}

template <bool GATED>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const uint16_t* __restrict__ x, const uint16_t* __restrict__ up, int K,
                                                            int G, int Q, uint64_t magic, uint32_t units,
                                                            uint8_t* __restrict__ codes, float* __restrict__ scale) {
    const int lane = threadIdx.x & 63, j = lane & 15;
    const uint32_t u = blockIdx.x * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (u >= units) return;
    const uint32_t m = (uint32_t)(((uint64_t)u * magic) >> 32);      // u / Q
    const int blk = 4 * (int)(u - m * Q) + (lane >> 4), col = 128 * blk + 8 * j;
    const bool in = col < K;
    const size_t at = (size_t)m * K + col;
    u32x4 xv{0, 0, 0, 0}, uv{0, 0, 0, 0};
    if (in) {
        xv = *reinterpret_cast<const u32x4*>(x + at);
        if (GATED) uv = *reinterpret_cast<const u32x4*>(up + at);
    }
    float h[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        h[2 * k] = bf16lo(xv[k]);
        h[2 * k + 1] = bf16hi(xv[k]);
        if (GATED) {
            h[2 * k] = gated(h[2 * k], bf16lo(uv[k]));
            h[2 * k + 1] = gated(h[2 * k + 1], bf16hi(uv[k]));
        }
    }
    // the bits of the largest |h| (integers order as the values; infinities
    // and NaNs are above every finite value)
    uint32_t top;
    if (GATED) {
        top = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float v = h[k];
            const uint32_t b = __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu;
            top = b > top ? b : top;
        }
    } else {
        const uint32_t p = pk_abs_max(pk_abs_max(xv.x, xv.y), pk_abs_max(xv.z, xv.w));
        const uint32_t hi = p & 0xFFFF0000u, lo = p << 16;
        top = hi > lo ? hi : lo;
    }
    const Codes8 e = e4m3_codes<16>(h, lanes_max<16>(top));
    if (in) *reinterpret_cast<uint2*>(codes + at) = e.codes;
    if (j == 0 && blk < G) scale[(size_t)m * G + blk] = e.scale;
}

template <bool GATED>
hipError_t launch(const uint16_t* x, const uint16_t* up, int M, int K, uint8_t* codes, float* scale, hipStream_t st) {
    const int G = (K + kFp8Block - 1) / kFp8Block, Q = (G + 3) / 4;
    const uint32_t units = (uint32_t)M * (uint32_t)Q;    // at most 2^19 * 64
    // u / Q = u * magic >> 32 for u < 2^25, Q <= 64 (u * Q < 2^32)
    const uint64_t magic = ((1ull << 32) / Q) + 1;
    constexpr uint32_t kWaves = kThreads / 64;
    return launch_kernel(quantize_kernel<GATED>, dim3((units + kWaves - 1) / kWaves), dim3(kThreads), 0, st, x, up, K, G, Q, magic, units,
                         codes, scale);
}

}  // namespace

hipError_t launch_fp8_quantize(const uint16_t* x, const uint16_t* up, int M, int K, uint8_t* codes, float* scale, hipStream_t s) {
    return up ? launch<true>(x, up, M, K, codes, scale, s) : launch<false>(x, nullptr, M, K, codes, scale, s);
}

}  // namespace q4
