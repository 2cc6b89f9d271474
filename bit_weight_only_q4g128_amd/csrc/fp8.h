// Host-side launchers of the 8-bit block-scaled operators (fp8_quant.hip,
// fp8_gemm.hip).  Everything here assumes the arguments were validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "q4gemv.h"

namespace q4 {

// One product y = RN_bf16(sum_g xs[m, g] ws[n / 128, g] sum_k x[m, k] w[n, k] (+ resid)).
struct Fp8Args {
    const uint8_t* x;        // e4m3 [M, K]
    const float* xs;         // [M, G], G = ceil(K / 128)
    const uint8_t* w;        // e4m3 [N, K]
    const float* ws;         // [ceil(N / 128), G]
    const uint16_t* resid;   // bf16 [M, N] or null; may equal y
    uint16_t* y;             // bf16 [M, N]
    int N, K;
    int ld;                  // elements from a row of y and resid to the next
};

constexpr int kFp8Block = 128;    // columns (and weight rows) that share a scale
constexpr int kFp8MaxTasks = 8;   // products of one call

// e4m3 codes and block scales of h = x (up null) or silu(x) * up, bf16 [M, K].
hipError_t launch_fp8_quantize(const uint16_t* x, const uint16_t* up, int M, int K, uint8_t* codes, float* scale, hipStream_t s);

// Up to kFp8MaxTasks products of one batch size M.  ws: a workspace whose
// first 64 KiB are arrival counters (zero, left zero), or null.
hipError_t launch_fp8_gemm(const Fp8Args* tasks, int count, int M, void* ws, size_t ws_bytes, hipStream_t s);
// The workspace with which a call has the launches that any larger one gives
// it (0: none), and the launches that a call with ws_bytes has: how many, and
// the first `most` of them into out.
size_t fp8_gemm_ws_bytes(const Fp8Args* tasks, int count, int M);
int fp8_gemm_launches(const Fp8Args* tasks, int count, int M, size_t ws_bytes, fp8b128_launch* out, int most);

}  // namespace q4
