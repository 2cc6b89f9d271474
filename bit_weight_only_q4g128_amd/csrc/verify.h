// Host-side launchers of the verification of drafted tokens (verify.hip).
// Everything here assumes the arguments were validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace q4 {

constexpr int kMaxDraft = 63;              // drafted tokens per sequence
constexpr int kMaxVerifyRows = 65536;      // B (D + 1)
constexpr int kMaxFullVocab = 1 << 20;     // logits per row of the whole-distribution form

struct VerifyArgs {
    const uint16_t* logits;        // bf16 [B, D + 1, V]: row i is the target's distribution after i drafted tokens
    const int32_t* draft;          // [B, D]
    const int32_t* n_draft;        // [B] or null (D each)
    const float* u;                // [B, D + 1]: D acceptance uniforms, then the draw's
    const int32_t* draft_index;    // top-k form: [B, D, draft_k], or null (the draft was certain of its token)
    const float* draft_prob;       // top-k form: [B, D, draft_k]
    const uint16_t* draft_logits;  // whole form: bf16 [B, D, V], or null (likewise)
    int32_t* token;                // [B, D + 1]
    int32_t* count;                // [B]
    float* accept_prob;            // [B, D] or null
    int B, D, V, top_k, draft_k;
    float temperature;
};

size_t verify_topk_ws_bytes(int B, int D, int V, int top_k);
hipError_t launch_verify_topk(const VerifyArgs& a, void* ws, hipStream_t s);
size_t verify_full_ws_bytes(int B, int D, int V);
hipError_t launch_verify_full(const VerifyArgs& a, void* ws, hipStream_t s);

}  // namespace q4
