// C ABI of the verification of drafted tokens: host-side argument checks and
// launches.  Declarations and the contract live in include/q4gemv.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q4gemv.h"
#include "api_util.h"
#include "internal.h"
#include "verify.h"

using q4::aligned;
using q4::overlaps;
using q4::Range;
using q4::range_of;
using q4::VerifyArgs;

namespace {

bool shape_ok(int B, int D, int V, int most) {
    return B >= 1 && D >= 1 && D <= q4::kMaxDraft && V >= 1 && V <= most && (long)B * (D + 1) <= q4::kMaxVerifyRows;
}

int check_verify(const VerifyArgs& a, int most_v, const void* workspace, size_t need, size_t given) {
    if (!a.logits || !a.draft || !a.u || !a.token || !a.count) return Q4_EINVAL_PTR;
    if (!shape_ok(a.B, a.D, a.V, most_v)) return Q4_EINVAL_SHAPE;
    if (!(a.temperature > 0.f) || !(a.temperature < __builtin_huge_valf())) return Q4_EINVAL_SHAPE;
    const size_t rows = (size_t)a.B * (a.D + 1), drafts = (size_t)a.B * a.D;
    if (!aligned(a.logits, 2) || !aligned(a.draft, 4) || !aligned(a.n_draft, 4) || !aligned(a.u, 4) || !aligned(a.draft_index, 4) ||
        !aligned(a.draft_prob, 4) || !aligned(a.draft_logits, 2) || !aligned(a.token, 4) || !aligned(a.count, 4) ||
        !aligned(a.accept_prob, 4))
        return Q4_EALIGN;
    if (need) {
        if (!workspace) return Q4_EINVAL_PTR;
        if (!aligned(workspace, 256)) return Q4_EALIGN;
        if (given < need) return Q4_ESCRATCH;
    }
    const Range none{0, 0};
    const Range in[7] = {range_of(a.logits, rows * a.V * 2), range_of(a.draft, drafts * 4),
                         a.n_draft ? range_of(a.n_draft, (size_t)a.B * 4) : none, range_of(a.u, rows * 4),
                         a.draft_index ? range_of(a.draft_index, drafts * a.draft_k * 4) : none,
                         a.draft_prob ? range_of(a.draft_prob, drafts * a.draft_k * 4) : none,
                         a.draft_logits ? range_of(a.draft_logits, drafts * a.V * 2) : none};
    const Range out[4] = {range_of(a.token, rows * 4), range_of(a.count, (size_t)a.B * 4),
                          a.accept_prob ? range_of(a.accept_prob, drafts * 4) : none, need ? range_of(workspace, need) : none};
    for (int i = 0; i < 4; ++i) {
        for (const Range& r : in)
            if (overlaps(out[i], r)) return Q4_EALIAS;
        for (int j = 0; j < i; ++j)
            if (overlaps(out[i], out[j])) return Q4_EALIAS;
    }
    return Q4_OK;
}

}  // namespace

extern "C" {

size_t q4_verify_topk_workspace_bytes(int B, int D, int V, int top_k) {
    if (!shape_ok(B, D, V, q4::kMaxVocab) || top_k < 1 || top_k > q4::kMaxTopK || top_k > V) return 0;
    return q4::verify_topk_ws_bytes(B, D, V, top_k);
}

int q4_verify_topk(const uint16_t* logits, int B, int D, int V, const int32_t* draft, const int32_t* draft_index,
                   const float* draft_prob, int draft_k, const int32_t* n_draft, const float* u, float temperature, int top_k,
                   int32_t* token, int32_t* count, float* accept_prob, void* workspace, size_t workspace_bytes, void* stream) {
    if (!draft_index != !draft_prob) return Q4_EINVAL_PTR;
    if (top_k < 1 || top_k > q4::kMaxTopK || top_k > V) return Q4_EINVAL_SHAPE;
    if (draft_index && (draft_k < 1 || draft_k > q4::kMaxTopK)) return Q4_EINVAL_SHAPE;
    const VerifyArgs a = {logits, draft, n_draft, u, draft_index, draft_prob, nullptr, token, count, accept_prob,
                          B, D, V, top_k, draft_index ? draft_k : 0, temperature};
    const int rc = check_verify(a, q4::kMaxVocab, workspace, q4_verify_topk_workspace_bytes(B, D, V, top_k), workspace_bytes);
    if (rc) return rc;
    const hipError_t e = q4::launch_verify_topk(a, workspace, reinterpret_cast<hipStream_t>(stream));
    return e == hipSuccess ? Q4_OK : Q4_ELAUNCH;
}

size_t q4_verify_full_workspace_bytes(int B, int D, int V) {
    return shape_ok(B, D, V, q4::kMaxFullVocab) ? q4::verify_full_ws_bytes(B, D, V) : 0;
}

int q4_verify_full(const uint16_t* logits, int B, int D, int V, const int32_t* draft, const uint16_t* draft_logits,
                   const int32_t* n_draft, const float* u, float temperature, int32_t* token, int32_t* count, float* accept_prob,
                   void* workspace, size_t workspace_bytes, void* stream) {
    const VerifyArgs a = {logits, draft, n_draft, u, nullptr, nullptr, draft_logits, token, count, accept_prob,
                          B, D, V, 0, 0, temperature};
    const int rc = check_verify(a, q4::kMaxFullVocab, workspace, q4_verify_full_workspace_bytes(B, D, V), workspace_bytes);
    if (rc) return rc;
    const hipError_t e = q4::launch_verify_full(a, workspace, reinterpret_cast<hipStream_t>(stream));
    return e == hipSuccess ? Q4_OK : Q4_ELAUNCH;
}

}  // extern "C"
