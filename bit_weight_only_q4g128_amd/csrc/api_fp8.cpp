// C ABI of the 8-bit block-scaled operators: host-side argument checks and
// launches.  Declarations and the contract live in include/q4gemv.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q4gemv.h"
#include "api_util.h"
#include "fp8.h"

using q4::aligned;
using q4::Fp8Args;
using q4::overlaps;
using q4::Range;
using q4::range_of;

namespace {

constexpr int kMaxM = 1 << 19;
constexpr int kMaxK = 32768;
constexpr int kMaxN = 1 << 24;

bool shape_ok(int M, int K) { return M >= 1 && M <= kMaxM && K >= 16 && K <= kMaxK && K % 16 == 0; }
size_t blocks(int n) { return ((size_t)n + q4::kFp8Block - 1) / q4::kFp8Block; }

// Validation of a group of products: fills a[].
int check_group(const fp8b128_task* tasks, int count, int M, Fp8Args* a) {
    if (!tasks) return Q4_EINVAL_PTR;
    if (count < 1 || count > q4::kFp8MaxTasks) return Q4_EINVAL_SHAPE;
    Range in[q4::kFp8MaxTasks][5], out[q4::kFp8MaxTasks];
    for (int i = 0; i < count; ++i) {
        const fp8b128_task& t = tasks[i];
        if (!t.x || !t.xscale || !t.w || !t.wscale || !t.y) return Q4_EINVAL_PTR;
        if (!shape_ok(M, t.K) || t.N < 1 || t.N > kMaxN) return Q4_EINVAL_SHAPE;
        if (!aligned(t.x, 16) || !aligned(t.w, 16) || !aligned(t.xscale, 4) || !aligned(t.wscale, 4) || !aligned(t.y, 2) ||
            (t.residual && !aligned(t.residual, 2)))
            return Q4_EALIGN;
        const size_t G = blocks(t.K), ybytes = (size_t)M * t.N * 2;
        in[i][0] = range_of(t.x, (size_t)M * t.K);
        in[i][1] = range_of(t.xscale, (size_t)M * G * 4);
        in[i][2] = range_of(t.w, (size_t)t.N * t.K);
        in[i][3] = range_of(t.wscale, blocks(t.N) * G * 4);
        // a residual that is exactly this task's y is read before each element is written
        in[i][4] = t.residual && t.residual != t.y ? range_of(t.residual, ybytes) : Range{0, 0};
        out[i] = range_of(t.y, ybytes);
        a[i] = Fp8Args{t.x, t.xscale, t.w, t.wscale, t.residual, t.y, t.N, t.K, t.N};
    }
    for (int i = 0; i < count; ++i)
        for (int j = 0; j < count; ++j) {
            for (const Range& r : in[j])
                if (overlaps(out[i], r)) return Q4_EALIAS;
            if (i != j && overlaps(out[i], out[j])) return Q4_EALIAS;
        }
    return Q4_OK;
}

// The workspace, where one is given, lies apart from every argument.
int check_workspace(const Fp8Args* a, int count, int M, const void* workspace, size_t bytes) {
    if (!workspace || !bytes) return Q4_OK;
    if (!aligned(workspace, 256)) return Q4_EALIGN;
    const Range w = range_of(workspace, bytes);
    for (int i = 0; i < count; ++i) {
        const size_t G = blocks(a[i].K);
        const Range all[6] = {range_of(a[i].x, (size_t)M * a[i].K), range_of(a[i].xs, (size_t)M * G * 4),
                              range_of(a[i].w, (size_t)a[i].N * a[i].K), range_of(a[i].ws, blocks(a[i].N) * G * 4),
                              a[i].resid ? range_of(a[i].resid, (size_t)M * a[i].N * 2) : Range{0, 0},
                              range_of(a[i].y, (size_t)M * a[i].N * 2)};
        for (const Range& r : all)
            if (overlaps(w, r)) return Q4_EALIAS;
    }
    return Q4_OK;
}

}  // namespace

extern "C" {

int fp8b128_quantize(const uint16_t* x, const uint16_t* up, int M, int K, uint8_t* codes, float* scale, void* stream) {
    if (!x || !codes || !scale) return Q4_EINVAL_PTR;
    if (!shape_ok(M, K)) return Q4_EINVAL_SHAPE;
    if (!aligned(x, 16) || (up && !aligned(up, 16)) || !aligned(codes, 16) || !aligned(scale, 4)) return Q4_EALIGN;
    const size_t n = (size_t)M * K;
    const Range cr = range_of(codes, n), sr = range_of(scale, (size_t)M * blocks(K) * 4), xr = range_of(x, n * 2),
                ur = up ? range_of(up, n * 2) : Range{0, 0};
    if (overlaps(cr, sr) || overlaps(cr, xr) || overlaps(cr, ur) || overlaps(sr, xr) || overlaps(sr, ur)) return Q4_EALIAS;
    const hipError_t e = q4::launch_fp8_quantize(x, up, M, K, codes, scale, reinterpret_cast<hipStream_t>(stream));
    return e == hipSuccess ? Q4_OK : Q4_ELAUNCH;
}

int fp8b128_gemm_grouped_ws(const fp8b128_task* tasks, int count, int M, void* workspace, size_t workspace_bytes, void* stream) {
    Fp8Args a[q4::kFp8MaxTasks];
    int rc = check_group(tasks, count, M, a);
    if (rc) return rc;
    rc = check_workspace(a, count, M, workspace, workspace_bytes);
    if (rc) return rc;
    const hipError_t e = q4::launch_fp8_gemm(a, count, M, workspace_bytes ? workspace : nullptr, workspace_bytes,
                                             reinterpret_cast<hipStream_t>(stream));
    return e == hipSuccess ? Q4_OK : Q4_ELAUNCH;
}

int fp8b128_workspace_bytes(const fp8b128_task* tasks, int count, int M, size_t* bytes) {
    if (!bytes) return Q4_EINVAL_PTR;
    Fp8Args a[q4::kFp8MaxTasks];
    const int rc = check_group(tasks, count, M, a);
    if (rc) return rc;
    *bytes = q4::fp8_gemm_ws_bytes(a, count, M);
    return Q4_OK;
}

int fp8b128_launches(const fp8b128_task* tasks, int count, int M, size_t workspace_bytes, fp8b128_launch* out, int most, int* launches) {
    if (!launches || (most > 0 && !out)) return Q4_EINVAL_PTR;
    Fp8Args a[q4::kFp8MaxTasks];
    const int rc = check_group(tasks, count, M, a);
    if (rc) return rc;
    *launches = q4::fp8_gemm_launches(a, count, M, workspace_bytes, out, most);
    return Q4_OK;
}

int fp8b128_gemm(const uint8_t* x, const float* xscale, int M, int K, const uint8_t* w, const float* wscale, int N,
                 const uint16_t* residual, uint16_t* y, void* stream) {
    const fp8b128_task t = {x, xscale, w, wscale, residual, y, N, K};
    return fp8b128_gemm_grouped_ws(&t, 1, M, nullptr, 0, stream);
}

}  // extern "C"
