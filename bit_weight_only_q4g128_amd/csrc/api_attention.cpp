// C ABI of the attention operators: host-side argument checks and launches.
// Declarations and the contract live in include/q4gemv.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q4gemv.h"
#include "api_util.h"
#include "attention.h"

using q4::aligned;
using q4::overlaps;
using q4::Range;
using q4::range_of;

namespace {

constexpr int kMaxTokens = 1 << 22;
constexpr int kMaxHeads = 256;
constexpr int kMaxNew = 64;                // new tokens of a sequence
constexpr long kMaxKeys = 1l << 24;        // of a sequence's table
constexpr long kMaxUnits = 1l << 31;       // of a decode call
constexpr size_t kMaxRows = 1ul << 31;     // of a cache, each head's counted
constexpr int64_t kMaxStride = 1l << 24;

bool heads_ok(int Hq, int Hk, int D) {
    return Hk >= 1 && Hq >= Hk && Hq <= kMaxHeads && Hq % Hk == 0 && (D == 64 || D == 128);
}
bool stride_ok(int64_t stride, int heads, int D) { return stride >= (int64_t)heads * D && stride <= kMaxStride && stride % 8 == 0; }
bool positive(float f) { return f > 0.f && f < __builtin_huge_valf(); }
bool scale_ok(float f) { return f > 0.f && f <= 0x1p127f; }      // times log2 e it is finite

// Rows of `width` elements, `stride` elements from one to the next.
struct Rows {
    const uint16_t* p;
    int64_t rows, stride, width;
};
Range range_of_rows(const Rows& r) { return r.p ? range_of(r.p, (size_t)((r.rows - 1) * r.stride + r.width) * 2) : Range{0, 0}; }
// Parts of one array of rows lie between each other and need not overlap.
bool rows_overlap(const Rows& a, const Rows& b) {
    if (!a.p || !b.p || !overlaps(range_of_rows(a), range_of_rows(b))) return false;
    if (a.stride != b.stride) return true;
    const int64_t apart = (reinterpret_cast<intptr_t>(b.p) - reinterpret_cast<intptr_t>(a.p)) / 2;
    const int64_t d = ((apart % a.stride) + a.stride) % a.stride;      // where b's row begins in a's
    return !(d >= a.width && d + b.width <= a.stride);
}

struct CacheRanges {
    Range r[4];
};
int check_cache(const q4_kv_cache* c, int Hk, int D, q4::Cache* out, CacheRanges* ranges) {
    if (!c->k || !c->v || !c->k_scale != !c->v_scale) return Q4_EINVAL_PTR;
    if (c->pages < 1 || c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1))) return Q4_EINVAL_SHAPE;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 16) || !aligned(c->v_scale, 16)) return Q4_EALIGN;
    const size_t rows = (size_t)c->pages * Hk * c->page_size;
    if (rows >= kMaxRows) return Q4_EINVAL_SHAPE;
    const size_t bytes = rows * D * (c->k_scale ? 1 : 2);
    *ranges = CacheRanges{{range_of(c->k, bytes), range_of(c->v, bytes), c->k_scale ? range_of(c->k_scale, rows * 4) : Range{0, 0},
                           c->v_scale ? range_of(c->v_scale, rows * 4) : Range{0, 0}}};
    *out = q4::Cache{static_cast<uint8_t*>(c->k), static_cast<uint8_t*>(c->v), c->k_scale, c->v_scale, c->pages,
                     __builtin_ctz((unsigned)c->page_size)};
    return Q4_OK;
}

}  // namespace

extern "C" {

int q4_rope_cache(const uint16_t* q, const uint16_t* k, const uint16_t* v, int T, int Hq, int Hk, int D, int64_t q_stride,
                  int64_t k_stride, int64_t v_stride, const uint16_t* q_norm, const uint16_t* k_norm, float eps,
                  const int32_t* positions, const float* inv_freq, int rot, int interleaved, uint16_t* q_out, uint16_t* k_out,
                  const q4_kv_cache* cache, const int64_t* slots, void* stream) {
    if (!q || !k || !q_out || (!k_out && !cache) || (cache && (!v || !slots)) || (rot && (!positions || !inv_freq))) return Q4_EINVAL_PTR;
    if (T < 1 || T > kMaxTokens || Hq < 1 || Hq > kMaxHeads || Hk < 1 || Hk > kMaxHeads || (D != 64 && D != 128)) return Q4_EINVAL_SHAPE;
    if (rot < 0 || rot > D || rot % 16 || ((q_norm || k_norm) && !positive(eps))) return Q4_EINVAL_SHAPE;
    if (!stride_ok(q_stride, Hq, D) || !stride_ok(k_stride, Hk, D) || (cache && !stride_ok(v_stride, Hk, D))) return Q4_EINVAL_SHAPE;
    if (!aligned(q, 16) || !aligned(k, 16) || (cache && !aligned(v, 16)) || !aligned(q_norm, 16) || !aligned(k_norm, 16) ||
        (rot && (!aligned(positions, 4) || !aligned(inv_freq, 4))) || !aligned(q_out, 16) || !aligned(k_out, 16) ||
        (cache && !aligned(slots, 8)))
        return Q4_EALIGN;
    q4::Cache c{};
    CacheRanges cr{};
    if (cache) {
        const int rc = check_cache(cache, Hk, D, &c, &cr);
        if (rc) return rc;
    }
    // in place means the input's rows; otherwise rows follow each other
    const Rows in[3] = {{q, T, q_stride, (int64_t)Hq * D}, {k, T, k_stride, (int64_t)Hk * D}, {cache ? v : nullptr, T, v_stride, (int64_t)Hk * D}};
    const Rows out[2] = {{q_out, T, q_out == q ? q_stride : (int64_t)Hq * D, (int64_t)Hq * D},
                         {k_out, T, k_out == k ? k_stride : (int64_t)Hk * D, (int64_t)Hk * D}};
    const Range small[5] = {q_norm ? range_of(q_norm, (size_t)D * 2) : Range{0, 0}, k_norm ? range_of(k_norm, (size_t)D * 2) : Range{0, 0},
                            rot ? range_of(positions, (size_t)T * 4) : Range{0, 0}, rot ? range_of(inv_freq, (size_t)rot * 2) : Range{0, 0},
                            cache ? range_of(slots, (size_t)T * 8) : Range{0, 0}};
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 3; ++j)
            if (!(i == j && out[i].p == in[j].p) && rows_overlap(out[i], in[j])) return Q4_EALIAS;
    if (rows_overlap(out[0], out[1])) return Q4_EALIAS;
    for (const Range& s : small) {
        if (overlaps(range_of_rows(out[0]), s) || (k_out && overlaps(range_of_rows(out[1]), s))) return Q4_EALIAS;
        for (const Range& r : cr.r)
            if (overlaps(r, s)) return Q4_EALIAS;
    }
    for (int i = 0; i < 4; ++i) {
        for (const Rows& r : in)
            if (r.p && overlaps(cr.r[i], range_of_rows(r))) return Q4_EALIAS;
        for (const Rows& r : out)
            if (r.p && overlaps(cr.r[i], range_of_rows(r))) return Q4_EALIAS;
        for (int j = 0; j < i; ++j)
            if (overlaps(cr.r[i], cr.r[j])) return Q4_EALIAS;
    }
    const q4::RopeArgs a{q, k, v, (long)q_stride, (long)k_stride, (long)v_stride, q_norm, k_norm, positions, inv_freq, slots, q_out, k_out,
                         (long)out[0].stride, (long)out[1].stride, T, Hq, Hk, D, rot, eps, interleaved != 0};
    const hipError_t e = q4::launch_rope_cache(a, cache ? &c : nullptr, reinterpret_cast<hipStream_t>(stream));
    return e == hipSuccess ? Q4_OK : Q4_ELAUNCH;
}

size_t q4_attention_decode_workspace_bytes(int T, int Hq, int Hk, int D) {
    return T >= 1 && T <= kMaxNew && heads_ok(Hq, Hk, D) ? q4::attention_decode_ws_bytes(T, Hq, Hk, D) : 0;
}

int q4_attention_decode(const uint16_t* q, int B, int T, int Hq, int Hk, int D, int64_t q_stride, const q4_kv_cache* cache,
                        const int32_t* table, int width, const int32_t* lengths, const int32_t* n_new, float scale, int window,
                        uint16_t* y, void* workspace, size_t workspace_bytes, void* stream) {
    if (!q || !cache || !table || !lengths || !y || !workspace) return Q4_EINVAL_PTR;
    if (B < 1 || B > q4::kMaxSequences || T < 1 || T > kMaxNew || !heads_ok(Hq, Hk, D) || !stride_ok(q_stride, Hq, D)) return Q4_EINVAL_SHAPE;
    if (width < 1 || window < 0 || !scale_ok(scale)) return Q4_EINVAL_SHAPE;
    q4::Cache c{};
    CacheRanges cr{};
    const int rc = check_cache(cache, Hk, D, &c, &cr);
    if (rc) return rc;
    if ((long)width << c.shift > kMaxKeys) return Q4_EINVAL_SHAPE;
    // a window of all keys is none
    const q4::DecodeArgs a{q, y, table, lengths, n_new, (long)q_stride, B, T, Hq, Hk, D, width, window >= kMaxKeys ? 0 : window, scale};
    if (q4::attention_decode_units(a, c) >= kMaxUnits) return Q4_EINVAL_SHAPE;
    if (!aligned(q, 16) || !aligned(table, 4) || !aligned(lengths, 4) || !aligned(n_new, 4) || !aligned(y, 16) || !aligned(workspace, 256))
        return Q4_EALIGN;
    const size_t need = q4::attention_decode_ws_bytes(T, Hq, Hk, D);
    if (workspace_bytes < need) return Q4_ESCRATCH;
    const long rows = (long)B * T;
    const Range in[8] = {range_of_rows(Rows{q, rows, q_stride, (int64_t)Hq * D}), range_of(table, (size_t)B * width * 4),
                         range_of(lengths, (size_t)B * 4), n_new ? range_of(n_new, (size_t)B * 4) : Range{0, 0}, cr.r[0], cr.r[1], cr.r[2], cr.r[3]};
    const Range out = range_of(y, (size_t)rows * Hq * D * 2), ws = range_of(workspace, need);
    for (const Range& r : in)
        if (overlaps(out, r) || overlaps(ws, r)) return Q4_EALIAS;
    if (overlaps(out, ws)) return Q4_EALIAS;
    const hipError_t e = q4::launch_attention_decode(a, c, workspace, reinterpret_cast<hipStream_t>(stream));
    return e == hipSuccess ? Q4_OK : Q4_ELAUNCH;
}

int q4_attention_prefill(const uint16_t* q, int T, const uint16_t* k, const uint16_t* v, int S, int Hq, int Hk, int D, int64_t q_stride,
                         int64_t k_stride, int64_t v_stride, const int32_t* starts, const int32_t* key_starts, int B, float scale,
                         int window, uint16_t* y, void* stream) {
    if (!q || !k || !v || !starts || !y) return Q4_EINVAL_PTR;
    if (T < 1 || T > kMaxTokens || S < 1 || S > kMaxTokens || B < 1 || B > q4::kMaxSequences || !heads_ok(Hq, Hk, D)) return Q4_EINVAL_SHAPE;
    if (!stride_ok(q_stride, Hq, D) || !stride_ok(k_stride, Hk, D) || !stride_ok(v_stride, Hk, D)) return Q4_EINVAL_SHAPE;
    if (window < 0 || !scale_ok(scale)) return Q4_EINVAL_SHAPE;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(starts, 4) || !aligned(key_starts, 4) || !aligned(y, 16))
        return Q4_EALIGN;
    const Rows out{y, T, (int64_t)Hq * D, (int64_t)Hq * D};
    const Range yr = range_of_rows(out);
    for (const Rows& r : {Rows{q, T, q_stride, (int64_t)Hq * D}, Rows{k, S, k_stride, (int64_t)Hk * D}, Rows{v, S, v_stride, (int64_t)Hk * D}})
        if (overlaps(yr, range_of_rows(r))) return Q4_EALIAS;
    if (overlaps(yr, range_of(starts, ((size_t)B + 1) * 4)) || (key_starts && overlaps(yr, range_of(key_starts, ((size_t)B + 1) * 4))))
        return Q4_EALIAS;
    const q4::PrefillArgs a{q, k, v, y, starts, key_starts, (long)q_stride, (long)k_stride, (long)v_stride, B, T, S, Hq, Hk, D,
                            window >= kMaxTokens ? 0 : window, scale};
    const hipError_t e = q4::launch_attention_prefill(a, reinterpret_cast<hipStream_t>(stream));
    return e == hipSuccess ? Q4_OK : Q4_ELAUNCH;
}

}  // extern "C"
