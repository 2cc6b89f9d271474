// Host-side launchers of the attention operators (rope_cache.hip,
// attn_decode.hip, attn_prefill.hip).  Everything here assumes the arguments
// were validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace q4 {

// A paged cache: k and v [pages, Hk, 1 << shift, D], bf16, or e4m3 codes with
// fp32 scales ks and vs [pages, Hk, 1 << shift] (null: bf16).
struct Cache {
    uint8_t* k;
    uint8_t* v;
    float* ks;
    float* vs;
    int pages, shift;
};

struct RopeArgs {
    const uint16_t *q, *k, *v;             // bf16 [T, heads, D], rows of a token qs, ks, vs elements apart
    long qs, ks, vs;
    const uint16_t *q_norm, *k_norm;       // bf16 [D] or null
    const int32_t* pos;                    // [T]; unused where rot is 0
    const float* inv_freq;                 // [rot / 2]
    const int64_t* slots;                  // [T]; unused without a cache
    uint16_t *q_out, *k_out;               // k_out may be null where there is a cache
    long qos, kos;                         // elements from a token of q_out, k_out to the next
    int T, Hq, Hk, D, rot;
    float eps;
    bool interleaved;
};
hipError_t launch_rope_cache(const RopeArgs& a, const Cache* cache, hipStream_t s);

struct DecodeArgs {
    const uint16_t* q;        // bf16 [B * T, Hq, D], rows qs elements apart
    uint16_t* out;            // bf16 [B, T, Hq, D]
    const int32_t* table;     // [B, width]
    const int32_t* lengths;   // [B]
    const int32_t* n_new;     // [B] or null
    long qs;
    int B, T, Hq, Hk, D, width, window;
    float scale;
};
// ws: a workspace whose first 64 KiB are arrival counters (zero, left zero).
// Tiles of work at the most: (sequence, key head, rows, 32 keys); they have to be below 2^31.
long attention_decode_units(const DecodeArgs& a, const Cache& cache);
size_t attention_decode_ws_bytes(int T, int Hq, int Hk, int D);
hipError_t launch_attention_decode(const DecodeArgs& a, const Cache& cache, void* ws, hipStream_t s);

struct PrefillArgs {
    const uint16_t *q, *k, *v;     // bf16 [T, Hq, D], [S, Hk, D], rows of a token qs, ks, vs elements apart
    uint16_t* out;                 // bf16 [T, Hq, D]
    const int32_t *starts, *key_starts;   // [B + 1]; key_starts null: starts
    long qs, ks, vs;
    int B, T, S, Hq, Hk, D, window;
    float scale;
};
hipError_t launch_attention_prefill(const PrefillArgs& a, hipStream_t s);

constexpr int kMaxSequences = 4096;

}  // namespace q4
