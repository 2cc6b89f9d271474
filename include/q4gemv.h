/*
 * q4gemv -- 4-bit weight-only dequantize-and-multiply for AMD MI355X (gfx950).
 *
 * C ABI of libq4gemv.so.  Every entry point computes
 *
 *     y[m, n] = sum_k x[m, k] * w[n, k]        (y = x . W^T, no bias)
 *
 * for a decode batch x of M rows against one weight matrix W of N rows
 * (output features) and K columns (input features), without ever writing the
 * dequantized W to memory.  Activations x and outputs y are BF16; the sum is
 * accumulated in fp32 and rounded to BF16 (round to nearest even) once.
 *
 * Types.  BF16 and fp16 values travel as uint16_t bit patterns and
 * float8_e4m3fn values as uint8_t, so C callers need no GPU half-precision
 * headers.  `stream` is a hipStream_t (NULL = the default stream).
 *
 * Memory and ownership.  All array arguments are DEVICE pointers to
 * contiguous, row-major arrays owned by the caller.  The library allocates
 * nothing, keeps no pointer after returning, and never synchronizes the host:
 * a call only enqueues kernels on `stream`, so it may be recorded into a HIP
 * graph.  Calls are thread-safe.  `y` is fully overwritten.
 *
 * Errors.  Arguments are checked on the host before anything is enqueued; a
 * rejected call returns a negative Q4_E* code and writes nothing.  A kernel
 * launch failure returns Q4_ELAUNCH.  Faults inside a kernel surface at the
 * caller's next synchronization, as with any HIP kernel.
 *
 * Common limits: 1 <= M <= 64, 1 <= N <= 2^24, 1 <= K <= 32768; x and the packed weights
 * 16-byte aligned; scale arrays 2-byte aligned (fp16) or 1-byte (e4m3); y
 * 2-byte aligned and not overlapping any input.
 */
#ifndef Q4GEMV_H
#define Q4GEMV_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* status codes */
#define Q4_OK 0
#define Q4_EINVAL_PTR (-1)   /* a required pointer is NULL */
#define Q4_EINVAL_SHAPE (-2) /* M, N or K out of range for the format */
#define Q4_EALIGN (-3)       /* a pointer is not aligned as documented */
#define Q4_EALIAS (-4)       /* the output overlaps an input */
#define Q4_ELAUNCH (-5)      /* the HIP runtime refused a kernel launch */
#define Q4_EVARIANT (-6)     /* unknown variant, or the variant cannot run this shape */
#define Q4_ESCRATCH (-7)     /* the call needs more scratch than the built-in array, or the given workspace, holds */

/* kernel variants (the *_gemv_variant entry points) */
#define Q4_VARIANT_AUTO 0 /* pick by (M, N, K) */
#define Q4_VARIANT_DOT2 1 /* wave-per-row packed-BF16 dot products; batch tiles of <= 8 rows */
#define Q4_VARIANT_MFMA 2 /* 16x16x32 BF16 matrix-core tiles, batch padded to 16 */
#define Q4_VARIANT_TILED 4  /* K % 128 == 0: 64-row workgroups, matrix cores, activations staged in LDS
                               per 128-column group; split over K when given a workspace
                               (the *_grouped_ws calls); the default for M >= 5 */
#define Q4_VARIANT_STREAM 3 /* M <= 4, rows of exactly 1, 2 or 4 KB (int4/NVFP4 K = 2048, 4096, 8192;
                               BF16 K = 512, 1024, 2048): every weight load issued at once, activations
                               and group parameters shared through LDS */
#define Q4_VARIANT_SKINNY 6 /* 5 <= M <= 48, K % 128 == 0: workgroups of up to 80 rows over a slice of at
                               most 16 groups of 128 columns (BF16: 8), each wave loading its own weights and
                               activation fragments straight into registers (no per-group barriers); split
                               over K when given a workspace, else int4/NVFP4 K <= 2048, BF16 K <= 1024; the
                               default for int4 at 5 <= M <= 48 and for mixed groups there */
#define Q4_VARIANT_GEMM 5   /* int4 prefill only (q4g128_gemm_variant): workgroup tiles of 128 batch
                               rows x 128 or 256 weight rows over all of K, codes unpacked from LDS
                               per wave, scale and min folded per 128-column group */

/* weight formats (q4gemv_variant_name) */
#define Q4_FMT_Q4G128 0
#define Q4_FMT_NVFP4G16 1
#define Q4_FMT_BF16 2

/*
 * int4 "g128 min/max" weights.
 * Format: rumik-oss-1-int4 model card, section "Format":
 *   qweight  uint8 [N, K/2]   two 4-bit codes per byte, LOW nibble = EVEN column
 *   scale    fp16  [N, K/128]
 *   min      fp16  [N, K/128]
 *   w[n, k] = code[n, k] * scale[n, k/128] + min[n, k/128]
 * x: bf16 [M, K]; y: bf16 [M, N].  Requires K % 128 == 0.
 */
int q4g128_gemv(const uint16_t* x, int M, int K, const uint8_t* qweight, const uint16_t* scale, const uint16_t* minv, int N,
                uint16_t* y, void* stream);

/* Same as q4g128_gemv with an explicit Q4_VARIANT_* choice. */
int q4g128_gemv_variant(const uint16_t* x, int M, int K, const uint8_t* qweight, const uint16_t* scale, const uint16_t* minv,
                        int N, uint16_t* y, int variant, void* stream);

/*
 * Several independent int4 g128 GEMVs with one batch size M, launched
 * together (as few kernel launches as the shapes allow).  This is how
 * projections that read the same activations (q, k, v, gate, up of a layer)
 * or that are independent of each other (o and down of a parallel block) go
 * out as one unit, as the Rumik TTS Fast Inference post ("What Made It
 * Faster") does by packing projections that share an input -- here without
 * re-laying out any weights.  1 <= count <= 8; every task obeys the
 * q4g128_gemv rules; no task's y may overlap any task's inputs or another y.
 */
typedef struct q4g128_task {
    const uint16_t* x;       /* bf16 [M, K] */
    const uint8_t* qweight;  /* uint8 [N, K/2] */
    const uint16_t* scale;   /* fp16 [N, K/128] */
    const uint16_t* minv;    /* fp16 [N, K/128] */
    uint16_t* y;             /* bf16 [M, N] */
    int N;
    int K;
} q4g128_task;

int q4g128_gemv_grouped(const q4g128_task* tasks, int count, int M, int variant, void* stream);

/*
 * Same as q4g128_gemv_grouped, with a caller-owned device workspace that lets
 * the Q4_VARIANT_TILED kernel split K over several workgroups when the row
 * blocks of the launch alone cannot fill the GPU (the o/down stage of a decode
 * layer at M = 48).  The partial tiles are summed in a fixed order by
 * whichever workgroup finishes a row block last, so results do not depend on
 * timing and equal those of the unsplit kernel within fp32 rounding.
 *   workspace        device memory, 256-byte aligned, ZERO-FILLED before its
 *                    first use; its first 64 KiB hold arrival counters, which
 *                    every call leaves at zero, the rest partial tiles, which
 *                    are scratch: the workspace can be reused, also by calls
 *                    with other tasks, without being cleared again
 *   workspace_bytes  at least what q4g128_workspace_bytes reports for the same
 *                    tasks and M (a workspace sized for the largest of several
 *                    calls serves them all); with less (or NULL) the call runs
 *                    unsplit
 * Calls that use one workspace must not overlap in time (same stream, or
 * ordered by events).
 */
int q4g128_gemv_grouped_ws(const q4g128_task* tasks, int count, int M, int variant, void* workspace,
                           size_t workspace_bytes, void* stream);

/* Workspace bytes q4g128_gemv_grouped_ws needs for these tasks (0 if no
 * split is planned).  Validates like the GEMV call; *bytes is set on Q4_OK. */
int q4g128_workspace_bytes(const q4g128_task* tasks, int count, int M, size_t* bytes);

/*
 * q4g128_gemv_grouped_ws without a workspace argument and without any
 * allocation, for callers that cannot allocate device memory: code recorded
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * allocation.  The split-K scratch is a built-in device array of 8 MiB per
 * GPU (Q4GEMV_NOALLOC_SCRATCH_BYTES), set up on the first call on a device
 * and held until the process ends; calls whose plan needs more than that
 * (q4g128_workspace_bytes > 8 MiB; no decode-layer shape at M <= 64 does)
 * return Q4_ESCRATCH before anything is enqueued.  Same kernels, plan and
 * results as q4g128_gemv_grouped_ws with a workspace of at least that size.
 * Every call on one GPU shares that GPU's array: calls on one GPU must not
 * overlap in time (same stream, or ordered by events), or they race.
 */
#define Q4GEMV_NOALLOC_SCRATCH_BYTES (8u << 20)
int q4g128_gemv_grouped_noalloc(const q4g128_task* tasks, int count, int M, int variant, void* stream);

/*
 * NVFP4 weight-only weights.
 * Format: VoxCPM2-NVFP4 model card, section "What was quantized": 4-bit float
 * (E2M1) codes, symmetric, group size 16, float8_e4m3fn group scales and one
 * fp32 global scale per matrix; activations stay BF16.
 *   qweight      uint8 [N, K/2]   E2M1 codes, LOW nibble = EVEN column
 *   scale_e4m3   uint8 [N, K/16]  OCP float8_e4m3fn bit patterns
 *   global_scale fp32            multiplier G
 *   w[n, k] = e2m1(code[n, k]) * e4m3(scale[n, k/16]) * G
 * x: bf16 [M, K]; y: bf16 [M, N].  Requires K % 32 == 0.
 */
int nvfp4g16_gemv(const uint16_t* x, int M, int K, const uint8_t* qweight, const uint8_t* scale_e4m3, float global_scale, int N,
                  uint16_t* y, void* stream);
int nvfp4g16_gemv_variant(const uint16_t* x, int M, int K, const uint8_t* qweight, const uint8_t* scale_e4m3, float global_scale,
                          int N, uint16_t* y, int variant, void* stream);

/*
 * Up to 8 independent NVFP4 GEMVs of one batch size M in one launch (the
 * NVFP4 q, k, gate, up projections of a decode layer read the same input;
 * Rumik TTS Fast Inference post, section "What Made It Faster": packing
 * projections that share an input).  Each task is validated as
 * nvfp4g16_gemv; outputs must not overlap any task's inputs or each other.
 * workspace / workspace_bytes: as for q4g128_gemv_grouped_ws (NULL / 0: no K
 * split); nvfp4g16_workspace_bytes gives the size (0 if no split is planned).
 */
typedef struct nvfp4g16_task {
    const uint16_t* x;          /* bf16 [M, K] */
    const uint8_t* qweight;     /* uint8 [N, K/2] E2M1 */
    const uint8_t* scale_e4m3;  /* uint8 [N, K/16] */
    float global_scale;         /* multiplier G */
    uint16_t* y;                /* bf16 [M, N] */
    int N;
    int K;
} nvfp4g16_task;

int nvfp4g16_gemv_grouped_ws(const nvfp4g16_task* tasks, int count, int M, int variant, void* workspace,
                             size_t workspace_bytes, void* stream);
int nvfp4g16_workspace_bytes(const nvfp4g16_task* tasks, int count, int M, size_t* bytes);

/*
 * Dense BF16 weights (the audio head head.audio_weight [16385, 2048] of the
 * rumik-oss-1-int4 card, section "Format"; its 2049-row codebook slice from
 * the Rumik TTS Fast Inference post, section "What Made It Faster"; and the
 * v/down projections the VoxCPM2-NVFP4 card keeps in BF16).
 *   w bf16 [N, K]; x bf16 [M, K]; y bf16 [M, N].  Requires K % 8 == 0.
 */
int bf16_gemv(const uint16_t* x, int M, int K, const uint16_t* w, int N, uint16_t* y, void* stream);
int bf16_gemv_variant(const uint16_t* x, int M, int K, const uint16_t* w, int N, uint16_t* y, int variant, void* stream);

/*
 * Up to 8 independent BF16 GEMVs of one batch size M in one launch, validated
 * as bf16_gemv; workspace as for q4g128_gemv_grouped_ws, sized by
 * bf16_workspace_bytes (0 if no split is planned).
 */
typedef struct bf16_task {
    const uint16_t* x;  /* bf16 [M, K] */
    const uint16_t* w;  /* bf16 [N, K] */
    uint16_t* y;        /* bf16 [M, N] */
    int N;
    int K;
} bf16_task;

int bf16_gemv_grouped_ws(const bf16_task* tasks, int count, int M, int variant, void* workspace, size_t workspace_bytes,
                         void* stream);
int bf16_workspace_bytes(const bf16_task* tasks, int count, int M, size_t* bytes);

/*
 * Grouped GEMVs of mixed weight formats: up to 8 independent GEMVs, each
 * int4, NVFP4 or BF16, with one batch size M.  When M <= 4 and every task is
 * a streaming shape (rows of 1, 2 or 4 KB: int4/NVFP4 K = 2048, 4096, 8192;
 * BF16 K = 512, 1024, 2048) they run as ONE launch -- the NVFP4 decode step's
 * BF16 v projection beside its NVFP4 q, k, gate, up (one launch per format
 * would otherwise be needed).  At 5 <= M <= 48 with K % 128 == 0 for every
 * task they run as one launch of the skinny matrix-core kernel (given a
 * workspace of at least q4gemv_mixed_workspace_bytes where a task's K needs
 * more than one slice: int4/NVFP4 K > 2048, BF16 K > 1024).  Above that, with
 * such a workspace, NVFP4 and BF16 tasks that all take the tiled matrix-core
 * kernel also run as one launch.  Otherwise the tasks run as one grouped
 * launch per format, in task order of first appearance, on the same stream
 * (sharing the workspace).
 * Streaming and per-format results equal those of the single-format calls bit
 * for bit; the one-launch matrix-core forms follow the group's plan (its K
 * slices), within the GEMV tolerance of the single calls.  Each task obeys its
 * format's single-call rules; no task's y may overlap any task's inputs or
 * another y.
 */
typedef struct q4gemv_mixed_task {
    int format;              /* Q4_FMT_Q4G128, Q4_FMT_NVFP4G16 or Q4_FMT_BF16 */
    const uint16_t* x;       /* bf16 [M, K], 16-byte aligned */
    const void* weight;      /* int4/NVFP4: uint8 codes [N, K/2]; BF16: bf16 [N, K]; 16-byte aligned */
    const void* scale;       /* int4: fp16 [N, K/128]; NVFP4: e4m3 bytes [N, K/16]; BF16: unused */
    const uint16_t* minv;    /* int4: fp16 [N, K/128]; otherwise unused */
    float global_scale;      /* NVFP4: per-matrix multiplier; otherwise unused */
    uint16_t* y;             /* bf16 [M, N] */
    int N;
    int K;
} q4gemv_mixed_task;

int q4gemv_grouped_mixed(const q4gemv_mixed_task* tasks, int count, int M, void* workspace, size_t workspace_bytes,
                         void* stream);
int q4gemv_mixed_workspace_bytes(const q4gemv_mixed_task* tasks, int count, int M, size_t* bytes);

/*
 * Fused int4 GEMVs for the decode step's elementwise neighbours.  The Rumik
 * TTS Fast Inference post ("What Made It Faster") fuses the residual and
 * normalization operations around its weight-only projections so that their
 * data movement disappears; here the two around the MLP and the residual
 * stream of a decoder layer:
 *
 *   up != NULL:        the activations of the product are
 *                          h[m, k] = RN_bf16(silu(x[m, k]) * up[m, k]),
 *                      silu(g) = g / (1 + e^-g) -- the gated MLP's
 *                      activation, formed while the activations are staged
 *                      (x holds the gate projection's output): down(h) with
 *                      no separate elementwise kernel and no h in memory;
 *   residual != NULL:  y[m, n] = RN_bf16(sum_k h[m, k] w[n, k] + residual[m, n]),
 *                      one rounding of the exact sum plus the residual (the
 *                      o and down projections adding into the residual
 *                      stream); residual may be y itself (in place).
 *
 * silu is evaluated in fp32 with the hardware exp2 and reciprocal (a few fp32
 * ulps), so h can differ from the exactly rounded value by one BF16 step when
 * the exact product lies within that error of a rounding boundary.  Kernels:
 * the streaming kernel when every task allows it (M <= 4, K = 2048, 4096 or
 * 8192), else the skinny or the tiled kernel (K % 128 == 0; see below);
 * shapes the tiled kernel cannot run return Q4_EVARIANT.  Tasks obey the q4g128_gemv rules; up is bf16 [M, K], 16-byte
 * aligned; residual is bf16 [M, N], 2-byte aligned; no y may overlap any
 * input of any task or another y, except that a task's y may be exactly its
 * own residual.  workspace / workspace_bytes as for q4g128_gemv_grouped_ws
 * (q4g128_fused_workspace_bytes sizes it; NULL runs unsplit).  Beyond the
 * streaming kernel, a workspace of that size also holds h: it is then formed
 * once by a separate pass (one extra launch), and for 5 <= M <= 48 the
 * skinny kernel (Q4_VARIANT_SKINNY) runs the GEMV with the residual in its
 * epilogue; without a workspace, or for M > 48, the tiled kernel runs, its
 * loader waves forming h for every 64-row block when no pass did (same h bit
 * for bit).
 */
typedef struct q4g128_fused_task {
    const uint16_t* x;         /* bf16 [M, K] (the gate activations when up is set) */
    const uint16_t* up;        /* NULL, or bf16 [M, K] */
    const uint8_t* qweight;    /* uint8 [N, K/2] */
    const uint16_t* scale;     /* fp16 [N, K/128] */
    const uint16_t* minv;      /* fp16 [N, K/128] */
    const uint16_t* residual;  /* NULL, or bf16 [M, N] (may equal y) */
    uint16_t* y;               /* bf16 [M, N] */
    int N;
    int K;
} q4g128_fused_task;

int q4g128_gemv_fused(const q4g128_fused_task* tasks, int count, int M, void* workspace, size_t workspace_bytes,
                      void* stream);
int q4g128_fused_workspace_bytes(const q4g128_fused_task* tasks, int count, int M, size_t* bytes);

/*
 * Prefill GEMM: y[M, N] = x[M, K] . W^T for int4 g128 weights and any M >= 1
 * (the prompt's tokens before the decode loop; the rumik-oss-1-int4 card's
 * engine lists a 4-bit prefill matrix multiply beside its decode kernels,
 * "Running it").  M <= 64 takes the q4g128_gemv choice.  Larger M runs one
 * of two kernels in one launch:
 *   - Q4_VARIANT_GEMM: workgroup tiles of 128 batch rows x 128 or 256 weight
 *     rows over all of K; the default once the 128 x 128 tiles number at
 *     least 256 (one per CU), and for K > 16384;
 *   - Q4_VARIANT_TILED: the tiled decode kernel over batch chunks of up to 64
 *     rows, every chunk an unsplit product over the same weights (chunks of
 *     64 rows up to K = 4096, 32 rows up to 12288, 16 rows up to 16384; above
 *     that Q4_EVARIANT); the default for fewer tiles.
 * Both compute sum over groups of scale * sum(code * x) + min * sum(x) in
 * fp32 with every product exact, then round to BF16 once.  Same layouts and
 * rules as q4g128_gemv, with 1 <= M <= 524288 and K % 128 == 0.
 */
int q4g128_gemm(const uint16_t* x, int M, int K, const uint8_t* qweight, const uint16_t* scale, const uint16_t* minv, int N,
                uint16_t* y, void* stream);
/* q4g128_gemm with an explicit variant: Q4_VARIANT_AUTO, Q4_VARIANT_TILED or
 * Q4_VARIANT_GEMM (any M >= 1 for these two; else Q4_EVARIANT). */
int q4g128_gemm_variant(const uint16_t* x, int M, int K, const uint8_t* qweight, const uint16_t* scale, const uint16_t* minv,
                        int N, uint16_t* y, int variant, void* stream);

/*
 * Sampling from the head: the step after the path.  The Rumik TTS Fast
 * Inference post samples each audio token at temperature 0.8 with top-k 30
 * ("The Result") from the head restricted to the current codebook, 2049 rows
 * ("What Made It Faster").  Per batch row m of BF16 logits [M, V]:
 *   1. the top_k largest logits, equal logits ordered by lower index (-0 and
 *      +0 are equal), in order of (logit descending, index ascending);
 *   2. p_i = softmax(logit_i / temperature) over those top_k, in fp32;
 *   3. token[m] = the first of that order whose running sum of p exceeds
 *      u[m] (the caller's uniform draw in [0, 1); the library draws no
 *      random numbers).
 * Outputs: token [M] int32; optionally topk_index [M, top_k] int32 and
 * topk_prob [M, top_k] fp32 (NULL to skip).  1 <= top_k <= 64 and
 * top_k <= V <= 30720; temperature finite and > 0; logits must hold no NaN.
 * The selection is exact; the probabilities and the draw are fp32 (a draw
 * can differ from exact arithmetic only when u lies within fp32 rounding of a
 * cumulative boundary).  Alignment: logits 2 bytes, u and the outputs 4 bytes;
 * outputs must not overlap each other or the inputs.
 *
 * q4_sample_topk samples from logits already in memory (one launch);
 * bf16_head_sample runs the BF16 head GEMV logits = x W^T (the bf16_gemv
 * rules, N = V; logits is the caller's [M, N] buffer) and then samples (two
 * launches).  Both return Q4_EINVAL_PTR / Q4_EINVAL_SHAPE / Q4_EALIGN /
 * Q4_EALIAS before enqueueing anything, Q4_ELAUNCH on a launch failure.
 */
int q4_sample_topk(const uint16_t* logits, int M, int V, float temperature, int top_k, const float* u, int32_t* token,
                   int32_t* topk_index, float* topk_prob, void* stream);
int bf16_head_sample(const uint16_t* x, int M, int K, const uint16_t* w, int N, uint16_t* logits, float temperature, int top_k,
                     const float* u, int32_t* token, int32_t* topk_index, float* topk_prob, void* stream);

/*
 * bf16_head_sample with a caller workspace.  Same arguments, rules, results
 * and status codes, plus a workspace of ws_bytes bytes, 4-byte aligned and
 * zero-filled before its first use: it holds arrival counters (every call
 * leaves them at zero) and per-block top-k candidates (scratch).  It must not
 * overlap any other argument (Q4_EALIAS, as are Q4_EALIGN and the sampling
 * checks, returned before anything is enqueued).  The logits and the
 * selection are bitwise those of bf16_head_sample.
 *
 * M = 1 (the single-stream decode of the pages, which replay the step,
 * sampling included, as one graph; "Rumik TTS Fast Inference", "What Made It
 * Faster"): the GEMV and the sampling run as ONE launch.  The streaming GEMV
 * workgroups store their logits; the last to finish in each block of
 * workgroups selects that block's top_k entries, and the last block selects
 * among the candidates, sorts and draws -- no workgroup waits for another.
 * Needs K in {512, 1024, 2048, 4096, 8192}.
 * 2 <= M <= 64 and N > 1024: the GEMV, then the sampler split over blocks of
 * 1024 logits per row (one workgroup each; the last of a row to finish
 * selects among the blocks' candidates and draws) -- two launches, the second
 * with M * ceil(N / 1024) workgroups instead of M.
 * Applies when bf16_head_sample_workspace_bytes(M, N, K, top_k) is nonzero
 * (top_k <= 64, heads up to 30720 rows, and the cases above) and ws_bytes is
 * at least that; otherwise the call runs bf16_head_sample.  Calls that share
 * a workspace must not overlap in time.
 */
size_t bf16_head_sample_workspace_bytes(int M, int N, int K, int top_k);
int bf16_head_sample_ws(const uint16_t* x, int M, int K, const uint16_t* w, int N, uint16_t* logits, float temperature, int top_k,
                        const float* u, int32_t* token, int32_t* topk_index, float* topk_prob, void* workspace, size_t ws_bytes,
                        void* stream);

/*
 * Products in 8-bit floating point with a scale for each block of 128: the
 * form for many rows at once (prompts; steps that verify several drafted
 * tokens per sequence), where activations in 8 bits run at the matrix cores'
 * 8-bit rate.
 *   x      uint8 [M, K] float8_e4m3fn    xscale  fp32 [M, G]
 *   w      uint8 [N, K] float8_e4m3fn    wscale  fp32 [ceil(N / 128), G]
 *   G = ceil(K / 128) blocks of 128 columns (the last may be shorter)
 *   y[m, n] = RN_bf16( sum_g xscale[m, g] wscale[n / 128, g] sum_{k in g} x[m, k] w[n, k]
 *                      + residual[m, n] )                       (residual NULL: without it)
 * The sum within a block is one 8-bit matrix instruction, which adds each 8
 * consecutive columns' products aligned to the largest of them (what lies below
 * 2^-13 of it is dropped) and those sums in fp32; blocks are added in fp32, in
 * a fixed order, so results do not change from call to call, and rounded to
 * bf16 once.  xscale wscale is an fp32 product: scales so far from 1 that
 * it leaves the normal range lose accuracy or give 0 or infinity.  NaN codes and
 * scales make the outputs they reach NaN.
 *
 * Limits: 1 <= M <= 524288, 1 <= N <= 2^24, 16 <= K <= 32768, K % 16 == 0;
 * x, w and codes 16-byte aligned, scales 4, y and residual 2.  residual may be
 * exactly y (in place); otherwise no output may overlap an input or another
 * output.
 */

/*
 * e4m3 codes and block scales of activations: h = x (up NULL), or
 * h = silu(x) * up in fp32 (the gated MLP's activation; silu(g) = g / (1 + e^-g),
 * taken as 0 for g below -87.3), x and up bf16 [M, K].  With a the largest |h|
 * of a block of 128 columns:
 *     scale[m, g] = RN(a / 448),  codes[m, k] = RN_e4m3(h[m, k] * 448 / a),
 * the quotient rounded once (exactly so without up; with up, h and its quotient
 * carry fp32 roundings, and about one code in 10^6 lies so near a tie that it
 * goes the other way than in exact arithmetic); nothing saturates.  A
 * block of zeros has scale 0 and codes 0.  A value that is not finite (x, or
 * x * up in fp32) gets the NaN code and takes no part in a.
 */
int fp8b128_quantize(const uint16_t* x, const uint16_t* up, int M, int K, uint8_t* codes, float* scale, void* stream);

int fp8b128_gemm(const uint8_t* x, const float* xscale, int M, int K, const uint8_t* w, const float* wscale, int N,
                 const uint16_t* residual, uint16_t* y, void* stream);

/*
 * Up to 8 independent products of one batch size M (the projections that read
 * one input, for instance), each under fp8b128_gemm's rules.  workspace:
 * optional device memory, 256-byte aligned, apart from every argument,
 * zero-filled before its first use; its first 64 KiB are arrival counters that
 * every call leaves at zero, the rest is scratch, so it can be shared with the
 * library's other calls that take a workspace of this kind.  It lets few rows
 * split K over workgroups (summed in slice order).  A call runs in the way that
 * is modelled fastest among those that the workspace holds: with
 * fp8b128_workspace_bytes (0: none is used) as with any larger one, with less
 * in fewer slices, without one unsplit.  Calls that use one workspace must not
 * overlap in time.
 */
typedef struct fp8b128_task {
    const uint8_t* x;          /* e4m3 [M, K] */
    const float* xscale;       /* fp32 [M, G] */
    const uint8_t* w;          /* e4m3 [N, K] */
    const float* wscale;       /* fp32 [ceil(N / 128), G] */
    const uint16_t* residual;  /* NULL, or bf16 [M, N] (may equal y) */
    uint16_t* y;               /* bf16 [M, N] */
    int N;
    int K;
} fp8b128_task;

int fp8b128_gemm_grouped_ws(const fp8b128_task* tasks, int count, int M, void* workspace, size_t workspace_bytes, void* stream);
int fp8b128_workspace_bytes(const fp8b128_task* tasks, int count, int M, size_t* bytes);

/*
 * Diagnostic: the kernel launches that a call with this many bytes of workspace
 * makes (nothing is launched): how many, and the first `most` of them.
 */
typedef struct fp8b128_launch {
    int tile_m, tile_n;        /* batch and weight rows of a workgroup */
    int count;                 /* products in it */
    int N[8], slices[8];       /* of each: weight rows, slices of K */
    size_t workspace_bytes;    /* that it uses */
} fp8b128_launch;
int fp8b128_launches(const fp8b128_task* tasks, int count, int M, size_t workspace_bytes, fp8b128_launch* out, int most, int* launches);

/*
 * Verification of drafted tokens (speculative decoding by rejection sampling,
 * from the caller's uniform numbers; the library draws none).  Sequence b has
 * n = n_draft[b] drafted tokens draft[b, 0 .. n) (n_draft NULL: D each; values
 * are taken within 0 .. D).  logits: bf16 [B, D + 1, V]; row i is the target's
 * distribution p_i after i drafted tokens, q_i the distribution that the draft
 * drew token i from.  u: fp32 [B, D + 1] in [0, 1).
 *   1. token i stands while u[b, i] * q_i(draft[b, i]) < p_i(draft[b, i]);
 *      count[b] = a, the tokens that stand from the first on;
 *   2. one more token is drawn: a < n: from max(p_a - q_a, 0) (from p_a where
 *      that is zero everywhere); a = n: from p_n.  It is the first entry, in the
 *      distribution's order, whose running sum exceeds u[b, D] times the total;
 *   3. token[b] (int32 [D + 1]) = the a tokens, the drawn one, then -1.
 * accept_prob (fp32 [B, D], or NULL): min(1, p_i / q_i) of each drafted token
 * (q_i = 0: 1 if p_i > 0, else 0), 0 behind the n-th.  Logits behind row n and
 * drafts behind the n-th are not read.
 *
 * q4_verify_topk: p is the distribution of q4_sample_topk at this temperature
 * and top_k (entries by larger logit, then lower index); the draft's is a list
 * of draft_k <= 64 entries per drafted token, draft_index int32 and draft_prob
 * fp32 [B, D, draft_k], as q4_sample_topk writes them (entries that repeat an
 * index add; an index below 0 never matches), or NULL for both: the draft was
 * certain of its token.  1 <= top_k <= 64, top_k <= V <= 30720.
 * q4_verify_full: p and q are softmax(row / temperature) of whole rows, in
 * index order; draft_logits bf16 [B, D, V], or NULL (as above).  V <= 2^20.
 *
 * A NaN logit counts as -inf (probability 0).  A row whose largest logit is
 * not finite has no distribution: nothing stands against it, and the token
 * drawn from it is -1.  A drafted token outside [0, V) never stands.  Masses
 * and running sums are fp64: a result differs from exact arithmetic only where
 * a uniform lies within about 1e-14 of a boundary, or, for a draw from
 * max(p - q, 0), within 1e-14 over that distribution's total (a draft close to
 * the target leaves little).
 *
 * 1 <= D <= 63, B (D + 1) <= 65536; temperature finite and > 0.  Alignment:
 * logits 2 bytes, everything else 4.  workspace: at least
 * q4_verify_*_workspace_bytes (where that is not 0), 256-byte aligned,
 * zero-filled before its first use; its first 64 KiB are arrival counters that
 * every call leaves at zero, the rest is scratch, so it can be shared with the
 * library's other calls that take a workspace of this kind.  Sizes grow with
 * every argument: the largest batch's workspace serves smaller ones.  Calls
 * that use one workspace must not overlap in time.  Returns Q4_EINVAL_PTR (no workspace where one is needed too), Q4_EINVAL_SHAPE,
 * Q4_EALIGN, Q4_ESCRATCH (workspace too small) or Q4_EALIAS before anything is
 * enqueued.
 */
size_t q4_verify_topk_workspace_bytes(int B, int D, int V, int top_k);
int q4_verify_topk(const uint16_t* logits, int B, int D, int V, const int32_t* draft, const int32_t* draft_index,
                   const float* draft_prob, int draft_k, const int32_t* n_draft, const float* u, float temperature, int top_k,
                   int32_t* token, int32_t* count, float* accept_prob, void* workspace, size_t workspace_bytes, void* stream);
size_t q4_verify_full_workspace_bytes(int B, int D, int V);
int q4_verify_full(const uint16_t* logits, int B, int D, int V, const int32_t* draft, const uint16_t* draft_logits,
                   const int32_t* n_draft, const float* u, float temperature, int32_t* token, int32_t* count, float* accept_prob,
                   void* workspace, size_t workspace_bytes, void* stream);

/*
 * A decoder layer's attention: what lies between its q, k, v projections and
 * its o projection.  The Rumik TTS Fast Inference post fuses "rotary position,
 * cache" operations ("What Made It Faster"), the rumik-oss-1-int4 card's engine
 * lists the decode steps' attention among its kernels ("Running it").
 *
 * Heads have D = 64 or 128 values; Hq query heads share Hk key heads, query
 * head h with key head h / (Hq / Hk).  Arrays of heads are bf16
 * [tokens, heads, D] whose tokens lie `stride` elements apart (at least
 * heads * D and at most 2^24, a multiple of 8), so that they may be parts of one
 * product's rows.
 *
 * The cache is paged: pages of page_size tokens (16, 32, 64, 128 or 256), each
 * head's part of a page in one piece; pages * Hk * page_size < 2^31.  bf16, or,
 * where scales are given, float8_e4m3fn codes with one fp32 scale per token and
 * head (value = code * scale).
 */
typedef struct q4_kv_cache {
    void* k;              /* bf16 or e4m3 [pages, Hk, page_size, D], 16-byte aligned */
    void* v;              /* as k */
    float* k_scale;       /* NULL, or fp32 [pages, Hk, page_size], 16-byte aligned */
    float* v_scale;       /* as k_scale; both or neither */
    int pages;
    int page_size;
} q4_kv_cache;

/*
 * Heads of q and k normalised, rotated to their positions, and k and v
 * appended to a cache; for prompts and decode steps alike (T tokens).
 * Per head x of q and k, in fp32, rounded once:
 *     h = x * w / sqrt(mean(x^2) + eps),  w = q_norm or k_norm, bf16 [D] (NULL: h = x)
 *     the first rot values of h in pairs (a, b), pair i turned by
 *     f = positions[t] * inv_freq[i]:  (a cos f - b sin f, b cos f + a sin f);
 *     pairs are elements (i, i + rot / 2), or (2 i, 2 i + 1) where interleaved
 * rot: a multiple of 16, 0 to D (0: no rotation, positions and inv_freq are not
 * used).  inv_freq fp32 [rot / 2]; angles are taken in fp64, whatever the
 * position (int32 [T]).
 * q_out: bf16 [T, Hq, D], or q itself (in place, with q's stride).  k_out: the
 * same for k, or NULL where there is a cache.
 * cache (NULL: none): token t's k and v go to slot slots[t] = page * page_size +
 * place (int64 [T]); a token whose slot is no slot of the cache (-1, say) is not
 * kept.  An e4m3 cache takes the unrounded h and v, with a the largest
 * finite |h| of the head: scale = RN(a / 448), code = RN_e4m3(h * 448 / a); a
 * value that is not finite becomes the NaN code.  v's codes round once; k's h is
 * an fp32 number, whose quotient rounds twice: a code whose quotient lies within
 * 2^-24 of it of a tie of e4m3 may be the other neighbour.  Slots must differ: of
 * a slot named twice the contents are not specified (nothing else is touched).
 *
 * 1 <= T <= 2^22, Hq and Hk 1 to 256, eps finite and > 0.  Alignment: arrays of
 * heads and norm weights 16 bytes, positions and inv_freq 4, slots 8.  No
 * output may overlap an input or another output but in place as said.
 */
int q4_rope_cache(const uint16_t* q, const uint16_t* k, const uint16_t* v, int T, int Hq, int Hk, int D, int64_t q_stride,
                  int64_t k_stride, int64_t v_stride, const uint16_t* q_norm, const uint16_t* k_norm, float eps,
                  const int32_t* positions, const float* inv_freq, int rot, int interleaved, uint16_t* q_out, uint16_t* k_out,
                  const q4_kv_cache* cache, const int64_t* slots, void* stream);

/*
 * Attention of new tokens over a paged cache that already holds them:
 *     y[b, i, h] = RN_bf16( sum_j p_j v_j ),  p = softmax over the seen keys j of scale * q[b, i, h] . k_j
 * T = 1: a decode step; T > 1: the rows that verify drafted tokens (q4_verify_*),
 * of which sequence b has n = n_new[b] (NULL: T each; taken within 0 .. T).
 * lengths[b] (int32): the sequence's tokens in the cache, the new ones the last
 * of them; row i sees the first lengths[b] - n + i + 1, and of those the last
 * `window` (0: all).  table int32 [B, width]: page numbers, token j on page
 * table[b, j / page_size]; an entry that is no page of the cache (-1, say)
 * holds nothing, and its tokens are not seen.  Lengths are taken within
 * 0 .. width * page_size.  Table entries behind a sequence's length are not read;
 * keys and values behind it on its last page may be, and have no effect.
 * q: rows b * T + i, q_stride apart; y [B, T, Hq, D] is fully overwritten: rows
 * that see no key (or only scores of -infinity), and rows behind the n-th, are 0.
 * Keys and values that a row does not see, and other rows' queries, have no effect
 * on it, to the last bit, whatever they hold.  Scores, softmax and sums are fp32 (a
 * score that leaves its range, before its scales or after them, is infinite); a
 * weight (times an 8-bit value's scale) is rounded to bf16 before it multiplies
 * its value, and, where values are bf16, before it is summed, so that a row is a
 * mean of its values.
 *
 * 1 <= B <= 4096, 1 <= T <= 64, Hq <= 256 a multiple of Hk, width * page_size <=
 * 2^24, and B * Hk * (ceil(width * page_size / 32) + 8), times ceil(T * Hq / Hk / 32)
 * where T * Hq / Hk is above 16, below 2^31; 0 < scale <= 2^127 (a k_scale's product
 * with it as well); window >= 0.
 * Alignment: q and y 16 bytes, table, lengths, n_new 4.
 * workspace: at least q4_attention_decode_workspace_bytes, 256-byte aligned,
 * zero-filled before its first use; its first 64 KiB are arrival counters that
 * every call leaves at zero, the rest is scratch, so it can be shared with the
 * library's other calls that take a workspace of this kind.  It does not depend on
 * B or the lengths.  Calls that use one workspace must not overlap in time.
 * Results do not depend on timing, but for one sequence they may differ in their
 * last bits with the others of its batch (the work is split by the lengths of
 * all).
 */
size_t q4_attention_decode_workspace_bytes(int T, int Hq, int Hk, int D);
int q4_attention_decode(const uint16_t* q, int B, int T, int Hq, int Hk, int D, int64_t q_stride, const q4_kv_cache* cache,
                        const int32_t* table, int width, const int32_t* lengths, const int32_t* n_new, float scale, int window,
                        uint16_t* y, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Causal attention over packed prompts: as above, with sequence b's queries in
 * rows starts[b] .. starts[b + 1] of q [T, Hq, D] and its keys and values in
 * rows key_starts[b] .. key_starts[b + 1] of k and v [S, Hk, D] (key_starts
 * NULL: starts, and S = T).  Its last query sees its last key, each query
 * before it one key less (so more keys than queries are a prefix that all
 * see, and with fewer keys than queries the first ones see nothing), and of
 * those the last `window` (0: all).  y [T, Hq, D]: rows that see nothing are 0;
 * rows of no sequence are left as they are.  starts, key_starts int32 [B + 1],
 * not decreasing; entries are taken within 0 .. T and 0 .. S.
 *
 * 1 <= T, S <= 2^22, 1 <= B <= 4096; the rest as above.  y must not overlap an
 * input.
 */
int q4_attention_prefill(const uint16_t* q, int T, const uint16_t* k, const uint16_t* v, int S, int Hq, int Hk, int D, int64_t q_stride,
                         int64_t k_stride, int64_t v_stride, const int32_t* starts, const int32_t* key_starts, int B, float scale,
                         int window, uint16_t* y, void* stream);

/*
 * Diagnostic dequantization of a whole matrix to fp32 w [N, K] (16-byte
 * aligned).  Bitwise equal to the format definitions above: int4 rounds
 * code*scale+min once; NVFP4 rounds e2m1*e4m3*G once (the first product is
 * exact).  Uses the device conversion helpers of the GEMV kernels.
 */
int q4g128_dequant_f32(const uint8_t* qweight, const uint16_t* scale, const uint16_t* minv, int N, int K, float* w, void* stream);
int nvfp4g16_dequant_f32(const uint8_t* qweight, const uint8_t* scale_e4m3, float global_scale, int N, int K, float* w,
                         void* stream);

/*
 * Diagnostic plain streaming read: the reference a GEMV launch of the same
 * bytes is compared with.  Reads `count` (1..32) device buffers bufs[i] of
 * bytes[i] bytes (each 4-byte aligned, 16 <= bytes[i] < 4 GiB) in one launch
 * with 16-byte loads and writes one XOR word per wave to the device buffer
 * `sink` of sink_words 32-bit words, which must be at least
 * q4gemv_stream_read_sink_words() and must not overlap the buffers.
 * Returns Q4_EINVAL_PTR, Q4_EINVAL_SHAPE, Q4_EALIGN or Q4_EALIAS before
 * enqueueing anything; Q4_ELAUNCH if the launch fails.
 */
int q4gemv_stream_read(const void* const* bufs, const size_t* bytes, int count, uint32_t* sink, size_t sink_words,
                       void* stream);
/* Sink words q4gemv_stream_read needs for these sizes (0 on invalid input). */
size_t q4gemv_stream_read_sink_words(const size_t* bytes, int count);

/*
 * Kernel timing without host gaps: the next kernel launched by the calling
 * thread through this library records start_event when it begins executing
 * and stop_event when it ends (hipExtLaunchKernel).  Both are caller-owned
 * hipEvent_t handles (either may be NULL); they apply to one launch only, so
 * time calls that launch one kernel.  Host only, always returns Q4_OK.
 */
int q4gemv_time_next_launch(void* start_event, void* stop_event);

/* Name of the kernel a call would run ("dot2", "mfma"); host only, never fails. */
const char* q4gemv_variant_name(int fmt, int variant, int M, int N, int K);

/* Static text for a status code; host only. */
const char* q4gemv_strerror(int status);

/* Library version, major*10000 + minor*100 + patch. */
int q4gemv_version(void);

#ifdef __cplusplus
}
#endif

#endif /* Q4GEMV_H */
