/*
 * fp8blk -- block-scaled ("fine-grained") FP8 linear layer for AMD MI355X (gfx950).
 *
 * What the library computes
 * -------------------------
 * Weights are stored as 8-bit floats with one fp32 scale per 2D block of
 * 128x128, and activations are quantized at run time with one fp32 scale per
 * token and per group of 128 input channels, the group matching the weight
 * block along the input channel ("Fine-grained FP8" page of the transformers
 * docs, introduction; run-time activation scales are the "dynamic"
 * activation scheme of its "DeepGEMM fast path" section; fp32 is the default
 * scale type, per its "UE8M0 scale format" section).  The linear layer's
 * value is that of dequantize-then-matmul ("BFL (fp8r / nvfp4)" page of the
 * diffusers docs, "Kernels").
 *
 * The readings this library fixes where the pages are silent:
 *   - the 8-bit format is OCP FP8 E4M3FN (bias 7, max 448, no infinities);
 *   - scale s = fl32(amax / 448) over the block or group (s is the
 *     dequantization multiplier: x ~= dec(q) * s);
 *   - code q = E4M3(fl32(x / s)): the IEEE fp32 quotient is rounded first,
 *     then rounded to nearest-even E4M3 and saturated to +-448;
 *   - an all-zero block or group gets s = 0 and signed-zero codes;
 *   - y[m,n] = bf16_RNE( sum_kb x_s[m,kb] * w_s[n/128,kb] *
 *                        sum_{k in block kb} dec(x_q[m,k]) * dec(w_q[n,k]) ),
 *     with fp32 accumulation; the 128-long inner sums run on fp8 matrix
 *     cores and the scale pair is applied once per K block.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *   - All tensor pointers are DEVICE pointers; the caller owns every buffer.
 *     The library never allocates, frees or keeps a pointer; it is stateless
 *     apart from a per-device architecture check that is cached.
 *   - Layouts are dense row-major: x [M,K], W [N,K] (the nn.Linear layout,
 *     K contiguous), x_s [M, K/128], w_s [ceil(N/128), K/128], y [M,N].
 *     bf16 tensors are raw 16-bit patterns; E4M3 codes are bytes.
 *   - K must be a positive multiple of 128.  N and M may be any size >= 0;
 *     a last weight block row with fewer than 128 rows covers only the rows
 *     that exist.  M == 0 or N == 0 (or E == 0) is a no-op returning OK.
 *   - Every tensor base pointer must be 16-byte aligned (expert_offsets:
 *     and expert_counts: 4-byte aligned, as int32 arrays; a single static scale: 4-byte
 *     aligned; E8M0 scale-byte arrays: any address).
 *   - Calls are asynchronous on `stream` (a hipStream_t; NULL = the default
 *     stream).  Inputs must stay valid until the stream reaches the launch.
 *     Outputs must not alias inputs.
 *   - Arguments are validated before any HIP runtime call, in the order
 *     null pointers, shapes, alignment; then the current device must be a
 *     gfx950, else FP8BLK_ERR_DEVICE.  A failed launch returns
 *     FP8BLK_ERR_LAUNCH.  Faults inside a kernel surface as HIP errors at
 *     the caller's next synchronisation.
 *   - Non-finite inputs (NaN, Inf) are outside the contract: results are
 *     unspecified, but the kernels stay in bounds.
 *   - Size limits: M, N <= 2^31 - 1 and K <= 2^24 per call.
 */
#ifndef FP8BLK_H
#define FP8BLK_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define FP8BLK_API __attribute__((visibility("default")))
#else
#define FP8BLK_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FP8BLK_OK = 0,
    FP8BLK_ERR_NULL = 1,    /* a required pointer is NULL                    */
    FP8BLK_ERR_SHAPE = 2,   /* negative size, K % 128 != 0, size over limit  */
    FP8BLK_ERR_ALIGN = 3,   /* a base pointer is not 16-byte aligned         */
    FP8BLK_ERR_DEVICE = 4,  /* no device, or the current device is not gfx950 */
    FP8BLK_ERR_LAUNCH = 5,  /* the kernel launch failed                      */
    FP8BLK_ERR_SCRATCH = 6  /* more device scratch needed than the library holds */
} fp8blk_status;

#define FP8BLK_BLOCK 128
#define FP8BLK_ABI_VERSION 1

/* Weight quantization, one fp32 scale per 128x128 block.
 * "Fine-grained FP8" page, introduction: weights are brought to 8 bits per
 * 2D block, weight_block_size = (128, 128).  Done once, when weights load.
 *   w_bf16  [N,K] bf16 in
 *   w_q     [N,K] E4M3 codes out
 *   w_scale [ceil(N/128), K/128] fp32 out; block (nb,kb) covers rows
 *           [128nb, min(N,128nb+128)) and columns [128kb, 128kb+128). */
FP8BLK_API fp8blk_status fp8_weight_block_quant(const void *w_bf16, int64_t N, int64_t K,
                                                void *w_q, float *w_scale, void *stream);

/* Dynamic activation quantization, one fp32 scale per token per 128 input
 * channels.  "Fine-grained FP8" page, introduction (per token, per group,
 * the group matching the weights' input-channel block, 128 by default) and
 * "DeepGEMM fast path" (activation_scheme = "dynamic": scales are computed
 * on every call).
 *   x_bf16  [M,K] bf16 in
 *   x_q     [M,K] E4M3 codes out
 *   x_scale [M, K/128] fp32 out; group (m,g) covers columns [128g, 128g+128). */
FP8BLK_API fp8blk_status fp8_act_quant_group(const void *x_bf16, int64_t M, int64_t K,
                                             void *x_q, float *x_scale, void *stream);

/* Block-scaled FP8 GEMM, y = x * W^T in bf16.  "Fine-grained FP8" page,
 * "DeepGEMM fast path": the FP8 linear layer with (128,128) weight blocks
 * and dynamic activation groups; value as dequantize-then-matmul ("BFL"
 * page, "Kernels").  The scale pair x_scale[m,kb] * w_scale[n/128,kb] is
 * applied to each 128-long partial sum inside the K loop.
 *   x_q [M,K], x_scale [M,K/128], w_q [N,K], w_scale [ceil(N/128),K/128] in
 *   y_bf16 [M,N] out (bf16, round to nearest even). */
FP8BLK_API fp8blk_status fp8_block_gemm(const void *x_q, const float *x_scale,
                                        const void *w_q, const float *w_scale,
                                        int64_t M, int64_t N, int64_t K,
                                        void *y_bf16, void *stream);

/* The same GEMM with a caller workspace, for shapes whose grid of output
 * tiles would leave compute units idle: small M and N with long K (e.g.
 * the DeepSeek-V3 q_a and kv_a projections at a few hundred tokens); large
 * grids of 256x256 tiles whose last round of 256 compute units is partly
 * empty (e.g. 8192 x 7168 x 16384: 896 tiles, 3.5 rounds), or that fill
 * less than one round with long K (e.g. 512 x 7168 x 16384); and decode
 * batches of 9 to 16 rows with long K (e.g. a 4096 x 14336 down
 * projection), where a workgroup covering 64 output columns over part of K
 * re-reads less of x than one covering 16 columns over all of it, and of
 * 33 to 64 rows with K >= 6144, where one row tile of 128 split over K
 * beats the decode kernel's per-workgroup re-reads of x.  The same
 * operation and passage as fp8_block_gemm: a workgroup runs one output tile
 * over one contiguous range of K blocks, promoting each 128-long partial
 * sum with its scale pair into fp32 as fp8_block_gemm does, and stores the
 * range's unrounded fp32 sums in the workspace; a second kernel adds a
 * tile's ranges in K order and rounds once to bf16.  In the partly empty
 * last round case only that round's tiles are split (their K blocks cut
 * into 256 equal ranges, "stream-K"); the whole rounds before it run
 * unsplit in the same launch.  The result meets the same tolerance; split
 * tiles are not bit-identical to fp8_block_gemm (the fp32 sums are
 * associated differently), unsplit ones are.
 *   fp8_block_gemm_workspace_bytes(M, N, K): bytes the split needs, 0 when
 *     it is not used for these sizes.  17 <= M <= 32 never splits.  M > 32
 *     (with K >= 6144 when M <= 64):
 *     either at most 128 output tiles of 128x128 and K long enough for the
 *     split to gain (a time model measured on MI355X picks the number of K
 *     ranges, 2 to min(256 / tiles, K / 512), or none): ranges x M x N x 4
 *     bytes; or at least 192 tiles of 256x256, not a whole number of rounds
 *     of 256, where a time model (1.9 us per K block of a tile against the
 *     partial sums' traffic) gains more than 8 us: (the ranges, at most
 *     256, plus the last round's tiles) x 256 KB (100.7 MB for 8192 x 7168
 *     x 16384); or 32 to 191 tiles of 256x256 with K >= 7168 and more than
 *     128 tiles of 128x128, run wholly as stream-K where the same model
 *     beats an estimate of the 128x128 kernels by 10 % (e.g. the
 *     DeepSeek-V3 o_proj, MLP up and MLP down at M = 512): (the ranges plus
 *     the tiles) x 256 KB (81.8 MB for 512 x 7168 x 16384).
 *     9 <= M <= 16: ceil(N / 64) column groups times the number of K ranges
 *     (at most 256 / groups and K / 2048) must reach 192, where N is too
 *     small for ceil(N / 64) groups alone to fill the chip and K is at most
 *     65536.  Invalid sizes: 0.  Host arithmetic only, no HIP call.
 *   fp8_block_gemm_ws: arguments as fp8_block_gemm, plus `workspace`
 *     (device, 16-byte aligned, owned by the caller, overwritten, not
 *     initialised by the caller) of `workspace_bytes` bytes.  When the
 *     workspace is NULL or smaller than fp8_block_gemm_workspace_bytes(M,
 *     N, K), or that is 0, the call is exactly fp8_block_gemm (bit-identical
 *     output) and the workspace is not touched.  Calls that share a
 *     workspace must be ordered on one stream.  Errors as fp8_block_gemm;
 *     a misaligned workspace that would be used is FP8BLK_ERR_ALIGN. */
FP8BLK_API size_t fp8_block_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K);
FP8BLK_API fp8blk_status fp8_block_gemm_ws(const void *x_q, const float *x_scale,
                                           const void *w_q, const float *w_scale,
                                           int64_t M, int64_t N, int64_t K, void *y_bf16,
                                           void *workspace, size_t workspace_bytes,
                                           void *stream);

/* fp8_block_gemm_ws without a caller workspace, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid allocation).  Same operation, plan and kernels as
 * fp8_block_gemm_ws given a large enough workspace (bit-identical output),
 * except that shapes fp8_block_gemm_ws would give the stream-K split of a
 * partly empty last round run unsplit, as fp8_block_gemm (bit-identical to
 * it; those partial sums take up to ~100 MB); the split's fp32 partial sums
 * go to a device array inside the library
 * of FP8BLK_SCRATCH_BYTES bytes, one per GPU, held until the process ends,
 * whose address is looked up once per device on the first call made with
 * that device current.  Allocates nothing.
 *   Arguments and errors as fp8_block_gemm; FP8BLK_ERR_SCRATCH if the split
 *   would need more than FP8BLK_SCRATCH_BYTES (no valid size does today:
 *   the largest plan is 16 MiB plus a few bytes).
 *   All calls on one GPU share its scratch array, which keeps the last
 *   call's contents (the split writes every partial it reads, so nothing
 *   needs clearing): calls that may overlap on one GPU (different streams,
 *   no ordering between them) race on it and must be serialised by the
 *   caller. */
#define FP8BLK_SCRATCH_BYTES ((size_t)16 * 1024 * 1024 + (size_t)64 * 1024)
FP8BLK_API fp8blk_status fp8_block_gemm_noalloc(const void *x_q, const float *x_scale,
                                                const void *w_q, const float *w_scale,
                                                int64_t M, int64_t N, int64_t K,
                                                void *y_bf16, void *stream);

/* Grouped block-scaled FP8 GEMM for mixture-of-experts layers: expert e
 * multiplies rows [off[e], off[e+1]) of x by its own W[e].  "Fine-grained
 * FP8" page, "UE8M0 scale format": expert matmuls run through grouped
 * back-ends that take fp32 scales directly; "DeepGEMM fast path" names the
 * expert back-ends.
 *   x_q [total_M,K], x_scale [total_M,K/128]
 *   w_q [E,N,K], w_scale [E, ceil(N/128), K/128]
 *   expert_offsets: DEVICE int32 [E+1], non-decreasing, off[0] = 0,
 *       off[E] <= total_M.  Trusted (read on the device, no host sync);
 *       row ranges are clamped to [0, total_M).
 *   y_bf16 [total_M,N] out; rows that belong to no expert are not written. */
FP8BLK_API fp8blk_status fp8_grouped_block_gemm(const void *x_q, const float *x_scale,
                                                const void *w_q, const float *w_scale,
                                                const int32_t *expert_offsets, int32_t E,
                                                int64_t total_M, int64_t N, int64_t K,
                                                void *y_bf16, void *stream);

/* The whole FP8 linear layer, y = x * W^T from bf16 x: dynamic activation
 * quantization then the block-scaled GEMM ("DeepGEMM fast path"; the
 * quantization "fused ahead of the GEMM").  For M <= 64 (decode) one kernel
 * can do both: the activation codes and scales are formed in registers
 * inside the weight-streaming GEMM and never reach memory.  It is used when
 * no workspaces are given (x_q_ws and x_scale_ws may be NULL for M <= 64;
 * they are then not touched), and with workspaces where it is the faster
 * path: M <= 16 with N * K <= 2^25, or with K <= 8192 and N wide enough for
 * the kernel to pack several 16-column slabs per workgroup; 16 < M <= 32
 * with N * K <= 2^24.
 * Otherwise the two kernels run back to back on `stream` through the
 * caller's workspaces x_q_ws [M,K] and x_scale_ws [M,K/128] (required for
 * M > 64, 16-byte aligned), which then hold the activation codes and
 * scales.  The activation codes and scales are always
 * those of fp8_act_quant_group; y is bit-identical to fp8_act_quant_group
 * followed by fp8_block_gemm wherever that GEMM runs its decode kernel
 * (M <= 32, and 32 < M <= 64 with N < 12288 and K <= 16384: the same K
 * split over the same waves); where it runs a tiled kernel instead
 * (32 < M <= 64 with N >= 12288 or K > 16384, reached by the fused kernel
 * only without workspaces) the fp32 partial sums are added in another
 * order.  It takes no GEMM workspace and so never the K splits of
 * fp8_block_gemm_ws (small grids, stream-K tail, decode with long K);
 * callers that want them run fp8_act_quant_group then fp8_block_gemm_ws.
 *   x_bf16 [M,K], w_q [N,K], w_scale [ceil(N/128),K/128] in; y_bf16 [M,N] out. */
FP8BLK_API fp8blk_status fp8_linear(const void *x_bf16, int64_t M, int64_t N, int64_t K,
                                    const void *w_q, const float *w_scale, void *x_q_ws,
                                    float *x_scale_ws, void *y_bf16, void *stream);

/* Batched (fixed-capacity) expert layout.  "Fine-grained FP8" page,
 * "UE8M0 scale format": the batched_mm expert back-end takes fp32 scales
 * directly.  Reading fixed here: expert e owns a slab of `capacity` rows of
 * which the first counts[e] (clamped to [0, capacity]) hold tokens.
 *   x_q [E*capacity, K], x_scale [E*capacity, K/128]  (i.e. [E, C, ...])
 *   w_q [E,N,K], w_scale [E, ceil(N/128), K/128]
 *   expert_counts: DEVICE int32 [E] (trusted, read on the device)
 *   y_bf16 [E*capacity, N] out; rows past an expert's count are not written. */
FP8BLK_API fp8blk_status fp8_batched_block_gemm(const void *x_q, const float *x_scale,
                                                const void *w_q, const float *w_scale,
                                                const int32_t *expert_counts, int32_t E,
                                                int64_t capacity, int64_t N, int64_t K,
                                                void *y_bf16, void *stream);

/* ------------------------------------------------------------------------
 * Row-wise scales ("fp8r").
 * "BFL (fp8r / nvfp4)" page of the diffusers docs, introduction: one fp32
 * weight scale per row, activations quantized row-wise at run time;
 * "Kernels": a row-scaled fp8 matrix product.  Readings fixed here: the
 * element map of the block scheme with the set = one whole row of K values
 * (s = fl32(amax_row / 448), q = E4M3_RNE(fl32(x / s)), all-zero rows get
 * s = 0); y[m,n] = bf16( x_scale[m] * w_scale[n] * sum_k dec(x_q[m,k])
 * dec(w_q[n,k]) ) with fp32 accumulation.  K must be a multiple of 128 as
 * everywhere else. */

/* Row-wise quantization (weights: R = N output rows; activations: R = M
 * tokens).  in_bf16 [R,K] in; q [R,K] E4M3 codes out; scale [R] fp32 out. */
FP8BLK_API fp8blk_status fp8_rowwise_quant(const void *in_bf16, int64_t R, int64_t K, void *q,
                                           float *scale, void *stream);

/* Row-scaled FP8 GEMM.  x_q [M,K], x_scale [M], w_q [N,K], w_scale [N] in;
 * y_bf16 [M,N] out. */
FP8BLK_API fp8blk_status fp8_rowwise_gemm(const void *x_q, const float *x_scale,
                                          const void *w_q, const float *w_scale,
                                          int64_t M, int64_t N, int64_t K,
                                          void *y_bf16, void *stream);

/* ------------------------------------------------------------------------
 * SwiGLU ahead of the activation quantizer (the quantized input of a
 * mixture-of-experts down projection).  "Fine-grained FP8" page: experts
 * run through grouped back-ends with fp32 scales, and activations are
 * quantized per token per 128-channel group at run time ("DeepGEMM fast
 * path").  The pages do not spell SwiGLU out; readings fixed here:
 *   gate_up_bf16 [M, 2I] in: gate g in columns [0, I), up u in [I, 2I);
 *   h = bf16_RNE(SiLU(g) * u), SiLU(g) = g / (1 + e^-g), evaluated in
 *   binary64 (its bf16 rounding is the exact value's except within ~2^-52
 *   of a rounding midpoint);
 *   x_q [M, I] E4M3 codes and x_scale [M, I/128] fp32 out: exactly
 *   fp8_act_quant_group applied to h (h itself is never written).
 * I must be a positive multiple of 128 and M * I / 128 < 2^31
 * (FP8BLK_ERR_SHAPE).  Every h must be finite (|SiLU(g) * u| below bf16's
 * overflow threshold); otherwise the codes of its group are unspecified. */
FP8BLK_API fp8blk_status fp8_swiglu_act_quant(const void *gate_up_bf16, int64_t M, int64_t I,
                                              void *x_q, float *x_scale, void *stream);

/* The same with power-of-two scales ("UE8M0 scale format"): x_scale [M, I/128]
 * E8M0 bytes (no alignment needed), exactly fp8_act_quant_group_ue8m0
 * applied to h. */
FP8BLK_API fp8blk_status fp8_swiglu_act_quant_ue8m0(const void *gate_up_bf16, int64_t M,
                                                    int64_t I, void *x_q, uint8_t *x_scale,
                                                    void *stream);

/* ------------------------------------------------------------------------
 * Static activation scale.
 * "Fine-grained FP8" page, "DeepGEMM fast path": besides the dynamic scheme
 * the page names static activation quantization (its back-ends keep it on
 * the Triton path).  Readings fixed here: one calibrated fp32 scale s for
 * the whole activation tensor, supplied by the caller in DEVICE memory (one
 * float, 4-byte aligned; it may change between calls without a host sync),
 * with the meaning of the dynamic scales (x ~= dec(q) * s);
 * q = E4M3_RNE(sat(fl32(x / s))), the IEEE quotient saturated to +-448 (the
 * inputs may exceed the calibrated range).  s must be positive and finite;
 * otherwise results are unspecified (the kernels stay in bounds). */

/* Static activation quantization.
 *   x_bf16 [M,K] bf16 in; x_scale DEVICE fp32 [1] in; x_q [M,K] E4M3 out. */
FP8BLK_API fp8blk_status fp8_act_quant_static(const void *x_bf16, int64_t M, int64_t K,
                                              const float *x_scale, void *x_q, void *stream);

/* Block-scaled FP8 GEMM with one static activation scale:
 * y[m,n] = bf16( sum_kb x_scale * w_scale[n/128,kb] * sum_{k in kb}
 *                dec(x_q[m,k]) dec(w_q[n,k]) ), fp32 accumulation.
 *   x_q [M,K], x_scale DEVICE fp32 [1], w_q [N,K], w_scale [ceil(N/128),K/128]
 *   in; y_bf16 [M,N] out. */
FP8BLK_API fp8blk_status fp8_block_gemm_static(const void *x_q, const float *x_scale,
                                               const void *w_q, const float *w_scale,
                                               int64_t M, int64_t N, int64_t K,
                                               void *y_bf16, void *stream);

/* ------------------------------------------------------------------------
 * Power-of-two scales stored as E8M0 bytes.
 * "Fine-grained FP8" page, "UE8M0 scale format": pre-quantized
 * DeepSeek-V4-style checkpoints keep their scales as packed float8_e8m0fnu
 * (scale_fmt = "ue8m0") instead of fp32.  Readings fixed here:
 *   - E8M0 is the OCP MX scale type: byte b encodes 2^(b - 127), 0xFF is NaN,
 *     there is no zero.  One byte per scale, in the same layouts as the fp32
 *     scales above ("packed" = 1 byte instead of 4).
 *   - The scale of a block or group is 2^e, e the smallest integer >= -127
 *     with amax <= 448 * 2^e (rounded up, so no code saturates); the byte is
 *     e + 127 (never 0xFF for finite input; an all-zero set gets 0x00).
 *   - q = E4M3_RNE(x * 2^-e), an exact quotient.
 *   - Activations are quantized with power-of-two scales too, so both GEMM
 *     operands carry E8M0 bytes and the matrix core applies them (each
 *     128-block product enters the fp32 accumulator already scaled).
 * Everything else (shapes, validation, errors, streams) is as above. */

/* Weight quantization with E8M0 block scales.
 *   w_bf16 [N,K] bf16 in; w_q [N,K] E4M3 codes out;
 *   w_scale [ceil(N/128), K/128] E8M0 bytes out (blocks as above). */
FP8BLK_API fp8blk_status fp8_weight_block_quant_ue8m0(const void *w_bf16, int64_t N, int64_t K,
                                                      void *w_q, uint8_t *w_scale,
                                                      void *stream);

/* Dynamic activation quantization with E8M0 group scales.
 *   x_bf16 [M,K] bf16 in; x_q [M,K] E4M3 codes out;
 *   x_scale [M, K/128] E8M0 bytes out (groups as above). */
FP8BLK_API fp8blk_status fp8_act_quant_group_ue8m0(const void *x_bf16, int64_t M, int64_t K,
                                                   void *x_q, uint8_t *x_scale, void *stream);

/* Block-scaled FP8 GEMM with E8M0 scales on both operands, y = x * W^T in
 * bf16: y[m,n] = sum_kb 2^(x_scale[m,kb]-127) * 2^(w_scale[n/128,kb]-127) *
 * sum_{k in kb} dec(x_q[m,k]) dec(w_q[n,k]), fp32 accumulation.
 *   x_q [M,K], x_scale [M,K/128] bytes, w_q [N,K],
 *   w_scale [ceil(N/128),K/128] bytes in; y_bf16 [M,N] out. */
FP8BLK_API fp8blk_status fp8_block_gemm_ue8m0(const void *x_q, const uint8_t *x_scale,
                                              const void *w_q, const uint8_t *w_scale,
                                              int64_t M, int64_t N, int64_t K,
                                              void *y_bf16, void *stream);

/* The E8M0 GEMM with K split over workgroups through a caller workspace,
 * exactly as fp8_block_gemm_ws is to fp8_block_gemm (same operation and
 * passage as fp8_block_gemm_ue8m0; the K ranges hold an even number of K
 * blocks, so shapes with an odd K/128 are never split).  Without a usable
 * workspace the call is fp8_block_gemm_ue8m0, bit for bit. */
FP8BLK_API size_t fp8_block_gemm_ue8m0_workspace_bytes(int64_t M, int64_t N, int64_t K);
FP8BLK_API fp8blk_status fp8_block_gemm_ue8m0_ws(const void *x_q, const uint8_t *x_scale,
                                                 const void *w_q, const uint8_t *w_scale,
                                                 int64_t M, int64_t N, int64_t K,
                                                 void *y_bf16, void *workspace,
                                                 size_t workspace_bytes, void *stream);

/* Grouped variant with E8M0 scales (mixture-of-experts; "UE8M0 scale
 * format": such checkpoints also run the expert matmuls).  Arguments as for
 * fp8_grouped_block_gemm, with x_scale [total_M,K/128] and
 * w_scale [E, ceil(N/128), K/128] as E8M0 bytes. */
FP8BLK_API fp8blk_status fp8_grouped_block_gemm_ue8m0(const void *x_q, const uint8_t *x_scale,
                                                      const void *w_q, const uint8_t *w_scale,
                                                      const int32_t *expert_offsets, int32_t E,
                                                      int64_t total_M, int64_t N, int64_t K,
                                                      void *y_bf16, void *stream);

/* ------------------------------------------------------------------------
 * Around the expert products and the shared projections: routing with its
 * balance loss, rows by group, the weighted return of the experts' rows, and
 * low-rank adapters of many requests.
 *
 * Conventions as above, except where an entry says otherwise: fp32 and int32
 * arrays other than logits need 4-byte alignment, byte masks none; rows of
 * bf16 matrices may have any width N >= 0 (odd ones too) and start at any
 * even address, only the base pointers are 16-byte aligned.  Workspaces are
 * 16-byte aligned device memory of at least the size the _workspace_bytes
 * function returns (0: may be NULL), overwritten, not initialised by the
 * caller (missing: FP8BLK_ERR_NULL, too small: FP8BLK_ERR_SHAPE); calls that
 * share one must be ordered on one stream.  None of these
 * calls synchronises, and no result depends on the order in which workgroups
 * run: the same inputs give the same bits. */

#define FP8BLK_F32 0
#define FP8BLK_BF16 1
#define FP8BLK_F16 2            /* gated projections and 4-bit weights */
#define FP8BLK_MAX_GROUPS 1024  /* experts, groups or adapters of one call */
#define FP8BLK_MAX_TOPK 32
#define FP8BLK_MAX_RANK 256

/* Routing of T tokens to k of E experts each, with the rows each expert gets
 * and the balance loss.
 *   logits [T,E] of logits_type (FP8BLK_F32 or FP8BLK_BF16) in
 *   mask [T] bytes in, or NULL (all set): rows with 0 are not routed, whatever
 *       their logits hold
 *   ids [T,k] int32 out: the k largest logits' experts, largest first, equal
 *       ones by the lowest expert; an expert whose logit is -infinity is never
 *       chosen, and slots left over hold -1
 *   weights [T,k] fp32 out: softmax over all experts at the chosen ones, or
 *       (renormalize != 0) softmax over the chosen ones alone; 0 in slots
 *       with id -1
 *   counts [E] int32 out: rows that chose each expert
 *   rows [1] int32 out, or NULL (not wanted): rows routed (mask set and some
 *       logit > -infinity) = n
 *   loss [1] fp32 out, or NULL (not computed):
 *       loss_coef * sum_e (counts_e * E / (k * n)) * (sum_t p_te / n),
 *       p the softmax over all experts of the routed rows; 0 if n = 0.
 * Sums are kept in fp32 in a fixed order.  NaN logits are never chosen and
 * make their row's weights and the loss unspecified; ids stay in range.
 * 1 <= E <= FP8BLK_MAX_GROUPS, 1 <= k <= min(E, FP8BLK_MAX_TOPK),
 * T * k < 2^31.  T = 0 clears counts, rows and loss. */
FP8BLK_API size_t fp8blk_moe_route_workspace_bytes(int64_t T, int32_t E);
FP8BLK_API fp8blk_status fp8blk_moe_route(const void *logits, int logits_type, const uint8_t *mask,
                                          int64_t T, int32_t E, int32_t k, int renormalize,
                                          float loss_coef, int32_t *ids, float *weights,
                                          int32_t *counts, int32_t *rows, float *loss,
                                          void *workspace, size_t workspace_bytes, void *stream);

/* Gradient of the logits, from the gradients of the weights and of the loss
 * (the choice and the counts carry none).  logits, ids, weights, counts, rows,
 * renormalize and loss_coef as in and out of fp8blk_moe_route; counts and rows
 * are read only with d_loss (rows may be NULL without it).
 *   d_weights [T,k] fp32 in, or NULL (zero); those of slots with id -1 are
 *       not read
 *   d_loss [1] fp32 in (device memory), or NULL (zero)
 *   d_logits [T,E] of logits_type out; rows not routed get 0. */
FP8BLK_API fp8blk_status fp8blk_moe_route_backward(
    const void *logits, int logits_type, int64_t T, int32_t E, int32_t k, int renormalize,
    float loss_coef, const int32_t *ids, const float *weights, const int32_t *counts,
    const int32_t *rows, const float *d_weights, const float *d_loss, void *d_logits,
    void *stream);

/* R rows listed by group (a stable counting sort), e.g. the slots of a routed
 * batch by expert (ids of fp8blk_moe_route, R = T * k) or rows by adapter.
 *   ids [R] int32 in: a row's group in [0, G); rows with any other number
 *       belong to no group
 *   order [R] int32 out: the rows group by group, in their own order within a
 *       group, rows of no group last
 *   positions [R] int32 out: a row's place in order, -1 for rows of no group
 *   offsets [G+1] int32 out: group g's rows are order[offsets[g] ..
 *       offsets[g+1]) -- the expert_offsets of the grouped GEMM.
 * 1 <= G <= FP8BLK_MAX_GROUPS, R < 2^31. */
FP8BLK_API size_t fp8blk_group_rows_workspace_bytes(int64_t R, int32_t G);
FP8BLK_API fp8blk_status fp8blk_group_rows(const int32_t *ids, int64_t R, int32_t G,
                                           int32_t *order, int32_t *positions, int32_t *offsets,
                                           void *workspace, size_t workspace_bytes, void *stream);

/* The experts' rows back to their tokens:
 * out[t] = bf16( base[t] + sum_j weights[t,j] * y[positions[t,j]] ), fp32 sums
 * in the order of j.
 *   y_bf16 [R,N], weights [T,k] fp32, positions [T,k] int32 in; a slot whose
 *       position is outside [0, R) adds nothing, and rows of y that no slot
 *       names are not read
 *   base_bf16 [T,N] in, or NULL (zero); out_bf16 [T,N] out, may be base_bf16.
 * 1 <= k <= FP8BLK_MAX_TOPK, T * k < 2^31. */
FP8BLK_API fp8blk_status fp8blk_moe_combine(const void *y_bf16, int64_t R, const float *weights,
                                            const int32_t *positions, const void *base_bf16,
                                            int64_t T, int32_t k, int64_t N, void *out_bf16,
                                            void *stream);

/* Gradients of fp8blk_moe_combine (that of base is d_out itself).
 *   rows_used [1] int32 in (device memory): the rows of y in use come first,
 *       e.g. offsets[G] of fp8blk_group_rows; positions names each of them
 *       once (the gradient of one that no slot names is not written)
 *   d_y_bf16 [R,N] out: bf16(weights[t,j] * d_out[t]) at positions[t,j]; rows
 *       from rows_used on get 0
 *   d_weights [T,k] fp32 out: <d_out[t], y[positions[t,j]]>, 0 for slots
 *       without a position. */
FP8BLK_API fp8blk_status fp8blk_moe_combine_backward(
    const void *d_out_bf16, const void *y_bf16, int64_t R, const float *weights,
    const int32_t *positions, const int32_t *rows_used, int64_t T, int32_t k, int64_t N,
    void *d_y_bf16, float *d_weights, void *stream);

/* Low-rank adapters of many requests at once, beside a shared projection:
 * out[t] = bf16( base[t] + scale[g] * (x[t] A[g]^T) B[g]^T ), g = ids[t];
 * rows with ids[t] outside [0, L) have no adapter: out[t] = base[t].
 * Products accumulate in fp32; x A^T enters the second product with every bit
 * of its fp32 value.
 *   base_bf16 [T,N], row stride base_stride elements, in, or NULL (zero)
 *   x_bf16 [T,K], row stride x_stride, in
 *   a_bf16 [L,r,K], b_bf16 [L,N,r], scale [L] fp32 (or NULL: 1) in.  Adapters
 *       of a smaller rank are padded with zeros.
 *   ids [T] int32 in
 *   order [T], offsets [L+1] int32 in, or both NULL: fp8blk_group_rows of ids,
 *       which a program with many projections computes once per batch; used
 *       (and needed inside, in the workspace) only for T > 64
 *   out_bf16 [T,N], row stride out_stride, out; may be base_bf16 (with the
 *       same stride), and rows without adapter are then left alone.
 * K a positive multiple of 128, r a multiple of 8 up to FP8BLK_MAX_RANK,
 * 1 <= L <= FP8BLK_MAX_GROUPS; strides at least the rows' widths.  A batch whose
 * launches would need 2^32 threads is refused (FP8BLK_ERR_SHAPE): with tiles =
 * min(T, T / 64 + L + 1), or T / 16 instead of T / 64 for T <= 64, sizes pass
 * while tiles * (N + 256) < 2^31 and tiles * (r + 32) < 2^29. */
FP8BLK_API size_t fp8blk_lora_add_workspace_bytes(int64_t T, int64_t K, int32_t r, int32_t L,
                                                  int listed);
FP8BLK_API fp8blk_status fp8blk_lora_add(const void *base_bf16, int64_t base_stride,
                                         const void *x_bf16, int64_t x_stride,
                                         const void *a_bf16, const void *b_bf16,
                                         const int32_t *ids, const float *scale,
                                         const int32_t *order, const int32_t *offsets, int64_t T,
                                         int64_t K, int64_t N, int32_t r, int32_t L,
                                         void *out_bf16, int64_t out_stride, void *workspace,
                                         size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------
 * The gated projections of a feed-forward block in 16 bits, with their
 * gradients: g = x Wg^T, u = x Wu^T, h = act(g) * u.
 *
 * Conventions as in the section before: rows of any width start at any even
 * address, base pointers are 16-byte aligned, workspaces likewise, nothing
 * synchronises, and the same inputs give the same bits.
 *   type: FP8BLK_BF16 or FP8BLK_F16, of every matrix of the call
 *   act: FP8BLK_SILU (g / (1 + e^-g)), FP8BLK_GELU (g times the normal
 *       distribution's function) or FP8BLK_GELU_TANH (its form by tanh,
 *       g (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3))) / 2)
 *   x [M,K], row stride x_stride elements
 *   w [2I,K]: the I gate rows first, then the I up rows (the order of
 *       fp8_swiglu_act_quant's columns)
 * Sums are kept in fp32; g, u and act(g) enter what follows unrounded.
 * 1 <= K <= 2^22, 0 <= I <= 2^21, K <= x_stride <= 2^22, M < 2^31, and fewer
 * than 2^23 tiles of 256 x 256 in any of the products (FP8BLK_ERR_SHAPE). */

#define FP8BLK_SILU 0
#define FP8BLK_GELU 1
#define FP8BLK_GELU_TANH 2

/*   h [M,I] out
 *   factors out, or NULL (not wanted): M rows of FP8BLK_FACTOR_ROW(I) bytes that
 *       fp8blk_gated_linear_backward takes: what the gradient of h is multiplied
 *       by, u act'(g) and act(g), in 24 bits each (of 16 the gradients would
 *       carry their rounding on top of dgu's). */
#define FP8BLK_FACTOR_ROW(I) (((I) + 3) / 4 * 24)
FP8BLK_API size_t fp8blk_gated_linear_workspace_bytes(int64_t M, int64_t I, int64_t K,
                                                      int64_t x_stride);
FP8BLK_API fp8blk_status fp8blk_gated_linear(const void *x, int64_t x_stride, const void *w,
                                             int type, int act, int64_t M, int64_t I, int64_t K,
                                             void *h, void *factors, void *workspace,
                                             size_t workspace_bytes, void *stream);

/* Gradients of fp8blk_gated_linear: dgu = (d_h u act'(g), d_h act(g)) rounded
 * once to type, d_x = dgu W, d_w = dgu^T x.  The rounding has type's range: in fp16 a
 * dgu past 65504 is an infinity, which d_x's row and d_w's row of it show (as infinities
 * or NaN), and one below 2^-25 is zero, so fp16 gradients want the loss scaled.
 *   d_h [M,I] in
 *   factors in, as the forward call wrote it, or NULL: g and u are then
 *       computed again (act is read only in this case)
 *   d_x [M,K], d_w [2I,K] out, either may be NULL (not wanted)
 * With M = 0 d_w, and with I = 0 d_x, is cleared. */
FP8BLK_API size_t fp8blk_gated_linear_backward_workspace_bytes(int64_t M, int64_t I, int64_t K,
                                                               int64_t x_stride, int want_d_x,
                                                               int want_d_w);
FP8BLK_API fp8blk_status fp8blk_gated_linear_backward(
    const void *d_h, const void *x, int64_t x_stride, const void *w, const void *factors, int type,
    int act, int64_t M, int64_t I, int64_t K, void *d_x, void *d_w, void *workspace,
    size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------
 * 4-bit weights with a scale, and if wanted a zero point, per group of K:
 *   W[n,k] = (q[n,k] - z[n,k/group]) * s[n,k/group]
 * Conventions, type and act as in the section before.
 *   codes [N,K/2] bytes: q in 0..15, two to a byte, the even k in the low half
 *   scale [N,K/group] of type
 *   zeros [N,K/group] bytes in 0..15, or NULL: every z is 8
 *   group: 32, 64 or 128; K a multiple of it, K <= 2^22
 * Products: N <= 2^26 rows (2I of them for the gated form), M < 2^31, K <= x_stride <=
 * 2^22, and fewer than 2^23 tiles of 256 x 256 in a product
 * (FP8BLK_ERR_SHAPE).  Codes meet x before the scale does: 15 |x| summed over a group
 * has to stay finite in fp32.  An infinity in x gives what (q - z) x does: an infinity,
 * or NaN where q = z; other rows are not touched by it. */

/* Weights [N,K] of type to 4 bits; per group
 *   with zero points: lo = min(0, least weight), hi = max(0, largest),
 *     s = type(fl32(fl32(hi - lo) / 15)), z = clamp(rint(-lo / s), 0, 15)
 *   zeros NULL: s = type(fl32(max |w| / 7)), z = 8
 *   q = clamp(rint(w / s) + z, 0, 15)
 * rint to the nearest whole number, ties to even.  A group that holds a NaN has a NaN
 * scale; one that holds an infinity, or whose hi - lo passes fp32's range, an infinite
 * one: the values that such a group stands for are NaN.  s = 0, infinite or NaN gives
 * q = z, with zero points z = 0. */
FP8BLK_API fp8blk_status fp8blk_w4_quant(const void *w, int type, int64_t N, int64_t K, int group,
                                         void *codes, void *scale, void *zeros, void *stream);

/* The weights that codes stand for, rounded once to type: w [N,K] out. */
FP8BLK_API fp8blk_status fp8blk_w4_dequant(const void *codes, const void *scale, const void *zeros,
                                           int type, int64_t N, int64_t K, int group, void *w,
                                           void *stream);

/* y = x W^T: x [M,K] of type with row stride x_stride, y [M,N] out, fp32 sums.
 * The codes enter the products as whole numbers and a group's sum is multiplied
 * by its scale in fp32, so no weight is rounded. */
FP8BLK_API size_t fp8blk_w4_linear_workspace_bytes(int64_t M, int64_t N, int64_t K,
                                                   int64_t x_stride);
FP8BLK_API fp8blk_status fp8blk_w4_linear(const void *x, int64_t x_stride, const void *codes,
                                          const void *scale, const void *zeros, int type, int group,
                                          int64_t M, int64_t N, int64_t K, void *y, void *workspace,
                                          size_t workspace_bytes, void *stream);

/* fp8blk_gated_linear's forward pass with 4-bit weights [2I,K], the gate rows
 * first: h [M,I] out. */
FP8BLK_API size_t fp8blk_w4_gated_linear_workspace_bytes(int64_t M, int64_t I, int64_t K,
                                                         int64_t x_stride);
FP8BLK_API fp8blk_status fp8blk_w4_gated_linear(const void *x, int64_t x_stride, const void *codes,
                                                const void *scale, const void *zeros, int type,
                                                int group, int act, int64_t M, int64_t I, int64_t K,
                                                void *h, void *workspace, size_t workspace_bytes,
                                                void *stream);

/* Human-readable name of a status code (static storage, never NULL). */
FP8BLK_API const char *fp8blk_status_string(int status);

/* FP8BLK_ABI_VERSION of the built library. */
FP8BLK_API int fp8blk_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FP8BLK_H */
