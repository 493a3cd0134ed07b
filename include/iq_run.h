/*
 * iq_run.h -- C ABI of libiq.so, continued: running tokens through encoded
 * weights (the payloads iq_quantize and iq_choice_search write) without
 * decoding them to memory first.
 *
 * The conventions, return codes, status bits and layouts of iq.h hold here as
 * well: caller-owned device buffers and workspaces, host-detected errors before
 * anything is enqueued, asynchronous work on `stream`, results that do not
 * depend on the launch and repeat bit for bit (no atomics on results).
 *
 * Arithmetic.  A weight is d * m * (signed codebook value), d the block's fp16
 * scale and m its odd integer multiplier (iq_dequantize; IQ1 adds the shift to
 * the codebook value, IQ2 divides by 8).  The products run on the fp16 matrix
 * cores with fp32 accumulation:
 *  - m * (codebook value) is formed in fp16.  It is exact when the value has at
 *    most 6 significant bits (IQ2; IQ1: value +- 1/8 at most 7), as {1,3,5} and
 *    {-1,0,1} have; any other codebook is rounded to fp16, and the product again
 *    (relative 2^-11 each; in steps of 2^-24 below 2^-14, infinite past 65,504),
 *    and IQ_STATUS_ROUNDED is raised.
 *  - each token is scaled by the power of two that brings its largest finite
 *    magnitude under 2^15 and held in fp16: exact for bf16 tokens (what lies 2^-29
 *    or more below the token's largest value is rounded by less than 2^-39 of it);
 *    fp32 tokens are held as the sum of two fp16 values (relative 2^-22 of the
 *    value, or 2^-39 of the token's largest).
 *  - the block scale d is applied in fp32 to each 256-column block's fp32 sum,
 *    blocks are added in fp32, and the power of two is taken back at the end (bf16
 *    prompts keep the running sum in units of the block's d instead, and rescale it
 *    in fp32 from block to block).
 * Infinities and NaN in a token reach that token's outputs only.
 */
#ifndef IQ_RUN_H
#define IQ_RUN_H

#include "iq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Device status bit of the calls below, beside those of iq.h. */
#define IQ_STATUS_ROUNDED 32 /* a codebook value times a multiplier is not exact in fp16 (see above) */

/* Tokens through an encoded projection, with the low-rank adapters of many
 * requests beside it:
 *
 *   y[t] = x[t] W^T + lora_scale[a] * (x[t] A_a^T) B_a^T,   a = lora_ids[t],
 *
 * W the weight iq_dequantize returns for `packed`.  Without adapters (rank 0)
 * the second term is absent.
 *
 *  packed   (device) [rows, cols/256, block_bytes] payload, at an even address.
 *           Whole aligned 4-byte words are read: of the words that hold its first
 *           and last bytes, the bytes outside the payload as well (and unused).
 *  grid     (device) [grid_size, 8] f32 codebook the payload was encoded with.
 *  x        (device) [T, cols] tokens, dtype f32 or bf16.
 *  lora_a   (device) [num_adapters, rank, cols], lora_b (device) [num_adapters,
 *           rows, rank], both of x's dtype; adapters of smaller rank are padded
 *           with zeros.  lora_scale (device, nullable: all ones) [num_adapters]
 *           f32.  lora_ids (device) [T] int32: the token's adapter, -1 for none;
 *           any other id outside [0, num_adapters) raises IQ_STATUS_BADID and
 *           adds nothing.  All are ignored when rank is 0.  An infinity in lora_b
 *           gives NaN (bf16: its factor is held as a sum of three values).
 *  y        (device) [T, rows] OUT, of x's dtype: the fp32 sum, rounded once.
 *           Must not overlap any input.
 *  workspace, workspace_bytes  (device) scratch of at least
 *           iq_linear_workspace_size(...) bytes: the codebook and the tokens in
 *           fp16, and the tokens' rank-wide products.
 *  status   (device, nullable): IQ_STATUS_BADID, IQ_STATUS_ROUNDED.
 * T == 0 or rows == 0 enqueues nothing and returns IQ_OK.
 * Errors: IQ_ERR_FMT, IQ_ERR_DTYPE, IQ_ERR_NULL (grid, packed, x, y; with
 * adapters lora_a, lora_b, lora_ids; a needed workspace), IQ_ERR_SHAPE (rows or
 * T negative, cols <= 0 or % 256, rows above 2^27, sizes whose launches would not
 * fit a grid), IQ_ERR_ARG (rank outside [0, 1024], num_adapters < 1 with a rank, packed at an
 * odd address),
 * IQ_ERR_WORKSPACE, IQ_ERR_HIP. */
int iq_linear(int fmt, const uint8_t *packed, int64_t rows, int64_t cols, const float *grid, const void *x,
              int dtype, int64_t T, const void *lora_a, const void *lora_b, const float *lora_scale,
              const int32_t *lora_ids, int num_adapters, int rank, void *y, void *workspace,
              size_t workspace_bytes, int32_t *status, hipStream_t stream);

/* Workspace bytes iq_linear needs.  *bytes (host).  Errors: IQ_ERR_FMT,
 * IQ_ERR_DTYPE, IQ_ERR_NULL, IQ_ERR_SHAPE, IQ_ERR_ARG. */
int iq_linear_workspace_size(int fmt, int64_t rows, int64_t cols, int dtype, int64_t T, int rank, size_t *bytes);

/* A mixture-of-experts layer on encoded experts:
 *
 *   logits[t] = x[t] R^T;  ids[t] = the top_k largest logits, largest first;
 *   p = softmax of logits[t] over the chosen ids (renormalize != 0) or over all
 *   experts;  h_s = silu(x[t] G_e^T) * (x[t] U_e^T),  e = ids[t][s];
 *   y[t] = sum_s p_s h_s D_e^T.
 *
 *  gate, up (device) [num_experts * inter, hidden/256, block_bytes(fmt)] payloads:
 *           expert e's rows are e * inter ... (the fused layout iq_quantize
 *           encodes with rows_per_expert = inter).  Payloads as in iq_linear.
 *  down     (device) [num_experts * hidden, inter/256, block_bytes(down_fmt)].
 *  grid, down_grid  (device) the codebooks of fmt and down_fmt (the same pointer
 *           where both are the same).
 *  x        (device) [T, hidden] tokens, dtype f32 or bf16.
 *  router   (device, nullable) [num_experts, hidden], router_dtype f32 or bf16.
 *           Given: ids and weights are OUT.  Logits are accumulated in fp64, in
 *           the same order for every expert: those further apart than that can
 *           round (2 hidden 2^-53 of the sum of |x R|) are ranked as exact ones
 *           are, equal rows of the router tie.  Equal logits take the lower id
 *           first, NaN logits come after all others.
 *           NULL: ids and weights are the caller's (any other routing); an id
 *           outside [0, num_experts) raises IQ_STATUS_BADID and adds nothing, an
 *           id repeated in one token counts per occurrence.
 *  ids      (device) [T, top_k] int32, weights (device) [T, top_k] f32.
 *  y        (device) [T, hidden] OUT, of x's dtype.  Must not overlap any input.
 *  h is held between the two products in fp32, and enters the second one as the
 *  sum of two fp16 values under a power of two per 256 columns, for tokens of
 *  either type (relative 2^-22 of the value, or 2^-39 of the block's largest).
 *  workspace, workspace_bytes  (device) at least iq_moe_workspace_size(...).
 *  status   (device, nullable): IQ_STATUS_BADID, IQ_STATUS_ROUNDED.
 * T == 0 enqueues nothing and returns IQ_OK.
 * Errors: IQ_ERR_FMT, IQ_ERR_DTYPE, IQ_ERR_NULL, IQ_ERR_SHAPE (T negative, hidden
 * or inter <= 0 or % 256, sizes whose launches would not fit a grid), IQ_ERR_ARG
 * (num_experts outside [1, 4096], top_k outside [1, 64], top_k > num_experts with
 * a router, a payload at an odd address), IQ_ERR_WORKSPACE, IQ_ERR_HIP. */
int iq_moe(int fmt, int down_fmt, const uint8_t *gate, const uint8_t *up, const uint8_t *down, int64_t hidden,
           int64_t inter, int num_experts, const float *grid, const float *down_grid, const void *x, int dtype,
           int64_t T, const void *router, int router_dtype, int top_k, int renormalize, int32_t *ids,
           float *weights, void *y, void *workspace, size_t workspace_bytes, int32_t *status, hipStream_t stream);

/* Workspace bytes iq_moe needs.  *bytes (host).  Errors: IQ_ERR_FMT,
 * IQ_ERR_DTYPE, IQ_ERR_NULL, IQ_ERR_SHAPE, IQ_ERR_ARG. */
int iq_moe_workspace_size(int fmt, int down_fmt, int64_t hidden, int64_t inter, int num_experts, int dtype,
                          int64_t T, int top_k, size_t *bytes);

#ifdef __cplusplus
}
#endif
#endif /* IQ_RUN_H */
