/*
 * iq_train.h -- C ABI of libiq.so, continued: adapting a model whose weights
 * stay encoded.  A gated feed-forward block's first half forward and backward,
 * the backward pass of iq_linear with its low-rank adapters, and activations
 * kept in 8 bits until their backward pass.
 *
 * The conventions of iq.h and iq_run.h hold here as well: return codes, status
 * bits, caller-owned device buffers and workspaces, errors that the host can
 * see before anything is enqueued, asynchronous work on `stream`, payloads at
 * even addresses of which whole aligned 4-byte words are read, outputs that
 * must not overlap inputs, and results that repeat bit for bit (no atomics but
 * for maxima).  A workspace for T tokens serves every smaller T: the sizes that the
 * queries give do not fall as T grows.
 *
 * Arithmetic.  Products over a weight's columns (g, u below) are iq_linear's:
 * exact fp16 operands, fp32 sums, the block scale applied in fp32.  Products
 * over its rows (dx) cannot take a block's scale d out of the sum, so there d
 * meets the gradient of its row: their fp32 product is held as the sum of two fp16
 * values (2^-23 of it, in steps of 2^-39 of the token's largest gradient times the
 * payload's largest finite scale), and m v is exact in fp16 (a codebook that fp16
 * does not hold raises IQ_STATUS_ROUNDED).  That holds for bf16 calls as for f32
 * ones: what a call forms on the way (g, u, the gradients by them, p and v) is fp32,
 * and bf16 outputs are rounded once.  Sums are fp32.
 * Infinities and NaN in a token reach that token's rows of the outputs, and the
 * gradients of its adapter.
 */
#ifndef IQ_TRAIN_H
#define IQ_TRAIN_H

#include "iq_run.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations of a gated block. */
enum {
  IQ_ACT_SILU = 0,      /* g / (1 + exp(-g)) */
  IQ_ACT_GELU = 1,      /* g * Phi(g), Phi the normal distribution function */
  IQ_ACT_GELU_TANH = 2, /* g / 2 * (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3))) */
};

/* Activations kept in 8 bits: for each block of 32 columns (the last one of a
 * row may be shorter) a power of two, for each value a code,
 *
 *   value = code * 2^(exponent - 133).
 *
 * The exponent is the biased fp32 exponent of the block's largest finite
 * magnitude (at least 1), one more where that magnitude would round to more than
 * 127, and codes are rounded to nearest even, so a value is off by half a unit at
 * most.  The largest exponent, 254, has no further one: there codes end at 127, a
 * unit from a magnitude that would round to 128.  An infinity or NaN gets code
 * -128, which iq_restore returns as NaN, and raises IQ_STATUS_NONFINITE.
 *
 *  x          (device) [T, cols] f32 or bf16.
 *  codes      (device) [T, cols] int8 OUT.
 *  exponents  (device) [T, ceil(cols / 32)] uint8 OUT.
 *  status     (device, nullable).
 * T == 0 or cols == 0 enqueues nothing and returns IQ_OK.  Errors: IQ_ERR_DTYPE,
 * IQ_ERR_SHAPE (a size negative, cols above 2^24, T above 2^24 or more
 * than a launch takes), IQ_ERR_NULL, IQ_ERR_HIP. */
int iq_checkpoint(const void *x, int dtype, int64_t T, int64_t cols, int8_t *codes, uint8_t *exponents,
                  int32_t *status, hipStream_t stream);

/* The values of a checkpoint (exact in either dtype).  y (device) [T, cols] OUT,
 * dtype f32 or bf16.  Errors as iq_checkpoint. */
int iq_restore(const int8_t *codes, const uint8_t *exponents, int64_t T, int64_t cols, void *y, int dtype,
               hipStream_t stream);

/* Both projections of a gated feed-forward block, its activation and product:
 *
 *   h[t] = act(x[t] G^T) * (x[t] U^T)
 *
 *  gate, up (device) [inter, hidden/256, block_bytes] payloads of G and U.
 *  grid     (device) [grid_size, 8] f32 codebook of both.
 *  x        (device) [T, hidden] tokens, dtype f32 or bf16.
 *  act      IQ_ACT_*.
 *  h        (device) [T, inter] OUT, of x's dtype, rounded once.
 *  workspace, workspace_bytes  (device) at least iq_glu_workspace_size(...).
 *  status   (device, nullable): IQ_STATUS_ROUNDED.
 * T == 0 or inter == 0 enqueues nothing and returns IQ_OK.
 * Errors: IQ_ERR_FMT, IQ_ERR_DTYPE, IQ_ERR_NULL, IQ_ERR_SHAPE (inter or T
 * negative, hidden <= 0 or % 256, inter above 2^24, hidden or T above 2^24, sizes
 * whose launches would not fit a grid), IQ_ERR_ARG (act, a payload at an odd
 * address), IQ_ERR_WORKSPACE, IQ_ERR_HIP. */
int iq_glu(int fmt, const uint8_t *gate, const uint8_t *up, int64_t inter, int64_t hidden, const float *grid,
           const void *x, int dtype, int64_t T, int act, void *h, void *workspace, size_t workspace_bytes,
           int32_t *status, hipStream_t stream);
int iq_glu_workspace_size(int fmt, int64_t inter, int64_t hidden, int dtype, int64_t T, size_t *bytes);

/* Its backward pass.  g and u are formed again from x, so x is all that has to
 * be kept of the forward pass, as it was or as a checkpoint:
 *
 *   g = x G^T, u = x U^T;  dx[t] = (dh act'(g) u) G + (dh act(g)) U
 *
 *  x, exponents  (device) x [T, hidden] of `dtype` with exponents NULL, or the
 *           codes [T, hidden] int8 and exponents [T, hidden/32] of a checkpoint.
 *  dh       (device) [T, inter] of `dtype` (f32 or bf16): the gradient by h.
 *  dx       (device) [T, hidden] OUT, of `dtype`, rounded once.
 * inter == 0: dx is zeros.  Otherwise as iq_glu. */
int iq_glu_backward(int fmt, const uint8_t *gate, const uint8_t *up, int64_t inter, int64_t hidden,
                    const float *grid, const void *x, const uint8_t *exponents, const void *dh, int dtype,
                    int64_t T, int act, void *dx, void *workspace, size_t workspace_bytes, int32_t *status,
                    hipStream_t stream);
int iq_glu_backward_workspace_size(int fmt, int64_t inter, int64_t hidden, int dtype, int64_t T, size_t *bytes);

/* The backward pass of iq_linear, a = lora_ids[t]:
 *
 *   dx[t] = dy[t] W + s_a (dy[t] B_a) A_a
 *   da[n] = sum of s_n (dy[t] B_n)^T x[t],  db[n] = sum of s_n dy[t]^T (x[t] A_n^T)
 *                                                      over the tokens with a = n
 *
 *  packed, grid, lora_a, lora_b, lora_scale, lora_ids, num_adapters, rank as in
 *           iq_linear; x and the adapters are ignored when rank is 0.
 *  dy       (device) [T, rows] of `dtype` (f32 or bf16): the gradient by y.
 *  x, exponents  as in iq_glu_backward.
 *  dx       (device, nullable) [T, cols] OUT, of `dtype`, rounded once.
 *  da, db   (device) [num_adapters, rank, cols] and [num_adapters, rows, rank]
 *           OUT, of `dtype`, rounded once; zeros for an adapter without tokens.
 *  status   (device, nullable): IQ_STATUS_BADID, IQ_STATUS_ROUNDED.
 * rows == 0 or T == 0: dx, da and db, where they have entries, are zeros.
 * Errors as iq_linear's. */
int iq_linear_backward(int fmt, const uint8_t *packed, int64_t rows, int64_t cols, const float *grid,
                       const void *dy, const void *x, const uint8_t *exponents, int dtype, int64_t T,
                       const void *lora_a, const void *lora_b, const float *lora_scale, const int32_t *lora_ids,
                       int num_adapters, int rank, void *dx, void *da, void *db, void *workspace,
                       size_t workspace_bytes, int32_t *status, hipStream_t stream);
int iq_linear_backward_workspace_size(int fmt, int64_t rows, int64_t cols, int dtype, int64_t T, int num_adapters,
                                      int rank, size_t *bytes);

#ifdef __cplusplus
}
#endif
#endif /* IQ_TRAIN_H */
