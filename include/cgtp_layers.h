/* cgtp_layers.h - the layers between equivariant convolutions and linear maps,
 * on irreps rows, for AMD Instinct MI355X (gfx950): group norm with its
 * activation, cross attention to a context of another length, and dropout.
 *
 * Conventions are those of cgtp.h: rows are ir_mul blocks ([2l+1][mul], channel
 * index fastest) concatenated in irreps order; tensor arguments are DEVICE
 * pointers of the handle's dtype unless stated; calls run on `stream` and
 * allocate nothing; outputs are overwritten; a NULL gradient is skipped;
 * results are bitwise reproducible (no floating-point atomics); errors are
 * status codes with a message in cgtp_last_error(). Degrees go up to CGTP_LMAX.
 * The compute calls only launch kernels, so they can be captured in a graph;
 * the create and destroy calls allocate, free or copy and cannot. Handles hold
 * tables on the device that was current when they were created and are used
 * with that device current (else INVALID_ARG); they are immutable and may be
 * shared between streams and threads.
 */
#ifndef CGTP_LAYERS_H
#define CGTP_LAYERS_H

#include "cgtp.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct cgtp_samples_s* cgtp_samples;
typedef struct cgtp_norm_s* cgtp_norm;
typedef struct cgtp_dropout_s* cgtp_dropout;
typedef struct cgtp_attn_s* cgtp_attn;
typedef struct cgtp_attn_batch_s* cgtp_attn_batch;

/* ------------------------------------------------------------------ samples */

/* The rows of S samples laid end to end: sample s owns rows ptr[s] ..
 * ptr[s+1]-1 (a molecule's atoms, a box's particles, a sequence's positions).
 * ptr is a HOST array of S + 1 offsets with ptr[0] = 0, non-decreasing; samples
 * may be empty. Copies the offsets (synchronously). At most 2^31 - 1 rows.
 * Errors: INDEX for bad offsets, UNSUPPORTED for too many rows, ALLOC. */
cgtp_status cgtp_samples_create(int64_t S, const int64_t* ptr, cgtp_samples* out);
cgtp_status cgtp_samples_destroy(cgtp_samples samples);

/* ------------------------------------------- group norm with its activation */

typedef enum { CGTP_ACT_NONE = 0, CGTP_ACT_SILU = 1, CGTP_ACT_GELU = 2 } cgtp_act;

/* Group norm of irreps rows, channels last. Every block's channels are split
 * into `groups` groups of mul / groups consecutive channels. Statistics are
 * taken per sample and group over the sample's rows, the 2l+1 components and
 * the group's channels:
 *   0e blocks: mu = mean x, var = mean (x - mu)^2, and y = act(xh w_c + b_c);
 *   others:    mu = 0,      var = mean x^2,        and y = xh w_c,
 * with xh = (x - mu) / sqrt(var + eps). Only the even scalars take a mean, a
 * bias and an activation, so the map commutes with rotations and inversion.
 * weight [channels] has one entry per channel of every block (channels = sum of
 * mul), bias [biases] one per channel of the 0e blocks. gelu is x Phi(x) with
 * the error function. fp32, bf16 (fp32 arithmetic) and fp64.
 * Errors: PARSE; UNSUPPORTED (groups does not divide a multiplicity, a degree
 * above CGTP_LMAX); INVALID_ARG (groups < 1, eps not positive or no normal number
 * of the arithmetic, bad enum). */
cgtp_status cgtp_norm_create(const char* irreps, int64_t groups, cgtp_act act, double eps, cgtp_dtype dtype,
                             cgtp_norm* out);
cgtp_status cgtp_norm_destroy(cgtp_norm norm);
/* Row size, channel count, bias count and number of groups over all blocks. */
cgtp_status cgtp_norm_query(cgtp_norm norm, int64_t* dim, int64_t* channels, int64_t* biases, int64_t* num_groups);
/* Workspace bytes of cgtp_norm_forward (backward = 0) or cgtp_norm_backward. */
cgtp_status cgtp_norm_workspace_size(cgtp_norm norm, cgtp_samples samples, int backward, size_t* bytes);
/* y [rows][dim] from x [rows][dim]. stats [S][num_groups][2] receives mu and
 * 1 / sqrt(var + eps) in the accumulation type (fp32; fp64 for fp64 norms) for
 * the backward (entries of empty samples are not written); NULL if not wanted.
 * weight and bias may each be NULL (1, 0).
 * ws is 16-byte aligned. Errors: WORKSPACE, INVALID_ARG. */
cgtp_status cgtp_norm_forward(cgtp_norm norm, cgtp_samples samples, const void* x, const void* weight,
                              const void* bias, void* y, void* stats, void* ws, size_t ws_bytes, void* stream);
/* Reverse mode. With gz = grad_y act'(z), n = the group's element count and
 * A_c = sum gz xh, B_c = sum gz over a sample's rows and components:
 *   grad_weight_c = sum over samples of A_c, grad_bias_c the same of B_c,
 *   grad_x = (gz w_c - sum_c(w_c B_c) / n [0e] - xh sum_c(w_c A_c) / n) / sqrt(var + eps). */
cgtp_status cgtp_norm_backward(cgtp_norm norm, cgtp_samples samples, const void* x, const void* weight,
                               const void* bias, const void* stats, const void* grad_y, void* grad_x,
                               void* grad_weight, void* grad_bias, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------ dropout */

/* Dropout of irreps rows from a counter-based generator: nothing is stored, the
 * backward draws the same mask again. The 2l+1 components of a channel share
 * one draw, so a rotated input gives the rotated output.
 *   y = residual + (draw >= t ? x 65536 / (65536 - t) : 0),  t = floor(65536 p + 1/2)
 * (t at most 65535; residual may be NULL; a dropped infinity or NaN gives 0).
 * Draws are the 16-bit halves of Philox 4x32 with 10 rounds (Salmon, Moraes,
 * Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011), key =
 * seed (low word first), counter = (chunk, row low, row high, offset): a chunk
 * is 8 consecutive channels of a block (the last one of a block may be short;
 * chunks are numbered through the blocks), channel i of a chunk takes half
 * i % 2 (low first) of word i / 2. Use another offset for every call and layer.
 * Errors of create: PARSE, UNSUPPORTED (degree above CGTP_LMAX), INVALID_ARG. */
cgtp_status cgtp_dropout_create(const char* irreps, cgtp_dtype dtype, cgtp_dropout* out);
cgtp_status cgtp_dropout_destroy(cgtp_dropout drop);
cgtp_status cgtp_dropout_query(cgtp_dropout drop, int64_t* dim);
/* Errors: INVALID_ARG (p outside [0, 1) or NaN, B < 0, null tensors with B > 0).
 * y may be x or residual itself. */
cgtp_status cgtp_dropout_forward(cgtp_dropout drop, int64_t B, const void* x, double p, uint64_t seed,
                                 uint32_t offset, const void* residual, void* y, void* stream);
/* grad_x for the same p, seed and offset (the residual's gradient is grad_y). */
cgtp_status cgtp_dropout_backward(cgtp_dropout drop, int64_t B, const void* grad_y, double p, uint64_t seed,
                                  uint32_t offset, void* grad_x, void* stream);

/* ---------------------------------------------------------- cross attention */

/* Attention of the rows of one set of samples (queries) to the rows of another
 * (the context) of different lengths, sample by sample. `irreps` are the
 * queries'; head h owns channels h mul/heads .. (h+1) mul/heads - 1 of every
 * block, all components, so a head's vector has D = dim / heads elements. The
 * context rows (k and v) have the same blocks with multiplicities
 * mul kv_heads / heads; query head h reads context head h / (heads / kv_heads).
 *   s_ij = scale q_i . k_j,  p = softmax over the sample's unmasked keys j,
 *   out_i = sum_j p_ij v_j,  lse_i = log sum_j exp s_ij
 * The products run over whole irreps, so s is invariant and out equivariant.
 * A query without any key gives out = 0, lse = -inf and zero gradients, and
 * masked keys' rows are never used (both may hold infinities or NaN; masked
 * keys' gradients are 0). fp32 (fp32 matrix cores) and bf16 (products of bf16 values
 * summed in fp32; softmax weights and the score gradients are rounded to bf16
 * as matrix operands, and the weights are normalised by the sum of what they
 * were rounded to, so a row that sees one key gets exactly its value). D <= 256.
 * Errors: PARSE; UNSUPPORTED (fp64, heads does not divide a multiplicity, D >
 * 256, a degree above CGTP_LMAX); INVALID_ARG (heads or kv_heads < 1, kv_heads
 * does not divide heads). */
cgtp_status cgtp_attn_create(const char* irreps, int64_t heads, int64_t kv_heads, cgtp_dtype dtype, cgtp_attn* out);
cgtp_status cgtp_attn_destroy(cgtp_attn attn);
/* Row sizes of q/out and of k/v, and D. */
cgtp_status cgtp_attn_query(cgtp_attn attn, int64_t* dim_q, int64_t* dim_kv, int64_t* head_dim);

/* The work lists of one pair of sample layouts (the same number of samples):
 * which workgroup takes which rows, and where a long context or a long run of
 * queries is split and joined. Keeps copies: attn must outlive it, the samples
 * need not. Host work and a synchronous upload; reusable for every call on
 * these layouts. Errors: INVALID_ARG, UNSUPPORTED (rows x heads beyond 2^31, or
 * tiles of 32 rows x kv_heads beyond 2^24; a sample of any rows has its own tiles). */
cgtp_status cgtp_attn_batch_create(cgtp_attn attn, cgtp_samples queries, cgtp_samples context, cgtp_attn_batch* out);
cgtp_status cgtp_attn_batch_destroy(cgtp_attn_batch batch);

typedef enum {
  CGTP_ATTN_FORWARD = 1,        /* workspace of cgtp_attn_forward        */
  CGTP_ATTN_BACKWARD = 2,       /* workspace of cgtp_attn_backward       */
  CGTP_ATTN_CONTEXT = 3,        /* the packed context's own bytes        */
  CGTP_ATTN_FORWARD_PACKED = 4  /* workspace of cgtp_attn_forward_packed */
} cgtp_attn_op;
cgtp_status cgtp_attn_workspace_size(cgtp_attn_batch batch, int op, size_t* bytes);

/* out [queries][dim_q] (contiguous rows) from q, k, v with row strides ldq, ldk,
 * ldv in elements (at least the row size; k and v may be slices of one row).
 * |scale| is at most 2e38 (else INVALID_ARG). key_mask [context rows]: one byte a row, nonzero = may be attended; NULL =
 * all. lse [queries][heads] fp32, or NULL. ws is 16-byte aligned. */
cgtp_status cgtp_attn_forward(cgtp_attn_batch batch, const void* q, int64_t ldq, const void* k, int64_t ldk,
                              const void* v, int64_t ldv, const uint8_t* key_mask, double scale, void* out, float* lse,
                              void* ws, size_t ws_bytes, void* stream);
/* Lay the context's keys and values out once in the order in which the matrix
 * cores read them (CGTP_ATTN_CONTEXT bytes, 16-byte aligned), for any number of
 * cgtp_attn_forward_packed calls: serving, where each new token's query reads
 * the same encoded context. */
cgtp_status cgtp_attn_pack(cgtp_attn_batch batch, const void* k, int64_t ldk, const void* v, int64_t ldv,
                           const uint8_t* key_mask, void* context, size_t context_bytes, void* stream);
/* cgtp_attn_forward on a packed context. The batch may be another one than the
 * one that packed it, as long as its context layout is the same. */
cgtp_status cgtp_attn_forward_packed(cgtp_attn_batch batch, const void* q, int64_t ldq, const void* context,
                                     size_t context_bytes, double scale, void* out, float* lse, void* ws,
                                     size_t ws_bytes, void* stream);
/* Reverse mode from the forward's out and lse. With P = exp(s - lse):
 *   grad_v = P^T grad_out,  dS = P (grad_out v^T - rowsum(grad_out out)),
 *   grad_q = scale dS k,    grad_k = scale dS^T q,
 * grad_k and grad_v summed over the query heads that share a context head.
 * (out as stored: in bf16 its rounding is in grad_q and grad_k, most with few keys.)
 * Gradients are contiguous rows. The summation orders are fixed. */
cgtp_status cgtp_attn_backward(cgtp_attn_batch batch, const void* q, int64_t ldq, const void* k, int64_t ldk,
                               const void* v, int64_t ldv, const uint8_t* key_mask, double scale, const void* out,
                               const float* lse, const void* grad_out, int64_t ldg, void* grad_q, void* grad_k,
                               void* grad_v, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CGTP_LAYERS_H */
