/*
 * moe_ops.h -- operators around and beside the routed block of moe.h:
 *
 *  - moe_norm_block: the norms before and after a block, fused with the
 *    block's gate and the residual scales;
 *  - moe_fp8_gemm, moe_fp8_gemm_grouped: matrix products of 8-bit floating
 *    point (e4m3) codes with one fp32 scale per block of 128, dense or grouped
 *    by expert;
 *  - moe_fp8_quant: bf16 rows to e4m3 codes with a scale per row and 128
 *    columns (the products' first operand);
 *  - moe_fp8_layer_forward: a whole MoE layer (router, top-k, SwiGLU experts,
 *    shared expert, weighted sum) whose experts are e4m3 with one scale per
 *    128 x 128 block.
 *
 * The Strata pages' experts are low-bit integer files (moe.h); e4m3 with block
 * scales is the form in which the same kind of layer is commonly distributed
 * before such a conversion, so a layer can be run from either.
 *
 * Conventions are those of moe.h: pointers marked "dev" are caller-owned
 * memory of the current device; nothing allocates, frees or synchronises;
 * arguments are checked on the host before anything is enqueued on `stream`;
 * MOE_OK means "enqueued".  Calls may be captured into graphs, and several
 * threads may call at once (on workspaces of their own).  Rows (T, M) are limited
 * to 2^31 - 256, else MOE_ERR_UNSUPPORTED_SHAPE.
 *
 * e4m3: sign, 4 exponent bits (bias 7), 3 mantissa bits, largest value 448, no
 * infinity; codes 0x7F and 0xFF are NaN.
 */
#ifndef MOE_OPS_H
#define MOE_OPS_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ norms */

/* moe_norm.flags */
#define MOE_NORM_F_POST 1u          /* the block's output is normalised before it is added */
#define MOE_NORM_F_ZERO_CENTRED 2u  /* weights are stored as w - 1: the factor is 1 + weight */
#define MOE_NORM_F_STREAM_F32 4u    /* the residual stream (x, x_out) is fp32 instead of bf16 */
#define MOE_NORM_F_SIGMOID 8u       /* the gate passes through a sigmoid */

/* moe_norm.gate_kind */
#define MOE_GATE_NONE 0
#define MOE_GATE_TOKEN 1    /* one value per token: bf16 [T] */
#define MOE_GATE_CHANNEL 2  /* one value per channel: bf16 [d] */
#define MOE_GATE_FULL 3     /* one value per token and channel: bf16 [T][d] */

/* Weights and constants of the norms between two blocks.  A host struct, read
 * only during the call. */
typedef struct moe_norm_s {
  int32_t d;            /* channels: a multiple of 8, 8 <= d <= 8192 */
  uint32_t flags;       /* MOE_NORM_F_* */
  int32_t gate_kind;    /* MOE_GATE_* */
  float eps;            /* > 0 */
  float stream_scale;   /* a: factor of the residual stream */
  float branch_scale;   /* b: factor of the block's (normalised, gated) output */
  const float* pre_w;   /* dev fp32 [d] or NULL (factor 1): the norm before the next block */
  const float* post_w;  /* dev fp32 [d] or NULL (factor 1): the norm after the block */
  /* row pitches in elements; 0 = d; otherwise >= d and a multiple of 8 */
  int64_t x_ld, y_ld, gate_ld, x_out_ld, h_ld;
} moe_norm;

/* For each of T rows, in fp32:
 *    u = y, or with MOE_NORM_F_POST  u = y * rsqrt(mean(y^2) + eps) * W(post_w)
 *    r = a * x + b * act(gate) * u          (y NULL: r = a * x, gate ignored)
 *    x_out = r rounded to the stream's type
 *    h = r * rsqrt(mean(r^2) + eps) * W(pre_w)
 * with W(w) = w, or 1 + w under MOE_NORM_F_ZERO_CENTRED, or 1 for a NULL
 * weight; act is the identity or the sigmoid, which is taken with the fast
 * exponential and division: off by at most 2^-21, and by (5 + 1.2 |gate|) 2^-23 of
 * its value down to -87 (0 or the value below).  h is taken from r before it is
 * rounded to the stream's type.  The outputs, each optional but at least one
 * given:
 *  x_out_or_null: dev [T][d] bf16 (fp32 under MOE_NORM_F_STREAM_F32);
 *  h_or_null: dev bf16 [T][d];
 *  codes_or_null, scales_or_null (both or neither): h in e4m3, dev uint8
 *    [T][d] (dense rows) and dev fp32 [T][ceil(d/128)]: for each 128 columns
 *    scale = max|h| / 448 and code = e4m3(h / scale), every step to nearest, ties
 *    to even (the quotients in fp32); a block of zeros has scale 0 and codes 0.
 *    The codes are taken from h before its rounding to bf16.
 * x: dev [T][d] of the stream's type; y_or_null: dev bf16 [T][d].
 * x_out may be x itself (same pitch), and h may be y itself (same pitch);
 * otherwise outputs may not overlap inputs or each other.
 * Sums of squares are fp32: rows with |value| above about 1e17 overflow.  A
 * NaN or infinity in a row stays in that row.
 * T = 0 enqueues nothing.  x, y, gate (CHANNEL, FULL), x_out, h, pre_w,
 * post_w: 16-byte aligned; codes: 8-byte aligned. */
moe_status moe_norm_block(const moe_norm* n, const void* x, const void* y_or_null,
                          const void* gate_or_null, int32_t T, void* x_out_or_null,
                          void* h_or_null, uint8_t* codes_or_null, float* scales_or_null,
                          void* stream);

/* --------------------------------------------------------------- products */

/* One weight matrix, or one per group (expert): e4m3 codes with a scale per
 * 128 x 128 block, row-major, K contracted.  A host struct, read only during
 * the call. */
typedef struct moe_fp8_mat_s {
  int32_t n;               /* N: rows of one matrix, output columns; 1 <= N <= 65536 */
  int32_t k;               /* K: a multiple of 16, 16 <= K <= 65536 */
  int32_t groups;          /* G: 1 <= G <= 1024; N*G < 2^31 */
  const uint8_t* codes;    /* dev [G][N][K], 16-byte aligned */
  const float* scales;     /* dev fp32 [G][ceil(N/128)][ceil(K/128)] */
} moe_fp8_mat;

/* bf16 rows to codes and scales, as moe_norm_block writes them.
 *  x: dev bf16 [T][d], rows ld elements apart (0 = d; >= d, a multiple of 8);
 *  d a multiple of 8, 8 <= d <= 65536; codes: dev [T][d], 8-byte aligned;
 *  scales: dev fp32 [T][ceil(d/128)].  x: 16-byte aligned.  Outputs may not overlap
 *  x or each other.  T = 0 enqueues nothing. */
moe_status moe_fp8_quant(const void* x, int64_t ld, int32_t T, int32_t d, uint8_t* codes,
                         float* scales, void* stream);

/* c[m][n] = sum over blocks b of 128 columns k of
 *           a_scales[m][b] * w->scales[n/128][b] * sum_{k in b} a[m][k] * w[n][k]
 * with products of codes summed in fp32 on the tensor cores, blocks joined in
 * fp32, one rounding to bf16.
 *  a: dev e4m3 [M][K] (dense rows), 16-byte aligned; a_scales: dev fp32
 *  [M][ceil(K/128)]; c: dev bf16 [M][N] (dense rows), 2-byte aligned (16-byte
 *  aligned with N a multiple of 8 stores faster), which may not overlap a or
 *  a_scales.  w->groups must be 1.
 *  A NaN code or scale in a row of a, or of the weights, stays in that row, or
 *  column, of c.  M = 0 enqueues nothing.
 *  ws_or_null: a workspace of at least 256 bytes, zeroed once with
 *  moe_workspace_init(), whose error word reports a bounded wait that ran out
 *  (moe_workspace_error); NULL: not reported. */
moe_status moe_fp8_gemm(const moe_fp8_mat* w, const uint8_t* a, const float* a_scales, int32_t M,
                        void* c_bf16, void* ws_or_null, void* stream);

/* The same with one matrix per group of rows: rows offsets[g] <= m <
 * offsets[g+1] of a are multiplied with group g's matrix (experts' rows in
 * bucket order).
 *  offsets: dev int32 [G+1], non-decreasing, 0 <= offsets[g] <= M.  Rows of c
 *  before offsets[0] and from offsets[G] on are left as they were.  Groups may
 *  be empty.  Offsets outside 0..M or decreasing are clamped to that range and
 *  order (nothing is read or written outside the M rows) and set the range bit
 *  of the workspace's error word. */
moe_status moe_fp8_gemm_grouped(const moe_fp8_mat* w, const uint8_t* a, const float* a_scales,
                                int32_t M, const int32_t* offsets, void* c_bf16, void* ws_or_null,
                                void* stream);

/* The kernel that a product of M >= 1 rows takes: plan[0] columns of a tile, plan[1]
 * rows of a staged for it, plan[2] stages of the operand ring.  Host only; for the
 * current device's SMs, or 148 where no call of the library has asked for them yet. */
moe_status moe_fp8_gemm_plan(const moe_fp8_mat* w, int32_t M, int32_t grouped, int32_t plan[3]);

/* ------------------------------------------------------------------ layer */

/* One MoE layer with e4m3 experts.  A host struct, read only during the call. */
typedef struct moe_fp8_layer_s {
  int32_t d_model;        /* d: a multiple of 32, 32 <= d <= 4096 */
  int32_t n_experts;      /* E: top_k <= E <= 1024 */
  int32_t ffn;            /* F: a multiple of 32, 32 <= F <= 4096 */
  int32_t top_k;          /* k: 1 <= k <= 16 */
  int32_t shared_ffn;     /* Fs: 0 = no shared expert, else as F */
  const float* router_w;         /* dev fp32 [E][d] */
  const float* router_bias;      /* dev fp32 [E] or NULL */
  const uint8_t* gate_up;        /* dev e4m3 [E][2][F][d]: gate rows, then up rows */
  const float* gate_up_scales;   /* dev fp32 [E][2][ceil(F/128)][ceil(d/128)] */
  const uint8_t* down;           /* dev e4m3 [E][d][F] */
  const float* down_scales;      /* dev fp32 [E][ceil(d/128)][ceil(F/128)] */
  const uint8_t* shared_gate_up; /* dev e4m3 [2][Fs][d], or NULL when Fs == 0 */
  const float* shared_gate_up_scales;
  const uint8_t* shared_down;    /* dev e4m3 [d][Fs], or NULL when Fs == 0 */
  const float* shared_down_scales;
} moe_fp8_layer;

/* Most tokens of one moe_fp8_layer_forward call. */
#define MOE_FP8_LAYER_MAX_T 32

/* Bytes of workspace moe_fp8_layer_forward needs for up to max_tokens tokens
 * (0 on invalid arguments); zero it once with moe_workspace_init(). */
size_t moe_fp8_layer_workspace_bytes(const moe_fp8_layer* layer, int32_t max_tokens);

/* The whole layer for a few tokens, 0 <= T <= MOE_FP8_LAYER_MAX_T:
 *   logits, ids, w as moe_route_topk (fp32 logits; largest first, equal values
 *   to the lower expert index, NaN below every number)
 *   y = FFN_shared(x) + sum_j w[j] * FFN_{ids[j]}(x)  -> bf16
 * with FFN as in moe.h and each weight = code * its block's scale.  Activations
 * are not quantised: a token's columns enter the gate/up products exactly, except
 * that in each 128 columns values below 2^-13 of the largest are off by up to
 * 2^-21 of it; the hidden values, with the routing weight folded in, enter the
 * down product as two fp16 terms after a power-of-two scale per expert and token:
 * 22 bits of each, or an error below 2^-39 of the token's largest.  Sums
 * are fp32.  An infinity or NaN in a token makes its row of y NaN; one in an
 * expert's weights reaches only the tokens that selected the expert.
 *  x: dev bf16 [T][d]; y: dev bf16 [T][d], which may not overlap x; both 16-byte
 *  aligned.
 *  ids_or_null: dev int32 [T][k]; w_or_null: dev fp32 [T][k]: the routing,
 *  written when non-NULL.
 * Windows of up to 8 tokens run as one kernel over all SMs, whose blocks wait
 * for one another between the router, the gate/up products and the down
 * product; more tokens run as consecutive windows of 8.  Those waits are
 * bounded as in moe.h (moe_workspace_set_wait_limit).  T = 0 enqueues nothing.
 * T above the limit returns MOE_ERR_UNSUPPORTED_SHAPE. */
moe_status moe_fp8_layer_forward(const moe_fp8_layer* layer, const void* x_bf16, int32_t T,
                                 void* y_bf16, int32_t* ids_or_null, float* w_or_null, void* ws,
                                 size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_OPS_H */
