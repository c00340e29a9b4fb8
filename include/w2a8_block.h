/*
 * w2a8_block.h — what stands around the ternary layers of a model, on int8
 * rows with one scale each (the rows of quant_act_int8): the norm that makes
 * them, products with 4-bit weights, and a mixture of ternary experts.
 *
 * Status codes, ownership, streams, device, limits and thread safety are those
 * of w2a8.h; float types are the w2a8_mx4_type of w2a8_mx4.h.  No entry point
 * keeps state between calls, so any number of calls may be in flight on any
 * streams (with workspaces of their own), and all may be recorded into HIP
 * graphs (kernels only).  Every result has a fixed order of sums, which
 * depends on the shape and the device alone.  An output must not share bytes
 * with another buffer of the call (W2A8_ERR_VALUE) unless stated.
 */
#ifndef W2A8_BLOCK_H
#define W2A8_BLOCK_H

#include "w2a8_mx4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * Root-mean-square norm into int8 rows.
 *
 * Per row, in fp32 unless stated (each step rounded once):
 *   h = x + residual, rounded to their type (h = x without a residual);
 *   v = h * weight (v = h without a weight);  a = max |v|;
 *   x_q = clamp(round_half_even(v * min(127 / a, FLT_MAX)), -127, 127);
 *   s_a = a / 127 / sqrt(mean(h^2) + eps), in fp64 and rounded once.
 * x_q * s_a is the normalised row: the codes are those of quant_act_int8 on
 * v, and the mean enters the scale alone, so the codes depend on no sum.  A
 * row whose v is all zero gives 0 and s_a = 0.  A row that holds a NaN or an
 * infinity, or whose h or v passes the range of its type, gives codes 0 and
 * s_a = NaN (its products are NaN).
 *
 * x, residual, h: device, [M][K] of `type`; residual may be NULL, and h is
 * given exactly when residual is.  h may be x or residual itself (in place).
 * weight: device, [K] of `type`, or NULL.  eps: at least 0, finite.
 * x_q: device, int8 [M][K].  s_a: device, fp32 [M].
 * ------------------------------------------------------------------------ */
int rmsnorm_quant_int8(const void *x, const void *residual, const void *weight, int type,
                       int64_t M, int64_t K, float eps, void *h, int8_t *x_q, float *s_a,
                       void *stream);

/* ------------------------------------------------------------------------
 * 4-bit weights with group scales.
 *
 * W[n][k] = s[n][g] * (q[n][k] - z[n][g]), q and z in 0..15, g = k / group,
 * group 32, 64 or 128 (the last group of a row may be shorter); z = 8 where
 * there are no zero points.  Scales are fp16 or bf16.
 *
 * Layout "W4T16x128".  Np = ceil(N/16)*16, KT = ceil(K/128), P = 128 / group,
 * GQ = ceil(ceil(K/group) / 4).
 *   Codes: 1 KiB tiles, tile (s, t) = rows 16s..16s+15, k 128t..128t+127, at
 *   byte (s*KT + t)*1024.  Lane slot l = 16c + r (c 0..3, r 0..15) is 16 bytes
 *   at 16l: 32 values of row 16s + r, value (32/P)*i + o (i < P) at
 *   k = 128t + (128/P)*i + (32/P)*c + o; byte 4j + b holds value 8j + b in its
 *   low and 8j + 4 + b in its high half, as q - 8 in two's complement.
 *   Scales behind them: 16 bits each, that of row 16s + r and group 4u + i at
 *   element ((s*GQ + u)*16 + r)*4 + i.
 *   Zero points (if any) behind them: z - 8 as int8, the same order.
 *   Rows past N, k past K and groups past the last hold 0.
 * ------------------------------------------------------------------------ */

/* Most activation rows of a product. */
#define W4A8_MAX_M 64

/* Bytes of the packed weights, or -1 if N, K or group is out of range. */
int64_t w4a8_packed_bytes(int64_t N, int64_t K, int64_t group, int zeros);

/* Host: from the interchange form.  codes: [N][ceil(K/2)] bytes, two values
 * q a byte, the lower k in the lower half.  scales: [N][ceil(K/group)] fp16 or
 * bf16 bit patterns.  zeros: [N][ceil(K/group)] bytes z, or NULL (none).
 * W2A8_ERR_VALUE for a group other than 32, 64, 128 or a z above 15 (packed is
 * then partly written), W2A8_ERR_BUFSIZE if packed_bytes is too small. */
int pack_w4a8(const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros, int64_t N,
              int64_t K, int64_t group, void *packed, int64_t packed_bytes);

/* Inverse of pack_w4a8 (host).  zeros: NULL if the packed weights have none. */
int unpack_w4a8(const void *packed, int64_t packed_bytes, int64_t N, int64_t K, int64_t group,
                uint8_t *codes, uint16_t *scales, uint8_t *zeros);

/* Device workspace bytes of w4a8_gemm, or -1 if a size is out of range: 0 for
 * one row and for rows of 1920 values or fewer, else room for the sums of up to
 * 8 parts of k. */
int64_t w4a8_workspace_bytes(int64_t M, int64_t N, int64_t K);

/* Product of int8 rows with them, 1 <= M <= W4A8_MAX_M (W2A8_ERR_SHAPE above):
 *   y[m][n] = s_a[m] * sum_g s[n][g] * sum_{k in g} (q[n][k] - z[n][g]) * x[m][k]
 * The sum over a group is exact, that over groups is in fp32.
 * x: device, int8 [M][K]; s_a: device, fp32 [M].  scale_type: W2A8_BF16 or
 * W2A8_F16.  zeros: whether w_packed has zero points.  y_f32, y_bf16: device,
 * [M][N], at least one of them.  workspace: device, at least
 * w4a8_workspace_bytes(M, N, K) bytes, 16-byte aligned (NULL when that is 0);
 * needs no clearing and holds nothing between calls. */
int w4a8_gemm(const void *w_packed, const int8_t *x, const float *s_a, int64_t M, int64_t N,
              int64_t K, int64_t group, int scale_type, int zeros, float *y_f32, uint16_t *y_bf16,
              void *workspace, int64_t ws_bytes, void *stream);

/* ------------------------------------------------------------------------
 * Mixture of ternary experts for a few tokens.
 *
 * Token m takes the top_k experts of its router logits (ties: the lower
 * index; a logit of -infinity is never taken), with weights
 *   p = exp(l - max l) / sum exp(l - max l),
 * the sum over the experts taken (renormalize) or over all.  For each of
 * them, the composition of this library's steps, e the expert:
 *   g = ((float)(w_gate[e] . x[m]) * s_a[m]) * s_gate[e],  u likewise (w_up);
 *   h = silu(g) * u, silu(g) = g / (1 + exp(-g))          (W2A8_ACT_SILU)
 *     = relu(g)^2 * u                                     (W2A8_ACT_RELU2);
 *   q, s_h: h quantized as quant_act_int8 does (on fp32 values);
 *   y[m] += p * (((float)(w_down[e] . q) * s_h) * s_down[e]),
 * added in the order of rank.  A token that takes no expert gives 0.  Logits
 * that hold a NaN or +infinity, and tokens that take an expert for which s_a or
 * a g, u or h of the row is not finite (a g of -infinity is no 0), give a row of
 * NaN.
 *
 * x: device, int8 [M][H]; s_a: device, fp32 [M]; logits: device, [M][E] of
 * logit_type.  w_gate, w_up: device, E matrices [I][H] in the T32x128 layout,
 * w2a8_packed_bytes(I, H) bytes apart; w_down: E matrices [H][I],
 * w2a8_packed_bytes(H, I) apart.  s_gate, s_up, s_down: device, fp32 [E].
 * y_f32, y_bf16: device, [M][H], at least one.  workspace: device, at least
 * w2a8_moe_workspace_bytes(M, H, I, E, top_k) bytes, 16-byte aligned; needs no
 * clearing and holds nothing between calls.
 * Limits: M <= W2A8_MOE_MAX_M, E <= W2A8_MOE_MAX_E, top_k <= E and
 * W2A8_MOE_MAX_TOP_K; H, I as K of w2a8.h (W2A8_ERR_SHAPE).
 * ------------------------------------------------------------------------ */
#define W2A8_MOE_MAX_M 64
#define W2A8_MOE_MAX_E 256
#define W2A8_MOE_MAX_TOP_K 16

enum w2a8_activation { W2A8_ACT_SILU = 0, W2A8_ACT_RELU2 = 1 };

/* Workspace bytes of w2a8_moe, or -1 if a size is out of range. */
int64_t w2a8_moe_workspace_bytes(int64_t M, int64_t H, int64_t I, int64_t E, int64_t top_k);

int w2a8_moe(const int8_t *x, const float *s_a, const void *logits, int logit_type,
             const void *w_gate, const void *w_up, const void *w_down, const float *s_gate,
             const float *s_up, const float *s_down, int64_t M, int64_t H, int64_t I, int64_t E,
             int64_t top_k, int activation, int renormalize, float *y_f32, uint16_t *y_bf16,
             void *workspace, int64_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* W2A8_BLOCK_H */
