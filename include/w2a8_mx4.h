/*
 * w2a8_mx4.h — microscaled 4-bit (MX4) rows, weights and products of
 * libw2a8.so.  Status codes, ownership, streams, device, limits and thread
 * safety are those of w2a8.h.  No entry point here takes a workspace: none
 * keeps state between calls, so any number of calls may be in flight on any
 * streams, and all may be recorded into HIP graphs (kernels only).  Results
 * do not depend on timing: every sum has a fixed order, which depends on the
 * shape and the device alone.  An output of a device entry point must not
 * share bytes with another buffer of the call (W2A8_ERR_VALUE): the kernels
 * write results while others of their workgroups still read.
 *
 * The format is the MXFP4 of the OCP Microscaling Formats specification
 * (version 1.0): 4-bit floats of 1 sign, 2 exponent and 1 mantissa bits
 * (magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6; codes 0..7, sign in bit 3) in
 * blocks of 32 consecutive k that share a power of two 2^e, held as the byte
 * e + 127 (byte 255: NaN, all 32 values of the block are NaN).
 *
 * Rounding of float values to MX4, shared by every quantizing entry point.
 * Per block b of 32 consecutive k of a row (the last one may be shorter):
 *   a = max |x|;  e = max(floor(log2 a) - 2, -127)  (a = 0: e = -127);
 *   q = x * 2^-e rounded half to even to a 4-bit float, magnitudes above 6
 *       becoming 6 (they are below 8).
 * The scaling is exact, so this is the only rounding.  A negative value that
 * rounds to zero keeps its sign (code 8).  A block that holds a NaN or an
 * infinity gets byte 255 and codes 0: it reads as 32 NaN.
 *
 * Row layout "MX4R" (activations).  Kp = ceil(K/128)*128, KT = Kp/128,
 * KU = ceil(KT/4).  Codes: 64*KT bytes per row, rows back to back, the
 * nibble order of A4I (w2a8.h): in a chunk of 16 values, byte j holds value j
 * in its low and 8+j in its high half, byte 4+j values 4+j and 12+j.  Scales:
 * 16*KU bytes per row, rows back to back; the byte of block g (0..3) of tile
 * t (k = 128t + 32g ..) is byte 16*(t/4) + 4*g + t%4.  Codes and scale bytes
 * of padding are 0.
 *
 * Weight layout "MX16x128".  NS = ceil(N/16) strips of 16 rows.  Codes: tile
 * (s, t) is 1024 bytes at (s*KT + t)*1024: slot l = 16*g + r is the 16 bytes
 * of row 16s + r, block g of tile t, in MX4R order.  Scales follow at
 * NS*KT*1024: 256 bytes per strip and four tiles, at (s*KU + t/4)*256 +
 * 4*l + t%4 the byte of slot l of tile t.  Padding is 0.
 */
#ifndef W2A8_MX4_H
#define W2A8_MX4_H

#include "w2a8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of float rows (x_type, w_type, y_type). */
enum w2a8_mx4_type { W2A8_F32 = 0, W2A8_BF16 = 1, W2A8_F16 = 2 };

/* Bytes of the codes / the scales of M rows (MX4R), or -1 if out of range. */
int64_t mx4_act_bytes(int64_t M, int64_t K);
int64_t mx4_scale_bytes(int64_t M, int64_t K);

/* Bytes of packed MX4 weights (MX16x128), or -1 if N or K is out of range. */
int64_t mx4_packed_bytes(int64_t N, int64_t K);

/* Host: pack MX4 weights from the interchange form.  codes: [N][ceil(K/2)]
 * bytes, value 2i in the low and 2i+1 in the high half of byte i.  scales:
 * [N][ceil(K/32)] bytes.  packed: at least mx4_packed_bytes(N, K) bytes
 * (packed_bytes is its capacity; W2A8_ERR_BUFSIZE). */
int pack_mx4(const uint8_t *codes, const uint8_t *scales, int64_t N, int64_t K, void *packed,
             int64_t packed_bytes);

/* Host: inverse of pack_mx4.  For odd K the last half byte of a row is 0. */
int unpack_mx4(const void *packed, int64_t packed_bytes, int64_t N, int64_t K, uint8_t *codes,
               uint8_t *scales);

/* Device: round M float rows to MX4R.  x: [M][K] of x_type, 16-byte aligned.
 * x_q: mx4_act_bytes(M, K), x_s: mx4_scale_bytes(M, K) bytes, both 16-byte
 * aligned.  W2A8_ERR_VALUE for an unknown x_type. */
int quant_act_mx4(const void *x, int x_type, int64_t M, int64_t K, uint8_t *x_q, uint8_t *x_s,
                  void *stream);

/* Device: the values of MX4R rows as floats, y: [M][K] of y_type, 16-byte
 * aligned.  Exact in fp32 and bf16, rounded half to even in fp16; magnitudes
 * past the type's range (65504 for fp16, some of scale bytes 253 and 254 for
 * the others) become infinity. */
int dequant_act_mx4(const uint8_t *x_q, const uint8_t *x_s, int64_t M, int64_t K, void *y,
                    int y_type, void *stream);

/* Device: round float weights W [N][K] of w_type to MX4 and pack them
 * (MX16x128).  w_packed: at least mx4_packed_bytes(N, K) bytes, 16-byte
 * aligned (packed_bytes is its capacity). */
int quant_pack_mx4(const void *W, int w_type, int64_t N, int64_t K, void *w_packed,
                   int64_t packed_bytes, void *stream);

/* Product of MX4 rows with MX4 weights, M >= 1 (decode, short batches,
 * prefill):
 *   y[m][n] = sum_b 2^(ex[m][b] + ew[n][b]) * sum_{k in b} qx[m][k] * qw[n][k]
 * accumulated in fp32.  w_packed: MX16x128 of W [N][K]; x_q, x_s: MX4R of M
 * rows; all 16-byte aligned.  y_f32: fp32 [M][N], y_bf16: bf16 [M][N] (the
 * fp32 result rounded half to even); at least one of them, both 16-byte
 * aligned, each element written once, nothing behind the last. */
int w4mx4_gemm(const void *w_packed, const uint8_t *x_q, const uint8_t *x_s, int64_t M, int64_t N,
               int64_t K, float *y_f32, uint16_t *y_bf16, void *stream);

/* The same product with ternary weights (T32x128 of w2a8.h, at least
 * w2a8_packed_bytes(N, K) bytes):
 *   y[m][n] = s_w * sum_b 2^(ex[m][b]) * sum_{k in b} qx[m][k] * w[n][k]
 * The sum is accumulated in fp32 and multiplied by s_w once. */
int w2mx4_gemm(const void *w_packed, const uint8_t *x_q, const uint8_t *x_s, int64_t M, int64_t N,
               int64_t K, float s_w, float *y_f32, uint16_t *y_bf16, void *stream);

/* Whole linear layer for one token, in one launch: bit-identical to
 * quant_act_mx4 (M = 1) followed by w4mx4_gemm / w2mx4_gemm.  x: [K] of
 * x_type, 16-byte aligned.  Every wave rounds the part of the row that it
 * consumes, so the 4-bit row never goes through memory. */
int w4mx4_linear_gemv(const void *w_packed, const void *x, int x_type, int64_t N, int64_t K,
                      float *y_f32, uint16_t *y_bf16, void *stream);
int w2mx4_linear_gemv(const void *w_packed, const void *x, int x_type, int64_t N, int64_t K,
                      float s_w, float *y_f32, uint16_t *y_bf16, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* W2A8_MX4_H */
