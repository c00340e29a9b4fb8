// Microscaled 4-bit (MX4) rows and weights: layout constants, the rounding
// shared by every quantizing kernel, and the launchers.
//
// Layouts MX4R (rows) and MX16x128 (weights) are described in w2a8_mx4.h.
// Both hold the 32 values of a block in the order of A4I chunks, and both
// give a lane of the scaled matrix instructions its operand by one 16-byte
// load: v_mfma_scale_f32_16x16x128_f8f6f4 takes row l % 16 and k-block l / 16
// of a 128-k tile from lane l (32 values of 4 bits, one scale byte).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device.h"
#include "w2a8_mx4.h"

namespace w2a8 {

constexpr int kMxRows = 16;                    // rows of a weight tile
constexpr int kMxTileBytes = kMxRows * kTileK / 2;   // 1024
constexpr int kMxRowTile = kTileK / 2;         // code bytes of a row's tile: 64
constexpr int kMxQuad = 4;                     // tiles whose scale bytes share a word

inline int64_t mx4_tiles(int64_t K) { return ceil_div(K, kTileK); }
inline int64_t mx4_quads(int64_t K) { return ceil_div(mx4_tiles(K), kMxQuad); }

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

// Operand register block of a scaled MFMA on 4-bit floats: the instruction
// reads the first four registers.
__device__ __forceinline__ v8i fp4_operand(v4u v) {
    return v8i{int(v[0]), int(v[1]), int(v[2]), int(v[3]), 0, 0, 0, 0};
}

// acc + a * b over one tile of 128 k; TILE picks the scale bytes.
template <int TILE>
__device__ __forceinline__ v4f mx4_mfma(v4u a, v4u b, v4f acc, uint32_t as, uint32_t bs) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(a), fp4_operand(b), acc, 4, 4,
                                                            TILE, int(as), TILE, int(bs));
}

// The two T32x128 words of a ternary row's block of 32 values -> the block as
// 4-bit floats of twice the weight, A4I order, to be used with the scale 2^-1.
// A word's codes c = w + 1 sit at bits 8b + 2j: with the bits inverted, bit 0
// of a code says that w is not 0 and bit 1 that it is not positive, which at
// bits 2 and 3 of a nibble is 2.0, -2.0 or -0.  The codes at bits 8b and
// 8b + 4 are values b and 8 + b of the chunk, those at 8b + 2 and 8b + 6
// values 4 + b and 12 + b.
// (Truth table 0x0C: not the first and the second operand.)
__device__ __forceinline__ uint32_t ternary_word(uint32_t w) {
    return __builtin_amdgcn_bitop3_b32(int(w), int(0xCCCCCCCCu), 0, 0x0C);
}
__device__ __forceinline__ v4u ternary_fp4(uint32_t w0, uint32_t w1) {
    return v4u{ternary_word(w0 << 2), ternary_word(w0), ternary_word(w1 << 2), ternary_word(w1)};
}
constexpr uint32_t kTernaryScale = 0x7E7E7E7Eu;   // 2^-1 in every byte

// Scale byte of a block from its largest magnitude's bits (an fp32 with the
// sign cleared; integer order is magnitude order, NaN above infinity above
// all numbers): floor(log2 a) is the exponent field less 127, so the byte
// (that - 2) + 127 is the field less 2, at least 0; 255 for a NaN or infinity.
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t amax_bits) {
    const int f = int(amax_bits >> 23);
    return f == 255 ? 255u : uint32_t(max(f - 2, 0));
}

// The power of two that a scale byte stands for (byte 0: 2^-127, a subnormal;
// 255: a NaN).
__device__ __forceinline__ float mx4_scale_value(uint32_t byte) {
    return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7FC00000u : byte << 23);
}

// Four bytes of codes: byte j holds lo[j] (low half) and hi[j], each divided
// by the scale and rounded half to even, saturating at 6 (v_cvt_scalef32_pk_
// fp4_f32: measured to round, saturate and take subnormal scales and values
// as w2a8_mx4.h states).  A block with a NaN or an infinity gets codes 0.
__device__ __forceinline__ uint32_t mx4_codes4(const float (&lo)[4], const float (&hi)[4],
                                               float scale) {
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, lo[0], hi[0], scale, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, lo[1], hi[1], scale, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, lo[2], hi[2], scale, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, lo[3], hi[3], scale, 3);
    return scale == scale ? w : 0u;
}

// Value i of a float row as fp32; TYPE is a w2a8_mx4_type.
template <int TYPE>
__device__ __forceinline__ float mx4_load1(const void *p, int64_t i) {
    if constexpr (TYPE == W2A8_F32)
        return static_cast<const float *>(p)[i];
    else if constexpr (TYPE == W2A8_BF16)
        return lo_bf16(static_cast<const uint16_t *>(p)[i]);
    else
        return float(static_cast<const _Float16 *>(p)[i]);
}

// Two fp32 -> two bf16 in one word, half to even; a NaN stays one
// (v_cvt_pk_bf16_f32: one instruction, where the integer form of the rounding
// took as long as a third of a 256 x 256 x 5120 product's instructions).
typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{a, b}), v2bf));
}
__device__ __forceinline__ uint32_t bf16_bits(float v) { return bf16_pair(v, 0.0f) & 0xFFFFu; }

// A product of MX4 rows (launch arguments by value).
struct Mx4Launch {
    const uint8_t *w;      // MX16x128 codes, or T32x128 ternary weights
    const uint8_t *ws;     // MX16x128 scales (null for ternary weights)
    const uint8_t *xq;     // MX4R codes and scales; unused by the fused kernels
    const uint8_t *xs;
    const void *x;         // fused kernels: one float row
    float *y_f32;
    uint16_t *y_bf16;
    float sw;
    int M, N, K, KT, KU;
    int strips, stages;    // stream kernel: row groups of the grid, LDS stages of a wave
};

// Result stores.  Rows of y start wherever N puts them, and global stores of
// 16 bytes need no more than their elements' alignment.
typedef v4f v4f_any __attribute__((aligned(4)));
typedef v4u v4u_any __attribute__((aligned(2)));
typedef v2u v2u_any __attribute__((aligned(2)));

// y[m][n..n+3] = v * sw where in range.
__device__ __forceinline__ void mx4_store4(const Mx4Launch &a, int m, int n, v4f v) {
    if (m >= a.M || n >= a.N) return;
    const int64_t at = int64_t(m) * a.N + n;
    v = v4f{v[0] * a.sw, v[1] * a.sw, v[2] * a.sw, v[3] * a.sw};
    if (n + 3 < a.N) {
        if (a.y_f32) *reinterpret_cast<v4f_any *>(a.y_f32 + at) = v;
        if (a.y_bf16)
            *reinterpret_cast<v2u_any *>(a.y_bf16 + at) =
                v2u{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
        return;
    }
#pragma unroll
    for (int e = 0; e < 3; ++e) {
        if (n + e >= a.N) break;
        if (a.y_f32) a.y_f32[at + e] = v[e];
        if (a.y_bf16) a.y_bf16[at + e] = uint16_t(bf16_bits(v[e]));
    }
}

hipError_t launch_quant_mx4(const void *x, int type, int64_t M, int K, uint8_t *xq, uint8_t *xs,
                            hipStream_t stream);
hipError_t launch_dequant_mx4(const uint8_t *xq, const uint8_t *xs, int64_t M, int K, void *y,
                              int type, hipStream_t stream);
hipError_t launch_quant_pack_mx4(const void *W, int type, int64_t N, int K, uint8_t *packed,
                                 hipStream_t stream);
// Weights streamed through LDS by single waves (mx4_stream.hip), M <= 32.
constexpr int kMx4StreamRows = 32;
hipError_t launch_mx4_stream(const Mx4Launch &a, int cus, hipStream_t stream);
// Waves of a workgroup of it.
int mx4_stream_waves(int M, int strips, int KU, int cus);
// Activations through LDS (mx4_gemm.hip), any M: the tile it takes (rows by
// columns over groups of waves that split k, and whether results pass the
// caches), and the launch.
struct Mx4TilePlan {
    int BM, BN, KS;
    bool pass;
};
Mx4TilePlan mx4_tile_plan(const Mx4Launch &a, int cus);
hipError_t launch_mx4_gemm(const Mx4Launch &a, int cus, hipStream_t stream);
// Its 256 x 256 form for MX4 weights (mx4_gemm_wide.hip), any M.  pass:
// results pass the caches.
hipError_t launch_mx4_gemm_wide(const Mx4Launch &a, bool pass, hipStream_t stream);
// One float row (x_type), rounded inside (M = 1).
hipError_t launch_mx4_fused(const Mx4Launch &a, int x_type, int cus, hipStream_t stream);

}  // namespace w2a8
