// Products of MX4 rows for few rows (decode and short batches) on gfx950:
// the weights go from HBM straight into the operand registers of
// v_mfma_scale_f32_16x16x128_f8f6f4.
//
//   y[m][n] = s_w * sum_b 2^(ex + ew) * sum_{k in b} qx * qw
//
// The instruction takes 16 weight rows x 128 k as its first operand and 16
// activation rows x 128 k as its second, multiplies each block of 32 by both
// scales and adds in fp32: one instruction per KiB of MX4 weights, so the
// matrix pipe is nearly idle and the kernel is bound by the weight stream.
//
//  * MX4 weights: a tile is 1 KiB in lane order, one 16-byte load per lane;
//    the scale bytes of four tiles are one 4-byte load, and the instruction
//    picks the tile's byte by its operand selector.
//  * Ternary weights (T32x128, 1 KiB = 32 rows x 128 k): a lane loads the two
//    words of its row and block for either half of the strip.  A word's codes
//    c = w + 1 of 16 k become 4-bit floats in three operations: with the bits
//    of c inverted, bit 0 says that w is not 0 and bit 1 that it is negative
//    (or zero), which put at bits 2 and 3 of a nibble is +-2.0 or a zero; the
//    weight scale is 2^-1.  Codes at bits 8b + 2j and 8b + 4 + 2j (j = 0, 1)
//    give nibbles in A4I order, the order of the MX4R rows.
//  * A workgroup takes one strip (16 rows of MX4, 32 of ternary weights) and
//    its waves interleave over groups of four tiles; their sums meet in LDS
//    and are added in wave order, so no workspace and no atomics.
//  * Rows past M repeat row M - 1 and are not stored.
//  * Fused form (one float row): every wave rounds the 512 values of its
//    group of tiles itself, 8 per lane, and passes the codes round by 272
//    bytes of LDS of its own: no barrier, and the row's rounding is repeated
//    by every strip (some 40 instructions per 4 KiB of weights).
#include "mx4.h"

namespace w2a8 {
namespace {

enum { kMx4Weights = 0, kTernary = 1 };
constexpr int kMx4Rows = 3;   // SRC: MX4R rows (0..2: one float row of that type)

// One group of up to four tiles as it was loaded.
template <int KIND, int MB, int SRC>
struct Quad {
    static constexpr int RB = KIND == kTernary ? 2 : 1;   // blocks of 16 weight rows
    v4u w[KIND == kTernary ? 1 : 4];
    uint32_t t[KIND == kTernary ? 16 : 1];   // ternary: [tile][row block][word]
    uint32_t ws;
    v4u x[SRC == kMx4Rows ? MB * 4 : SRC == W2A8_F32 ? 2 : 1];
    uint32_t xs[MB];
};

template <int KIND, int MB, int SRC>
__device__ __forceinline__ void load_quad(const Mx4Launch &a, int64_t s, int m0, int u, int lane,
                                          Quad<KIND, MB, SRC> &q) {
    const int r = lane & 15, g = lane >> 4;
    const int last = a.KT - 1;
    if constexpr (KIND == kTernary) {
        const uint32_t *base = reinterpret_cast<const uint32_t *>(a.w) + s * a.KT * kTileWords;
        const int at = 32 * (r >> 2) + 8 * g + (r & 3);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t *t = base + int64_t(min(4 * u + i, last)) * kTileWords + at;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    q.t[4 * i + 2 * j + h] = __builtin_nontemporal_load(t + 128 * j + 4 * h);
        }
    } else {
        const uint8_t *base = a.w + s * a.KT * kMxTileBytes + 16 * lane;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            q.w[i] = __builtin_nontemporal_load(
                reinterpret_cast<const v4u *>(base + int64_t(min(4 * u + i, last)) * kMxTileBytes));
        q.ws = __builtin_nontemporal_load(
            reinterpret_cast<const uint32_t *>(a.ws + (s * a.KU + u) * 256) + lane);
    }
    if constexpr (SRC == kMx4Rows) {
#pragma unroll
        for (int b = 0; b < MB; ++b) {
            const int64_t m = min(m0 + 16 * b + r, a.M - 1);
            const uint8_t *row = a.xq + m * a.KT * kMxRowTile + 16 * g;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                q.x[4 * b + i] =
                    *reinterpret_cast<const v4u *>(row + min(4 * u + i, last) * kMxRowTile);
            q.xs[b] = *reinterpret_cast<const uint32_t *>(a.xs + (m * a.KU + u) * 16 + 4 * g);
        }
    } else {
        // Block lane / 4 of the group, values 16c + 4h + {0..3} and 8 more
        // of it (part c = bit 1, h = bit 0 of the lane): one code word.
        const int k = 512 * u + 32 * (lane >> 2) + 16 * ((lane >> 1) & 1) + 4 * (lane & 1);
        const int64_t size = SRC == W2A8_F32 ? 4 : 2;
        const uint8_t *p = static_cast<const uint8_t *>(a.x) + size * k;
        if (512 * u + 512 <= a.K) {
            if constexpr (SRC == W2A8_F32) {
                q.x[0] = *reinterpret_cast<const v4u *>(p);
                q.x[1] = *reinterpret_cast<const v4u *>(p + 32);
            } else {
                const v2u lo = *reinterpret_cast<const v2u *>(p);
                const v2u hi = *reinterpret_cast<const v2u *>(p + 16);
                q.x[0] = v4u{lo[0], lo[1], hi[0], hi[1]};
            }
        } else {
            // The row's end: values past K read as 0.
#pragma unroll
            for (int i = 0; i < (SRC == W2A8_F32 ? 2 : 1); ++i) q.x[i] = v4u{0u, 0u, 0u, 0u};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int at = k + (i & 3) + 8 * (i >> 2);
                if (at < a.K) {
                    if constexpr (SRC == W2A8_F32)
                        q.x[i >> 2][i & 3] = static_cast<const uint32_t *>(a.x)[at];
                    else
                        q.x[0][i >> 1] |=
                            uint32_t(static_cast<const uint16_t *>(a.x)[at]) << (16 * (i & 1));
                }
            }
        }
    }
}

// Rounds the wave's 512 float values and leaves their codes (256 bytes, block
// by block) and scale bytes (4g + tile) in `sh`.
template <int KIND, int MB, int SRC>
__device__ __forceinline__ void round_quad(const Quad<KIND, MB, SRC> &q, int lane, uint8_t *sh) {
    float lo[4], hi[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (SRC == W2A8_F32) {
            lo[i] = __uint_as_float(q.x[0][i]);
            hi[i] = __uint_as_float(q.x[1][i]);
        } else {
            const uint32_t l = q.x[0][i >> 1], h = q.x[0][2 + (i >> 1)];
            const uint32_t lb = (i & 1) ? l >> 16 : l & 0xFFFFu, hb = (i & 1) ? h >> 16 : h & 0xFFFFu;
            if constexpr (SRC == W2A8_BF16) {
                lo[i] = __uint_as_float(lb << 16);
                hi[i] = __uint_as_float(hb << 16);
            } else {
                lo[i] = float(__builtin_bit_cast(_Float16, uint16_t(lb)));
                hi[i] = float(__builtin_bit_cast(_Float16, uint16_t(hb)));
            }
        }
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        m = max(m, max(__float_as_uint(lo[i]) & 0x7FFFFFFFu, __float_as_uint(hi[i]) & 0x7FFFFFFFu));
    m = max(m, uint32_t(__builtin_amdgcn_update_dpp(0, int(m), 0xB1, 0xF, 0xF, false)));
    m = max(m, uint32_t(__builtin_amdgcn_update_dpp(0, int(m), 0x4E, 0xF, 0xF, false)));
    const uint32_t byte = mx4_scale_byte(m);
    const uint32_t w = mx4_codes4(lo, hi, mx4_scale_value(byte));
    // Ordered after the reads of the group before (LDS keeps a wave's order).
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    reinterpret_cast<uint32_t *>(sh)[lane] = w;
    const int blk = lane >> 2;
    if ((lane & 3) == 0) sh[256 + 4 * (blk & 3) + (blk >> 2)] = uint8_t(byte);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

template <int KIND, int MB, int SRC, int T>
__device__ __forceinline__ void mma_tile(const Quad<KIND, MB, SRC> &q, const v4u *x,
                                         const uint32_t *xs,
                                         v4f (&acc)[Quad<KIND, MB, SRC>::RB][MB]) {
    constexpr int RB = Quad<KIND, MB, SRC>::RB;
#pragma unroll
    for (int j = 0; j < RB; ++j) {
        v4u w;
        uint32_t ws;
        if constexpr (KIND == kTernary) {
            w = ternary_fp4(q.t[4 * T + 2 * j], q.t[4 * T + 2 * j + 1]);
            ws = kTernaryScale;
        } else {
            w = q.w[T];
            ws = q.ws;
        }
#pragma unroll
        for (int b = 0; b < MB; ++b)
            acc[j][b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                fp4_operand(w), fp4_operand(x[4 * b + T]), acc[j][b], 4, 4, T, int(ws), T,
                int(xs[b]));
    }
}

template <int KIND, int MB, int SRC>
__device__ __forceinline__ void use_quad(const Mx4Launch &a, int u, int lane,
                                         const Quad<KIND, MB, SRC> &q, uint8_t *sh,
                                         v4f (&acc)[Quad<KIND, MB, SRC>::RB][MB]) {
    v4u x[MB * 4];
    uint32_t xs[MB];
    if constexpr (SRC == kMx4Rows) {
#pragma unroll
        for (int i = 0; i < MB * 4; ++i) x[i] = q.x[i];
#pragma unroll
        for (int b = 0; b < MB; ++b) xs[b] = q.xs[b];
    } else {
        round_quad(q, lane, sh);
        const int g = lane >> 4;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = reinterpret_cast<const v4u *>(sh)[4 * i + g];
        xs[0] = reinterpret_cast<const uint32_t *>(sh + 256)[g];
    }
    // The last group may have fewer tiles (their loads repeated the last one).
    const int n = a.KT - 4 * u;
    mma_tile<KIND, MB, SRC, 0>(q, x, xs, acc);
    if (n > 1) mma_tile<KIND, MB, SRC, 1>(q, x, xs, acc);
    if (n > 2) mma_tile<KIND, MB, SRC, 2>(q, x, xs, acc);
    if (n > 3) mma_tile<KIND, MB, SRC, 3>(q, x, xs, acc);
}

constexpr int kMaxWaves = 8;
constexpr int kRoundBytes = 288;   // LDS per wave of the fused form: 256 + 16, padded

template <int KIND, int MB, int SRC>
__global__ __launch_bounds__(64 * kMaxWaves) void mx4_stream_kernel(Mx4Launch a) {
    using Q = Quad<KIND, MB, SRC>;
    constexpr int RB = Q::RB;
    __shared__ v4f red[kMaxWaves * RB * MB * 64];
    __shared__ __attribute__((aligned(16))) uint8_t rnd[SRC == kMx4Rows ? 16
                                                                        : kMaxWaves * kRoundBytes];
    const int lane = int(threadIdx.x) & 63;
    const int wv = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const int nw = int(blockDim.x) >> 6;
    const int64_t s = blockIdx.x + int64_t(blockIdx.y) * gridDim.x;
    if (s >= a.strips) return;
    const int m0 = int(blockIdx.z) * (16 * MB);
    uint8_t *sh = SRC == kMx4Rows ? rnd : rnd + wv * kRoundBytes;

    v4f acc[RB][MB];
#pragma unroll
    for (int j = 0; j < RB; ++j)
#pragma unroll
        for (int b = 0; b < MB; ++b) acc[j][b] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

    // Two groups in flight: the next is loaded before this one is used.
    Q q0, q1;
    int u = wv;
    if (u < a.KU) load_quad(a, s, m0, u, lane, q0);
    while (u < a.KU) {
        int v = u + nw;
        if (v < a.KU) load_quad(a, s, m0, v, lane, q1);
        use_quad(a, u, lane, q0, sh, acc);
        if (v >= a.KU) break;
        u = v + nw;
        if (u < a.KU) load_quad(a, s, m0, u, lane, q0);
        use_quad(a, v, lane, q1, sh, acc);
    }

    if (nw > 1) {
#pragma unroll
        for (int j = 0; j < RB; ++j)
#pragma unroll
            for (int b = 0; b < MB; ++b) red[((wv * RB + j) * MB + b) * 64 + lane] = acc[j][b];
        __syncthreads();
    }
    // Lane l of block (j, b): rows 16j + 4(l/16) .. + 3 of the strip, activation
    // row m0 + 16b + l%16.  Wave w adds up blocks w, w + nw, ...
#pragma unroll
    for (int i = 0; i < RB * MB; ++i) {
        if (i % nw != wv) continue;
        v4f v = acc[i / MB][i % MB];
        if (nw > 1) {
            v = red[i * 64 + lane];
            for (int w = 1; w < nw; ++w) {
                const v4f p = red[(w * RB * MB + i) * 64 + lane];
                v = v4f{v[0] + p[0], v[1] + p[1], v[2] + p[2], v[3] + p[3]};
            }
        }
        mx4_store4(a, m0 + 16 * (i % MB) + (lane & 15),
                   int(s) * (16 * RB) + 16 * (i / MB) + 4 * (lane >> 4), v);
    }
}

// Waves per workgroup: one per group of four tiles, at most 8.
int stream_waves(const Mx4Launch &a) { return std::min(kMaxWaves, a.KU); }

template <int KIND, int MB, int SRC>
hipError_t stream_launch(Mx4Launch a, hipStream_t stream) {
    constexpr int RB = Quad<KIND, MB, SRC>::RB;
    a.strips = int(ceil_div(a.N, 16 * RB));
    const int64_t gx = std::min<int64_t>(a.strips, int64_t(1) << 20);
    const dim3 grid(unsigned(gx), unsigned(ceil_div(a.strips, gx)),
                    unsigned(ceil_div(a.M, 16 * MB)));
    void *args[] = {&a};
    return hipLaunchKernel(reinterpret_cast<const void *>(&mx4_stream_kernel<KIND, MB, SRC>), grid,
                           dim3(unsigned(64 * stream_waves(a))), args, 0, stream);
}

template <int KIND>
hipError_t stream_rows(const Mx4Launch &a, hipStream_t stream) {
    if (a.M <= 16) return stream_launch<KIND, 1, kMx4Rows>(a, stream);
    if (a.M <= 32) return stream_launch<KIND, 2, kMx4Rows>(a, stream);
    return stream_launch<KIND, 4, kMx4Rows>(a, stream);
}

template <int KIND>
hipError_t stream_fused(const Mx4Launch &a, int type, hipStream_t stream) {
    return type == W2A8_F32    ? stream_launch<KIND, 1, W2A8_F32>(a, stream)
           : type == W2A8_BF16 ? stream_launch<KIND, 1, W2A8_BF16>(a, stream)
                               : stream_launch<KIND, 1, W2A8_F16>(a, stream);
}

}  // namespace

hipError_t launch_mx4_stream(const Mx4Launch &a, int cus, hipStream_t stream) {
    (void)cus;
    return a.ws ? stream_rows<kMx4Weights>(a, stream) : stream_rows<kTernary>(a, stream);
}

hipError_t launch_mx4_fused(const Mx4Launch &a, int x_type, int cus, hipStream_t stream) {
    (void)cus;
    return a.ws ? stream_fused<kMx4Weights>(a, x_type, stream)
                : stream_fused<kTernary>(a, x_type, stream);
}

}  // namespace w2a8
