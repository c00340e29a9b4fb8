// Products of MX4 rows for few rows (decode and short batches, M <= 32) on
// gfx950: a stream of weights through LDS into
// v_mfma_scale_f32_16x16x128_f8f6f4.
//
//   y[m][n] = s_w * sum_b 2^(ex + ew) * sum_{k in b} qx * qw
//
// The instruction takes 16 weight rows x 128 k as its first operand and 16
// activation rows x 128 k as its second, multiplies each block of 32 by both
// scales and adds in fp32: one or two instructions per KiB of weights, so the
// matrix pipe is nearly idle and the kernel is bound by the weight stream.
//
//  * A workgroup takes one strip (16 rows of MX4, 32 of ternary weights); its
//    waves interleave over the strip's quads (four tiles, 4 KiB of weights).
//    Their sums meet in LDS and are added in wave order: no workspace, no
//    atomics, and a result that does not depend on timing.
//  * Every wave has a ring of LDS stages of its own, one quad each, filled by
//    direct global->LDS loads two quads ahead; nothing is shared before
//    the sums, so the loop has no barrier, and the bytes in flight (what
//    bounds a stream) need no registers.
//  * MX4 weights: a tile is 1 KiB in operand order.  Ternary weights
//    (T32x128): a slot holds four rows of 16 k, so lane r stands for rows
//    4 (r / 2) + 2 (r % 2) + j of the strip, j = 0, 1 for the two
//    instructions, and two 8-byte reads give it both; slot kg of row group rg
//    sits at 8 rg + (kg ^ rg), which spreads the reads over the banks.
//  * Rows: M = 1 loads the quad's 256 code bytes, 4 bytes a lane, and every
//    column of the instruction repeats the row.  Otherwise 64-byte row pieces
//    land in operand order but for a swizzle; rows past M repeat row M - 1
//    and are not stored.
//  * Fused form (one float row): the quad's 512 values arrive as they are,
//    and every wave rounds them itself, 8 per lane, and passes the codes
//    round by 272 bytes of LDS of its own.  The rounding is repeated by every
//    strip (some 40 instructions per 4 KiB of weights) and never leaves the
//    compute unit.
#include "mx4.h"
#include "mx4_device.h"

namespace w2a8 {
namespace {

// Where the activations come from: one float row of that w2a8_mx4_type, one
// MX4R row, up to 16 and up to 32 MX4R rows.
enum { kOneRow = 3, kRows16 = 4, kRows32 = 5 };
constexpr int kMaxWaves = 8;
constexpr int kDepth = 2;     // stages of a wave: quads loaded ahead

template <int KIND, int SRC>
struct Stream {
    static constexpr bool kFloat = SRC < kOneRow;
    static constexpr int RB = KIND == kTernary ? 2 : 1;   // blocks of 16 weight rows
    static constexpr int MB = SRC == kRows32 ? 2 : 1;     // blocks of 16 activation rows
    // A stage: weights, their scales, activations, their scales.
    static constexpr int W = 0, WS = 4096, X = WS + (KIND == kTernary ? 0 : 256);
    static constexpr int XBYTES = SRC == W2A8_F32 ? 2048 : kFloat ? 1024 : SRC == kOneRow ? 256 : MB * 4096;
    static constexpr int XS = X + XBYTES;
    static constexpr int XSBYTES = kFloat ? 0 : SRC == kOneRow ? 256 : MB * 1024;
    static constexpr int STAGE = XS + XSBYTES;
    // Its loads.
    static constexpr int LOADS = 4 + (KIND == kTernary ? 0 : 1) +
                                 (SRC == W2A8_F32 ? 2 : kFloat ? 1 : SRC == kOneRow ? 2 : 5 * MB);
    static constexpr int ROUND = kFloat ? 288 : 0;        // rounding exchange: 256 + 16, padded
    static constexpr int SUM = RB * MB * 1024;            // a wave's sums
};

// The last quad of a float row that ends inside it: values past K are 0.
template <int TYPE>
__device__ __forceinline__ void load_tail(const void *x, int k0, int K, int lane, uint8_t *dst) {
    constexpr int kSize = TYPE == W2A8_F32 ? 4 : 2;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int k = k0 + 64 * i + lane;
        if constexpr (kSize == 4)
            reinterpret_cast<uint32_t *>(dst)[64 * i + lane] =
                k < K ? static_cast<const uint32_t *>(x)[k] : 0u;
        else
            reinterpret_cast<uint16_t *>(dst)[64 * i + lane] =
                k < K ? static_cast<const uint16_t *>(x)[k] : uint16_t(0);
    }
}

// Rounds the 512 values of a float stage, 8 per lane, and leaves the codes
// (256 bytes, block by block) and scale bytes (4g + tile) in `sh`.
template <int TYPE>
__device__ __forceinline__ void round_quad(const uint8_t *x, int lane, uint8_t *sh) {
    // Block lane / 4 of the quad, values 16c + 4h + {0..3} and 8 more of it
    // (c = bit 1, h = bit 0 of the lane): one code word.
    const int k = 32 * (lane >> 2) + 16 * ((lane >> 1) & 1) + 4 * (lane & 1);
    float lo[4], hi[4];
    if constexpr (TYPE == W2A8_F32) {
        const v4f a = *reinterpret_cast<const v4f *>(x + 4 * k);
        const v4f b = *reinterpret_cast<const v4f *>(x + 4 * k + 32);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = a[i];
            hi[i] = b[i];
        }
    } else {
        const v2u a = *reinterpret_cast<const v2u *>(x + 2 * k);
        const v2u b = *reinterpret_cast<const v2u *>(x + 2 * k + 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t l = (i & 1) ? a[i >> 1] >> 16 : a[i >> 1] & 0xFFFFu;
            const uint32_t h = (i & 1) ? b[i >> 1] >> 16 : b[i >> 1] & 0xFFFFu;
            if constexpr (TYPE == W2A8_BF16) {
                lo[i] = __uint_as_float(l << 16);
                hi[i] = __uint_as_float(h << 16);
            } else {
                lo[i] = float(__builtin_bit_cast(_Float16, uint16_t(l)));
                hi[i] = float(__builtin_bit_cast(_Float16, uint16_t(h)));
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
    reinterpret_cast<uint32_t *>(sh)[lane] = w;
    const int blk = lane >> 2;
    if ((lane & 3) == 0) sh[256 + 4 * (blk & 3) + (blk >> 2)] = uint8_t(byte);
}

template <int KIND, int SRC>
__global__ __launch_bounds__(64 * kMaxWaves) void mx4_stream_kernel(Mx4Launch a) {
    using S = Stream<KIND, SRC>;
    constexpr int RB = S::RB, MB = S::MB;
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const int lane = int(threadIdx.x) & 63;
    const int wv = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const int nw = int(blockDim.x) >> 6;
    const int64_t s = blockIdx.x + int64_t(blockIdx.y) * gridDim.x;
    if (s >= a.strips) return;
    const int r = lane & 15, g = lane >> 4;
    uint8_t *ring = lds + wv * (a.stages * S::STAGE + S::ROUND);
    uint8_t *rnd = ring + a.stages * S::STAGE;

    const int last = a.KT - 1;
    const int64_t wstrip = int64_t(a.KT) * 1024;      // a tile of either kind is 1 KiB
    const auto wbuf = mx4_buffer(a.w + s * wstrip, wstrip);
    const int woff = 16 * (KIND == kTernary ? (lane & 56) + ((lane & 7) ^ (lane >> 3)) : lane);
    const auto wsbuf = mx4_buffer(KIND == kTernary ? a.w : a.ws + s * a.KU * 256, int64_t(a.KU) * 256);
    const int xrow = a.KT * kMxRowTile, srow = a.KU * 16;
    const auto xbuf = S::kFloat ? mx4_buffer(static_cast<const uint8_t *>(a.x),
                                             int64_t(a.K) * (SRC == W2A8_F32 ? 4 : 2))
                                : mx4_buffer(a.xq, int64_t(a.M) * xrow);
    const auto xsbuf = mx4_buffer(S::kFloat ? a.w : a.xs, int64_t(a.M) * srow);
    int xoff[MB], xsoff[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) {
        // Lane l brings row 16b + l/4, block (l%4) ^ (l/8%4); its scales' 16
        // bytes of row 16b + l%16.
        xoff[b] = min(16 * b + (lane >> 2), a.M - 1) * xrow + 16 * ((lane & 3) ^ ((lane >> 3) & 3));
        xsoff[b] = min(16 * b + r, a.M - 1) * srow;
    }

    // Loads of quad u into a stage (tiles past the last: of the last).
    auto issue = [&](int u, uint8_t *st) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
            mx4_load_lds16(wbuf, st + S::W + 1024 * t, woff, min(4 * u + t, last) * 1024);
        if constexpr (KIND != kTernary) mx4_load_lds4(wsbuf, st + S::WS, 4 * lane, u * 256);
        if constexpr (S::kFloat) {
            if (512 * u + 512 <= a.K) {
#pragma unroll
                for (int i = 0; i < S::XBYTES / 1024; ++i)
                    mx4_load_lds16(xbuf, st + S::X + 1024 * i, 16 * lane, u * S::XBYTES + 1024 * i);
            } else {
                load_tail<SRC>(a.x, 512 * u, a.K, lane, st + S::X);
            }
        } else if constexpr (SRC == kOneRow) {
            // (The last quad may end before 256 bytes.)
            mx4_load_lds4(xbuf, st + S::X, min(u * 256 + 4 * lane, xrow - 4), 0);
            mx4_load_lds4(xsbuf, st + S::XS, 4 * (lane & 3), u * 16);
        } else {
#pragma unroll
            for (int b = 0; b < MB; ++b) {
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    mx4_load_lds16(xbuf, st + S::X + 4096 * b + 1024 * t, xoff[b],
                                   min(4 * u + t, last) * kMxRowTile);
                mx4_load_lds16(xsbuf, st + S::XS + 1024 * b, xsoff[b], u * 16);
            }
        }
    };

    v4f acc[RB][MB];
#pragma unroll
    for (int j = 0; j < RB; ++j)
#pragma unroll
        for (int b = 0; b < MB; ++b) acc[j][b] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

    const int wswz = 128 * (r >> 1) + 8 * (r & 1);
    const int xfrag = 16 * (4 * r + (g ^ ((r >> 1) & 3)));
    auto use = [&](int u, const uint8_t *st) __attribute__((always_inline)) {
        uint32_t ws = kTernaryScale, xs[MB];
        if constexpr (KIND != kTernary) ws = *reinterpret_cast<const uint32_t *>(st + S::WS + 4 * lane);
        if constexpr (S::kFloat) {
            round_quad<SRC>(st + S::X, lane, rnd);
            mx4_wave_sync();
            xs[0] = *reinterpret_cast<const uint32_t *>(rnd + 256 + 4 * g);
        } else if constexpr (SRC == kOneRow) {
            xs[0] = *reinterpret_cast<const uint32_t *>(st + S::XS + 4 * g);
        } else {
#pragma unroll
            for (int b = 0; b < MB; ++b)
                xs[b] = *reinterpret_cast<const uint32_t *>(st + S::XS + 1024 * b + 16 * r + 4 * g);
        }
        auto tile = [&](auto tt) __attribute__((always_inline)) {
            constexpr int T = decltype(tt)::value;
            v4u w[RB], x[MB];
            const uint8_t *wt = st + S::W + 1024 * T;
            if constexpr (KIND == kTernary) {
                const v2u h0 = *reinterpret_cast<const v2u *>(wt + wswz + 16 * ((2 * g) ^ (r >> 1)));
                const v2u h1 = *reinterpret_cast<const v2u *>(wt + wswz + 16 * ((2 * g + 1) ^ (r >> 1)));
#pragma unroll
                for (int j = 0; j < RB; ++j) w[j] = ternary_fp4(h0[j], h1[j]);
            } else {
                w[0] = *reinterpret_cast<const v4u *>(wt + 16 * lane);
            }
#pragma unroll
            for (int b = 0; b < MB; ++b)
                x[b] = *reinterpret_cast<const v4u *>(
                    S::kFloat          ? rnd + 64 * T + 16 * g
                    : SRC == kOneRow   ? st + S::X + 64 * T + 16 * g
                                       : st + S::X + 4096 * b + 1024 * T + xfrag);
#pragma unroll
            for (int j = 0; j < RB; ++j)
#pragma unroll
                for (int b = 0; b < MB; ++b)
                    acc[j][b] = mx4_mfma<T>(w[j], x[b], acc[j][b], ws, xs[b]);
        };
        const int n = a.KT - 4 * u;      // the last quad may have fewer tiles
        tile(std::integral_constant<int, 0>{});
        if (n > 1) tile(std::integral_constant<int, 1>{});
        if (n > 2) tile(std::integral_constant<int, 2>{});
        if (n > 3) tile(std::integral_constant<int, 3>{});
    };

    // This wave's quads: wv, wv + nw, ...
    const int count = wv < a.KU ? (a.KU - wv + nw - 1) / nw : 0;
#pragma unroll
    for (int i = 0; i < kDepth; ++i)
        if (i < count) issue(wv + i * nw, ring + i * S::STAGE);
    int slot = 0;
#pragma unroll 1
    for (int i = 0; i < count; ++i) {
        // The quad's loads have landed: at most those of the kDepth - 1 quads
        // after it are on their way.  (The tail of a float row is waited for
        // where it is loaded, and with it all loads before it.)
        const int ahead = count - 1 - i;
        if (ahead >= kDepth - 1)
            mx4_wait_loads<(kDepth - 1) * S::LOADS>();
        else
            mx4_wait_loads<0>();
        uint8_t *st = ring + slot * S::STAGE;
        const int u = wv + i * nw;
        use(u, st);
        if (ahead >= kDepth) {
            // The stage's reads are done before it is filled again.
            mx4_wait_lds();
            issue(u + kDepth * nw, st);
        }
        slot = slot + 1 == kDepth ? 0 : slot + 1;
    }

    // Lane (r, g) of block (j, b): activation row 16b + r, and weight rows
    // 4g + e (MX4) or 8g + 2e + j (ternary), e = 0..3.
    if (nw > 1) {
        v4f *red = reinterpret_cast<v4f *>(lds);
        __syncthreads();                  // every stage has been read
#pragma unroll
        for (int j = 0; j < RB; ++j)
#pragma unroll
            for (int b = 0; b < MB; ++b) red[((wv * MB + b) * RB + j) * 64 + lane] = acc[j][b];
        __syncthreads();
#pragma unroll
        for (int b = 0; b < MB; ++b) {
            if (b % nw != wv) continue;
#pragma unroll
            for (int j = 0; j < RB; ++j) {
                v4f v = red[(b * RB + j) * 64 + lane];
                for (int w = 1; w < nw; ++w) {
                    const v4f p = red[((w * MB + b) * RB + j) * 64 + lane];
                    v = v4f{v[0] + p[0], v[1] + p[1], v[2] + p[2], v[3] + p[3]};
                }
                acc[j][b] = v;
            }
        }
    }
#pragma unroll
    for (int b = 0; b < MB; ++b) {
        if (b % nw != wv) continue;
        const int m = 16 * b + r, n = int(s) * (16 * RB) + 4 * RB * g;
        if constexpr (KIND == kTernary) {
            const v4f p = acc[0][b], q = acc[1][b];
            mx4_store4(a, m, n, v4f{p[0], q[0], p[1], q[1]});
            mx4_store4(a, m, n + 4, v4f{p[2], q[2], p[3], q[3]});
        } else {
            mx4_store4(a, m, n, acc[0][b]);
        }
    }
}

template <int KIND, int SRC>
hipError_t stream_launch(Mx4Launch a, int cus, hipStream_t stream) {
    using S = Stream<KIND, SRC>;
    a.strips = int(ceil_div(a.N, 16 * S::RB));
    const int nw = mx4_stream_waves(a.M, a.strips, a.KU, cus);
    a.stages = int(std::min<int64_t>(kDepth, ceil_div(a.KU, nw)));
    const int64_t gx = std::min<int64_t>(a.strips, int64_t(1) << 20);
    const dim3 grid(unsigned(gx), unsigned(ceil_div(a.strips, gx)));
    const size_t bytes = size_t(nw) * std::max(a.stages * S::STAGE + S::ROUND, S::SUM);
    void *args[] = {&a};
    return hipLaunchKernel(reinterpret_cast<const void *>(&mx4_stream_kernel<KIND, SRC>), grid,
                           dim3(unsigned(64 * nw)), args, bytes, stream);
}

template <int KIND>
hipError_t stream_rows(const Mx4Launch &a, int cus, hipStream_t stream) {
    if (a.M == 1) return stream_launch<KIND, kOneRow>(a, cus, stream);
    if (a.M <= 16) return stream_launch<KIND, kRows16>(a, cus, stream);
    return stream_launch<KIND, kRows32>(a, cus, stream);
}

template <int KIND>
hipError_t stream_fused(const Mx4Launch &a, int type, int cus, hipStream_t stream) {
    return type == W2A8_F32    ? stream_launch<KIND, W2A8_F32>(a, cus, stream)
           : type == W2A8_BF16 ? stream_launch<KIND, W2A8_BF16>(a, cus, stream)
                               : stream_launch<KIND, W2A8_F16>(a, cus, stream);
}

}  // namespace

// Waves of a workgroup.  A CU holds as many waves as its LDS holds pairs of
// stages (16, 8 or 5 by M).  With a strip or less for every CU the waves of a
// strip are all there is to keep loads on their way; beyond, few waves to a
// strip (shorter sums, and a wave that streams on).  For short batches that
// lets all strips of most matrices start at once; at M = 1 the strips of the
// largest start in turns (55296 rows: 3456 strips of three waves, 2.5 turns).
// Measured (MI355X, us, cold weights): M = 1, 5120 x
// 27648 MX4, 320 strips: 3 waves 16.7, 8 waves 17.9; 55296 x 5120 28.4 against
// 30.9; ternary, 160 strips: 8 waves 10.2, 4 waves 11.7.  M = 16, 55296 x 5120
// ternary: 1 wave 16.7, 2 waves 19.6, 5 waves 27 or more; 13824 x 2560 MX4: 2
// waves 6.6, 5 waves 7.8; 8192 x 27648 ternary, 256 strips: 5 waves 15.8, 2
// waves 18.5.  M = 17, 256 strips: 8192 x 13824 ternary: 3 waves 9.8, 2 waves
// 11.7, 1 wave 17.4; 290 strips, 9280 x 5120: 2 waves 7.4, 1 wave 8.6, 3 waves
// 9.4; 563 strips, 9000 x 2560 MX4: 1 wave 6.2, 2 waves 7.6.
int mx4_stream_waves(int M, int strips, int KU, int cus) {
    const bool many = strips > cus;
    const int nw = M == 1    ? (many ? 3 : kMaxWaves)
                   : M <= 16 ? (strips >= 4 * cus ? 1 : many ? 2 : 5)
                             : (strips > 2 * cus ? 1 : many ? 2 : 3);
    return std::min(nw, KU);
}

hipError_t launch_mx4_stream(const Mx4Launch &a, int cus, hipStream_t stream) {
    return a.ws ? stream_rows<kMx4Weights>(a, cus, stream) : stream_rows<kTernary>(a, cus, stream);
}

hipError_t launch_mx4_fused(const Mx4Launch &a, int x_type, int cus, hipStream_t stream) {
    return a.ws ? stream_fused<kMx4Weights>(a, x_type, cus, stream)
                : stream_fused<kTernary>(a, x_type, cus, stream);
}

}  // namespace w2a8
