// Products of int8 rows with 4-bit weights and group scales (decode and short
// batches, M <= 64) on gfx950.
//
//   y[m][n] = s_a[m] * sum_g s[n][g] * sum_{k in g} (q[n][k] - z[n][g]) * x[m][k]
//
// int8 matrix instructions take the activations as their first operand (16
// rows) and the weights as their second (16 rows of W): lane l brings row
// l % 16 and the bytes of k-part l / 16, and holds results of weight row
// l % 16, so one scale a lane and group serves all its sums.  A group of 128
// is two instructions of 64 k, one of 64 one, one of 32 one of 32 k.
//
// Two values share a byte.  In the high half, as two's complement of q - 8, a
// value is a signed byte of 16 times itself: the high values are one AND, the
// low ones a shift and an AND, and the 16 goes out with the scale (a power of
// two, so exactly).  A group's sum is at most 16 * 15 * 127 * 128 < 2^22, exact
// as int32 and as fp32.  With zero points, one more instruction with a
// constant operand of ones gives sum x of the group for every lane.
//
// A workgroup takes one strip of 16 weight rows; its waves take the strip's
// tiles (16 x 128, 1 KiB) in turn and add their sums in LDS in wave order.
#include "block.h"
#include "mx4_device.h"

namespace w2a8 {
namespace {

constexpr int kMaxWaves = 8;

// The 8 values of a word as signed bytes of 16 times themselves.
__device__ __forceinline__ uint32_t low_values(uint32_t w) { return (w << 4) & 0xF0F0F0F0u; }
__device__ __forceinline__ uint32_t high_values(uint32_t w) { return w & 0xF0F0F0F0u; }

__device__ __forceinline__ v4i mfma64(v4u x, v4u w, v4i acc) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(v4i, x), __builtin_bit_cast(v4i, w),
                                                 acc, 0, 0, 0);
}
__device__ __forceinline__ v4i mfma32(v2u x, v2u w, v4i acc) {
    return __builtin_amdgcn_mfma_i32_16x16x32_i8(__builtin_bit_cast(long, x), __builtin_bit_cast(long, w),
                                                 acc, 0, 0, 0);
}

// What a tile needs: codes, activations of MB blocks of 16 rows, scales and
// zero points of its P groups.
template <int P, int MB, bool ZEROS>
struct Tile {
    v4u w;
    uint32_t x[MB][8];
    uint32_t s[(P + 1) / 2];
    uint32_t z;
};

template <int P, int MB, bool ZEROS, bool ONE>
__global__ __launch_bounds__(64 * kMaxWaves) void w4a8_kernel(W4Launch a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    using T = Tile<P, MB, ZEROS>;
    constexpr int D = MB == 4 ? 2 : 4;       // tiles of a wave on their way
    constexpr int RES = ONE ? 1 : 4;         // results of a lane and block (ONE: all rows are the same)
    const int lane = int(threadIdx.x) & 63;
    const int wv = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const int nw = int(blockDim.x) >> 6;
    const int s = int(blockIdx.x + blockIdx.y * gridDim.x);
    if (s >= a.strips) return;
    const int r = lane & 15, c = lane >> 4;

    const uint8_t *wp = a.w + int64_t(s) * a.KT * kW4TileBytes + 16 * lane;
    const uint16_t *sp = a.scales + (int64_t(s) * a.GQ * 16 + r) * 4;
    const uint8_t *zp = ZEROS ? a.zeros + (int64_t(s) * a.GQ * 16 + r) * 4 : nullptr;
    const int8_t *xp[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) xp[b] = a.x + int64_t(min(16 * b + r, a.M - 1)) * a.K;

    // Tile t: groups P t .. P t + P - 1, which share a quad of groups.
    auto load_w = [&](int t, T &d) __attribute__((always_inline)) {
        d.w = __builtin_nontemporal_load(reinterpret_cast<const v4u *>(wp + int64_t(t) * kW4TileBytes));
        const int g = P * t, at = (g >> 2) * 64 + (g & 3);
        if constexpr (P == 1)
            d.s[0] = sp[at];
        else
#pragma unroll
            for (int i = 0; i < P / 2; ++i) d.s[i] = reinterpret_cast<const uint32_t *>(sp + at)[i];
        if constexpr (ZEROS)
            d.z = P == 1   ? zp[at]
                  : P == 2 ? *reinterpret_cast<const uint16_t *>(zp + at)
                           : *reinterpret_cast<const uint32_t *>(zp + at);
    };
    auto load_x = [&](int t, T &d) __attribute__((always_inline)) {
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
            for (int i = 0; i < (P == 4 ? 4 : 2); ++i) {
                const int8_t *p = xp[b] + t * kTileK + (P == 1 ? 32 * c + 16 * i : P == 2 ? 64 * i + 16 * c : 32 * i + 8 * c);
                if constexpr (P == 4) {
                    const v2u v = *reinterpret_cast<const v2u_b *>(p);
                    d.x[b][2 * i] = v[0];
                    d.x[b][2 * i + 1] = v[1];
                } else {
                    const v4u v = *reinterpret_cast<const v4u_b *>(p);
#pragma unroll
                    for (int j = 0; j < 4; ++j) d.x[b][4 * i + j] = v[j];
                }
            }
    };
    auto load_x_tail = [&](int t, T &d) __attribute__((always_inline)) {
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
            for (int i = 0; i < (P == 4 ? 4 : 2); ++i) {
                const int k = t * kTileK + (P == 1 ? 32 * c + 16 * i : P == 2 ? 64 * i + 16 * c : 32 * i + 8 * c);
                if constexpr (P == 4)
                    load_int8_tail<8>(xp[b], k, a.K, d.x[b] + 2 * i);
                else
                    load_int8_tail<16>(xp[b], k, a.K, d.x[b] + 4 * i);
            }
    };

    float y[MB][RES];
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
        for (int e = 0; e < RES; ++e) y[b][e] = 0.0f;

    auto use = [&](const T &d) __attribute__((always_inline)) {
        const v4i none = {0, 0, 0, 0};
        const v4u ones = {0x01010101u, 0x01010101u, 0x01010101u, 0x01010101u};
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const uint32_t sb = (d.s[i >> 1] >> (16 * (i & 1))) & 0xFFFFu;
            const float sc = (a.bf16_scales ? __uint_as_float(sb << 16)
                                            : float(__builtin_bit_cast(_Float16, uint16_t(sb)))) * 0.0625f;
            const int z16 = ZEROS ? int(d.z << (24 - 8 * i)) >> 24 << 4 : 0;
#pragma unroll
            for (int b = 0; b < MB; ++b) {
                v4i acc = none, sum = none;
                const uint32_t *x = d.x[b];
                if constexpr (P == 4) {
                    const v2u xo = {x[2 * i], x[2 * i + 1]};
                    acc = mfma32(xo, v2u{low_values(d.w[i]), high_values(d.w[i])}, acc);
                    if constexpr (ZEROS) sum = mfma32(xo, v2u{ones[0], ones[1]}, sum);
                } else {
#pragma unroll
                    for (int j = (P == 1 ? 0 : i); j < (P == 1 ? 2 : i + 1); ++j) {
                        const v4u xo = {x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]};
                        const uint32_t w0 = d.w[2 * j], w1 = d.w[2 * j + 1];
                        acc = mfma64(xo, v4u{low_values(w0), high_values(w0), low_values(w1), high_values(w1)}, acc);
                        if constexpr (ZEROS) sum = mfma64(xo, ones, sum);
                    }
                }
#pragma unroll
                for (int e = 0; e < RES; ++e)
                    y[b][e] = __builtin_fmaf(float(ZEROS ? acc[e] - z16 * sum[e] : acc[e]), sc, y[b][e]);
            }
        }
    };

    // This wave's whole tiles: wv, wv + nw, ...; the ragged one behind them.
    const int whole = a.K / kTileK;
    const int n = wv < whole ? (whole - wv + nw - 1) / nw : 0;
    T d[D];
#pragma unroll
    for (int j = 0; j < D; ++j)
        if (j < n) {
            load_w(wv + j * nw, d[j]);
            load_x(wv + j * nw, d[j]);
        }
    for (int i = 0; i < n; i += D) {
#pragma unroll
        for (int j = 0; j < D; ++j) {
            if (i + j < n) use(d[j]);
            if (i + j + D < n) {
                load_w(wv + (i + j + D) * nw, d[j]);
                load_x(wv + (i + j + D) * nw, d[j]);
            }
        }
    }
    if (whole < a.KT && wv == whole % nw) {
        load_w(whole, d[0]);
        load_x_tail(whole, d[0]);
        use(d[0]);
    }

    // Lane (r, c) of block b: weight row r, activation rows 16b + 4c + e.
    float *red = reinterpret_cast<float *>(lds);
    constexpr int PER = MB * RES;
    if (nw > 1) {
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
            for (int e = 0; e < RES; ++e) red[(wv * PER + b * RES + e) * 64 + lane] = y[b][e];
        __syncthreads();
    }
    const int row = s * kW4Rows + r;
#pragma unroll
    for (int b = 0; b < MB; ++b) {
        if (b % nw != wv) continue;
#pragma unroll
        for (int e = 0; e < RES; ++e) {
            float v = y[b][e];
            if (nw > 1) {
                v = red[(b * RES + e) * 64 + lane];
                for (int w = 1; w < nw; ++w) v += red[(w * PER + b * RES + e) * 64 + lane];
            }
            const int m = ONE ? c : 16 * b + 4 * c + e;
            if (m >= a.M || row >= a.N) continue;
            v *= a.sa[m];
            const int64_t at = int64_t(m) * a.N + row;
            if (a.y_f32) a.y_f32[at] = v;
            if (a.y_bf16) a.y_bf16[at] = uint16_t(bf16_bits(v));
        }
    }
}

template <int P, bool ZEROS>
hipError_t w4_launch(const W4Launch &a, int cus, hipStream_t stream) {
    const void *fn = a.M == 1    ? reinterpret_cast<const void *>(&w4a8_kernel<P, 1, ZEROS, true>)
                     : a.M <= 16 ? reinterpret_cast<const void *>(&w4a8_kernel<P, 1, ZEROS, false>)
                     : a.M <= 32 ? reinterpret_cast<const void *>(&w4a8_kernel<P, 2, ZEROS, false>)
                                 : reinterpret_cast<const void *>(&w4a8_kernel<P, 4, ZEROS, false>);
    const int per = a.M == 1 ? 1 : a.M <= 16 ? 4 : a.M <= 32 ? 8 : 16;
    const int nw = std::min(kMaxWaves, a.KT);
    W4Launch l = a;
    void *args[] = {&l};
    const int gx = std::min(a.strips, 1 << 20);
    return hipLaunchKernel(fn, dim3(unsigned(gx), unsigned(ceil_div(a.strips, gx))), dim3(unsigned(64 * nw)), args,
                           size_t(nw) * per * 256, stream);
}

template <int P>
hipError_t w4_zeros(const W4Launch &a, int cus, hipStream_t stream) {
    return a.zeros ? w4_launch<P, true>(a, cus, stream) : w4_launch<P, false>(a, cus, stream);
}

}  // namespace

hipError_t launch_w4a8(const W4Launch &a, int cus, hipStream_t stream) {
    return a.group == 128 ? w4_zeros<1>(a, cus, stream)
           : a.group == 64 ? w4_zeros<2>(a, cus, stream)
                           : w4_zeros<4>(a, cus, stream);
}

}  // namespace w2a8
