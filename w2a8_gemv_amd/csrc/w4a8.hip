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
// low ones a shift and an AND, and the 16 goes out in the end (a power of two,
// so exactly).  With zero points a byte is q - z itself, three to four
// operations a word.  A group's sum is at most 16 * 8 * 127 * 128 < 2^22, exact
// as int32 and as fp32.  What is left of the work, and the most of it, is one
// conversion and one multiply-add for every result and group.
//
// A workgroup takes one strip of 16 weight rows; its waves take the strip's
// tiles (16 x 128, 1 KiB) in turn and add their sums in LDS in wave order.
#include "block.h"
#include "mx4_device.h"

namespace w2a8 {
namespace {

constexpr int kMaxWaves = 8;

// The low and high values of a word (bytes of q - 8, two each) as signed bytes:
// 16 (q - 8), or with a zero point (in every byte of z) q - z.  The latter takes
// 128 + q - z, from which no byte borrows, and the sign bit back out.
template <bool ZEROS>
__device__ __forceinline__ uint32_t low_values(uint32_t w, uint32_t z) {
    if constexpr (!ZEROS) return (w << 4) & 0xF0F0F0F0u;
    return (((w & 0x0F0F0F0Fu) ^ 0x88888888u) - z) ^ 0x80808080u;
}
template <bool ZEROS>
__device__ __forceinline__ uint32_t high_values(uint32_t w, uint32_t z) {
    if constexpr (!ZEROS) return w & 0xF0F0F0F0u;
    return low_values<true>(w >> 4, z);
}
// What the sums of such bytes are multiplied by, in the end.
template <bool ZEROS>
constexpr float kBack = ZEROS ? 1.0f : 0.0625f;
// Zero point byte i (z - 8) of a word, as z in every byte.
__device__ __forceinline__ uint32_t zero_bytes(uint32_t z, int i) {
    return __builtin_amdgcn_perm(0u, (z & 0x0F0F0F0Fu) ^ 0x08080808u, 0x01010101u * uint32_t(i));
}
__device__ __forceinline__ float scale_value(uint32_t bits, int bf16) {
    return bf16 ? __uint_as_float(bits << 16) : float(__builtin_bit_cast(_Float16, uint16_t(bits)));
}

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
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const float sc = scale_value((d.s[i >> 1] >> (16 * (i & 1))) & 0xFFFFu, a.bf16_scales);
            const uint32_t z = ZEROS ? zero_bytes(d.z, i) : 0u;
#pragma unroll
            for (int b = 0; b < MB; ++b) {
                v4i acc = {0, 0, 0, 0};
                const uint32_t *x = d.x[b];
                if constexpr (P == 4) {
                    acc = mfma32(v2u{x[2 * i], x[2 * i + 1]}, v2u{low_values<ZEROS>(d.w[i], z), high_values<ZEROS>(d.w[i], z)}, acc);
                } else {
#pragma unroll
                    for (int j = (P == 1 ? 0 : i); j < (P == 1 ? 2 : i + 1); ++j) {
                        const uint32_t w0 = d.w[2 * j], w1 = d.w[2 * j + 1];
                        acc = mfma64(v4u{x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]},
                                     v4u{low_values<ZEROS>(w0, z), high_values<ZEROS>(w0, z), low_values<ZEROS>(w1, z),
                                         high_values<ZEROS>(w1, z)}, acc);
                    }
                }
#pragma unroll
                for (int e = 0; e < RES; ++e) y[b][e] = __builtin_fmaf(float(acc[e]), sc, y[b][e]);
            }
        }
    };

    // This wave's whole tiles: wv, wv + nw, ...; the ragged one behind them.
    const int whole = a.K / kTileK;
    const int n = wv < whole ? (whole - wv + nw - 1) / nw : 0;
    T d[D];
    auto load = [&](int i, T &t) __attribute__((always_inline)) {
        load_w(wv + i * nw, t);
        load_x(wv + i * nw, t);
    };
#pragma unroll
    for (int j = 0; j < D; ++j)
        if (j < n) load(j, d[j]);
    for (int i = 0; i < n; i += D) {
#pragma unroll
        for (int j = 0; j < D; ++j) {
            if (i + j < n) use(d[j]);
            if (i + j + D < n) load(i + j + D, d[j]);
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
            v *= kBack<ZEROS> * a.sa[m];
            const int64_t at = int64_t(m) * a.N + row;
            if (a.y_f32) a.y_f32[at] = v;
            if (a.y_bf16) a.y_bf16[at] = uint16_t(bf16_bits(v));
        }
    }
}

// More rows (17 to 64): activations through LDS.  A workgroup of four waves
// takes 4 * STRIPS strips, each wave STRIPS of them, and walks a range of the
// tiles of k together; the rows' part of a tile (MB blocks of 16 rows x 128 k)
// is staged once for all of them.  LDS holds it as [block][chunk of 16 k][row],
// where every operand is 16 (or, for groups of 32, 8) bytes of a lane and a
// quarter of a wave reads 256 bytes in a row; chunks are 16 bytes apart from
// that, so that the stores of a row's chunks fall in different banks.  Rows
// start anywhere, so they are staged through registers, a tile ahead.
#ifndef TS
#define TS 1
#define WGC 2
#define TG 2
#define TD 2
#endif
constexpr int kChunkBytes = 272;

template <int P, int MB, bool ZEROS, int STRIPS, int GROUPS>
__global__ __launch_bounds__(256 * GROUPS, 2) void w4a8_tile_kernel(W4Launch a) {
    constexpr int STAGE = MB * 8 * kChunkBytes, PER = (MB * 128 + 255) / 256;
    constexpr int D = TD;                    // tiles of weights on their way
    __shared__ __attribute__((aligned(16))) uint8_t stages[GROUPS][2][STAGE];
    const int tid = int(threadIdx.x) & 255, lane = tid & 63, r = lane & 15, c = lane >> 4;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int group = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 8);
    uint8_t(&lds)[2][STAGE] = stages[group];
    const int s0 = (int(blockIdx.x) * 4 + wv) * STRIPS, part = int(blockIdx.y);
    // The part's tiles of k from t0 on; this group's are t0 + group + i * GROUPS,
    // i < n (steps: the most that a group has).
    const int t0 = int(int64_t(a.KT) * part / a.parts), t1 = int(int64_t(a.KT) * (part + 1) / a.parts);
    const int steps = (t1 - t0 + GROUPS - 1) / GROUPS, n = (t1 - t0 - group + GROUPS - 1) / GROUPS;

    const uint8_t *wp[STRIPS], *zp[STRIPS];
    const uint16_t *sp[STRIPS];
#pragma unroll
    for (int k = 0; k < STRIPS; ++k) {
        const int64_t s = min(s0 + k, a.strips - 1);       // (past the last: not stored)
        wp[k] = a.w + s * a.KT * kW4TileBytes + 16 * lane;
        sp[k] = a.scales + (s * a.GQ * 16 + r) * 4;
        zp[k] = ZEROS ? a.zeros + (s * a.GQ * 16 + r) * 4 : nullptr;
    }
    struct Weights {
        v4u w;
        uint32_t s[(P + 1) / 2], z;
    };
    auto load_w = [&](int t, Weights (&d)[STRIPS]) __attribute__((always_inline)) {
        const int g = P * t, at = (g >> 2) * 64 + (g & 3);
#pragma unroll
        for (int k = 0; k < STRIPS; ++k) {
            d[k].w = __builtin_nontemporal_load(reinterpret_cast<const v4u *>(wp[k] + int64_t(t) * kW4TileBytes));
            if constexpr (P == 1)
                d[k].s[0] = sp[k][at];
            else
#pragma unroll
                for (int i = 0; i < P / 2; ++i) d[k].s[i] = reinterpret_cast<const uint32_t *>(sp[k] + at)[i];
            if constexpr (ZEROS)
                d[k].z = P == 1   ? zp[k][at]
                         : P == 2 ? *reinterpret_cast<const uint16_t *>(zp[k] + at)
                                  : *reinterpret_cast<const uint32_t *>(zp[k] + at);
        }
    };
    // This thread's chunks of the rows: row id / 8, chunk id % 8 (rows past M
    // repeat the last one).
    const int8_t *xp[PER];
    int to[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int id = tid + 256 * j, row = min(id >> 3, 16 * MB - 1), q = id & 7;
        xp[j] = a.x + int64_t(min(row, a.M - 1)) * a.K;
        to[j] = ((row >> 4) * 8 + q) * kChunkBytes + 16 * (row & 15);
    }
    const int q16 = 16 * (tid & 7);
    auto load_x = [&](int t, v4u (&xv)[PER]) __attribute__((always_inline)) {
        const int k = t * kTileK + q16;
        if ((t + 1) * kTileK <= a.K) {
#pragma unroll
            for (int j = 0; j < PER; ++j) xv[j] = *reinterpret_cast<const v4u_b *>(xp[j] + k);
        } else {
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                uint32_t w[4];
                load_int8_tail<16>(xp[j], k, a.K, w);
                xv[j] = v4u{w[0], w[1], w[2], w[3]};
            }
        }
    };
    auto store_x = [&](uint8_t *stage, const v4u (&xv)[PER]) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (MB * 128 % 256 == 0 || tid + 256 * j < MB * 128) *reinterpret_cast<v4u *>(stage + to[j]) = xv[j];
    };

    float y[STRIPS][MB][4];
#pragma unroll
    for (int k = 0; k < STRIPS; ++k)
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) y[k][b][e] = 0.0f;

    auto use = [&](const Weights (&d)[STRIPS], const uint8_t *stage) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            float sc[STRIPS];
            uint32_t z[STRIPS];
#pragma unroll
            for (int k = 0; k < STRIPS; ++k) {
                sc[k] = scale_value((d[k].s[i >> 1] >> (16 * (i & 1))) & 0xFFFFu, a.bf16_scales);
                z[k] = ZEROS ? zero_bytes(d[k].z, i) : 0u;
            }
#pragma unroll
            for (int b = 0; b < MB; ++b) {
                v4i acc[STRIPS];
#pragma unroll
                for (int k = 0; k < STRIPS; ++k) acc[k] = v4i{0, 0, 0, 0};
                if constexpr (P == 4) {
                    const v2u x = *reinterpret_cast<const v2u *>(stage + (b * 8 + 2 * i + (c >> 1)) * kChunkBytes + 16 * r + 8 * (c & 1));
#pragma unroll
                    for (int k = 0; k < STRIPS; ++k)
                        acc[k] = mfma32(x, v2u{low_values<ZEROS>(d[k].w[i], z[k]), high_values<ZEROS>(d[k].w[i], z[k])}, acc[k]);
                } else {
#pragma unroll
                    for (int j = (P == 1 ? 0 : i); j < (P == 1 ? 2 : i + 1); ++j) {
                        const v4u x = *reinterpret_cast<const v4u *>(stage + (b * 8 + (P == 1 ? 2 * c + j : 4 * j + c)) * kChunkBytes + 16 * r);
#pragma unroll
                        for (int k = 0; k < STRIPS; ++k) {
                            const uint32_t w0 = d[k].w[2 * j], w1 = d[k].w[2 * j + 1];
                            acc[k] = mfma64(x, v4u{low_values<ZEROS>(w0, z[k]), high_values<ZEROS>(w0, z[k]),
                                                   low_values<ZEROS>(w1, z[k]), high_values<ZEROS>(w1, z[k])}, acc[k]);
                        }
                    }
                }
#pragma unroll
                for (int k = 0; k < STRIPS; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[k][b][e] = __builtin_fmaf(float(acc[k][e]), sc[k], y[k][b][e]);
            }
        }
    };

    // Weights D tiles ahead; rows D + 1, the nearest of them in the other stage.
    Weights d[D][STRIPS];
    v4u xv[D][PER];
    const auto tile = [&](int i) { return t0 + group + i * GROUPS; };
    if (n > 0) load_x(tile(0), xv[0]);
#pragma unroll
    for (int j = 0; j < D; ++j)
        if (j < n) load_w(tile(j), d[j]);
    if (n > 0) store_x(lds[0], xv[0]);
#pragma unroll
    for (int j = 1; j <= D; ++j)
        if (j < n) load_x(tile(j), xv[j % D]);
    __syncthreads();
    // While no load can be past the end none is asked for it: a load that may
    // be skipped makes the compiler wait for all before it.
    static_assert(D % 2 == 0, "stages and weight sets turn together");
    int i = 0;
    for (; i + 2 * D < (t1 - t0) / GROUPS; i += D) {
#pragma unroll
        for (int j = 0; j < D; ++j) {
            store_x(lds[(j + 1) & 1], xv[(j + 1) % D]);
            load_x(tile(i + j + 1 + D), xv[(j + 1) % D]);
            use(d[j], lds[j & 1]);
            load_w(tile(i + j + D), d[j]);
            __syncthreads();
        }
    }
    for (; i < steps; i += D) {
#pragma unroll
        for (int j = 0; j < D; ++j) {
            if (i + j < steps) {
                if (i + j + 1 < n) store_x(lds[(j + 1) & 1], xv[(j + 1) % D]);
                if (i + j + 1 + D < n) load_x(tile(i + j + 1 + D), xv[(j + 1) % D]);
                if (i + j < n) use(d[j], lds[j & 1]);
                if (i + j + D < n) load_w(tile(i + j + D), d[j]);
                __syncthreads();
            }
        }
    }

    // The groups' sums, added in their order by the first one.
    if constexpr (GROUPS > 1) {
        static_assert(STRIPS * MB * 4096 <= 2 * STAGE, "a group's sums fit its stages");
        float *mine = reinterpret_cast<float *>(&lds[0][0]);
#pragma unroll
        for (int k = 0; k < STRIPS; ++k)
#pragma unroll
            for (int b = 0; b < MB; ++b)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (group > 0) mine[((k * MB + b) * 4 + e) * 256 + tid] = y[k][b][e];
        __syncthreads();
        if (group > 0) return;
#pragma unroll
        for (int g = 1; g < GROUPS; ++g)
#pragma unroll
            for (int k = 0; k < STRIPS; ++k)
#pragma unroll
                for (int b = 0; b < MB; ++b)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        y[k][b][e] += reinterpret_cast<const float *>(&stages[g][0][0])[((k * MB + b) * 4 + e) * 256 + tid];
    }

    // Lane (r, c) of strip k and block b: weight row r, activation rows 16b + 4c + e.
#pragma unroll
    for (int k = 0; k < STRIPS; ++k) {
        const int row = (s0 + k) * kW4Rows + r;
        if (row >= a.N) continue;
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int m = 16 * b + 4 * c + e;
                if (m >= a.M) continue;
                const int64_t at = int64_t(m) * a.N + row;
                if (a.parts > 1) {
                    a.ws[part * (int64_t(a.M) * a.N) + at] = y[k][b][e];
                    continue;
                }
                const float v = y[k][b][e] * (kBack<ZEROS> * a.sa[m]);
                if (a.y_f32) a.y_f32[at] = v;
                if (a.y_bf16) a.y_bf16[at] = uint16_t(bf16_bits(v));
            }
    }
}

// The parts of k, added in order.
__global__ __launch_bounds__(256) void w4a8_join_kernel(W4Launch a) {
    const int n = int(blockIdx.x) * 256 + int(threadIdx.x), m = int(blockIdx.y);
    if (n >= a.N) return;
    const int64_t at = int64_t(m) * a.N + n, all = int64_t(a.M) * a.N;
    float v = 0.0f;
#pragma unroll 8
    for (int p = 0; p < a.parts; ++p) v += a.ws[p * all + at];
    v *= (a.zeros ? kBack<true> : kBack<false>) * a.sa[m];
    if (a.y_f32) a.y_f32[at] = v;
    if (a.y_bf16) a.y_bf16[at] = uint16_t(bf16_bits(v));
}

template <int P, bool ZEROS>
hipError_t w4_tiles_launch(const W4Launch &la, int cus, hipStream_t stream) {
    W4Launch a = la;
    const int blocks = int(ceil_div(a.strips, 4 * TS));
    a.parts = 2 * blocks > cus ? 1 : std::max(1, std::min({WGC * cus / blocks, a.KT / 8, kW4Parts}));
    const void *fn = a.M <= 32   ? reinterpret_cast<const void *>(&w4a8_tile_kernel<P, 2, ZEROS, TS, TG>)
                     : a.M <= 48 ? reinterpret_cast<const void *>(&w4a8_tile_kernel<P, 3, ZEROS, TS, TG>)
                                 : reinterpret_cast<const void *>(&w4a8_tile_kernel<P, 4, ZEROS, TS, TG>);
    void *args[] = {&a};
    const hipError_t e = hipLaunchKernel(fn, dim3(unsigned(blocks), unsigned(a.parts)), dim3(256 * TG), args, 0, stream);
    if (e != hipSuccess || a.parts == 1) return e;
    return hipLaunchKernel(reinterpret_cast<const void *>(&w4a8_join_kernel),
                           dim3(unsigned(ceil_div(a.N, 256)), unsigned(a.M)), dim3(256), args, 0, stream);
}

template <int P, bool ZEROS>
hipError_t w4_launch(const W4Launch &a, int cus, hipStream_t stream) {
    if (a.M > 16) return w4_tiles_launch<P, ZEROS>(a, cus, stream);
    const void *fn = a.M == 1 ? reinterpret_cast<const void *>(&w4a8_kernel<P, 1, ZEROS, true>)
                              : reinterpret_cast<const void *>(&w4a8_kernel<P, 1, ZEROS, false>);
    const int per = a.M == 1 ? 1 : 4;
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
