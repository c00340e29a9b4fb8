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
// low ones a shift and an AND, and the 16 goes out with the group's scale, one
// multiplication each: exactly (the least bit of a bf16 scale is 2^-133, of fp32
// 2^-149), and no sum is larger than the formula's.  With zero points a byte is
// q - z itself, three to four operations a word.  A group's sum is at most
// 16 * 8 * 128 * 128 = 2^21, exact as int32 and as fp32.  What is left of the work,
// and the most of it, is one conversion and one multiply-add for every result and
// group.
//
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
// Zero point byte i (z - 8) of a word, as z in every byte.
__device__ __forceinline__ uint32_t zero_bytes(uint32_t z, int i) {
    return __builtin_amdgcn_perm(0u, (z & 0x0F0F0F0Fu) ^ 0x08080808u, 0x01010101u * uint32_t(i));
}
// A group's scale, for sums of such bytes: divided by 16 where these are.
template <bool ZEROS>
__device__ __forceinline__ float scale_value(uint32_t bits, int bf16) {
    const float s = bf16 ? __uint_as_float(bits << 16) : float(__builtin_bit_cast(_Float16, uint16_t(bits)));
    return ZEROS ? s : s * 0.0625f;
}

__device__ __forceinline__ v4i mfma64(v4u x, v4u w, v4i acc) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(v4i, x), __builtin_bit_cast(v4i, w),
                                                 acc, 0, 0, 0);
}
__device__ __forceinline__ v4i mfma32(v2u x, v2u w, v4i acc) {
    return __builtin_amdgcn_mfma_i32_16x16x32_i8(__builtin_bit_cast(long, x), __builtin_bit_cast(long, w),
                                                 acc, 0, 0, 0);
}

// A lane's part of a tile of weights: codes, and the scales and zero points of
// its row in the tile's P groups, which share a quad of groups.
template <int P>
struct Weights {
    v4u w;
    uint32_t s[(P + 1) / 2], z;

    template <bool ZEROS>
    __device__ __forceinline__ void load(const uint8_t *wp, const uint16_t *sp, const uint8_t *zp, int t) {
        w = __builtin_nontemporal_load(reinterpret_cast<const v4u *>(wp + int64_t(t) * kW4TileBytes));
        const int g = P * t, at = (g >> 2) * 64 + (g & 3);
        if constexpr (P == 1)
            s[0] = sp[at];
        else
#pragma unroll
            for (int i = 0; i < P / 2; ++i) s[i] = reinterpret_cast<const uint32_t *>(sp + at)[i];
        if constexpr (ZEROS)
            z = P == 1   ? zp[at]
                : P == 2 ? *reinterpret_cast<const uint16_t *>(zp + at)
                         : *reinterpret_cast<const uint32_t *>(zp + at);
    }
    // The 16 values of piece j (of two).
    template <bool ZEROS>
    __device__ __forceinline__ v4u operand(int j, uint32_t zero) const {
        return v4u{low_values<ZEROS>(w[2 * j], zero), high_values<ZEROS>(w[2 * j], zero),
                   low_values<ZEROS>(w[2 * j + 1], zero), high_values<ZEROS>(w[2 * j + 1], zero)};
    }
    template <bool ZEROS>
    __device__ __forceinline__ float scale(int i, int bf16) const {
        return scale_value<ZEROS>((s[i >> 1] >> (16 * (i & 1))) & 0xFFFFu, bf16);
    }
};

// One row.  A workgroup takes one strip; its waves take the strip's tiles in
// turn, each asked for D tiles ahead, and add their sums in LDS in wave order.
// (Compiled, a round of D begins with a wait for every load of the round before, its
// last one among them: other waves hide the latency more than D does.)  The
// row is staged once (kRowChunk values at a time, zeros past its end), so the
// loop loads weights alone and knows no ragged tile.  Every row of the first
// operand is that row, so all results of a lane are the same: one is scaled.
constexpr int kRowChunk = 32768;

template <int P, bool ZEROS>
__global__ __launch_bounds__(64 * kMaxWaves) void w4a8_row_kernel(W4Launch a) {
    constexpr int D = 4;
    extern __shared__ __attribute__((aligned(16))) uint8_t row[];
    __shared__ float red[kMaxWaves][16];
    const int tid = int(threadIdx.x), lane = tid & 63, r = lane & 15, c = lane >> 4;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6), nw = int(blockDim.x) >> 6;
    const int s = int(blockIdx.x + blockIdx.z * gridDim.x);
    if (s >= a.strips) return;
    const uint8_t *wp = a.w + int64_t(s) * a.KT * kW4TileBytes + 16 * lane;
    const uint16_t *sp = a.scales + (int64_t(s) * a.GQ * 16 + r) * 4;
    const uint8_t *zp = ZEROS ? a.zeros + (int64_t(s) * a.GQ * 16 + r) * 4 : nullptr;
    Weights<P> d[D];
    float y = 0.0f;
    for (int t0 = 0; t0 < a.KT; t0 += kRowChunk / kTileK) {
        // This wave's tiles of the chunk: t0 + wv + i * nw, i < n.
        const int tiles = min(kRowChunk / kTileK, a.KT - t0);
        const int n = wv < tiles ? (tiles - wv + nw - 1) / nw : 0;
        const auto load = [&](int i, Weights<P> &t) __attribute__((always_inline)) {
            t.template load<ZEROS>(wp, sp, zp, t0 + wv + i * nw);
        };
#pragma unroll
        for (int j = 0; j < D; ++j)
            if (j < n) load(j, d[j]);
        if (t0 > 0) __syncthreads();        // the chunk before has been read
        for (int k = 16 * tid; k < tiles * kTileK; k += 16 * int(blockDim.x))
            *reinterpret_cast<v4u *>(row + k) = load_int8_tail(a.x, t0 * kTileK + k, a.K);
        __syncthreads();
        const auto use = [&](int i, const Weights<P> &t) __attribute__((always_inline)) {
            const uint8_t *x = row + (wv + i * nw) * kTileK;
#pragma unroll
            for (int g = 0; g < P; ++g) {
                const uint32_t z = ZEROS ? zero_bytes(t.z, g) : 0u;
                v4i acc = {0, 0, 0, 0};
                if constexpr (P == 4) {
                    acc = mfma32(*reinterpret_cast<const v2u *>(x + 32 * g + 8 * c),
                                 v2u{low_values<ZEROS>(t.w[g], z), high_values<ZEROS>(t.w[g], z)}, acc);
                } else {
#pragma unroll
                    for (int j = (P == 1 ? 0 : g); j < (P == 1 ? 2 : g + 1); ++j)
                        acc = mfma64(*reinterpret_cast<const v4u *>(x + (P == 1 ? 32 * c + 16 * j : 64 * j + 16 * c)),
                                     t.template operand<ZEROS>(j, z), acc);
                }
                y = __builtin_fmaf(float(acc[0]), t.template scale<ZEROS>(g, a.bf16_scales), y);
            }
        };
        // While no load can be past the end none is asked for it: a load that may
        // be skipped makes the compiler wait for all before it at every tile.
        int i = 0;
        for (; i + 2 * D <= n; i += D) {
#pragma unroll
            for (int j = 0; j < D; ++j) {
                use(i + j, d[j]);
                load(i + j + D, d[j]);
            }
        }
        for (; i < n; i += D) {
#pragma unroll
            for (int j = 0; j < D; ++j) {
                if (i + j < n) use(i + j, d[j]);
                if (i + j + D < n) load(i + j + D, d[j]);
            }
        }
    }
    if (c == 0) red[wv][r] = y;
    __syncthreads();
    const int n = s * kW4Rows + tid;
    if (tid >= 16 || n >= a.N) return;
    float v = 0.0f;
    for (int w = 0; w < nw; ++w) v += red[w][tid];
    v *= a.sa[0];
    if (a.y_f32) a.y_f32[n] = v;
    if (a.y_bf16) a.y_bf16[n] = uint16_t(bf16_bits(v));
}

constexpr int kFewWaves = 8;

// Few strips, 2 to 64 rows.  A workgroup takes one strip, up to eight waves take
// its tiles in turn and add their sums in LDS in wave order; a wave reads the
// rows' part of a tile as operands, without LDS.  A ragged tile is the last of
// the wave whose turn it is.  Bound by latency: a launch, two loads, one sum
// (16 x 2560 x 2560: 4.3 us, 3.4 for one row of it; 16 waves 4.4).
template <int P, int MB>
struct Rows {
    v4u v[MB][2];                       // P = 4: 8 bytes for every group

    template <bool TAIL>
    __device__ __forceinline__ void load(const int8_t *const (&xp)[MB], int t, int c, int K) {
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
            for (int j = 0; j < (P == 4 ? 4 : 2); ++j) {
                const int k = t * kTileK + (P == 4 ? 32 * j + 8 * c : P == 2 ? 64 * j + 16 * c : 32 * c + 16 * j);
                if constexpr (P == 4) {
                    v2u x = TAIL ? v2u(load_int8_tail(xp[b], k, K).xy) : v2u(*reinterpret_cast<const v2u_b *>(xp[b] + k));
                    v[b][j >> 1][2 * (j & 1)] = x[0];
                    v[b][j >> 1][2 * (j & 1) + 1] = x[1];
                } else {
                    v[b][j] = TAIL ? load_int8_tail(xp[b], k, K) : v4u(*reinterpret_cast<const v4u_b *>(xp[b] + k));
                }
            }
    }
};

template <int P, int MB, bool ZEROS>
__global__ __launch_bounds__(64 * kFewWaves) void w4a8_few_kernel(W4Launch a) {
    constexpr int D = 2;
    extern __shared__ __attribute__((aligned(16))) float part[];       // [wave][block][e][lane]
    const int tid = int(threadIdx.x), lane = tid & 63, r = lane & 15, c = lane >> 4;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6), nw = int(blockDim.x) >> 6;
    const int s = int(blockIdx.x);
    const uint8_t *wp = a.w + int64_t(s) * a.KT * kW4TileBytes + 16 * lane;
    const uint16_t *sp = a.scales + (int64_t(s) * a.GQ * 16 + r) * 4;
    const uint8_t *zp = ZEROS ? a.zeros + (int64_t(s) * a.GQ * 16 + r) * 4 : nullptr;
    const int8_t *xp[MB];
    float y[MB][4];
#pragma unroll
    for (int b = 0; b < MB; ++b) {
        xp[b] = a.x + int64_t(min(16 * b + r, a.M - 1)) * a.K;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[b][e] = 0.0f;
    }
    const auto use = [&](const Weights<P> &t, const Rows<P, MB> &x) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const float sc = t.template scale<ZEROS>(i, a.bf16_scales);
            const uint32_t z = ZEROS ? zero_bytes(t.z, i) : 0u;
#pragma unroll
            for (int b = 0; b < MB; ++b) {
                v4i acc = {0, 0, 0, 0};
                if constexpr (P == 4) {
                    acc = mfma32(v2u{x.v[b][i >> 1][2 * (i & 1)], x.v[b][i >> 1][2 * (i & 1) + 1]},
                                 v2u{low_values<ZEROS>(t.w[i], z), high_values<ZEROS>(t.w[i], z)}, acc);
                } else {
#pragma unroll
                    for (int j = (P == 1 ? 0 : i); j < (P == 1 ? 2 : i + 1); ++j)
                        acc = mfma64(x.v[b][j], t.template operand<ZEROS>(j, z), acc);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) y[b][e] = __builtin_fmaf(float(acc[e]), sc, y[b][e]);
            }
        }
    };
    const int whole = a.K / kTileK, n = wv < whole ? (whole - wv + nw - 1) / nw : 0;
    Weights<P> d[D];
    Rows<P, MB> x[D];
    const auto load = [&](int i, int j) __attribute__((always_inline)) {
        d[j].template load<ZEROS>(wp, sp, zp, wv + i * nw);
        x[j].template load<false>(xp, wv + i * nw, c, a.K);
    };
#pragma unroll
    for (int j = 0; j < D; ++j)
        if (j < n) load(j, j);
    int i = 0;
    for (; i + 2 * D <= n; i += D) {
#pragma unroll
        for (int j = 0; j < D; ++j) {
            use(d[j], x[j]);
            load(i + j + D, j);
        }
    }
    for (; i < n; i += D) {
#pragma unroll
        for (int j = 0; j < D; ++j) {
            if (i + j < n) use(d[j], x[j]);
            if (i + j + D < n) load(i + j + D, j);
        }
    }
    if (whole < a.KT && wv == whole % nw) {
        d[0].template load<ZEROS>(wp, sp, zp, whole);
        x[0].template load<true>(xp, whole, c, a.K);
        use(d[0], x[0]);
    }
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) part[((wv * MB + b) * 4 + e) * 64 + lane] = y[b][e];
    __syncthreads();
    // Place o is lane o % 64's result e of block b: weight row o % 16, activation
    // row 16b + 4c + e.
    for (int o = tid; o < 256 * MB; o += 64 * nw) {
        float v = 0.0f;
        for (int w = 0; w < nw; w += 4) {
            float t[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) t[q] = part[min(w + q, nw - 1) * 256 * MB + o];
#pragma unroll
            for (int q = 0; q < 4; ++q) v += w + q < nw ? t[q] : 0.0f;
        }
        const int n = s * kW4Rows + (o & 15), m = 16 * (o >> 8) + 4 * ((o >> 4) & 3) + ((o >> 6) & 3);
        if (m >= a.M || n >= a.N) continue;
        const int64_t at = int64_t(m) * a.N + n;
        v *= a.sa[m];
        if (a.y_f32) a.y_f32[at] = v;
        if (a.y_bf16) a.y_bf16[at] = uint16_t(bf16_bits(v));
    }
}

// More strips: activations through LDS.  A workgroup takes four strips
// and a range of the tiles of k, in GROUPS groups of four waves that take its
// tiles in turn, a strip a wave; a group stages the rows' part of a tile (MB
// blocks of 16 rows x 128 k) once for its four waves.  LDS holds it as
// [block][chunk of 16 k][row], where every operand is 16 (or, for groups of 32,
// 8) bytes of a lane and a quarter of a wave reads 256 bytes in a row; chunks
// are 16 bytes apart from that, so that the stores of a row's chunks fall in
// different banks.  Rows start anywhere, so they are staged through registers.
//
// Bound by the results' conversions and multiply-adds and by the loop's waits (64 x
// 5120 x 27648, groups of 64: some 105 vector instructions a tile, 8 of them on the
// matrix pipe; 27 us, of which the instructions are 12 and the weights 15, side by
// side; half of the waves' cycles are waits).  Each strip
// reading its rows from the L2 by itself took 106 us for that product.
constexpr int kChunkBytes = 272;

template <int P, int MB, bool ZEROS, int GROUPS>
__global__ __launch_bounds__(256 * GROUPS, 2) void w4a8_tile_kernel(W4Launch a) {
    constexpr int STAGE = MB * 8 * kChunkBytes, PER = (MB * 128 + 255) / 256;
    constexpr int D = 2;                     // tiles that a wave's weights are asked for ahead
    __shared__ __attribute__((aligned(16))) uint8_t stages[GROUPS][2][STAGE];
    const int tid = int(threadIdx.x) & 255, lane = tid & 63, r = lane & 15, c = lane >> 4;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int group = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 8);
    uint8_t(&lds)[2][STAGE] = stages[group];
    const int strip = int(blockIdx.x + blockIdx.z * gridDim.x) * 4 + wv, part = int(blockIdx.y);
    // The part's tiles of k from t0 on; this group's are t0 + group + i * GROUPS,
    // i < n (steps: the most that a group has).
    const int t0 = int(int64_t(a.KT) * part / a.parts), t1 = int(int64_t(a.KT) * (part + 1) / a.parts);
    const int steps = (t1 - t0 + GROUPS - 1) / GROUPS, n = (t1 - t0 - group + GROUPS - 1) / GROUPS;

    const int64_t s = min(strip, a.strips - 1);       // (past the last: not stored)
    const uint8_t *wp = a.w + s * a.KT * kW4TileBytes + 16 * lane;
    const uint16_t *sp = a.scales + (s * a.GQ * 16 + r) * 4;
    const uint8_t *zp = ZEROS ? a.zeros + (s * a.GQ * 16 + r) * 4 : nullptr;
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
            for (int j = 0; j < PER; ++j) xv[j] = load_int8_tail(xp[j], k, a.K);
        }
    };
    auto store_x = [&](uint8_t *stage, const v4u (&xv)[PER]) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (MB * 128 % 256 == 0 || tid + 256 * j < MB * 128) *reinterpret_cast<v4u *>(stage + to[j]) = xv[j];
    };

    float y[MB][4];
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) y[b][e] = 0.0f;

    auto use = [&](const Weights<P> &d, const uint8_t *stage) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const float sc = d.template scale<ZEROS>(i, a.bf16_scales);
            const uint32_t z = ZEROS ? zero_bytes(d.z, i) : 0u;
#pragma unroll
            for (int b = 0; b < MB; ++b) {
                v4i acc = {0, 0, 0, 0};
                if constexpr (P == 4) {
                    acc = mfma32(*reinterpret_cast<const v2u *>(stage + (b * 8 + 2 * i + (c >> 1)) * kChunkBytes + 16 * r + 8 * (c & 1)),
                                 v2u{low_values<ZEROS>(d.w[i], z), high_values<ZEROS>(d.w[i], z)}, acc);
                } else {
#pragma unroll
                    for (int j = (P == 1 ? 0 : i); j < (P == 1 ? 2 : i + 1); ++j)
                        acc = mfma64(*reinterpret_cast<const v4u *>(stage + (b * 8 + (P == 1 ? 2 * c + j : 4 * j + c)) * kChunkBytes + 16 * r),
                                     d.template operand<ZEROS>(j, z), acc);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) y[b][e] = __builtin_fmaf(float(acc[e]), sc, y[b][e]);
            }
        }
    };

    // Weights are asked for D tiles ahead; rows D + 1, the nearest of them in the other
    // stage.  (Compiled, all weights asked for are waited for once in a round of D, ahead
    // of its stages' stores: load_x may take its ragged side, which has loads of its own.)
    Weights<P> d[D];
    v4u xv[D][PER];
    const auto tile = [&](int i) { return t0 + group + i * GROUPS; };
    const auto load_w = [&](int t, Weights<P> &w) __attribute__((always_inline)) { w.template load<ZEROS>(wp, sp, zp, t); };
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
    // be skipped makes the compiler wait for all before it at every tile.
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
    static_assert(MB * 4096 <= 2 * STAGE, "a group's sums fit its stages");
    float *mine = reinterpret_cast<float *>(&lds[0][0]);
    if (group > 0) {
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) mine[(b * 4 + e) * 256 + tid] = y[b][e];
    }
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int g = 1; g < GROUPS; ++g)
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                y[b][e] += reinterpret_cast<const float *>(&stages[g][0][0])[(b * 4 + e) * 256 + tid];

    // Lane (r, c) of block b: weight row r, activation rows 16b + 4c + e.
    const int row = strip * kW4Rows + r;
    if (row >= a.N) return;
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int m = 16 * b + 4 * c + e;
            if (m >= a.M) continue;
            const int64_t at = int64_t(m) * a.N + row;
            if (a.parts > 1) {
                a.ws[part * (int64_t(a.M) * a.N) + at] = y[b][e];
                continue;
            }
            const float v = y[b][e] * a.sa[m];
            if (a.y_f32) a.y_f32[at] = v;
            if (a.y_bf16) a.y_bf16[at] = uint16_t(bf16_bits(v));
        }
}

// The parts of k, added in order.
__global__ __launch_bounds__(256) void w4a8_join_kernel(W4Launch a) {
    const int n = int(blockIdx.x) * 256 + int(threadIdx.x), m = int(blockIdx.y);
    if (n >= a.N) return;
    const int64_t at = int64_t(m) * a.N + n, all = int64_t(a.M) * a.N;
    float v = 0.0f;
    // Eight parts a wait; those past the last are read as the last.
    for (int p = 0; p < a.parts; p += 8) {
        float t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = a.ws[min(p + i, a.parts - 1) * all + at];
#pragma unroll
        for (int i = 0; i < 8; ++i) v += p + i < a.parts ? t[i] : 0.0f;
    }
    v *= a.sa[m];
    if (a.y_f32) a.y_f32[at] = v;
    if (a.y_bf16) a.y_bf16[at] = uint16_t(bf16_bits(v));
}

template <int P, bool ZEROS>
const void *w4_kernel(const W4Plan &p) {
    const auto fn = [](auto *k) { return reinterpret_cast<const void *>(k); };
    if (p.few)
        return p.blocks == 1   ? fn(&w4a8_few_kernel<P, 1, ZEROS>)
               : p.blocks == 2 ? fn(&w4a8_few_kernel<P, 2, ZEROS>)
               : p.blocks == 3 ? fn(&w4a8_few_kernel<P, 3, ZEROS>)
                               : fn(&w4a8_few_kernel<P, 4, ZEROS>);
    const bool four = p.groups == 4;
    switch (p.blocks) {
    case 0: return fn(&w4a8_row_kernel<P, ZEROS>);
    case 1: return four ? fn(&w4a8_tile_kernel<P, 1, ZEROS, 4>) : fn(&w4a8_tile_kernel<P, 1, ZEROS, 2>);
    case 2: return four ? fn(&w4a8_tile_kernel<P, 2, ZEROS, 4>) : fn(&w4a8_tile_kernel<P, 2, ZEROS, 2>);
    case 3: return fn(&w4a8_tile_kernel<P, 3, ZEROS, 2>);
    default: return fn(&w4a8_tile_kernel<P, 4, ZEROS, 2>);
    }
}

template <int P, bool ZEROS>
hipError_t w4_launch(const W4Launch &la, int cus, hipStream_t stream) {
    W4Launch a = la;
    const W4Plan p = w4_plan(a.M, a.strips, a.KT, a.K, a.group, cus);
    a.parts = p.parts;
    const int units = p.blocks ? int(ceil_div(a.strips, 4)) : a.strips, gx = std::min(units, 1 << 20);
    const unsigned far = unsigned(ceil_div(units, gx)), threads = unsigned((p.blocks ? 256 : 64) * p.groups);
    void *args[] = {&a};
    if (p.few)
        return hipLaunchKernel(w4_kernel<P, ZEROS>(p), dim3(unsigned(a.strips)), dim3(unsigned(64 * p.groups)), args,
                               size_t(p.groups * p.blocks) * 1024, stream);
    const hipError_t e = hipLaunchKernel(w4_kernel<P, ZEROS>(p), dim3(unsigned(gx), unsigned(a.parts), far), dim3(threads),
                                         args, p.blocks ? 0 : size_t(std::min(a.KT * kTileK, kRowChunk)), stream);
    if (e != hipSuccess || a.parts == 1) return e;
    return hipLaunchKernel(reinterpret_cast<const void *>(&w4a8_join_kernel),
                           dim3(unsigned(ceil_div(a.N, 256)), unsigned(a.M)), dim3(256), args, 0, stream);
}

template <int P>
hipError_t w4_zeros(const W4Launch &a, int cus, hipStream_t stream) {
    return a.zeros ? w4_launch<P, true>(a, cus, stream) : w4_launch<P, false>(a, cus, stream);
}

}  // namespace

// One row: waves of a strip, all that the sums bear where strips are few, and
// four where they are many (us, eight and four waves: 2560 x 2560 3.7 and 4.1,
// 5120 x 27648 19.2 and 23.3; 13824 x 2560 6.6 and 6.2, 27648 x 5120 19.0 and 15.3,
// 55296 x 5120 26.6 and 24.7; 8640 x 3200, 540 strips, 5.6 and 5.7).
//
// More rows: workgroups of four strips.  Where these are half the compute units
// or fewer, k is split into parts, about two workgroups to a compute unit, with
// four tiles for every wave; the sums of parts go through memory (4.5 us for
// their joining, so not for grids that fill most of the device: 19 x 13824 x 2570
// 13.5 us whole, 16.5 + 4 in two parts).  Four groups of waves share a
// workgroup's k where it has a compute unit to itself: 16 x 13824 x 2560 7.8 us
// against 9.8, 32 x 5120 x 5120 10.9 against 13.3; two otherwise: 16 x 55296 x
// 5120 32.5 against 34.3, 32 x 5120 x 27648 24.0 against 26.8, and beyond 32
// rows, whose stages are larger: 64 x 5120 x 27648 30.2 against 34.3.
//
// Few strips and 2 rows or more: a workgroup for each strip, while its waves have
// few steps to make (tiles of a wave, by blocks of rows, by strips to a compute
// unit).  Its waves read the rows from the L2 as operands, all strips the same, so
// that no step may be one of many (us, this and workgroups of four strips; groups of
// 128, 64 and 32: 16 x 2560 x 2560, 3 steps, 4.3, 4.3, 5.4 and 7.0, 7.3, 8.1; 64 rows,
// 12 steps, 8.3, 8.6, 13.2 and 10.0, 10.5, 12.2; 32 x 2560 x 6912, 14 steps, 10.7, 10.2,
// 16.2 and 10.2, 10.8, 12.4; two strips to a unit: 16 x 5120 x 1280, 4 steps, 4.2, 4.2,
// 5.5 and 5.2, 5.5, 6.0; 32 x 8192 x 640, 4 steps, 4.8, 4.8, 7.5 and 5.2, 5.5, 6.0, 64
// rows, 8 steps, 9.1, 9.3, 11.8 and 7.0, 7.4, 8.3; four: 16 x 13824 x 1024 5.4, 5.4, 8.0
// and 5.2, 5.4, 6.0; rows that begin at odd addresses: 16 x 2560 x 2565, 3 steps, 6.9,
// 6.9, 7.3 and 8.8, 9.0, 9.7, 32 rows, 6 steps, 10.1, 10.3, 10.7 and 9.6, 9.7, 10.9).
static bool few_strips(int M, int strips, int KT, int K, int group, int cus) {
    const int blocks = (M + 15) / 16, rounds = int(ceil_div(strips, cus));
    const int steps = std::min(rounds, 3) * blocks * int(ceil_div(KT, kFewWaves));
    if (rounds > 2 || (rounds == 2 && (K % 8 || blocks > (group == 32 ? 1 : 2)))) return false;
    return steps <= (K % 8 ? 4 : (group == 32 ? 8 : 12) - 4 * (rounds - 1));
}

W4Plan w4_plan(int M, int strips, int KT, int K, int group, int cus) {
    if (M == 1) return {0, std::min(strips > 2 * cus ? 4 : kMaxWaves, KT), 1, false};
    if (few_strips(M, strips, KT, K, group, cus)) return {(M + 15) / 16, std::min(kFewWaves, KT), 1, true};
    const int units = int(ceil_div(strips, 4));
    const auto parts = [&](int groups) {
        return 2 * units > cus ? 1 : std::max(1, std::min({2 * cus / units, KT / (4 * groups), kW4Parts}));
    };
    const bool four = M <= 16 ? units <= cus : M <= 32 && units * parts(4) <= cus;
    const int groups = four ? 4 : 2;
    return {(M + 15) / 16, groups, parts(groups), false};
}

hipError_t launch_w4a8(const W4Launch &a, int cus, hipStream_t stream) {
    return a.group == 128 ? w4_zeros<1>(a, cus, stream)
           : a.group == 64 ? w4_zeros<2>(a, cus, stream)
                           : w4_zeros<4>(a, cus, stream);
}

}  // namespace w2a8
