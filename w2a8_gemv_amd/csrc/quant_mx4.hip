// MX4 rounding of float rows (activations, MX4R) and of weights (MX16x128),
// and back (gfx950).
//
// Per block of 32 values: a = max|x|, 2^e from a's exponent field, and
// x * 2^-e rounded half to even to a 4-bit float (w2a8_mx4.h).  A lane holds
// one chunk of 16 values, the pair of lanes of a block exchange their maxima
// with one DPP move, and v_cvt_scalef32_pk_fp4_f32 makes a code byte of two
// values.  The row is read once and nothing but the codes is written.
#include "mx4.h"

namespace w2a8 {
namespace {

constexpr int kChunk = 16;                 // values per lane
constexpr int kChunksPerTile = kTileK / kChunk;   // 8

template <int TYPE> struct Elem;
template <> struct Elem<W2A8_F32> { typedef float T; };
template <> struct Elem<W2A8_BF16> { typedef uint16_t T; };
template <> struct Elem<W2A8_F16> { typedef uint16_t T; };

// Values k0 .. k0+15 of a row as fp32 (0 at k >= K).
template <int TYPE>
__device__ __forceinline__ void load_chunk(const typename Elem<TYPE>::T *row, int k0, int K,
                                           float (&v)[kChunk]) {
    if (k0 + kChunk <= K) {
        // Four-byte (or two-byte) aligned rows: the global loads need no more
        // than the element's own alignment.
        if constexpr (TYPE == W2A8_F32) {
            float t[kChunk];
            __builtin_memcpy(t, row + k0, sizeof t);
#pragma unroll
            for (int i = 0; i < kChunk; ++i) v[i] = t[i];
        } else {
            uint32_t t[kChunk / 2];
            __builtin_memcpy(t, row + k0, sizeof t);
#pragma unroll
            for (int i = 0; i < kChunk / 2; ++i) {
                if constexpr (TYPE == W2A8_BF16) {
                    v[2 * i] = lo_bf16(t[i]);
                    v[2 * i + 1] = hi_bf16(t[i]);
                } else {
                    v[2 * i] = float(__builtin_bit_cast(_Float16, uint16_t(t[i])));
                    v[2 * i + 1] = float(__builtin_bit_cast(_Float16, uint16_t(t[i] >> 16)));
                }
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < kChunk; ++i) v[i] = k0 + i < K ? mx4_load1<TYPE>(row, k0 + i) : 0.0f;
}

// The two code words of this lane's chunk and its block's scale byte (the
// block's two chunks sit in lanes 2j and 2j + 1).
__device__ __forceinline__ v2u round_chunk(const float (&v)[kChunk], uint32_t *byte) {
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < kChunk; ++i) a = max(a, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    a = max(a, uint32_t(__builtin_amdgcn_update_dpp(0, int(a), 0xB1, 0xF, 0xF, false)));
    *byte = mx4_scale_byte(a);
    const float s = mx4_scale_value(*byte);
    const float l0[4] = {v[0], v[1], v[2], v[3]}, h0[4] = {v[8], v[9], v[10], v[11]};
    const float l1[4] = {v[4], v[5], v[6], v[7]}, h1[4] = {v[12], v[13], v[14], v[15]};
    return v2u{mx4_codes4(l0, h0, s), mx4_codes4(l1, h1, s)};
}

// How rows are dealt to workgroups: 2^shift lanes to a row and the rest of the
// workgroup's 256 to other rows (short rows), or `segs` workgroups to a row;
// one item (a chunk, or a group of values) to a lane.  (Two or four items to a
// lane were no faster: 2045 x 6907 fp32 14.5 and 14.7 us, back 12.6, 14.1 and
// 13.9.)
struct Rows {
    int64_t rows;
    uint32_t segs;
    int shift, K, KT;
};
__device__ __forceinline__ void place_item(const Rows &t, int64_t *row, int *item) {
    const int64_t blk = blockIdx.x + int64_t(blockIdx.y) * gridDim.x;
    const int64_t seg = blk / t.segs;
    *row = seg * (256 >> t.shift) + (int(threadIdx.x) >> t.shift);
    *item = int(blk - seg * t.segs) * 256 + (int(threadIdx.x) & ((1 << t.shift) - 1));
}

// PACK: the row is row m of the weights and goes to MX16x128 (rows N ..
// 16*NS - 1 are padding), otherwise to MX4R.  A row's 16 bytes of a block lie
// 256 bytes apart there, and its scale bytes 256: 13824 x 5120 takes 68 us in
// bf16 and 101 in fp32, where the same rows to MX4R take 39 and 68 (5125 GB/s,
// a large copy's rate: 35 and 63).  It is done once for a matrix.
template <int TYPE, bool PACK>
__global__ __launch_bounds__(256) void quant_mx4_kernel(const void *x, Rows t, uint8_t *xq,
                                                        uint8_t *xs) {
    const int KT = t.KT, KU = (KT + kMxQuad - 1) / kMxQuad;
    int64_t m;
    int c;
    place_item(t, &m, &c);
    // Chunks of whole groups of four tiles: those past the last tile only
    // clear their scale byte.
    if (c >= KU * kMxQuad * kChunksPerTile) return;
    if (m >= (PACK ? (t.rows + kMxRows - 1) / kMxRows * kMxRows : t.rows)) return;
    float v[kChunk];
    load_chunk<TYPE>(static_cast<const typename Elem<TYPE>::T *>(x) + m * t.K, c * kChunk,
                     !PACK || m < t.rows ? t.K : 0, v);
    uint32_t byte;
    const v2u w = round_chunk(v, &byte);
    const int tile = c / kChunksPerTile, g = (c % kChunksPerTile) / 2;
    const int64_t s = m / kMxRows;
    const int l = 16 * g + int(m % kMxRows);
    if (tile < KT) {
        uint8_t *q = PACK ? xq + (s * KT + tile) * kMxTileBytes + 16 * l + 8 * (c & 1)
                          : xq + m * KT * kMxRowTile + c * 8;
        *reinterpret_cast<v2u *>(q) = w;
    }
    if ((c & 1) == 0) {
        uint8_t *q = PACK ? xs + (s * KU + tile / kMxQuad) * 256 + 4 * l + tile % kMxQuad
                          : xs + m * KU * 16 + 16 * (tile / kMxQuad) + 4 * g + tile % kMxQuad;
        *q = uint8_t(byte);
    }
}

// The values of the low halves of a word's four bytes times a block's power of
// two (v_cvt_scalef32_pk_f32_fp4 makes both halves of a byte; exact down to
// fp32's subnormals, NaN for a NaN scale).
__device__ __forceinline__ void low_values(uint32_t w, float scale, float *v) {
    v[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 0)[0];
    v[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 1)[0];
    v[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 2)[0];
    v[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 3)[0];
}

// A lane writes 16 bytes of the row, four or eight values, so that a wave's
// stores are whole lines, and non-temporal ones: 12.6 us for 2045 x 6907 fp32,
// 22.5 us with ordinary stores, 35 us with 16 values a lane, 64 bytes apart.
// Values 4i .. 4i + 3 of a chunk are the low (i < 2) or high halves of its word
// i % 2.
template <int TYPE>
__global__ __launch_bounds__(256) void dequant_mx4_kernel(const uint8_t *xq, const uint8_t *xs, Rows t,
                                                          void *y) {
    constexpr int V = TYPE == W2A8_F32 ? 4 : 8;
    typedef typename Elem<TYPE>::T E;
    int64_t m;
    int i;
    place_item(t, &m, &i);
    const int k = i * V;
    if (m >= t.rows || k >= t.K) return;
    const int KU = (t.KT + kMxQuad - 1) / kMxQuad;
    const int tile = k / kTileK, g = k % kTileK / 32;
    const v2u w = reinterpret_cast<const v2u *>(xq + m * t.KT * kMxRowTile)[k / kChunk];
    const float s = mx4_scale_value(xs[m * KU * 16 + 16 * (tile / kMxQuad) + 4 * g + tile % kMxQuad]);
    const int part = k % kChunk / 4, half = 2 * (part & 2);
    float v[V];
    if constexpr (V == 4) {
        low_values((part & 1 ? w[1] : w[0]) >> half, s, v);
    } else {
        low_values(w[0] >> half, s, v);
        low_values(w[1] >> half, s, v + 4);
    }
    v4u o;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (TYPE == W2A8_F32)
            o[j] = __float_as_uint(v[j]);
        else if constexpr (TYPE == W2A8_BF16)
            o[j] = bf16_pair(v[2 * j], v[2 * j + 1]);
        else
            o[j] = uint32_t(__builtin_bit_cast(uint16_t, _Float16(v[2 * j]))) |
                   (uint32_t(__builtin_bit_cast(uint16_t, _Float16(v[2 * j + 1]))) << 16);
    }
    E *at = static_cast<E *>(y) + m * t.K + k;
    if (k + V <= t.K) {
        __builtin_nontemporal_store(o, reinterpret_cast<v4u_any *>(at));
        return;
    }
#pragma unroll
    for (int j = 0; j < V - 1; ++j)
        if (k + j < t.K) {
            if constexpr (TYPE == W2A8_F32)
                at[j] = __uint_as_float(o[j]);
            else
                at[j] = uint16_t(o[j / 2] >> (16 * (j & 1)));
        }
}

// Rows of `items` items: as many rows to a workgroup as fit side by side, or
// 256 items of one row.  A grid of more than 2^20 in x folds into y (a launch
// holds fewer than 2^32 lanes in x).
Rows row_plan(int64_t rows, int64_t padded, int64_t items, int K, dim3 *grid) {
    Rows t;
    t.rows = rows;
    t.K = K;
    t.KT = int(mx4_tiles(K));
    t.shift = 8;
    while (t.shift > 5 && items <= (1 << (t.shift - 1))) --t.shift;
    t.segs = uint32_t(ceil_div(items, 256));
    const int64_t blocks = ceil_div(padded, 256 >> t.shift) * t.segs;
    const int64_t gx = std::min<int64_t>(blocks, int64_t(1) << 20);
    *grid = dim3(unsigned(gx), unsigned(ceil_div(blocks, gx)));
    return t;
}

template <int TYPE, bool PACK>
hipError_t quant_launch(const void *x, int64_t rows, int K, uint8_t *q, uint8_t *s,
                        hipStream_t stream) {
    dim3 grid;
    Rows t = row_plan(rows, PACK ? round_up(rows, kMxRows) : rows,
                      mx4_quads(K) * kMxQuad * kChunksPerTile, K, &grid);
    void *args[] = {&x, &t, &q, &s};
    return hipLaunchKernel(reinterpret_cast<const void *>(&quant_mx4_kernel<TYPE, PACK>), grid,
                           dim3(256), args, 0, stream);
}

template <int TYPE>
hipError_t dequant_launch(const uint8_t *q, const uint8_t *s, int64_t rows, int K, void *y,
                          hipStream_t stream) {
    dim3 grid;
    Rows t = row_plan(rows, rows, ceil_div(K, TYPE == W2A8_F32 ? 4 : 8), K, &grid);
    void *args[] = {&q, &s, &t, &y};
    return hipLaunchKernel(reinterpret_cast<const void *>(&dequant_mx4_kernel<TYPE>), grid, dim3(256),
                           args, 0, stream);
}

}  // namespace

hipError_t launch_quant_mx4(const void *x, int type, int64_t M, int K, uint8_t *xq, uint8_t *xs,
                            hipStream_t stream) {
    return type == W2A8_F32    ? quant_launch<W2A8_F32, false>(x, M, K, xq, xs, stream)
           : type == W2A8_BF16 ? quant_launch<W2A8_BF16, false>(x, M, K, xq, xs, stream)
                               : quant_launch<W2A8_F16, false>(x, M, K, xq, xs, stream);
}

hipError_t launch_quant_pack_mx4(const void *W, int type, int64_t N, int K, uint8_t *packed,
                                 hipStream_t stream) {
    uint8_t *s = packed + ceil_div(N, kMxRows) * mx4_tiles(K) * kMxTileBytes;
    return type == W2A8_F32    ? quant_launch<W2A8_F32, true>(W, N, K, packed, s, stream)
           : type == W2A8_BF16 ? quant_launch<W2A8_BF16, true>(W, N, K, packed, s, stream)
                               : quant_launch<W2A8_F16, true>(W, N, K, packed, s, stream);
}

hipError_t launch_dequant_mx4(const uint8_t *xq, const uint8_t *xs, int64_t M, int K, void *y,
                              int type, hipStream_t stream) {
    return type == W2A8_F32    ? dequant_launch<W2A8_F32>(xq, xs, M, K, y, stream)
           : type == W2A8_BF16 ? dequant_launch<W2A8_BF16>(xq, xs, M, K, y, stream)
                               : dequant_launch<W2A8_F16>(xq, xs, M, K, y, stream);
}

}  // namespace w2a8
