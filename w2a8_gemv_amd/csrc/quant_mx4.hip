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

// blockIdx.x = row * segs + segment; a workgroup takes blockDim.x chunks of
// one row.  PACK: the row is row m of the weights and goes to MX16x128 (rows
// N .. 16*NS - 1 are padding), otherwise to MX4R.
template <int TYPE, bool PACK>
__global__ __launch_bounds__(256) void quant_mx4_kernel(const void *x, uint32_t segs, int64_t rows,
                                                        int K, int KT, uint8_t *xq, uint8_t *xs) {
    const int64_t blk = blockIdx.x + int64_t(blockIdx.y) * gridDim.x;
    const int64_t m = blk / segs;
    const int c = int(blk - m * segs) * int(blockDim.x) + int(threadIdx.x);   // chunk of the row
    const int KU = (KT + kMxQuad - 1) / kMxQuad;
    // Chunks of whole groups of four tiles: those past the last tile only
    // clear their scale byte.
    if (c >= KU * kMxQuad * kChunksPerTile) return;
    if (PACK ? m >= (rows + kMxRows - 1) / kMxRows * kMxRows : m >= rows) return;
    const int t = c / kChunksPerTile, g = (c % kChunksPerTile) / 2;
    float v[kChunk];
    if (PACK && m >= rows) {
#pragma unroll
        for (int i = 0; i < kChunk; ++i) v[i] = 0.0f;
    } else {
        load_chunk<TYPE>(static_cast<const typename Elem<TYPE>::T *>(x) + m * K, c * kChunk, K, v);
    }
    uint32_t byte;
    const v2u w = round_chunk(v, &byte);
    const int64_t s = m / kMxRows;
    const int l = 16 * g + int(m % kMxRows);
    if (t < KT) {
        uint8_t *q = PACK ? xq + (s * KT + t) * kMxTileBytes + 16 * l + 8 * (c & 1)
                          : xq + m * KT * kMxRowTile + c * 8;
        *reinterpret_cast<v2u *>(q) = w;
    }
    if ((c & 1) == 0) {
        uint8_t *q = PACK ? xs + (s * KU + t / kMxQuad) * 256 + 4 * l + t % kMxQuad
                          : xs + m * KU * 16 + 16 * (t / kMxQuad) + 4 * g + t % kMxQuad;
        *q = uint8_t(byte);
    }
}

template <int TYPE>
__device__ __forceinline__ uint32_t narrow_bits(float v) {
    if constexpr (TYPE == W2A8_BF16) return bf16_bits(v);
    return __builtin_bit_cast(uint16_t, _Float16(v));
}

// Value of a 4-bit code times a block's power of two, each exact in fp32
// down to its subnormals.
__device__ __forceinline__ float code_value(uint32_t c, float scale) {
    // Twice the magnitude, 0 1 2 3 4 6 8 12, out of a table of nibbles.
    const uint32_t twice = (0xC8643210u >> (4 * (c & 7))) & 15u;
    const float r = (0.5f * float(twice)) * scale;
    return (c & 8) ? -r : r;
}

template <int TYPE>
__global__ __launch_bounds__(256) void dequant_mx4_kernel(const uint8_t *xq, const uint8_t *xs,
                                                          uint32_t segs, int64_t rows, int K, int KT,
                                                          void *y) {
    const int64_t blk = blockIdx.x + int64_t(blockIdx.y) * gridDim.x;
    const int64_t m = blk / segs;
    const int c = int(blk - m * segs) * int(blockDim.x) + int(threadIdx.x);
    const int KU = (KT + kMxQuad - 1) / kMxQuad;
    const int k0 = c * kChunk;
    if (m >= rows || k0 >= K) return;
    const int t = c / kChunksPerTile, g = (c % kChunksPerTile) / 2;
    const v2u w = *reinterpret_cast<const v2u *>(xq + m * KT * kMxRowTile + c * 8);
    const uint32_t byte = xs[m * KU * 16 + 16 * (t / kMxQuad) + 4 * g + t % kMxQuad];
    const float s = mx4_scale_value(byte);
    float v[kChunk];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[j] = code_value(w[0] >> (8 * j), s);
        v[8 + j] = code_value(w[0] >> (8 * j + 4), s);
        v[4 + j] = code_value(w[1] >> (8 * j), s);
        v[12 + j] = code_value(w[1] >> (8 * j + 4), s);
    }
    typename Elem<TYPE>::T *row = static_cast<typename Elem<TYPE>::T *>(y) + m * K + k0;
    if (k0 + kChunk <= K) {
        if constexpr (TYPE == W2A8_F32) {
            __builtin_memcpy(row, v, sizeof v);
        } else {
            uint32_t o[kChunk / 2];
#pragma unroll
            for (int i = 0; i < kChunk / 2; ++i)
                o[i] = narrow_bits<TYPE>(v[2 * i]) | (narrow_bits<TYPE>(v[2 * i + 1]) << 16);
            __builtin_memcpy(row, o, sizeof o);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < kChunk; ++i)
        if (k0 + i < K) {
            if constexpr (TYPE == W2A8_F32)
                row[i] = v[i];
            else
                row[i] = uint16_t(narrow_bits<TYPE>(v[i]));
        }
}

// Workgroups of up to 256 chunks of one row; a grid of more than 2^20 in x
// folds into y (a launch holds fewer than 2^32 lanes in x).
struct RowGrid {
    dim3 grid, block;
    uint32_t segs;
};
RowGrid row_grid(int64_t rows, int64_t chunks) {
    RowGrid r;
    const int64_t b = std::min<int64_t>(256, round_up(chunks, 64));
    r.segs = uint32_t(ceil_div(chunks, b));
    const int64_t blocks = rows * r.segs;
    const int64_t gx = std::min<int64_t>(blocks, int64_t(1) << 20);
    r.grid = dim3(unsigned(gx), unsigned(ceil_div(blocks, gx)));
    r.block = dim3(unsigned(b));
    return r;
}

template <int TYPE, bool PACK>
hipError_t quant_launch(const void *x, int64_t rows, int K, uint8_t *q, uint8_t *s,
                        hipStream_t stream) {
    int KT = int(mx4_tiles(K));
    RowGrid r = row_grid(PACK ? round_up(rows, kMxRows) : rows,
                         mx4_quads(K) * kMxQuad * kChunksPerTile);
    void *args[] = {&x, &r.segs, &rows, &K, &KT, &q, &s};
    return hipLaunchKernel(reinterpret_cast<const void *>(&quant_mx4_kernel<TYPE, PACK>), r.grid,
                           r.block, args, 0, stream);
}

template <int TYPE>
hipError_t dequant_launch(const uint8_t *q, const uint8_t *s, int64_t rows, int K, void *y,
                          hipStream_t stream) {
    int KT = int(mx4_tiles(K));
    RowGrid r = row_grid(rows, ceil_div(K, kChunk));
    void *args[] = {&q, &s, &r.segs, &rows, &K, &KT, &y};
    return hipLaunchKernel(reinterpret_cast<const void *>(&dequant_mx4_kernel<TYPE>), r.grid,
                           r.block, args, 0, stream);
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
