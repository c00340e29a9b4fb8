// C ABI of the MX4 rows, weights and products (w2a8_mx4.h): size queries,
// host packers and device entry points.  Validation happens on the host
// before any HIP call.
#include <cstring>

#include "mx4.h"
#include "w2a8_tuning.h"

namespace w2a8 {
namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool rows_ok(int64_t M, int64_t K) { return M >= 1 && M <= kMaxM && K >= 1 && K <= W2A8_MAX_K; }
bool matrix_ok(int64_t N, int64_t K) { return N >= 1 && N <= kMaxN && K >= 1 && K <= W2A8_MAX_K; }
bool type_ok(int t) { return t == W2A8_F32 || t == W2A8_BF16 || t == W2A8_F16; }

// Do two buffers share bytes?  A kernel reads what others of its workgroups
// have written by then, so outputs have to be apart from all other buffers.
bool meet(const void *a, int64_t na, const void *b, int64_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && x < y + uint64_t(nb) && y < x + uint64_t(na);
}
int64_t type_bytes(int type) { return type == W2A8_F32 ? 4 : 2; }

// Byte and half of value i (0..31) of a block's 16 code bytes.
int code_byte(int i) { return (i / 16) * 8 + (i % 16 / 4 % 2) * 4 + i % 4; }
int code_shift(int i) { return i % 16 >= 8 ? 4 : 0; }

// Offsets in the packed weights of a block's codes and scale byte.
struct Place {
    int64_t codes, scale;
};
Place place(int64_t n, int64_t b, int64_t NS, int64_t KT, int64_t KU) {
    const int64_t s = n / kMxRows, t = b / 4, l = 16 * (b % 4) + n % kMxRows;
    return {(s * KT + t) * kMxTileBytes + 16 * l,
            NS * KT * kMxTileBytes + (s * KU + t / kMxQuad) * 256 + 4 * l + t % kMxQuad};
}

// Rows of activations up to which the weight stream serves a product.  It
// reads every weight once, but every strip reads all rows: with many weight
// rows to a CU the tiles of the other kernel share them, and where strips
// are a few more than CUs, and long, they fall behind its split of k.
// Measured (MI355X, us, stream and tiles): 13824 x 2560, M = 32: MX4 7.5 and
// 9.1, ternary 5.7 and 6.9; 55296 x 5120: MX4, M = 4, 16 and 32: 32.2 and 32.3,
// 36.7 and 33.0, 46.0 and 34.4; ternary, M = 16, 17 and 32: 16.7 and 19.9, 21.7
// and 20.2, 27.1 and 20.5; 27648 columns, MX4, 320 strips, M = 16, 24 and 32:
// 25.4 and 32.3, 32.0 and 29.9, 35.8 and 31.2, 256 strips: 17.1 and 30.8, 19.5
// and 27.5, 20.9 and 29.4; ternary, 320 strips, M = 32: 34.7 and 31.1.  With
// three and five strips to a compute unit and k = 27648, MX4, the two are close:
// M = 24: 43.6 and 47.6, 80.1 and 79.3, M = 32: 48.8 and 50.7, 87.9 and 84.6.
// The limits are coarse where a matrix is larger still.  On the stream's side
// of them, but faster in tiles: 40000 columns, MX4, M = 32: k = 13824 86.5 and
// 72.1, 27648 165 and 134.  In tiles, but faster in the stream: 40960 x 2560,
// MX4, M = 8 and 16: 13.4 and 16.1, 14.1 and 17.0; ternary, M = 17: 10.9 and
// 12.7.
int stream_rows(const Mx4Launch &a, int cus) {
    const bool ternary = !a.ws;
    if (a.N >= 160 * int64_t(cus)) return ternary ? 16 : 4;
    const int64_t strips = ceil_div(a.N, ternary ? kTileRows : kMxRows);
    return a.KU >= 40 && strips > cus && strips <= 2 * cus ? 16 : kMx4StreamRows;
}

// Shared by the four product entry points.  x_type < 0: MX4R rows.
int product(const void *w, bool ternary, const uint8_t *xq, const uint8_t *xs, const void *x,
            int x_type, int64_t M, int64_t N, int64_t K, float s_w, float *y_f32, uint16_t *y_bf16,
            void *stream) {
    const bool rows = x_type < 0;
    if (!w || (rows ? !xq || !xs : !x) || (!y_f32 && !y_bf16)) return W2A8_ERR_NULL;
    if (!rows_ok(M, K) || !matrix_ok(N, K)) return W2A8_ERR_SHAPE;
    if (!rows && !type_ok(x_type)) return W2A8_ERR_VALUE;
    if (!aligned16(w) || !aligned16(xq) || !aligned16(xs) || !aligned16(x) || !aligned16(y_f32) ||
        !aligned16(y_bf16))
        return W2A8_ERR_ALIGN;
    const int64_t nw = ternary ? ceil_div(N, kTileRows) * mx4_tiles(K) * 1024 : mx4_packed_bytes(N, K);
    const int64_t nq = M * mx4_tiles(K) * kMxRowTile, ns = M * mx4_quads(K) * 16;
    const int64_t nx = rows ? 0 : K * type_bytes(x_type);
    const auto clear = [&](const void *y, int64_t ny) {
        return !meet(y, ny, w, nw) && !meet(y, ny, xq, nq) && !meet(y, ny, xs, ns) &&
               !meet(y, ny, x, nx);
    };
    if (!clear(y_f32, M * N * 4) || !clear(y_bf16, M * N * 2) ||
        meet(y_f32, M * N * 4, y_bf16, M * N * 2))
        return W2A8_ERR_VALUE;
    DeviceInfo dev;
    const int st = current_device(&dev);
    if (st != W2A8_OK) return st;
    Mx4Launch a;
    a.KT = int(mx4_tiles(K));
    a.KU = int(mx4_quads(K));
    a.w = static_cast<const uint8_t *>(w);
    a.ws = ternary ? nullptr : a.w + ceil_div(N, kMxRows) * a.KT * kMxTileBytes;
    a.xq = xq;
    a.xs = xs;
    a.x = x;
    a.y_f32 = y_f32;
    a.y_bf16 = y_bf16;
    a.sw = s_w;
    a.M = int(M);
    a.N = int(N);
    a.K = int(K);
    a.strips = a.stages = 0;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = !rows                             ? launch_mx4_fused(a, x_type, dev.cus, s)
                         : M <= stream_rows(a, dev.cus) ? launch_mx4_stream(a, dev.cus, s)
                                                        : launch_mx4_gemm(a, dev.cus, s);
    return e == hipSuccess ? W2A8_OK : W2A8_ERR_LAUNCH;
}

}  // namespace
}  // namespace w2a8

using namespace w2a8;

extern "C" {

int64_t mx4_act_bytes(int64_t M, int64_t K) {
    return rows_ok(M, K) ? M * mx4_tiles(K) * kMxRowTile : -1;
}

int64_t mx4_scale_bytes(int64_t M, int64_t K) { return rows_ok(M, K) ? M * mx4_quads(K) * 16 : -1; }

int64_t mx4_packed_bytes(int64_t N, int64_t K) {
    if (!matrix_ok(N, K)) return -1;
    return ceil_div(N, kMxRows) * (mx4_tiles(K) * kMxTileBytes + mx4_quads(K) * 256);
}

int pack_mx4(const uint8_t *codes, const uint8_t *scales, int64_t N, int64_t K, void *packed,
             int64_t packed_bytes) {
    if (!codes || !scales || !packed) return W2A8_ERR_NULL;
    const int64_t need = mx4_packed_bytes(N, K);
    if (need < 0) return W2A8_ERR_SHAPE;
    if (packed_bytes < need) return W2A8_ERR_BUFSIZE;
    uint8_t *out = static_cast<uint8_t *>(packed);
    memset(out, 0, size_t(need));
    const int64_t NS = ceil_div(N, kMxRows), KT = mx4_tiles(K), KU = mx4_quads(K);
    const int64_t blocks = ceil_div(K, 32), row = ceil_div(K, 2);
    for (int64_t n = 0; n < N; ++n)
        for (int64_t b = 0; b < blocks; ++b) {
            const Place p = place(n, b, NS, KT, KU);
            out[p.scale] = scales[n * blocks + b];
            for (int i = 0; i < 32 && 32 * b + i < K; ++i) {
                const int64_t k = 32 * b + i;
                const unsigned c = (codes[n * row + k / 2] >> (4 * (k & 1))) & 15u;
                out[p.codes + code_byte(i)] |= uint8_t(c << code_shift(i));
            }
        }
    return W2A8_OK;
}

int unpack_mx4(const void *packed, int64_t packed_bytes, int64_t N, int64_t K, uint8_t *codes,
               uint8_t *scales) {
    if (!codes || !scales || !packed) return W2A8_ERR_NULL;
    const int64_t need = mx4_packed_bytes(N, K);
    if (need < 0) return W2A8_ERR_SHAPE;
    if (packed_bytes < need) return W2A8_ERR_BUFSIZE;
    const uint8_t *in = static_cast<const uint8_t *>(packed);
    const int64_t NS = ceil_div(N, kMxRows), KT = mx4_tiles(K), KU = mx4_quads(K);
    const int64_t blocks = ceil_div(K, 32), row = ceil_div(K, 2);
    memset(codes, 0, size_t(N * row));
    for (int64_t n = 0; n < N; ++n)
        for (int64_t b = 0; b < blocks; ++b) {
            const Place p = place(n, b, NS, KT, KU);
            scales[n * blocks + b] = in[p.scale];
            for (int i = 0; i < 32 && 32 * b + i < K; ++i) {
                const int64_t k = 32 * b + i;
                const unsigned c = (in[p.codes + code_byte(i)] >> code_shift(i)) & 15u;
                codes[n * row + k / 2] |= uint8_t(c << (4 * (k & 1)));
            }
        }
    return W2A8_OK;
}

int quant_act_mx4(const void *x, int x_type, int64_t M, int64_t K, uint8_t *x_q, uint8_t *x_s,
                  void *stream) {
    if (!x || !x_q || !x_s) return W2A8_ERR_NULL;
    if (!rows_ok(M, K)) return W2A8_ERR_SHAPE;
    if (!type_ok(x_type)) return W2A8_ERR_VALUE;
    if (!aligned16(x) || !aligned16(x_q) || !aligned16(x_s)) return W2A8_ERR_ALIGN;
    const int64_t nx = M * K * type_bytes(x_type), nq = mx4_act_bytes(M, K), ns = mx4_scale_bytes(M, K);
    if (meet(x, nx, x_q, nq) || meet(x, nx, x_s, ns) || meet(x_q, nq, x_s, ns)) return W2A8_ERR_VALUE;
    DeviceInfo dev;
    const int st = current_device(&dev);
    if (st != W2A8_OK) return st;
    const hipError_t e =
        launch_quant_mx4(x, x_type, M, int(K), x_q, x_s, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? W2A8_OK : W2A8_ERR_LAUNCH;
}

int dequant_act_mx4(const uint8_t *x_q, const uint8_t *x_s, int64_t M, int64_t K, void *y,
                    int y_type, void *stream) {
    if (!x_q || !x_s || !y) return W2A8_ERR_NULL;
    if (!rows_ok(M, K)) return W2A8_ERR_SHAPE;
    if (!type_ok(y_type)) return W2A8_ERR_VALUE;
    if (!aligned16(x_q) || !aligned16(x_s) || !aligned16(y)) return W2A8_ERR_ALIGN;
    const int64_t ny = M * K * type_bytes(y_type);
    if (meet(y, ny, x_q, mx4_act_bytes(M, K)) || meet(y, ny, x_s, mx4_scale_bytes(M, K)))
        return W2A8_ERR_VALUE;
    DeviceInfo dev;
    const int st = current_device(&dev);
    if (st != W2A8_OK) return st;
    const hipError_t e =
        launch_dequant_mx4(x_q, x_s, M, int(K), y, y_type, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? W2A8_OK : W2A8_ERR_LAUNCH;
}

int quant_pack_mx4(const void *W, int w_type, int64_t N, int64_t K, void *w_packed,
                   int64_t packed_bytes, void *stream) {
    if (!W || !w_packed) return W2A8_ERR_NULL;
    const int64_t need = mx4_packed_bytes(N, K);
    if (need < 0) return W2A8_ERR_SHAPE;
    if (!type_ok(w_type)) return W2A8_ERR_VALUE;
    if (!aligned16(W) || !aligned16(w_packed)) return W2A8_ERR_ALIGN;
    if (packed_bytes < need) return W2A8_ERR_BUFSIZE;
    if (meet(W, N * K * type_bytes(w_type), w_packed, need)) return W2A8_ERR_VALUE;
    DeviceInfo dev;
    const int st = current_device(&dev);
    if (st != W2A8_OK) return st;
    const hipError_t e = launch_quant_pack_mx4(W, w_type, N, int(K), static_cast<uint8_t *>(w_packed),
                                               static_cast<hipStream_t>(stream));
    return e == hipSuccess ? W2A8_OK : W2A8_ERR_LAUNCH;
}

int w4mx4_gemm(const void *w_packed, const uint8_t *x_q, const uint8_t *x_s, int64_t M, int64_t N,
               int64_t K, float *y_f32, uint16_t *y_bf16, void *stream) {
    return product(w_packed, false, x_q, x_s, nullptr, -1, M, N, K, 1.0f, y_f32, y_bf16, stream);
}

int w2mx4_gemm(const void *w_packed, const uint8_t *x_q, const uint8_t *x_s, int64_t M, int64_t N,
               int64_t K, float s_w, float *y_f32, uint16_t *y_bf16, void *stream) {
    return product(w_packed, true, x_q, x_s, nullptr, -1, M, N, K, s_w, y_f32, y_bf16, stream);
}

int w2a8_mx4_plan(int64_t M, int64_t N, int64_t K, int ternary, int outputs, int cus, int *kernel,
                  int *rows, int *cols, int *groups, int *pass) {
    if (!kernel || !rows || !cols || !groups || !pass) return W2A8_ERR_NULL;
    if (!rows_ok(M, K) || !matrix_ok(N, K)) return W2A8_ERR_SHAPE;
    if (cus < 1 || cus > 65536 || outputs < 1 || outputs > 3) return W2A8_ERR_VALUE;
    // (The plans ask whether there are MX4 scales and which outputs, not where.)
    alignas(16) static uint8_t some[16];
    Mx4Launch a = {};
    a.KT = int(mx4_tiles(K));
    a.KU = int(mx4_quads(K));
    a.ws = ternary ? nullptr : some;
    a.y_f32 = outputs & 1 ? reinterpret_cast<float *>(some) : nullptr;
    a.y_bf16 = outputs & 2 ? reinterpret_cast<uint16_t *>(some) : nullptr;
    a.M = int(M);
    a.N = int(N);
    a.K = int(K);
    if (M <= stream_rows(a, cus)) {
        *kernel = 1;
        *rows = M == 1 ? 1 : M <= 16 ? 16 : 32;
        *cols = ternary ? kTileRows : kMxRows;
        *groups = mx4_stream_waves(a.M, int(ceil_div(N, *cols)), a.KU, cus);
        *pass = 0;
        return W2A8_OK;
    }
    const Mx4TilePlan p = mx4_tile_plan(a, cus);
    *kernel = 2;
    *rows = p.BM;
    *cols = p.BN;
    *groups = p.KS;
    *pass = p.pass;
    return W2A8_OK;
}

int w4mx4_linear_gemv(const void *w_packed, const void *x, int x_type, int64_t N, int64_t K,
                      float *y_f32, uint16_t *y_bf16, void *stream) {
    // An unknown type must not read as "rows".
    return product(w_packed, false, nullptr, nullptr, x, x_type < 0 ? 99 : x_type, 1, N, K, 1.0f,
                   y_f32, y_bf16, stream);
}

int w2mx4_linear_gemv(const void *w_packed, const void *x, int x_type, int64_t N, int64_t K,
                      float s_w, float *y_f32, uint16_t *y_bf16, void *stream) {
    return product(w_packed, true, nullptr, nullptr, x, x_type < 0 ? 99 : x_type, 1, N, K, s_w,
                   y_f32, y_bf16, stream);
}

}  // extern "C"
