// C ABI of w2a8_block.h: size queries, host packers and device entry points.
// Validation happens on the host before any HIP call.
#include <cmath>
#include <cstring>

#include "block.h"
#include "host_checks.h"
#include "w2a8_tuning.h"

namespace w2a8 {
namespace {

bool matrix_ok(int64_t N, int64_t K) { return N >= 1 && N <= kMaxN && K >= 1 && K <= W2A8_MAX_K; }
bool group_ok(int64_t group) { return group == 32 || group == 64 || group == 128; }

// Where the packed 4-bit weights hold value (n, k): its byte and the shift of
// its half; and the element of group g of row n among the scales.
struct W4Place {
    int64_t byte;
    int shift;
};
W4Place w4_place(int64_t n, int64_t k, int64_t KT, int64_t group) {
    const int64_t part = group, o_len = group / 4;       // a part's k and a lane's of them
    const int64_t in = k % kTileK, i = in / part, c = in % part / o_len, o = in % o_len;
    const int64_t v = o_len * i + o;
    return {((n / kW4Rows) * KT + k / kTileK) * kW4TileBytes + 16 * (16 * c + n % kW4Rows) + v / 8 * 4 + v % 4,
            v % 8 < 4 ? 0 : 4};
}
int64_t w4_group_at(int64_t n, int64_t g, int64_t GQ) {
    return (((n / kW4Rows) * GQ + g / 4) * kW4Rows + n % kW4Rows) * 4 + g % 4;
}
// Offsets of the scales and zero points, and the whole.
struct W4Size {
    int64_t scales, zeros, total;
};
W4Size w4_size(int64_t N, int64_t K, int64_t group, bool zeros) {
    const int64_t NS = ceil_div(N, kW4Rows), per = NS * w4_group_quads(K, group) * kW4Rows * 4;
    W4Size s;
    s.scales = NS * w4_tiles(K) * kW4TileBytes;
    s.zeros = s.scales + 2 * per;
    s.total = s.zeros + (zeros ? per : 0);
    return s;
}

// Space for the parts of k of the products that may split it.
int64_t w4_workspace(int64_t M, int64_t N, int64_t K) {
    return M < kW4PartRows || w4_tiles(K) < 16 ? 0 : 4 * M * N * std::min<int64_t>(kW4Parts, w4_tiles(K) / 8);
}

bool moe_ok(int64_t M, int64_t H, int64_t I, int64_t E, int64_t top_k) {
    return M >= 1 && M <= W2A8_MOE_MAX_M && H >= 1 && H <= W2A8_MAX_K && I >= 1 && I <= W2A8_MAX_K &&
           E >= 1 && E <= W2A8_MOE_MAX_E && top_k >= 1 && top_k <= E && top_k <= W2A8_MOE_MAX_TOP_K;
}

}  // namespace
}  // namespace w2a8

using namespace w2a8;

extern "C" {

int rmsnorm_quant_int8(const void *x, const void *residual, const void *weight, int type, int64_t M,
                       int64_t K, float eps, void *h, int8_t *x_q, float *s_a, void *stream) {
    if (!x || !x_q || !s_a || (residual && !h)) return W2A8_ERR_NULL;
    if (M < 1 || M > kMaxM || K < 1 || K > W2A8_MAX_K) return W2A8_ERR_SHAPE;
    if (!type_ok(type) || (h && !residual) || !(eps >= 0.0f) || !std::isfinite(eps))
        return W2A8_ERR_VALUE;
    if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(h) ||
        !aligned16(x_q) || !aligned4(s_a))
        return W2A8_ERR_ALIGN;
    const int64_t t = type_bytes(type), nx = M * K * t, nw = K * t, nq = M * K, ns = M * 4;
    // h may be x or residual itself: a lane reads what it then writes.
    const auto clear = [&](const void *y, int64_t ny) {
        return !meet(y, ny, x, nx) && !meet(y, ny, residual, nx) && !meet(y, ny, weight, nw);
    };
    if (!clear(x_q, nq) || !clear(s_a, ns) || meet(x_q, nq, s_a, ns) || meet(h, nx, x_q, nq) ||
        meet(h, nx, s_a, ns) || meet(h, nx, weight, nw) || (h != x && meet(h, nx, x, nx)) ||
        (h != residual && meet(h, nx, residual, nx)))
        return W2A8_ERR_VALUE;
    DeviceInfo dev;
    const int st = current_device(&dev);
    if (st != W2A8_OK) return st;
    const NormLaunch a = {x, residual, weight, h, x_q, s_a, eps, int(M), int(K)};
    const hipError_t e = launch_rmsnorm_quant(a, type, dev.cus, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? W2A8_OK : W2A8_ERR_LAUNCH;
}

int64_t w4a8_packed_bytes(int64_t N, int64_t K, int64_t group, int zeros) {
    return matrix_ok(N, K) && group_ok(group) ? w4_size(N, K, group, zeros != 0).total : -1;
}

int pack_w4a8(const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros, int64_t N, int64_t K,
              int64_t group, void *packed, int64_t packed_bytes) {
    if (!codes || !scales || !packed) return W2A8_ERR_NULL;
    if (!matrix_ok(N, K)) return W2A8_ERR_SHAPE;
    if (!group_ok(group)) return W2A8_ERR_VALUE;
    const W4Size z = w4_size(N, K, group, zeros != nullptr);
    if (packed_bytes < z.total) return W2A8_ERR_BUFSIZE;
    uint8_t *out = static_cast<uint8_t *>(packed);
    memset(out, 0, size_t(z.total));
    const int64_t KT = w4_tiles(K), GQ = w4_group_quads(K, group);
    const int64_t groups = ceil_div(K, group), row = ceil_div(K, 2);
    for (int64_t n = 0; n < N; ++n) {
        for (int64_t k = 0; k < K; ++k) {
            const W4Place p = w4_place(n, k, KT, group);
            const unsigned q = (codes[n * row + k / 2] >> (4 * (k & 1))) & 15u;
            out[p.byte] |= uint8_t((q ^ 8u) << p.shift);
        }
        for (int64_t g = 0; g < groups; ++g) {
            const int64_t at = w4_group_at(n, g, GQ);
            memcpy(out + z.scales + 2 * at, scales + n * groups + g, 2);
            if (!zeros) continue;
            if (zeros[n * groups + g] > 15) return W2A8_ERR_VALUE;
            out[z.zeros + at] = uint8_t(zeros[n * groups + g] - 8);
        }
    }
    return W2A8_OK;
}

int unpack_w4a8(const void *packed, int64_t packed_bytes, int64_t N, int64_t K, int64_t group,
                uint8_t *codes, uint16_t *scales, uint8_t *zeros) {
    if (!codes || !scales || !packed) return W2A8_ERR_NULL;
    if (!matrix_ok(N, K)) return W2A8_ERR_SHAPE;
    if (!group_ok(group)) return W2A8_ERR_VALUE;
    const W4Size z = w4_size(N, K, group, zeros != nullptr);
    if (packed_bytes < z.total) return W2A8_ERR_BUFSIZE;
    const uint8_t *in = static_cast<const uint8_t *>(packed);
    const int64_t KT = w4_tiles(K), GQ = w4_group_quads(K, group);
    const int64_t groups = ceil_div(K, group), row = ceil_div(K, 2);
    memset(codes, 0, size_t(N * row));
    for (int64_t n = 0; n < N; ++n) {
        for (int64_t k = 0; k < K; ++k) {
            const W4Place p = w4_place(n, k, KT, group);
            const unsigned q = ((in[p.byte] >> p.shift) & 15u) ^ 8u;
            codes[n * row + k / 2] |= uint8_t(q << (4 * (k & 1)));
        }
        for (int64_t g = 0; g < groups; ++g) {
            const int64_t at = w4_group_at(n, g, GQ);
            memcpy(scales + n * groups + g, in + z.scales + 2 * at, 2);
            if (zeros) zeros[n * groups + g] = uint8_t(in[z.zeros + at] + 8);
        }
    }
    return W2A8_OK;
}

int64_t w4a8_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (M < 1 || M > W4A8_MAX_M || !matrix_ok(N, K)) return -1;
    return w4_workspace(M, N, K);
}

int w4a8_gemm(const void *w_packed, const int8_t *x, const float *s_a, int64_t M, int64_t N, int64_t K,
              int64_t group, int scale_type, int zeros, float *y_f32, uint16_t *y_bf16, void *workspace,
              int64_t ws_bytes, void *stream) {
    if (!w_packed || !x || !s_a || (!y_f32 && !y_bf16)) return W2A8_ERR_NULL;
    if (M < 1 || M > W4A8_MAX_M || !matrix_ok(N, K)) return W2A8_ERR_SHAPE;
    if (!group_ok(group) || (scale_type != W2A8_BF16 && scale_type != W2A8_F16)) return W2A8_ERR_VALUE;
    if (!aligned16(w_packed) || !aligned16(x) || !aligned4(s_a) || !aligned16(y_f32) || !aligned16(y_bf16))
        return W2A8_ERR_ALIGN;
    const int64_t need = w4_workspace(M, N, K);
    if (need > 0) {
        if (!workspace) return W2A8_ERR_NULL;
        if (!aligned16(workspace)) return W2A8_ERR_ALIGN;
        if (ws_bytes < need) return W2A8_ERR_BUFSIZE;
    }
    const W4Size z = w4_size(N, K, group, zeros != 0);
    const auto clear = [&](const void *y, int64_t ny) {
        return !meet(y, ny, w_packed, z.total) && !meet(y, ny, x, M * K) && !meet(y, ny, s_a, M * 4);
    };
    const int64_t nf = M * N * 4, nb = M * N * 2;
    if (!clear(y_f32, nf) || !clear(y_bf16, nb) || meet(y_f32, nf, y_bf16, nb) ||
        (need > 0 && (!clear(workspace, need) || meet(workspace, need, y_f32, nf) || meet(workspace, need, y_bf16, nb))))
        return W2A8_ERR_VALUE;
    DeviceInfo dev;
    const int st = current_device(&dev);
    if (st != W2A8_OK) return st;
    W4Launch a;
    a.w = static_cast<const uint8_t *>(w_packed);
    a.scales = reinterpret_cast<const uint16_t *>(a.w + z.scales);
    a.zeros = zeros ? a.w + z.zeros : nullptr;
    a.x = x;
    a.sa = s_a;
    a.y_f32 = y_f32;
    a.y_bf16 = y_bf16;
    a.M = int(M);
    a.N = int(N);
    a.K = int(K);
    a.KT = int(w4_tiles(K));
    a.GQ = int(w4_group_quads(K, group));
    a.group = int(group);
    a.bf16_scales = scale_type == W2A8_BF16;
    a.strips = int(ceil_div(N, kW4Rows));
    a.ws = static_cast<float *>(workspace);
    a.parts = 1;
    const hipError_t e = launch_w4a8(a, dev.cus, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? W2A8_OK : W2A8_ERR_LAUNCH;
}

int64_t w2a8_moe_workspace_bytes(int64_t M, int64_t H, int64_t I, int64_t E, int64_t top_k) {
    return moe_ok(M, H, I, E, top_k) ? moe_space(M, H, I, E, top_k).total : -1;
}

int w2a8_moe(const int8_t *x, const float *s_a, const void *logits, int logit_type, const void *w_gate,
             const void *w_up, const void *w_down, const float *s_gate, const float *s_up,
             const float *s_down, int64_t M, int64_t H, int64_t I, int64_t E, int64_t top_k,
             int activation, int renormalize, float *y_f32, uint16_t *y_bf16, void *workspace,
             int64_t ws_bytes, void *stream) {
    if (!x || !s_a || !logits || !w_gate || !w_up || !w_down || !s_gate || !s_up || !s_down ||
        (!y_f32 && !y_bf16) || !workspace)
        return W2A8_ERR_NULL;
    if (!moe_ok(M, H, I, E, top_k)) return W2A8_ERR_SHAPE;
    if (!type_ok(logit_type) || (activation != W2A8_ACT_SILU && activation != W2A8_ACT_RELU2))
        return W2A8_ERR_VALUE;
    const void *const wide[] = {x, logits, w_gate, w_up, w_down, y_f32, y_bf16, workspace};
    for (const void *p : wide)
        if (!aligned16(p)) return W2A8_ERR_ALIGN;
    const void *const narrow[] = {s_a, s_gate, s_up, s_down};
    for (const void *p : narrow)
        if (!aligned4(p)) return W2A8_ERR_ALIGN;
    MoeLaunch a;
    a.sp = moe_space(M, H, I, E, top_k);
    if (ws_bytes < a.sp.total) return W2A8_ERR_BUFSIZE;
    a.wb1 = w2a8_packed_bytes(I, H);
    a.wb2 = w2a8_packed_bytes(H, I);
    // What the call writes has to be apart from what it reads and from one another.
    const struct {
        const void *p;
        int64_t n;
    } in[] = {{x, M * H}, {s_a, 4 * M}, {logits, M * E * type_bytes(logit_type)}, {w_gate, E * a.wb1},
              {w_up, E * a.wb1}, {w_down, E * a.wb2}, {s_gate, 4 * E}, {s_up, 4 * E}, {s_down, 4 * E}},
      out[] = {{y_f32, 4 * M * H}, {y_bf16, 2 * M * H}, {workspace, a.sp.total}};
    for (int i = 0; i < 3; ++i) {
        for (const auto &b : in)
            if (meet(out[i].p, out[i].n, b.p, b.n)) return W2A8_ERR_VALUE;
        for (int j = 0; j < i; ++j)
            if (meet(out[i].p, out[i].n, out[j].p, out[j].n)) return W2A8_ERR_VALUE;
    }
    DeviceInfo dev;
    const int st = current_device(&dev);
    if (st != W2A8_OK) return st;
    a.x = x;
    a.sa = s_a;
    a.logits = logits;
    a.logit_type = logit_type;
    a.w_gate = static_cast<const uint8_t *>(w_gate);
    a.w_up = static_cast<const uint8_t *>(w_up);
    a.w_down = static_cast<const uint8_t *>(w_down);
    a.s_gate = s_gate;
    a.s_up = s_up;
    a.s_down = s_down;
    a.y_f32 = y_f32;
    a.y_bf16 = y_bf16;
    a.ws = static_cast<uint8_t *>(workspace);
    a.M = int(M);
    a.H = int(H);
    a.I = int(I);
    a.E = int(E);
    a.top_k = int(top_k);
    a.act = activation;
    a.renormalize = renormalize != 0;
    const hipError_t e = launch_moe(a, dev.cus, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? W2A8_OK : W2A8_ERR_LAUNCH;
}

int w2a8_w4a8_plan(int64_t M, int64_t N, int64_t K, int64_t group, int cus, int *kernel, int *rows, int *groups,
                   int *parts) {
    if (!kernel || !rows || !groups || !parts) return W2A8_ERR_NULL;
    if (M < 1 || M > W4A8_MAX_M || !matrix_ok(N, K)) return W2A8_ERR_SHAPE;
    if (!group_ok(group) || cus < 1 || cus > 65536) return W2A8_ERR_VALUE;
    const W4Plan p = w4_plan(int(M), int(ceil_div(N, kW4Rows)), int(w4_tiles(K)), int(K), int(group), cus);
    *kernel = p.few ? 3 : p.blocks ? 2 : 1;
    *rows = p.blocks ? 16 * p.blocks : 1;
    *groups = p.groups;
    *parts = p.parts;
    return W2A8_OK;
}

int w2a8_moe_plan(int64_t M, int64_t H, int64_t I, int64_t E, int64_t top_k, int cus, int *kernel, int *up,
                  int *down) {
    if (!kernel || !up || !down) return W2A8_ERR_NULL;
    if (!moe_ok(M, H, I, E, top_k)) return W2A8_ERR_SHAPE;
    if (cus < 1 || cus > 65536) return W2A8_ERR_VALUE;
    const MoePlan p = moe_plan(M, H, I, E, top_k, cus);
    *kernel = p.one ? 1 : 2;
    *up = p.one ? 1 : p.up;
    *down = p.one ? 1 : p.down;
    return W2A8_OK;
}

int w2a8_tune_moe(int kernel) {
    if (kernel < 0 || kernel > 4) return W2A8_ERR_VALUE;
    set_moe_mode(kernel);
    return W2A8_OK;
}

}  // extern "C"
