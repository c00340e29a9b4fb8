// Launchers and shared pieces of the operators of w2a8_block.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device.h"
#include "mx4.h"
#include "w2a8_block.h"

namespace w2a8 {

// Vectors at any alignment: rows of K bytes start wherever K puts them, and
// global loads and stores of any width need no alignment on gfx950.
typedef v4u v4u_b __attribute__((aligned(1)));
typedef v2u v2u_b __attribute__((aligned(1)));
typedef v4f v4f_b __attribute__((aligned(4)));

// 16 consecutive int8 of a row of K from k on; those past K are 0.  One load of
// the 16 that end with the row at the latest, shifted; rows below 16 by bytes.
__device__ __forceinline__ v4u load_int8_tail(const int8_t *row, int k, int K) {
    uint64_t lo = 0, hi = 0;
    if (K >= 16) {
        const int at = min(k, K - 16), s = 8 * min(k - at, 16);
        const v4u v = *reinterpret_cast<const v4u_b *>(row + at);
        const uint64_t a = (uint64_t(v[1]) << 32) | v[0], b = (uint64_t(v[3]) << 32) | v[2];
        lo = s >= 128 ? 0 : s >= 64 ? b >> (s - 64) : s > 0 ? (a >> s) | (b << (64 - s)) : a;
        hi = s >= 64 ? 0 : b >> s;
    } else {
#pragma unroll 1
        for (int i = 0; k + i < K; ++i) {
            const uint64_t byte = uint64_t(uint8_t(row[k + i])) << (8 * (i & 7));
            if (i < 8)
                lo |= byte;
            else
                hi |= byte;
        }
    }
    return v4u{uint32_t(lo), uint32_t(lo >> 32), uint32_t(hi), uint32_t(hi >> 32)};
}

struct NormLaunch {
    const void *x, *residual, *weight;
    void *h;
    int8_t *xq;
    float *sa;
    float eps;
    int M, K;
};
hipError_t launch_rmsnorm_quant(const NormLaunch &a, int type, int cus, hipStream_t stream);

// Products with 4-bit weights (W4T16x128).
constexpr int kW4Rows = 16;
constexpr int kW4TileBytes = 1024;
inline int64_t w4_tiles(int64_t K) { return ceil_div(K, kTileK); }
inline int64_t w4_group_quads(int64_t K, int64_t group) { return ceil_div(ceil_div(K, group), 4); }
struct W4Launch {
    const uint8_t *w;          // codes
    const uint16_t *scales;
    const uint8_t *zeros;      // or null
    const int8_t *x;
    const float *sa;
    float *y_f32;
    uint16_t *y_bf16;
    int M, N, K, KT, GQ;
    int group, bf16_scales, strips;
    float *ws;                 // sums of parts of k, [part][M][N]
    int parts;
};
// Most parts that k is split into (and the rows from which it may be).
constexpr int kW4Parts = 8, kW4PartRows = 2;
// How a product is run (w2a8_w4a8_plan): blocks of 16 activation rows (0: the
// one-row kernel), waves of a strip or groups of waves, parts of k; few: a strip
// to a workgroup.
struct W4Plan {
    int blocks, groups, parts;
    bool few;
};
W4Plan w4_plan(int M, int strips, int KT, int K, int group, int cus);
hipError_t launch_w4a8(const W4Launch &a, int cus, hipStream_t stream);

// Mixture of experts: offsets into the workspace, all multiples of 256.
struct MoeSpace {
    int64_t picked, tops, slot, row_of, scales, code_sums, row_sums, rows, codes, hidden, part, total;
};
MoeSpace moe_space(int64_t M, int64_t H, int64_t I, int64_t E, int64_t top_k);
struct MoeLaunch {
    const int8_t *x;
    const float *sa;
    const void *logits;
    const uint8_t *w_gate, *w_up, *w_down;
    const float *s_gate, *s_up, *s_down;
    float *y_f32;
    uint16_t *y_bf16;
    uint8_t *ws;
    MoeSpace sp;
    int64_t wb1, wb2;          // bytes of an expert's w_gate or w_up, w_down
    int M, H, I, E, top_k, act, renormalize, logit_type;
};
// How a mixture is run (w2a8_moe_plan), and the knob over it (w2a8_tune_moe).
struct MoePlan {
    bool one;           // a token at a time
    int up, down;       // together: strips of a workgroup
};
MoePlan moe_plan(int64_t M, int64_t H, int64_t I, int64_t E, int64_t top_k, int cus);
int moe_mode();
void set_moe_mode(int mode);
hipError_t launch_moe(const MoeLaunch &a, int cus, hipStream_t stream);

}  // namespace w2a8
