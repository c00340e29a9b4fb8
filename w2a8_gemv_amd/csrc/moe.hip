// Mixture of ternary experts for a few tokens (gfx950): the layer of w2a8_moe.
//
// One token at a time, two launches (few tokens, which share few experts):
//   up_one    routes inside every workgroup; hidden = act(g) * u of one expert
//   down_one  hidden to int8 in every workgroup, w_down of all the token's
//             experts, and their weighted sum
// Token rows together, five launches (more tokens):
//   route     every token's experts and weights, every expert's tokens: pairs
//             (token, expert) in the order of experts; rows padded to tiles
//   up        hidden[pair]          quant  hidden to int8
//   down      part[token][rank]     combine  y[token], ranks in order
//
// All sums of products are integers, so how they are split and joined does
// not show.  Weights are in the T32x128 layout, one matrix an expert.
#include <atomic>

#include "block.h"

namespace w2a8 {
namespace {

constexpr int kMoeRows = 16;       // tokens of a pass of the matrix kernels
constexpr int kMoeWaves = 4;       // waves of a workgroup of them
constexpr int kRouteThreads = 1024;
constexpr int kRouteWaves = kRouteThreads / 64;
constexpr int kRouteTokens = W2A8_MOE_MAX_M / kRouteWaves;   // of a wave
constexpr int kPerLane = W2A8_MOE_MAX_E / 64;

// What the route leaves behind.
struct Slot {
    int expert, begin;                  // -1: none; the first of its pairs
    uint32_t mask[2];                   // its tokens
};
struct Picked {                         // [token][rank]
    int expert;                         // -1: none, -2: a broken token
    float weight;
};

// ---------------------------------------------------------------------------
// Routing
// ---------------------------------------------------------------------------
// Order of floats as unsigned integers; 0 stands for an expert that cannot be taken.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(v);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
    v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0xB1, 0xF, 0xF, false)));
    v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x4E, 0xF, 0xF, false)));
    v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x124, 0xF, 0xF, false)));
    v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x128, 0xF, 0xF, false)));
    const uint32_t a = uint32_t(__builtin_amdgcn_readlane(int(v), 0)), b = uint32_t(__builtin_amdgcn_readlane(int(v), 16));
    const uint32_t c = uint32_t(__builtin_amdgcn_readlane(int(v), 32)), d = uint32_t(__builtin_amdgcn_readlane(int(v), 48));
    return max(max(a, b), max(c, d));
}
__device__ __forceinline__ float wave_sum_f32(float v) {
    for (int o = 1; o < 64; o *= 2) v += __shfl_xor(v, o);
    return v;
}
__device__ __forceinline__ float logit(const MoeLaunch &a, int64_t i) {
    return a.logit_type == W2A8_F32    ? mx4_load1<W2A8_F32>(a.logits, i)
           : a.logit_type == W2A8_BF16 ? mx4_load1<W2A8_BF16>(a.logits, i)
                                       : mx4_load1<W2A8_F16>(a.logits, i);
}

// A token's logits over the lanes of a wave: expert lane + 64 i.
struct Router {
    float l[kPerLane];
    uint32_t key[kPerLane];
    bool bad;

    __device__ __forceinline__ void load(const MoeLaunch &a, int m, int lane) {
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) {
            const int e = lane + 64 * i;
            l[i] = -__builtin_inff();
            if (e < a.E) l[i] = logit(a, int64_t(m) * a.E + e);
        }
    }
    __device__ __forceinline__ void keys() {
        bool b = false;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) {
            b |= !(l[i] < __builtin_inff());
            key[i] = l[i] == -__builtin_inff() ? 0u : order_key(l[i] + 0.0f);   // (-0 ties with 0)
        }
        bad = __any(b);
    }
    // The next expert by rank (-1: none is left) and its logit.
    __device__ __forceinline__ int next(int E, int lane, float *value) {
        uint32_t best = key[0];
        if (E > 64) {
#pragma unroll
            for (int i = 1; i < kPerLane; ++i) best = max(best, key[i]);
        }
        best = wave_max_u32(best);
        if (best == 0 || bad) return -1;
        *value = key_value(best);
        // The first 64 experts that hold it, and the first lane of them.
        uint64_t hit = __ballot(key[0] == best);
        int e = __builtin_ctzll(hit);
        if (E > 64) {
#pragma unroll
            for (int i = 1; i < kPerLane; ++i) {
                const uint64_t more = __ballot(key[i] == best);
                if (!hit) {
                    e = 64 * i + __builtin_ctzll(more);
                    hit = more;
                }
            }
#pragma unroll
            for (int i = 1; i < kPerLane; ++i)
                if (lane + 64 * i == e) key[i] = 0;
        }
        if (lane == e) key[0] = 0;
        return e;
    }
    // All ranks: lane j is left with rank j's expert and weight.
    __device__ __forceinline__ void all(const MoeLaunch &a, int lane, int *expert, float *weight) {
        float top = 0.0f, sum = 0.0f, whole = 0.0f;
        *expert = bad ? -2 : -1;
        *weight = 0.0f;
        for (int j = 0; j < a.top_k; ++j) {
            float v;
            const int e = next(a.E, lane, &v);
            if (e < 0) break;
            if (j == 0) {
                top = v;
#pragma unroll
                for (int i = 0; i < kPerLane; ++i) whole += expf(l[i] - top);
                if (!a.renormalize) whole = wave_sum_f32(whole);
            }
            const float p = expf(v - top);
            sum += p;
            if (lane == j) {
                *expert = e;
                *weight = p;
            }
        }
        if (*expert >= 0) *weight /= a.renormalize ? sum : whole;
    }
};

// ---------------------------------------------------------------------------
// One token at a time
// ---------------------------------------------------------------------------
// Lane l of a wave reads 16 bytes of a step of eight tiles: tile l / 8, k-part
// l % 8, four weight rows (a slice of 128 bytes a tile).  Codes c = w + 1
// against activations by dot products, less the activations' sum; masks leave
// c, 4c and 16c, divided out at the end.
struct Dots {
    int a1[4], a4[4], a16[4];

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int q = 0; q < 4; ++q) a1[q] = a4[q] = a16[q] = 0;
    }
    __device__ __forceinline__ void add(v4u w, v4u x) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            a1[q] = dot4(w[q] & 0x03030303u, x[0], a1[q]);
            a4[q] = dot4(w[q] & 0x0C0C0C0Cu, x[1], a4[q]);
            a16[q] = dot4(w[q] & 0x30303030u, x[2], a16[q]);
            a16[q] = dot4((w[q] >> 2) & 0x30303030u, x[3], a16[q]);
        }
    }
    // Row q's sum over the 8 k-parts of a tile.
    __device__ __forceinline__ int row(int q) const { return sum8(a1[q] + (a4[q] >> 2) + (a16[q] >> 4)); }
    // The same less the activations' (sx, a lane's), row kg, and of `other` row kg - 4.
    __device__ __forceinline__ int rows(int sx, int kg, const Dots &other) const {
        int v = row(0);
#pragma unroll
        for (int q = 1; q < 8; ++q) {
            const int n = q < 4 ? row(q) : other.row(q - 4);
            v = kg == q ? n : v;
        }
        return v - sum8(sx);
    }
};
// Sum over the eight tiles of a step: lanes of the same k-part.
__device__ __forceinline__ int sum_over_tiles(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x128, 0xF, 0xF, false);   // row_ror:8
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}
__device__ __forceinline__ int add16(v4u x, int s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s = dot4(x[i], 0x01010101u, s);
    return s;
}

// A g that is not finite gives no finite value: silu of it is infinite or NaN by
// its own steps, and relu, whose maximum drops a NaN and -infinity, has 0 * g for it.
__device__ __forceinline__ float activate(int act, float g, float u) {
    if (act == W2A8_ACT_SILU) return (g / (1.0f + expf(-g))) * u;
    const float p = fmaxf(g, 0.0f) + 0.0f * g;
    return (p * p) * u;
}

// Workgroup (strip, rank, token) of eight waves, one slice of four rows each (the
// strip past the last only routes).
// A wave's loads are its own, so nothing is shared but the strip's largest
// hidden value.  Every wave routes by itself: up to `rank` + 1 maxima.
constexpr int kOneDepth = 3;

__global__ __launch_bounds__(512) void moe_up_one_kernel(MoeLaunch a) {
    __shared__ uint32_t most[8];
    const int s = int(blockIdx.x), rank = int(blockIdx.y), m = int(blockIdx.z);
    const int lane = int(threadIdx.x) & 63;
    const int sl = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    Router route;
    route.load(a, m, lane);
    route.keys();
    const int strips = int(gridDim.x) - 1;
    if (s == strips) {
        // What the second launch needs of the route, once a token.
        if (rank > 0 || sl > 0) return;
        int expert;
        float weight;
        route.all(a, lane, &expert, &weight);
        Picked *out = reinterpret_cast<Picked *>(a.ws + a.sp.picked) + m * a.top_k;
        if (lane < a.top_k) out[lane] = Picked{expert, weight};
        return;
    }
    int e = -1;
    float v;
    for (int j = 0; j <= rank; ++j) e = route.next(a.E, lane, &v);
    if (e < 0) return;      // (the same for all waves)
    const int pair = m * a.top_k + rank;
    float *tops = reinterpret_cast<float *>(a.ws + a.sp.tops);
    {
        const float sa = a.sa[m], sg = a.s_gate[e], su = a.s_up[e];
        const int u = lane >> 3, kg = lane & 7;
        const int KT = (a.H + kTileK - 1) / kTileK, nst = (KT + 7) / 8;
        const int64_t off = int64_t(e) * a.wb1 + int64_t(s) * KT * kTileBytes + 16 * (8 * sl + kg);
        const uint8_t *wg = a.w_gate + off, *wu = a.w_up + off;
        const int8_t *x = a.x + int64_t(m) * a.H;
        v4u g[kOneDepth], p[kOneDepth], xv[kOneDepth];
        auto load = [&](int i, int d) __attribute__((always_inline)) {
            const int t = 8 * i + u, at = min(t, KT - 1) * kTileBytes;
            g[d] = __builtin_nontemporal_load(reinterpret_cast<const v4u *>(wg + at));
            p[d] = __builtin_nontemporal_load(reinterpret_cast<const v4u *>(wu + at));
            const int k = t * kTileK + 16 * kg;
            xv[d] = v4u{0u, 0u, 0u, 0u};
            if (k + 16 <= a.H) {
                xv[d] = *reinterpret_cast<const v4u_b *>(x + k);
            } else if (k < a.H) {
                xv[d] = load_int8_tail(x, k, a.H);
            }
        };
        Dots dg, du;
        dg.clear();
        du.clear();
        int sx = 0;
#pragma unroll
        for (int d = 0; d < kOneDepth; ++d)
            if (d < nst) load(d, d);
        for (int i = 0; i < nst; i += kOneDepth) {
#pragma unroll
            for (int d = 0; d < kOneDepth; ++d) {
                if (i + d < nst) {
                    sx = add16(xv[d], sx);
                    dg.add(g[d], xv[d]);
                    du.add(p[d], xv[d]);
                }
                if (i + d + kOneDepth < nst) load(i + d + kOneDepth, d);
            }
        }
        // Lane kg of eight takes row kg % 4 of the gate's or the up weights' sums;
        // lanes 0 .. 3 then have the wave's.
        const int v = sum_over_tiles(dg.rows(sx, kg, du));
        const int up = __builtin_amdgcn_ds_swizzle(v, 0x101F);      // lane ^ 4
        const float h = activate(a.act, (float(v) * sa) * sg, (float(up) * sa) * su);
        const int row = s * kTileRows + 4 * sl + lane;
        const bool mine = lane < 4 && row < a.I;
        if (mine) reinterpret_cast<float *>(a.ws + a.sp.hidden)[int64_t(pair) * a.I + row] = h;
        const uint32_t top = wave_max_u32(mine ? __float_as_uint(h) & 0x7FFFFFFFu : 0u);
        if (lane == 0) most[sl] = top;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        uint32_t t = most[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) t = max(t, most[i]);
        tops[int64_t(pair) * strips + s] = __uint_as_float(t);
    }
}

// Four fp32 of a row to codes, values past the row 0.
__device__ __forceinline__ v4f load4(const float *h, int k, int K) {
    v4f f = {0.0f, 0.0f, 0.0f, 0.0f};
    if (k + 4 <= K) return *reinterpret_cast<const v4f_b *>(h + k);
#pragma unroll
    for (int i = 0; i < 3; ++i)
        if (k + i < K) f[i] = h[k + i];
    return f;
}
__device__ __forceinline__ uint32_t codes4(v4f f, float inv) {
    return q8(f[0], inv) | (q8(f[1], inv) << 8) | (q8(f[2], inv) << 16) | (q8(f[3], inv) << 24);
}
// The factor of the codes and the scale of a row of largest magnitude `top`
// (a row that is not finite has no codes: NaN).
__device__ __forceinline__ float code_factor(float top) {
    return top == 0.0f || !(top < __builtin_inff()) ? 0.0f : fminf(127.0f / top, __FLT_MAX__);
}
__device__ __forceinline__ float code_scale(float top) {
    return top < __builtin_inff() ? top / 127.0f : __builtin_nanf("");
}

// Workgroup (16 rows of y, token) of 16 waves: wave w takes slice w % 4 of the
// rows and quarter w / 4 of the steps of all the token's experts.  Every
// workgroup rounds all of the token's hidden rows, which is as many bytes to
// read as its weights: eight rows to a workgroup made it slower (8 experts of
// 2560 x 6912, two taken, both launches: 16.9 us, 16 rows 15.2, 32 rows 17.1;
// with eight waves 16.0).
constexpr int kDownDepth = 4;       // steps that a wave's weights are asked for ahead
constexpr int kDownAhead = 4;       // groups of four hidden values that a lane loads ahead
constexpr int kDownThreads = 1024, kDownWaves = kDownThreads / 64;
constexpr int kDownSlices = 4, kDownParts = kDownWaves / kDownSlices, kDownRows = 4 * kDownSlices;

__global__ __launch_bounds__(kDownThreads) void moe_down_one_kernel(MoeLaunch a) {
    extern __shared__ __attribute__((aligned(16))) int8_t q[];     // [rank][tiles * 128]
    __shared__ float factor[W2A8_MOE_MAX_TOP_K], scale[W2A8_MOE_MAX_TOP_K];
    __shared__ int sums[W2A8_MOE_MAX_TOP_K][kDownRows];
    const int m = int(blockIdx.y), tid = int(threadIdx.x), lane = tid & 63;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6), part = wv / kDownSlices, slice = wv % kDownSlices;
    const int KT = (a.I + kTileK - 1) / kTileK, nst = (KT + 7) / 8, stride = KT * kTileK;
    const Picked *picked = reinterpret_cast<const Picked *>(a.ws + a.sp.picked) + m * a.top_k;
    const float *hidden = reinterpret_cast<const float *>(a.ws + a.sp.hidden) + int64_t(m) * a.top_k * a.I;
    const int strips = (a.I + kTileRows - 1) / kTileRows;
    const float *tops = reinterpret_cast<const float *>(a.ws + a.sp.tops) + int64_t(m) * a.top_k * strips;
    Picked mine = {-1, 0.0f};
    if (lane < a.top_k) mine = picked[lane];

    // Hidden values, four at a time over all ranks: the first ones now.
    const int per = stride / 4, groups = a.top_k * per;
    v4f ahead[kDownAhead];
#pragma unroll
    for (int i = 0; i < kDownAhead; ++i) {
        const int g = tid + kDownThreads * i, j = g / per;
        if (g < groups) ahead[i] = load4(hidden + int64_t(j) * a.I, 4 * (g - j * per), a.I);
    }
    // Each rank's largest hidden value, from the strips': a rank a wave.
    static_assert(W2A8_MOE_MAX_TOP_K <= kDownWaves);
    uint32_t most = 0;
    if (wv < a.top_k)
        for (int n = lane; n < strips; n += 64) most = max(most, __float_as_uint(tops[int64_t(wv) * strips + n]));
    if (tid < W2A8_MOE_MAX_TOP_K * kDownRows) (&sums[0][0])[tid] = 0;

    // This wave's steps, and the first of its weights.
    const int ranks = __popcll(__ballot(mine.expert >= 0));
    const int total = ranks * nst, u0 = total * part / kDownParts, u1 = total * (part + 1) / kDownParts;
    const int u = lane >> 3, kg = lane & 7;
    const int s = int(blockIdx.x) / (8 / kDownSlices), sl = kDownSlices * (int(blockIdx.x) % (8 / kDownSlices)) + slice;
    const uint8_t *wd = a.w_down + int64_t(s) * KT * kTileBytes + 16 * (8 * sl + kg);
    v4u w[kDownDepth];
    auto load = [&](int n, int d) __attribute__((always_inline)) {
        const int j = n / nst, t = min(8 * (n - j * nst) + u, KT - 1);
        const int e = __builtin_amdgcn_readlane(mine.expert, j);
        w[d] = __builtin_nontemporal_load(reinterpret_cast<const v4u *>(wd + int64_t(e) * a.wb2 + t * kTileBytes));
    };
#pragma unroll
    for (int d = 0; d < kDownDepth; ++d)
        if (u0 + d < u1) load(u0 + d, d);

    const float sd = mine.expert >= 0 ? a.s_down[mine.expert] : 0.0f;     // of rank `lane`
    const float top = __uint_as_float(wave_max_u32(most));
    if (wv < ranks && lane == 0) {
        factor[wv] = code_factor(top);
        scale[wv] = code_scale(top);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kDownAhead; ++i) {
        const int g = tid + kDownThreads * i, j = g / per;
        if (g < groups && j < ranks) *reinterpret_cast<uint32_t *>(q + 4 * g) = codes4(ahead[i], factor[j]);
    }
    for (int g = tid + kDownThreads * kDownAhead; g < groups; g += kDownThreads) {
        const int j = g / per;
        if (j < ranks)
            *reinterpret_cast<uint32_t *>(q + 4 * g) =
                codes4(load4(hidden + int64_t(j) * a.I, 4 * (g - j * per), a.I), factor[j]);
    }
    __syncthreads();

    Dots acc;
    acc.clear();
    int sx = 0, j = u0 / nst, st = u0 - j * nst;
    auto flush = [&]() __attribute__((always_inline)) {
        const int x = sum8(sx);
        int r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = acc.row(i) - x;
        const int mine = kg == 0 ? r[0] : kg == 1 ? r[1] : kg == 2 ? r[2] : r[3];
        if (kg < 4) atomicAdd(&sums[j][4 * slice + kg], mine);
        acc.clear();
        sx = 0;
    };
    for (int n = u0; n < u1; n += kDownDepth) {
#pragma unroll
        for (int d = 0; d < kDownDepth; ++d) {
            if (n + d < u1) {
                const int t = 8 * st + u;
                v4u x = {0u, 0u, 0u, 0u};
                if (t < KT) x = *reinterpret_cast<const v4u *>(q + j * stride + t * kTileK + 16 * kg);
                sx = add16(x, sx);
                acc.add(w[d], x);
                if (++st == nst || n + d + 1 == u1) {
                    flush();
                    st = 0;
                    ++j;
                }
            }
            if (n + d + kDownDepth < u1) load(n + d + kDownDepth, d);
        }
    }
    __syncthreads();
    if (tid >= 64) return;
    const int row = kDownRows * int(blockIdx.x) + lane;
    float y = __builtin_amdgcn_readfirstlane(mine.expert) == -2 ? __builtin_nanf("") : 0.0f;
    for (int j = 0; j < ranks; ++j) {
        const float p = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(mine.weight), j));
        const float d = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(sd), j));
        if (lane < kDownRows) y += p * ((float(sums[j][lane]) * scale[j]) * d);
    }
    if (lane >= kDownRows || row >= a.H) return;
    const int64_t at = int64_t(m) * a.H + row;
    if (a.y_f32) a.y_f32[at] = y;
    if (a.y_bf16) a.y_bf16[at] = uint16_t(bf16_bits(y));
}

// ---------------------------------------------------------------------------
// Token rows together
// ---------------------------------------------------------------------------
// Sum over a workgroup.
__device__ __forceinline__ int block_sum(int *red, int v) {
    v = wave_sum(v);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0;
    for (int i = 0; i < int(blockDim.x) >> 6; ++i) v += red[i];
    return v;
}

// Block 1 + m: the experts of token m and their weights, and its row, padded
// with zeros to whole tiles (where the matrix kernel reads it without asking
// for its end), and the row's sum.  Block 0: the experts' tokens.
__global__ __launch_bounds__(kRouteThreads) void moe_route_kernel(MoeLaunch a, int slots) {
    __shared__ uint32_t mask[W2A8_MOE_MAX_E][2];      // tokens of an expert
    __shared__ int begins[W2A8_MOE_MAX_E], red[kRouteWaves];
    const int tid = int(threadIdx.x), lane = tid & 63, wv = tid >> 6;
    if (blockIdx.x > 0) {
        const int m = int(blockIdx.x) - 1, Hp = (a.H + kTileK - 1) / kTileK * kTileK;
        const int8_t *row = a.x + int64_t(m) * a.H;
        uint8_t *out = a.ws + a.sp.rows + int64_t(m) * Hp;
        if (wv == kRouteWaves - 1) {      // (the wave that has least of the row)
            Router r;
            r.load(a, m, lane);
            r.keys();
            int expert;
            float weight;
            r.all(a, lane, &expert, &weight);
            Picked *to = reinterpret_cast<Picked *>(a.ws + a.sp.picked) + m * a.top_k;
            if (lane < a.top_k) to[lane] = Picked{expert, weight};
        }
        int sum = 0;
        for (int k = 16 * tid; k < Hp; k += 16 * kRouteThreads) {
            const v4u v = k + 16 <= a.H ? v4u(*reinterpret_cast<const v4u_b *>(row + k)) : load_int8_tail(row, k, a.H);
            *reinterpret_cast<v4u *>(out + k) = v;
            sum = add16(v, sum);
        }
        sum = block_sum(red, sum);
        if (tid == 0) reinterpret_cast<int *>(a.ws + a.sp.row_sums)[m] = sum;
        return;
    }
    Slot *slot = reinterpret_cast<Slot *>(a.ws + a.sp.slot);
    int *row_of = reinterpret_cast<int *>(a.ws + a.sp.row_of);     // a pair's token * top_k + rank
    Router r[kRouteTokens];
#pragma unroll
    for (int i = 0; i < kRouteTokens; ++i)
        if (wv + i * kRouteWaves < a.M) r[i].load(a, wv + i * kRouteWaves, lane);
    if (tid < W2A8_MOE_MAX_E) mask[tid][0] = mask[tid][1] = 0;
    __syncthreads();
    int expert[kRouteTokens];           // of rank `lane`, of this wave's tokens
#pragma unroll
    for (int i = 0; i < kRouteTokens; ++i) {
        const int m = wv + i * kRouteWaves;
        expert[i] = -1;
        if (m >= a.M) continue;
        r[i].keys();
        for (int j = 0; j < a.top_k; ++j) {
            float v;
            const int e = r[i].next(a.E, lane, &v);
            if (e < 0) break;
            if (lane == j) expert[i] = e;
        }
        if (expert[i] >= 0) atomicOr(&mask[expert[i]][m >> 5], 1u << (m & 31));
    }
    __syncthreads();
    // Places of the experts' pairs and slots: sums of (pairs, experts) over
    // the experts before, in one word.  One wave, four experts a lane.
    if (wv == 0) {
        int n[kPerLane], before = 0;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) {
            const int e = kPerLane * lane + i;
            n[i] = __popc(mask[e][0]) + __popc(mask[e][1]);
            before += n[i] + (n[i] ? 1 << 16 : 0);
        }
        const int mine = before;
        for (int o = 1; o < 64; o *= 2) {
            const int up = __shfl_up(before, o);
            before += lane >= o ? up : 0;
        }
        const int used = __shfl(before, 63);
        before -= mine;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) {
            const int e = kPerLane * lane + i;
            begins[e] = before & 0xFFFF;
            if (n[i]) {
                slot[before >> 16] = Slot{e, before & 0xFFFF, {mask[e][0], mask[e][1]}};
                before += n[i] + (1 << 16);
            }
            if (e >= used >> 16 && e < slots) slot[e] = Slot{-1, 0, {0, 0}};
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRouteTokens; ++i) {
        const int m = wv + i * kRouteWaves, e = expert[i];
        if (e < 0) continue;
        const uint32_t lo = mask[e][0], hi = mask[e][1];
        const int at = begins[e] + (m < 32 ? __popc(lo & ((1u << m) - 1u))
                                           : __popc(lo) + __popc(hi & ((1u << (m - 32)) - 1u)));
        row_of[at] = m * a.top_k + lane;
    }
}

// The matrix instruction (16x16x64, int8) takes activation rows as its first
// operand and weight rows as its second: lane (r, c) brings row r and the 16
// bytes of k-part c of both, and holds results of weight row r and activation
// rows 4c .. 4c + 3.  A T32x128 slot holds four rows of 16 k.  Lane r stands for
// rows 2r and 2r + 1 of the strip and reads the slot of row group r / 2 and
// k-part c + 4 (r % 2): its own two rows of one half of k, and two rows of its
// neighbour's, which has those that it lacks.  A wave so reads a whole tile in
// one load of 16 bytes a lane (64 tokens, 16 experts of 5120 x 6912: up 48 us,
// down 27; with 8 bytes a lane, half a line at a time, 62 and 37 where this had
// 51 and 29).  The instruction multiplies the codes w + 1 as they are; the sums
// are less the row's sum at the end.
typedef v4u Words;
__device__ __forceinline__ Words load_words(const uint8_t *w) {
    return __builtin_nontemporal_load(reinterpret_cast<const v4u *>(w));
}
__device__ __forceinline__ int words_at(int r, int c) { return 16 * (8 * (r >> 1) + c + 4 * (r & 1)); }
__device__ __forceinline__ uint32_t beside(uint32_t v) {      // lane ^ 1
    return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0xB1, 0xF, 0xF, false));
}
// The 16 codes w + 1 of a word as bytes, in the order of k.
__device__ __forceinline__ v4i code_bytes(uint32_t w) {
    return v4i{int(w & 0x03030303u), int((w >> 2) & 0x03030303u), int((w >> 4) & 0x03030303u),
               int((w >> 6) & 0x03030303u)};
}
__device__ __forceinline__ void add_tile(const Words &w, const v4u (&x)[2], v4i (&acc)[2]) {
    const bool odd = threadIdx.x & 1;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint32_t lo = beside(w[2 + j]), hi = beside(w[j]);
        const uint32_t h[2] = {odd ? lo : w[j], odd ? w[2 + j] : hi};
#pragma unroll
        for (int i = 0; i < 2; ++i)
            acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(v4i, x[i]), code_bytes(h[i]), acc[j], 0, 0, 0);
    }
}

// Sums over tiles wv, wv + kMoeWaves, ... of a strip of MATS matrices, against row x
// (padded to whole tiles), a wave's tiles asked for D ahead.  Compiled, a round of
// D begins with a wait for every load of the round before, its last one among them,
// so that other waves hide the latency more than D does (64 tokens: 38% of the waves'
// cycles are waits, at 5.9 TB/s; 13 tokens 46%, at 3.7).
template <int MATS, int D>
__device__ __forceinline__ void strip_sums(const uint8_t *const (&w)[MATS], const int8_t *x, int KT, int wv,
                                           v4i (&acc)[MATS][2]) {
    Words d[D][MATS];
    v4u xv[D][2];
    const int n = wv < KT ? (KT - wv + kMoeWaves - 1) / kMoeWaves : 0;
    auto load = [&](int i, int j) __attribute__((always_inline)) {
        const int t = wv + i * kMoeWaves;
#pragma unroll
        for (int k = 0; k < MATS; ++k) d[j][k] = load_words(w[k] + int64_t(t) * kTileBytes);
#pragma unroll
        for (int h = 0; h < 2; ++h) xv[j][h] = *reinterpret_cast<const v4u *>(x + t * kTileK + 64 * h);
    };
#pragma unroll
    for (int k = 0; k < MATS; ++k) acc[k][0] = acc[k][1] = v4i{0, 0, 0, 0};
    auto use = [&](int j) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < MATS; ++k) add_tile(d[j][k], xv[j], acc[k]);
    };
#pragma unroll
    for (int j = 0; j < D; ++j)
        if (j < n) load(j, j);
    // While no load can be past the end none is asked for it: a load that may
    // be skipped makes the compiler wait for all before it at every tile.
    int i = 0;
    for (; i + 2 * D <= n; i += D) {
#pragma unroll
        for (int j = 0; j < D; ++j) {
            use(j);
            load(i + j + D, j);
        }
    }
    for (; i < n; i += D) {
#pragma unroll
        for (int j = 0; j < D; ++j) {
            if (i + j < n) use(j);
            if (i + j + D < n) load(i + j + D, j);
        }
    }
}

// Sums of the waves' results; wave w is left with those of rows 4c + w.
template <int BLOCKS>
__device__ __forceinline__ void join_waves(int *red, int lane, int wv, const v4i (&v)[BLOCKS], int (&sum)[BLOCKS]) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < BLOCKS; ++k)
#pragma unroll
        for (int i = 0; i < kMoeWaves; ++i) red[((i * BLOCKS + k) * kMoeWaves + wv) * 64 + lane] = v[k][i];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < BLOCKS; ++k) {
        sum[k] = 0;
#pragma unroll
        for (int w = 0; w < kMoeWaves; ++w) sum[k] += red[((wv * BLOCKS + k) * kMoeWaves + w) * 64 + lane];
    }
}

// The place of the n-th set bit of a 64-bit mask, for n = first + (lane's r);
// the last one for n past the last.
__device__ __forceinline__ int token_of(uint64_t mask, int first, int r) {
    for (int i = 0; i < first; ++i) mask &= mask - 1;
    int at = 0;
    for (int i = 0; i < kMoeRows && mask; ++i) {
        const int b = __builtin_ctzll(mask);
        if (i <= r) at = b;
        mask &= mask - 1;
    }
    return at;
}

typedef v2f v2f_a __attribute__((aligned(4)));

// STRIPS strips of a slot's expert to a workgroup (those past the last are
// read as the last, and not stored): its rows are read once for all of them.
template <int STRIPS, int D>
__global__ __launch_bounds__(64 * kMoeWaves) void moe_up_kernel(MoeLaunch a) {
    extern __shared__ __attribute__((aligned(16))) int red[];
    const Slot slot = reinterpret_cast<const Slot *>(a.ws + a.sp.slot)[blockIdx.y];
    if (slot.expert < 0) return;
    const int s0 = STRIPS * int(blockIdx.x);
    float *hidden = reinterpret_cast<float *>(a.ws + a.sp.hidden);
    const uint64_t mask = (uint64_t(slot.mask[1]) << 32) | slot.mask[0];
    const int tokens = __popcll(mask);
    const int lane = int(threadIdx.x) & 63, r = lane & 15, c = lane >> 4;
    const int wv = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const int KT = (a.H + kTileK - 1) / kTileK, last = (a.I - 1) / kTileRows;
    const uint8_t *w[2 * STRIPS];
#pragma unroll
    for (int k = 0; k < STRIPS; ++k) {
        const int64_t off = int64_t(slot.expert) * a.wb1 + int64_t(min(s0 + k, last)) * KT * kTileBytes + words_at(r, c);
        w[2 * k] = a.w_gate + off;
        w[2 * k + 1] = a.w_up + off;
    }
    const int8_t *rows = reinterpret_cast<const int8_t *>(a.ws + a.sp.rows) + 16 * c;
    const int *row_sums = reinterpret_cast<const int *>(a.ws + a.sp.row_sums);
    const float sg = a.s_gate[slot.expert], su = a.s_up[slot.expert];

    for (int m0 = 0; m0 < tokens; m0 += kMoeRows) {
        const int token = token_of(mask, m0, r);
        const float mine = a.sa[token];            // of row r
        const int sum = row_sums[token];
        v4i acc[2 * STRIPS][2];
        strip_sums<2 * STRIPS, D>(w, rows + int64_t(token) * KT * kTileK, KT, wv, acc);
        v4i v[4 * STRIPS];
#pragma unroll
        for (int k = 0; k < 4 * STRIPS; ++k) v[k] = acc[k >> 1][k & 1];
        int all[4 * STRIPS];
        join_waves(red, lane, wv, v, all);
        // Lane (r, c): weight rows 2r + j, pair m.
        const float sa = __shfl(mine, 4 * c + wv);
        const int sx = __shfl(sum, 4 * c + wv), m = m0 + 4 * c + wv;
        float *out = hidden + int64_t(slot.begin + m) * a.I;
#pragma unroll
        for (int k = 0; k < STRIPS; ++k) {
            const int row = (s0 + k) * kTileRows + 2 * r;
            float h[2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
                h[j] = activate(a.act, (float(all[4 * k + j] - sx) * sa) * sg, (float(all[4 * k + 2 + j] - sx) * sa) * su);
            if (m < tokens && row + 1 < a.I)
                *reinterpret_cast<v2f_a *>(out + row) = v2f{h[0], h[1]};
            else if (m < tokens && row < a.I)
                out[row] = h[0];
        }
    }
}

// One workgroup per pair: its hidden row to int8, padded with zeros to whole
// tiles; the first values stay in registers between the two walks.  (Places of
// pairs that tokens left are rounded too, and not read: their number would
// be a load ahead of all others, 0.3 us.)
constexpr int kQuantThreads = 512, kQuantWaves = kQuantThreads / 64, kQuantKept = 4;

__global__ __launch_bounds__(kQuantThreads) void moe_quant_kernel(MoeLaunch a) {
    __shared__ uint32_t most[kQuantWaves];
    const int pair = int(blockIdx.x), tid = int(threadIdx.x);
    const float *h = reinterpret_cast<const float *>(a.ws + a.sp.hidden) + int64_t(pair) * a.I;
    const int Ip = (a.I + kTileK - 1) / kTileK * kTileK;
    v4f kept[kQuantKept];
    uint32_t top = 0;
    auto largest = [&](v4f f) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, __float_as_uint(f[i]) & 0x7FFFFFFFu);
    };
#pragma unroll
    for (int i = 0; i < kQuantKept; ++i) kept[i] = load4(h, 4 * (tid + kQuantThreads * i), a.I);
#pragma unroll
    for (int i = 0; i < kQuantKept; ++i) largest(kept[i]);
    for (int k = 4 * (tid + kQuantThreads * kQuantKept); k < a.I; k += 4 * kQuantThreads) largest(load4(h, k, a.I));
    top = wave_max_u32(top);
    if ((tid & 63) == 0) most[tid >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kQuantWaves; ++i) top = max(top, most[i]);
    const float factor = code_factor(__uint_as_float(top));
    uint32_t *out = reinterpret_cast<uint32_t *>(a.ws + a.sp.codes + int64_t(pair) * Ip);
    int sum = 0;
    auto store = [&](int g, v4f f) __attribute__((always_inline)) {
        const uint32_t w = codes4(f, factor);
        out[g] = w;
        sum = dot4(w, 0x01010101u, sum);
    };
#pragma unroll
    for (int i = 0; i < kQuantKept; ++i)
        if (4 * (tid + kQuantThreads * i) < Ip) store(tid + kQuantThreads * i, kept[i]);
    for (int g = tid + kQuantThreads * kQuantKept; 4 * g < Ip; g += kQuantThreads) store(g, load4(h, 4 * g, a.I));
    // (The waves' sums as they are: their reader adds them.)
    sum = wave_sum(sum);
    if ((tid & 63) == 0) reinterpret_cast<int *>(a.ws + a.sp.code_sums)[pair * kQuantWaves + (tid >> 6)] = sum;
    if (tid == 0) reinterpret_cast<float *>(a.ws + a.sp.scales)[pair] = code_scale(__uint_as_float(top));
}

template <int STRIPS, int D>
__global__ __launch_bounds__(64 * kMoeWaves) void moe_down_kernel(MoeLaunch a) {
    extern __shared__ __attribute__((aligned(16))) int red[];
    const Slot slot = reinterpret_cast<const Slot *>(a.ws + a.sp.slot)[blockIdx.y];
    if (slot.expert < 0) return;
    const int s0 = STRIPS * int(blockIdx.x);
    const float *scales = reinterpret_cast<const float *>(a.ws + a.sp.scales);
    const int *code_sums = reinterpret_cast<const int *>(a.ws + a.sp.code_sums);
    const int *row_of = reinterpret_cast<const int *>(a.ws + a.sp.row_of);
    float *part = reinterpret_cast<float *>(a.ws + a.sp.part);
    const int tokens = __popc(slot.mask[0]) + __popc(slot.mask[1]);
    const int lane = int(threadIdx.x) & 63, r = lane & 15, c = lane >> 4;
    const int wv = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const int KT = (a.I + kTileK - 1) / kTileK, last = (a.H - 1) / kTileRows;
    const uint8_t *w[STRIPS];
#pragma unroll
    for (int k = 0; k < STRIPS; ++k)
        w[k] = a.w_down + int64_t(slot.expert) * a.wb2 + int64_t(min(s0 + k, last)) * KT * kTileBytes + words_at(r, c);
    const int8_t *codes = reinterpret_cast<const int8_t *>(a.ws + a.sp.codes) + 16 * c;
    const float sd = a.s_down[slot.expert];

    for (int m0 = 0; m0 < tokens; m0 += kMoeRows) {
        const int at = slot.begin + min(m0 + r, tokens - 1);
        const float mine = scales[at];
        const int my_row = row_of[at];             // of row r
        int sum = 0;
#pragma unroll
        for (int i = 0; i < kQuantWaves; ++i) sum += code_sums[at * kQuantWaves + i];
        v4i acc[STRIPS][2];
        strip_sums<STRIPS, D>(w, codes + int64_t(at) * KT * kTileK, KT, wv, acc);
        v4i v[2 * STRIPS];
#pragma unroll
        for (int k = 0; k < 2 * STRIPS; ++k) v[k] = acc[k >> 1][k & 1];
        int all[2 * STRIPS];
        join_waves(red, lane, wv, v, all);
        const float sh = __shfl(mine, 4 * c + wv);
        const int sx = __shfl(sum, 4 * c + wv), m = m0 + 4 * c + wv;
        float *out = part + int64_t(__shfl(my_row, 4 * c + wv)) * a.H;
#pragma unroll
        for (int k = 0; k < STRIPS; ++k) {
            const int row = (s0 + k) * kTileRows + 2 * r;
            const v2f y = {(float(all[2 * k] - sx) * sh) * sd, (float(all[2 * k + 1] - sx) * sh) * sd};
            if (m < tokens && row + 1 < a.H)
                *reinterpret_cast<v2f_a *>(out + row) = y;
            else if (m < tokens && row < a.H)
                out[row] = y[0];
        }
    }
}

__global__ __launch_bounds__(256) void moe_combine_kernel(MoeLaunch a) {
    const int n = int(blockIdx.x) * 256 + int(threadIdx.x), m = int(blockIdx.y);
    const Picked *picked = reinterpret_cast<const Picked *>(a.ws + a.sp.picked) + m * a.top_k;
    const float *part = reinterpret_cast<const float *>(a.ws + a.sp.part) + int64_t(m) * a.top_k * a.H + n;
    if (n >= a.H) return;
    float y = picked[0].expert == -2 ? __builtin_nanf("") : 0.0f;
    // Four ranks a wait; those past the last are read as the last.  (Nothing was
    // written for a rank that has no expert.)
    for (int j = 0; j < a.top_k; j += 4) {
        Picked of[4];
        float p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = min(j + i, a.top_k - 1);
            of[i] = picked[k];
            p[i] = part[int64_t(k) * a.H];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) y += j + i < a.top_k && of[i].expert >= 0 ? of[i].weight * p[i] : 0.0f;
    }
    const int64_t at = int64_t(m) * a.H + n;
    if (a.y_f32) a.y_f32[at] = y;
    if (a.y_bf16) a.y_bf16[at] = uint16_t(bf16_bits(y));
}

hipError_t launch(const void *fn, dim3 grid, int threads, size_t lds, void **args, hipStream_t stream) {
    return hipLaunchKernel(fn, grid, dim3(unsigned(threads)), args, lds, stream);
}

// Most LDS of the hidden rows of a token (the kernel has some of its own).
constexpr int64_t kOneLds = 49152;
std::atomic<int> g_mode{0};

}  // namespace

MoeSpace moe_space(int64_t M, int64_t H, int64_t I, int64_t E, int64_t top_k) {
    MoeSpace s;
    const int64_t pairs = M * top_k;
    int64_t at = 0;
    const auto take = [&](int64_t bytes) {
        const int64_t from = at;
        at += round_up(bytes, 256);
        return from;
    };
    s.picked = take(pairs * sizeof(Picked));
    s.tops = take(4 * pairs * ceil_div(I, kTileRows));
    s.slot = take(W2A8_MOE_MAX_E * sizeof(Slot));
    s.row_of = take(4 * pairs);
    s.scales = take(4 * pairs);
    s.code_sums = take(4 * kQuantWaves * pairs);
    s.row_sums = take(4 * M);
    s.rows = take(M * round_up(H, kTileK));
    s.codes = take(pairs * round_up(I, kTileK));
    s.hidden = take(4 * pairs * I);
    s.part = take(4 * pairs * H);
    s.total = at;
    return s;
}

int moe_mode() { return g_mode.load(std::memory_order_relaxed); }
void set_moe_mode(int mode) { g_mode.store(mode, std::memory_order_relaxed); }

// One token at a time reads an expert's weights once for every token that
// takes it, in two launches; token rows together read them once, in five (us
// below: one at a time and together).
//
// Several tokens go by themselves while the first launch is one round of
// workgroups (two to a compute unit) and the second is no more than four to a
// compute unit (8 experts of 2560 x 6912, two taken: two tokens, 868 workgroups,
// 24.9 and 24.1; 64 of 2560 x 640, eight taken: three tokens, 480, 18.3 and 22.4,
// four, 640, 25.5 and 23.6; 8 of 2560 x 2560, one taken: six tokens, 480, 18.9 and
// 20.2, seven, 560, 23.5 and 20.4; 16 of 5120 x 1280, two taken, four tokens, 320
// and 1280 of the second launch, 25.4 and 23.5; 32 of 1024 x 512, two taken: twelve
// tokens, 384 and 768, 14.2 and 17.0, 24 tokens 22.9 and 18.0).
//
// One token shares no expert.  Where it takes one or two, together is the slower
// wherever the hidden rows fit LDS, but for a few sizes within 6%: its products have a
// strip of few experts to a workgroup, and its other launches little to do (8 experts
// of 512 x 40960, one taken, 1280 workgroups, 30.0 and 45.3, of 5120 x 12288 25.2 and
// 30.2; two taken, 512 x 20480, 27.1 and 29.9, 5120 x 20480 52.9 and 54.2; 5 of
// 8192 x 13600, two taken, 49.2 and 46.4).  Where it takes more, every workgroup of
// the first launch takes up to top_k maxima one after the other, on top of work that
// is worth some eight of them, so their sum is bounded (16 of 2560 x 6400, four taken,
// 800 workgroups, 24.3 and 25.7, 2560 x 8192, 1024, 28.5 and 28.0; 32 of 512 x 2048,
// eight taken, 512, 16.2 and 17.0, 512 x 4096, 1024, 23.9 and 18.7, 2048 x 2560,
// 640, 20.2 and 22.2, 2048 x 4096, 1024, 27.4 and 25.7; 64 of 2048 x 768, sixteen
// taken, 384, 17.9 and 21.8, 2048 x 1536, 768, 26.2 and 25.2.  Over 252 sizes the
// choice costs 0.6% on average, 10% at most, and 4.2% and 56% if all are bounded by
// four workgroups to a compute unit).
//
// Together, a workgroup takes two strips of an expert where that leaves four
// workgroups to a compute unit, so that a wave reads its rows for twice the
// weights (the layer, us, two strips and one; 64 tokens, 16 experts of 5120 x
// 6912: 93.9 and 99.2, 128 of 5120 x 1536, eight taken: 147 and 159), and one where
// strips are fewer (8 tokens, 16 experts of 2560 x 2560, four taken: 30.1 and
// 29.3; 8 of 2560 x 6912, two taken: four tokens 30.6 and 30.0, 64 tokens 57.3 and
// 58.4).
MoePlan moe_plan(int64_t M, int64_t H, int64_t I, int64_t E, int64_t top_k, int cus) {
    MoePlan p;
    const int mode = moe_mode();
    const bool fits = top_k * round_up(I, kTileK) <= kOneLds;
    const int64_t first = M * top_k * ceil_div(I, kTileRows);
    const bool few = (M > 1 ? first <= 2 * cus : top_k <= 2 || first * (top_k + 8) <= 40 * cus) &&
                     M * ceil_div(H, kDownRows) <= 4 * cus;
    p.one = fits && (mode == 0 ? few : mode == 1);
    const int64_t slots = std::min(E, M * top_k);
    const auto strips = [&](int64_t N) { return ceil_div(ceil_div(N, kTileRows), 2) * slots >= 4 * int64_t(cus) ? 2 : 1; };
    p.up = mode == 3 ? 1 : mode == 4 ? 2 : strips(I);
    p.down = mode == 3 ? 1 : mode == 4 ? 2 : strips(H);
    return p;
}

hipError_t launch_moe(const MoeLaunch &la, int cus, hipStream_t stream) {
    MoeLaunch a = la;
    const auto fn = [](auto *k) { return reinterpret_cast<const void *>(k); };
    const MoePlan p = moe_plan(a.M, a.H, a.I, a.E, a.top_k, cus);
    const int64_t up = ceil_div(a.I, kTileRows), down = ceil_div(a.H, kTileRows);
    int slots = std::min(a.E, a.M * a.top_k);
    void *args[] = {&a, &slots};
    hipError_t e;
    if (p.one) {
        e = launch(fn(&moe_up_one_kernel), dim3(unsigned(up + 1), unsigned(a.top_k), unsigned(a.M)), 512, 0, args,
                   stream);
        if (e != hipSuccess) return e;
        return launch(fn(&moe_down_one_kernel), dim3(unsigned(ceil_div(a.H, kDownRows)), unsigned(a.M)), kDownThreads,
                      size_t(a.top_k * round_up(a.I, kTileK)), args, stream);
    }
    e = launch(fn(&moe_route_kernel), dim3(unsigned(1 + a.M)), kRouteThreads, 0, args, stream);
    if (e != hipSuccess) return e;
    e = launch(p.up == 2 ? fn(&moe_up_kernel<2, 2>) : fn(&moe_up_kernel<1, 3>),
               dim3(unsigned(ceil_div(up, p.up)), unsigned(slots)), 64 * kMoeWaves, size_t(kMoeWaves * p.up) * 4096, args,
               stream);
    if (e != hipSuccess) return e;
    e = launch(fn(&moe_quant_kernel), dim3(unsigned(a.M * a.top_k)), kQuantThreads, 0, args, stream);
    if (e != hipSuccess) return e;
    e = launch(p.down == 2 ? fn(&moe_down_kernel<2, 3>) : fn(&moe_down_kernel<1, 4>),
               dim3(unsigned(ceil_div(down, p.down)), unsigned(slots)), 64 * kMoeWaves, size_t(kMoeWaves * p.down) * 2048,
               args, stream);
    if (e != hipSuccess) return e;
    return launch(fn(&moe_combine_kernel), dim3(unsigned(ceil_div(a.H, 256)), unsigned(a.M)), 256, 0, args, stream);
}

}  // namespace w2a8
