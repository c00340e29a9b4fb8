// Mixture of ternary experts for a few tokens (gfx950): the layer of w2a8_moe
// in four launches.
//
//   route     every token's top_k experts and their weights, and every
//             expert's tokens: pairs (token, expert) in the order of experts
//   gate, up  hidden[pair] = act(g) * u, and its largest magnitude
//   down      hidden quantized to int8 by it, part[pair] = p * (w_down . q) ...
//   combine   y[token] = the sum of its pairs' parts, in order of rank
//
// The weights of an expert are read once for 16 of its tokens: a workgroup
// takes a strip of 32 weight rows of one expert, its waves the strip's tiles
// in turn.  The matrix instruction (16x16x64, int8) takes activation rows as
// its first operand and weight rows as its second; lane (r, c) reads 8 bytes
// of the T32x128 slots of k-parts c and 4 + c: two words, of weight rows 2r
// and 2r + 1.  Sums are integers, so waves add up in any order; the pair's
// maximum is an atomic maximum, which has no order either.
#include "block.h"

namespace w2a8 {
namespace {

constexpr int kMoeRows = 16;       // tokens of a pass
constexpr int kMoeWaves = 8;
constexpr int kRouteThreads = 1024;
constexpr int kMaxPairs = W2A8_MOE_MAX_M * W2A8_MOE_MAX_TOP_K;
constexpr int kPerLane = W2A8_MOE_MAX_E / 64;

// What the route leaves behind, at the start of the workspace.
struct Slots {
    int count;                          // experts that have tokens
    int bad[W2A8_MOE_MAX_M];            // tokens whose logits are no numbers
    int expert[W2A8_MOE_MAX_E], begin[W2A8_MOE_MAX_E], tokens[W2A8_MOE_MAX_E];
};
// Pairs: the token and weight of each, and each token's pairs by rank.
struct Pairs {
    int token[kMaxPairs];
    float weight[kMaxPairs];
    int of[kMaxPairs];                  // [token][rank]: pair or -1
};

// Order of floats as unsigned integers; 0 stands for an expert that cannot be taken.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(v);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
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

__global__ __launch_bounds__(kRouteThreads) void moe_route_kernel(MoeLaunch a) {
    __shared__ uint32_t mask[W2A8_MOE_MAX_E][2];      // tokens of an expert
    __shared__ short taken[kMaxPairs];                // [token][rank]
    __shared__ int ends[2][W2A8_MOE_MAX_E], begins[W2A8_MOE_MAX_E];
    const int tid = int(threadIdx.x), lane = tid & 63, wv = tid >> 6;
    Slots *slots = reinterpret_cast<Slots *>(a.ws + a.sp.slot);
    Pairs *pairs = reinterpret_cast<Pairs *>(a.ws + a.sp.pair);
    uint32_t *amax = reinterpret_cast<uint32_t *>(a.ws + a.sp.amax);
    if (tid < W2A8_MOE_MAX_E) mask[tid][0] = mask[tid][1] = 0;
    for (int i = tid; i < a.M * a.top_k; i += kRouteThreads) amax[i] = 0;
    __syncthreads();

    float weight[W2A8_MOE_MAX_M / (kRouteThreads / 64)];     // of rank `lane`, of this wave's tokens
#pragma unroll
    for (int q = 0; q < W2A8_MOE_MAX_M / (kRouteThreads / 64); ++q) {
        const int m = wv + q * (kRouteThreads / 64);
        weight[q] = 0.0f;
        if (m >= a.M) continue;
        float l[kPerLane];
        uint32_t key[kPerLane];
        bool bad = false;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) {
            const int e = lane + 64 * i;
            l[i] = e < a.E ? logit(a, int64_t(m) * a.E + e) : -__builtin_inff();
            bad |= !(l[i] < __builtin_inff());
            key[i] = l[i] == -__builtin_inff() ? 0u : order_key(l[i] + 0.0f);   // (-0 ties with 0)
        }
        bad = __any(bad);
        float top = 0.0f, sum = 0.0f, all = 0.0f;
        for (int j = 0; j < a.top_k; ++j) {
            uint32_t best = 0;
#pragma unroll
            for (int i = 0; i < kPerLane; ++i) best = max(best, key[i]);
            best = wave_max_u32(best);
            if (bad) best = 0;
            int e = -1;
#pragma unroll
            for (int i = 0; i < kPerLane; ++i) {
                const uint64_t hit = __ballot(best != 0 && key[i] == best);
                if (e < 0 && hit) e = 64 * i + __builtin_ctzll(hit);
            }
            float p = 0.0f;
            if (e >= 0) {
#pragma unroll
                for (int i = 0; i < kPerLane; ++i)
                    if (lane + 64 * i == e) key[i] = 0;
                const float v = __uint_as_float(best & 0x80000000u ? best & 0x7FFFFFFFu : ~best);
                if (j == 0) {
                    top = v;
#pragma unroll
                    for (int i = 0; i < kPerLane; ++i) all += expf(l[i] - top);
                    all = wave_sum_f32(all);
                }
                p = expf(v - top);
                sum += p;
                if (lane == 0) {
                    taken[m * a.top_k + j] = short(e);
                    atomicOr(&mask[e][m >> 5], 1u << (m & 31));
                }
            } else if (lane == 0) {
                taken[m * a.top_k + j] = -1;
            }
            if (lane == j) weight[q] = p;
        }
        weight[q] /= a.renormalize ? sum : all;
        if (lane == 0) slots->bad[m] = bad;
    }
    __syncthreads();

    // Places of the experts' pairs and slots: sums of (pairs, experts) over
    // the experts before, in one word each.
    const int n = tid < W2A8_MOE_MAX_E ? __popc(mask[tid][0]) + __popc(mask[tid][1]) : 0;
    int v = n + (n ? 1 << 16 : 0);
    if (tid < W2A8_MOE_MAX_E) ends[0][tid] = v;
    __syncthreads();
    int from = 0;
    for (int o = 1; o < W2A8_MOE_MAX_E; o *= 2) {
        if (tid < W2A8_MOE_MAX_E) ends[from ^ 1][tid] = ends[from][tid] + (tid >= o ? ends[from][tid - o] : 0);
        from ^= 1;
        __syncthreads();
    }
    if (tid < W2A8_MOE_MAX_E) {
        const int before = ends[from][tid] - v;
        begins[tid] = before & 0xFFFF;
        if (n) {
            slots->expert[before >> 16] = tid;
            slots->begin[before >> 16] = before & 0xFFFF;
            slots->tokens[before >> 16] = n;
        }
        if (tid == W2A8_MOE_MAX_E - 1) slots->count = ends[from][tid] >> 16;
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < W2A8_MOE_MAX_M / (kRouteThreads / 64); ++q) {
        const int m = wv + q * (kRouteThreads / 64);
        if (m >= a.M || lane >= a.top_k) continue;
        const int e = taken[m * a.top_k + lane];
        int at = -1;
        if (e >= 0) {
            const uint32_t lo = mask[e][0], hi = mask[e][1];
            at = begins[e] + (m < 32 ? __popc(lo & ((1u << m) - 1u))
                                     : __popc(lo) + __popc(hi & ((1u << (m - 32)) - 1u)));
            pairs->token[at] = m;
            pairs->weight[at] = weight[q];
        }
        pairs->of[m * a.top_k + lane] = at;
    }
}

// The weight words of a tile that a lane brings: rows 2r, 2r + 1 of k-parts c
// and 4 + c.
struct Words {
    v2u h[2];
};
__device__ __forceinline__ Words load_words(const uint8_t *tile, int r, int c) {
    Words w;
#pragma unroll
    for (int h = 0; h < 2; ++h)
        w.h[h] = __builtin_nontemporal_load(
            reinterpret_cast<const v2u *>(tile + 16 * (8 * (r >> 1) + c + 4 * h) + 8 * (r & 1)));
    return w;
}
__device__ __forceinline__ void add_tile(const Words &w, const v4i (&x)[2], v4i (&acc)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 2; ++j)
            acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(x[h], expand_word(w.h[h][j]), acc[j], 0, 0, 0);
}

// Sums of the waves' results (COUNT words a lane) in wave 0 .. nw - 1: wave w
// is left with words i % nw == w, the others' are stale.
template <int COUNT>
__device__ __forceinline__ void add_waves(int *red, int lane, int wv, int nw, int (&v)[COUNT]) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < COUNT; ++i) red[(wv * COUNT + i) * 64 + lane] = v[i];
    __syncthreads();
    if (wv != 0) return;
#pragma unroll
    for (int i = 0; i < COUNT; ++i)
        for (int w = 1; w < nw; ++w) v[i] += red[(w * COUNT + i) * 64 + lane];
}

__device__ __forceinline__ float activate(int act, float g, float u) {
    if (act == W2A8_ACT_SILU) return (g / (1.0f + expf(-g))) * u;
    const float p = fmaxf(g, 0.0f);
    return (p * p) * u;
}

__global__ __launch_bounds__(64 * kMoeWaves) void moe_up_kernel(MoeLaunch a) {
    extern __shared__ __attribute__((aligned(16))) int red[];
    const Slots *slots = reinterpret_cast<const Slots *>(a.ws + a.sp.slot);
    const int slot = int(blockIdx.y), s = int(blockIdx.x);
    if (slot >= slots->count) return;
    const Pairs *pairs = reinterpret_cast<const Pairs *>(a.ws + a.sp.pair);
    uint32_t *amax = reinterpret_cast<uint32_t *>(a.ws + a.sp.amax);
    float *hidden = reinterpret_cast<float *>(a.ws + a.sp.hidden);
    const int e = slots->expert[slot], begin = slots->begin[slot], tokens = slots->tokens[slot];
    const int lane = int(threadIdx.x) & 63, r = lane & 15, c = lane >> 4;
    const int wv = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6), nw = int(blockDim.x) >> 6;
    const int KT = (a.H + kTileK - 1) / kTileK, whole = a.H / kTileK;
    const int64_t off = int64_t(e) * a.wb1 + int64_t(s) * KT * kTileBytes;
    const uint8_t *wg = a.w_gate + off, *wu = a.w_up + off;
    const float sg = a.s_gate[e], su = a.s_up[e];

    for (int m0 = 0; m0 < tokens; m0 += kMoeRows) {
        const int8_t *xr = a.x + int64_t(pairs->token[begin + min(m0 + r, tokens - 1)]) * a.H;
        v4i acc[2][2];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i >> 1][i & 1] = v4i{0, 0, 0, 0};
#pragma unroll 2
        for (int t = wv; t < whole; t += nw) {
            const Words g = load_words(wg + int64_t(t) * kTileBytes, r, c);
            const Words u = load_words(wu + int64_t(t) * kTileBytes, r, c);
            v4i x[2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
                x[h] = __builtin_bit_cast(v4i, *reinterpret_cast<const v4u_b *>(xr + t * kTileK + 64 * h + 16 * c));
            add_tile(g, x, acc[0]);
            add_tile(u, x, acc[1]);
        }
        if (whole < KT && wv == whole % nw) {
            uint32_t w[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) load_int8_tail<16>(xr, whole * kTileK + 64 * h + 16 * c, a.H, w[h]);
            const v4i x[2] = {v4i{int(w[0][0]), int(w[0][1]), int(w[0][2]), int(w[0][3])},
                              v4i{int(w[1][0]), int(w[1][1]), int(w[1][2]), int(w[1][3])}};
            add_tile(load_words(wg + int64_t(whole) * kTileBytes, r, c), x, acc[0]);
            add_tile(load_words(wu + int64_t(whole) * kTileBytes, r, c), x, acc[1]);
        }
        int v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = acc[i >> 3][(i >> 2) & 1][i & 3];
        if (nw > 1) add_waves(red, lane, wv, nw, v);
        if (wv != 0) continue;
        // Lane (r, c): weight rows 2r + j, pairs 4c + i.
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int m = m0 + 4 * c + i;
            const int at = begin + m;
            const float sa = m < tokens ? a.sa[pairs->token[at]] : 0.0f;
            uint32_t most = 0;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int row = s * kTileRows + 2 * r + j;
                const float g = (float(v[4 * j + i]) * sa) * sg, u = (float(v[8 + 4 * j + i]) * sa) * su;
                const float h = activate(a.act, g, u);
                if (m < tokens && row < a.I) {
                    hidden[int64_t(at) * a.I + row] = h;
                    most = max(most, __float_as_uint(h) & 0x7FFFFFFFu);
                }
            }
            // The largest of the strip's 32 rows: one atomic a pair.
            for (int o = 1; o < 16; o *= 2) most = max(most, uint32_t(__shfl_xor(int(most), o)));
            if (r == 0 && m < tokens) atomicMax(&amax[at], most);
        }
    }
}

__global__ __launch_bounds__(64 * kMoeWaves) void moe_down_kernel(MoeLaunch a, int chunk, int rows) {
    extern __shared__ __attribute__((aligned(16))) int8_t lds[];
    const Slots *slots = reinterpret_cast<const Slots *>(a.ws + a.sp.slot);
    const int slot = int(blockIdx.y), s = int(blockIdx.x);
    if (slot >= slots->count) return;
    const Pairs *pairs = reinterpret_cast<const Pairs *>(a.ws + a.sp.pair);
    const uint32_t *amax = reinterpret_cast<const uint32_t *>(a.ws + a.sp.amax);
    const float *hidden = reinterpret_cast<const float *>(a.ws + a.sp.hidden);
    float *part = reinterpret_cast<float *>(a.ws + a.sp.part);
    const int e = slots->expert[slot], begin = slots->begin[slot], tokens = slots->tokens[slot];
    const int tid = int(threadIdx.x), lane = tid & 63, r = lane & 15, c = lane >> 4;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6), nw = int(blockDim.x) >> 6;
    const int KT = (a.I + kTileK - 1) / kTileK;
    const uint8_t *wd = a.w_down + int64_t(e) * a.wb2 + int64_t(s) * KT * kTileBytes;
    const float sd = a.s_down[e];
    const int stride = chunk + 16;        // rows of LDS start in banks of their own
    int *red = reinterpret_cast<int *>(lds);

    for (int m0 = 0; m0 < tokens; m0 += kMoeRows) {
        const int mt = min(tokens - m0, rows);
        v4i acc[2] = {v4i{0, 0, 0, 0}, v4i{0, 0, 0, 0}};
        for (int k0 = 0; k0 < a.I; k0 += chunk) {
            const int kn = min(chunk, KT * kTileK - k0);
            __syncthreads();
            // int8 rows of the chunk, four values a lane; zeros past I.
            for (int j = 0; j < mt; ++j) {
                const int at = begin + m0 + j;
                const float most = __uint_as_float(amax[at]);
                const float inv = most == 0.0f ? 0.0f : fminf(127.0f / most, __FLT_MAX__);
                const float *h = hidden + int64_t(at) * a.I + k0;
                for (int k = 4 * tid; k < kn; k += 4 * int(blockDim.x)) {
                    v4f f = {0.0f, 0.0f, 0.0f, 0.0f};
                    if (k0 + k + 4 <= a.I)
                        f = *reinterpret_cast<const v4f_b *>(h + k);
                    else
#pragma unroll
                        for (int i = 0; i < 3; ++i)
                            if (k0 + k + i < a.I) f[i] = h[k + i];
                    *reinterpret_cast<uint32_t *>(lds + j * stride + k) =
                        q8(f[0], inv) | (q8(f[1], inv) << 8) | (q8(f[2], inv) << 16) | (q8(f[3], inv) << 24);
                }
            }
            __syncthreads();
            const int8_t *xr = lds + min(r, mt - 1) * stride;
#pragma unroll 2
            for (int t = wv; t < kn / kTileK; t += nw) {
                const Words w = load_words(wd + int64_t(k0 / kTileK + t) * kTileBytes, r, c);
                v4i x[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) x[h] = *reinterpret_cast<const v4i *>(xr + t * kTileK + 64 * h + 16 * c);
                add_tile(w, x, acc);
            }
        }
        int v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = acc[i >> 2][i & 3];
        if (nw > 1) add_waves(red, lane, wv, nw, v);
        if (wv != 0) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int m = m0 + 4 * c + i;
            if (m >= tokens) continue;
            const int at = begin + m;
            const float most = __uint_as_float(amax[at]);
            // (A hidden row that is not finite has no codes.)
            const float sh = most < __builtin_inff() ? most / 127.0f : __builtin_nanf("");
            const float p = pairs->weight[at];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int row = s * kTileRows + 2 * r + j;
                if (row < a.H) part[int64_t(at) * a.H + row] = p * ((float(v[4 * j + i]) * sh) * sd);
            }
        }
    }
}

__global__ __launch_bounds__(256) void moe_combine_kernel(MoeLaunch a) {
    const int n = int(blockIdx.x) * 256 + int(threadIdx.x), m = int(blockIdx.y);
    if (n >= a.H) return;
    const Slots *slots = reinterpret_cast<const Slots *>(a.ws + a.sp.slot);
    const Pairs *pairs = reinterpret_cast<const Pairs *>(a.ws + a.sp.pair);
    const float *part = reinterpret_cast<const float *>(a.ws + a.sp.part);
    float y = slots->bad[m] ? __builtin_nanf("") : 0.0f;
    for (int j = 0; j < a.top_k; ++j) {
        const int at = pairs->of[m * a.top_k + j];
        if (at >= 0) y += part[int64_t(at) * a.H + n];
    }
    const int64_t at = int64_t(m) * a.H + n;
    if (a.y_f32) a.y_f32[at] = y;
    if (a.y_bf16) a.y_bf16[at] = uint16_t(bf16_bits(y));
}

}  // namespace

MoeSpace moe_space(int64_t M, int64_t H, int64_t I, int64_t E, int64_t top_k) {
    MoeSpace s;
    const int64_t pairs = M * top_k;
    s.slot = 0;
    s.pair = s.slot + round_up(sizeof(Slots), 256);
    s.amax = s.pair + round_up(sizeof(Pairs), 256);
    s.hidden = s.amax + round_up(4 * pairs, 256);
    s.part = s.hidden + round_up(4 * pairs * I, 256);
    s.total = s.part + round_up(4 * pairs * H, 256);
    return s;
}

hipError_t launch_moe(const MoeLaunch &la, int cus, hipStream_t stream) {
    MoeLaunch a = la;
    void *args[] = {&a};
    const unsigned slots = unsigned(std::min(a.E, a.M * a.top_k));
    hipError_t e = hipLaunchKernel(reinterpret_cast<const void *>(&moe_route_kernel), dim3(1),
                                   dim3(kRouteThreads), args, 0, stream);
    if (e != hipSuccess) return e;
    const int nw1 = int(std::min<int64_t>(kMoeWaves, ceil_div(a.H, kTileK)));
    e = hipLaunchKernel(reinterpret_cast<const void *>(&moe_up_kernel),
                        dim3(unsigned(ceil_div(a.I, kTileRows)), slots), dim3(unsigned(64 * nw1)), args,
                        size_t(nw1) * 4096, stream);
    if (e != hipSuccess) return e;
    const int64_t KT = ceil_div(a.I, kTileK);
    const int nw2 = int(std::min<int64_t>(kMoeWaves, KT));
    // Rows of a pass and the part of I that they have in LDS: 64 KiB at most.
    int rows = std::min(a.M, kMoeRows);
    int chunk = int(std::min<int64_t>(KT, (65536 / rows - 16) / kTileK) * kTileK);
    const size_t bytes = std::max(size_t(rows) * (chunk + 16), size_t(nw2) * 2048);
    void *args2[] = {&a, &chunk, &rows};
    e = hipLaunchKernel(reinterpret_cast<const void *>(&moe_down_kernel),
                        dim3(unsigned(ceil_div(a.H, kTileRows)), slots), dim3(unsigned(64 * nw2)), args2,
                        bytes, stream);
    if (e != hipSuccess) return e;
    return hipLaunchKernel(reinterpret_cast<const void *>(&moe_combine_kernel),
                           dim3(unsigned(ceil_div(a.H, 256)), unsigned(a.M)), dim3(256), args, 0, stream);
}

}  // namespace w2a8
