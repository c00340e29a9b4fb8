// Root-mean-square norm with the residual's addition, into int8 rows (gfx950).
//
//   h = x + residual;  v = h * weight;  a = max |v|;
//   q = rint(v * 127 / a);  s = a / 127 / sqrt(mean(h^2) + eps)
//
// The mean cancels from the codes (v / rms over max |v| / rms), so they need
// one maximum and no sum, and come out the same in any order of reduction.
// The sum of squares is in fp64: squares of fp32 values are exact there, and
// none passes its range.
//
// Bound by memory: a row is read once, held in registers as v (fp32), reduced
// over the workgroup, rounded and stored.  Rows past 4096 chunks of 8 values are
// walked twice, the second time from h.
#include "block.h"

namespace w2a8 {
namespace {

typedef v4u v4u_f __attribute__((aligned(4)));

constexpr int kMaxChunks = 4096;       // 4 for each of 1024 lanes

__device__ __forceinline__ float half_value(uint32_t bits) {
    return float(__builtin_bit_cast(_Float16, uint16_t(bits)));
}
__device__ __forceinline__ uint32_t half_bits(float v) {
    return uint32_t(__builtin_bit_cast(uint16_t, _Float16(v)));
}

// Values i..i+7 of a float row (at any alignment of its elements), as they are.
template <int TYPE>
struct Raw8 {
    v4u w[TYPE == W2A8_F32 ? 2 : 1];

    __device__ __forceinline__ void load(const void *p, int64_t i) {
        if constexpr (TYPE == W2A8_F32) {
            const v4u_f *f = reinterpret_cast<const v4u_f *>(static_cast<const float *>(p) + i);
            w[0] = f[0];
            w[1] = f[1];
        } else {
            w[0] = *reinterpret_cast<const v4u_any *>(static_cast<const uint16_t *>(p) + i);
        }
    }
    __device__ __forceinline__ float value(int j) const {
        if constexpr (TYPE == W2A8_F32) return __uint_as_float(w[j >> 2][j & 3]);
        const uint32_t u = w[0][j >> 1];
        if constexpr (TYPE == W2A8_BF16) return j & 1 ? hi_bf16(u) : lo_bf16(u);
        return half_value(j & 1 ? u >> 16 : u & 0xFFFFu);
    }
};

// Rounds v to TYPE, stores it as values i..i+7, and leaves the rounded values.
template <int TYPE>
__device__ __forceinline__ void store8(void *p, int64_t i, float (&v)[8]) {
    if constexpr (TYPE == W2A8_F32) {
        float *f = static_cast<float *>(p) + i;
        *reinterpret_cast<v4f_b *>(f) = v4f{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<v4f_b *>(f + 4) = v4f{v[4], v[5], v[6], v[7]};
    } else {
        v4u w;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w[j] = TYPE == W2A8_BF16 ? bf16_pair(v[2 * j], v[2 * j + 1])
                                     : half_bits(v[2 * j]) | half_bits(v[2 * j + 1]) << 16;
            v[2 * j] = TYPE == W2A8_BF16 ? lo_bf16(w[j]) : half_value(w[j] & 0xFFFFu);
            v[2 * j + 1] = TYPE == W2A8_BF16 ? hi_bf16(w[j]) : half_value(w[j] >> 16);
        }
        *reinterpret_cast<v4u_any *>(static_cast<uint16_t *>(p) + i) = w;
    }
}

template <int TYPE>
__device__ __forceinline__ float store1(void *p, int64_t i, float v) {
    if constexpr (TYPE == W2A8_F32) {
        static_cast<float *>(p)[i] = v;
        return v;
    } else {
        const uint32_t b = TYPE == W2A8_BF16 ? bf16_bits(v) : half_bits(v);
        static_cast<uint16_t *>(p)[i] = uint16_t(b);
        return TYPE == W2A8_BF16 ? lo_bf16(b) : half_value(b);
    }
}

// The operands of 8 values from k on, 0 <= k <= K - 8.
template <int TYPE>
struct Chunk {
    Raw8<TYPE> x, r, w;

    __device__ __forceinline__ void load(const NormLaunch &a, int64_t row, int k) {
        x.load(a.x, row + k);
        if (a.residual) r.load(a.residual, row + k);
        if (a.weight) w.load(a.weight, k);
    }
    // h, stored, and v.
    __device__ __forceinline__ void use(const NormLaunch &a, int64_t row, int k, float (&v)[8], double &sum) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = x.value(j);
        if (a.residual) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] += r.value(j);
            store8<TYPE>(a.h, row + k, v);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += double(v[j]) * double(v[j]);
        if (a.weight) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= w.value(j);
        }
    }
};

__device__ __forceinline__ float abs_max(float amax, float v) {
    return __int_as_float(max(__float_as_int(amax), __float_as_int(v) & 0x7FFFFFFF));
}

__device__ __forceinline__ void store_codes(const NormLaunch &a, int64_t at, const float (&v)[8], float inv) {
    uint32_t o[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        o[i] = q8(v[4 * i], inv) | (q8(v[4 * i + 1], inv) << 8) | (q8(v[4 * i + 2], inv) << 16) |
               (q8(v[4 * i + 3], inv) << 24);
    *reinterpret_cast<v2u_b *>(a.xq + at) = v2u{o[0], o[1]};
}

// Chunks begin at multiples of 8 values of the whole buffer, so that rows of any
// length are read and written at aligned addresses (their weight is not).  The
// values of a row ahead of its chunks, and those behind them, are one each to the
// workgroup's last 16 lanes (8191 x 1287 fp16 with a residual 20.0 us; from the
// row's start on 22.4; that with all ends by one lane 29.3; 8191 x 1288 18.5).
template <int TYPE>
struct Ends {
    float x, r, w;
    int k;                              // -1: none

    __device__ __forceinline__ void load(const NormLaunch &a, int64_t row, int head, int nc) {
        const int j = int(threadIdx.x) - int(blockDim.x) + 16;
        k = j < 0 ? -1 : j < 8 ? (j < head ? j : -1) : head + 8 * nc + j - 8;
        if (k >= a.K) k = -1;
        if (k < 0) return;
        x = mx4_load1<TYPE>(a.x, row + k);
        r = a.residual ? mx4_load1<TYPE>(a.residual, row + k) : 0.0f;
        w = a.weight ? mx4_load1<TYPE>(a.weight, k) : 1.0f;
    }
    // h, stored, and v, left in w.
    __device__ __forceinline__ void use(const NormLaunch &a, int64_t row, double &sum, float &amax) {
        if (k < 0) return;
        if (a.residual) x = store1<TYPE>(a.h, row + k, x + r);
        sum += double(x) * double(x);
        w *= x;
        amax = abs_max(amax, w);
    }
    __device__ __forceinline__ void store(const NormLaunch &a, int64_t row, float inv) const {
        if (k >= 0) a.xq[row + k] = int8_t(q8(inv == 0.0f ? 0.0f : w, inv));
    }
};

template <int CTRL>
__device__ __forceinline__ double add_moved(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = uint32_t(__builtin_amdgcn_update_dpp(0, int(uint32_t(b)), CTRL, 0xF, 0xF, false));
    const uint32_t hi = uint32_t(__builtin_amdgcn_update_dpp(0, int(uint32_t(b >> 32)), CTRL, 0xF, 0xF, false));
    return v + __builtin_bit_cast(double, (uint64_t(hi) << 32) | lo);
}
__device__ __forceinline__ double lane_value(double v, int lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = uint32_t(__builtin_amdgcn_readlane(int(uint32_t(b)), lane));
    const uint32_t hi = uint32_t(__builtin_amdgcn_readlane(int(uint32_t(b >> 32)), lane));
    return __builtin_bit_cast(double, (uint64_t(hi) << 32) | lo);
}
// Sum over the 64 lanes of a wave, wave-uniform (the moves of wave_max_nonneg).
__device__ __forceinline__ double wave_sum64(double v) {
    v = add_moved<0xB1>(v);
    v = add_moved<0x4E>(v);
    v = add_moved<0x124>(v);
    v = add_moved<0x128>(v);
    return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}

// Maximum and sum over a workgroup of up to 16 waves.  amax is taken as bits:
// a NaN is above infinity and infinity above all numbers.
struct NormSums {
    double sum[16];
    float amax[16];
};
__device__ __forceinline__ void block_norm(NormSums &s, float &amax, double &sum) {
    amax = wave_max_nonneg(amax);
    sum = wave_sum64(sum);
    const int nw = int(blockDim.x) >> 6;
    if (nw == 1) return;
    const int wv = int(threadIdx.x) >> 6;
    if ((threadIdx.x & 63) == 0) {
        s.amax[wv] = amax;
        s.sum[wv] = sum;
    }
    __syncthreads();
    int b = 0;
    sum = 0.0;
    for (int i = 0; i < nw; ++i) {
        b = max(b, __float_as_int(s.amax[i]));
        sum += s.sum[i];
    }
    amax = __int_as_float(b);
}

// The factor of the codes, and the row's scale by one lane.
__device__ __forceinline__ float norm_scale(const NormLaunch &a, int m, float amax, double sum) {
    const bool fine = amax < __builtin_inff() && sum < __builtin_inf();
    if (threadIdx.x == 0) {
        const double rms = sqrt(sum / double(a.K) + double(a.eps));
        a.sa[m] = !fine ? __builtin_nanf("") : amax == 0.0f ? 0.0f : float(double(amax) / 127.0 / rms);
    }
    return fine && amax != 0.0f ? fminf(127.0f / amax, __FLT_MAX__) : 0.0f;
}

// One workgroup per row, CPL chunks of 8 values per lane, and ENDS by the last lanes.
template <int TYPE, int CPL, bool ENDS>
__global__ __launch_bounds__(1024) void norm_rows_kernel(NormLaunch a) {
    __shared__ NormSums red;
    const int tid = int(threadIdx.x), bd = int(blockDim.x), m = int(blockIdx.x);
    const int64_t row = int64_t(m) * a.K;
    const int head = ENDS ? min(int(-row) & 7, a.K) : 0, nc = (a.K - head) >> 3;
    float v[CPL][8], amax = 0.0f;
    double sum = 0.0;
    // All loads first (2045 x 6912 fp32 17.5 us, 19.7 a chunk after the other);
    // lanes without a chunk read the row's last.
    Chunk<TYPE> q[CPL];
    Ends<TYPE> ends;
    if (nc > 0) {
#pragma unroll
        for (int i = 0; i < CPL; ++i) q[i].load(a, row, head + 8 * min(tid + i * bd, nc - 1));
    }
    if (ENDS) ends.load(a, row, head, nc);
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
        const int c = tid + i * bd;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
        if (c < nc) q[i].use(a, row, head + 8 * c, v[i], sum);
    }
#pragma unroll
    for (int i = 0; i < CPL; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = abs_max(amax, v[i][j]);
    if (ENDS) ends.use(a, row, sum, amax);
    block_norm(red, amax, sum);
    const float inv = norm_scale(a, m, amax, sum);
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
        if (inv == 0.0f) {
            // (a NaN times 0 is no code 0)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
        }
        if (tid + i * bd < nc) store_codes(a, row + head + 8 * (tid + i * bd), v[i], inv);
    }
    if (ENDS) ends.store(a, row, inv);
}

// Rows of any length: the second walk reads h, which this lane wrote (x
// where there is no residual).
template <int TYPE>
__global__ __launch_bounds__(1024) void norm_long_kernel(NormLaunch a) {
    __shared__ NormSums red;
    const int tid = int(threadIdx.x), bd = int(blockDim.x), m = int(blockIdx.x);
    const int64_t row = int64_t(m) * a.K;
    const int head = min(int(-row) & 7, a.K), nc = (a.K - head) >> 3;
    float amax = 0.0f, v[8];
    double sum = 0.0;
    Chunk<TYPE> q;
    Ends<TYPE> ends;
    ends.load(a, row, head, nc);
    for (int c = tid; c < nc; c += bd) {
        q.load(a, row, head + 8 * c);
        q.use(a, row, head + 8 * c, v, sum);
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = abs_max(amax, v[j]);
    }
    ends.use(a, row, sum, amax);
    block_norm(red, amax, sum);
    const float inv = norm_scale(a, m, amax, sum);
    NormLaunch again = a;
    if (a.residual) again.x = a.h;
    again.residual = nullptr;
    for (int c = tid; c < nc; c += bd) {
        q.load(again, row, head + 8 * c);
        q.use(again, row, head + 8 * c, v, sum);
        if (inv == 0.0f) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = 0.0f;
        }
        store_codes(a, row + head + 8 * c, v, inv);
    }
    ends.store(a, row, inv);
}

// Lanes of a row: with a row or less for every compute unit, one chunk to a
// lane; beyond, lanes of up to four chunks, so that more rows are on their way
// (us, rows of 1024, 512 and 256 lanes where these are enough: 8192 x 5120 bf16
// with a residual 60.5, 56.5 and 56.0, 2048 x 6912 26.5, 23.7 and 23.4, 2045 x 6912
// fp32 without 22.1, 17.8 and 17.4, 8192 x 2560 30.1, 30.4 and 30.7).
template <int TYPE>
hipError_t norm_type(const NormLaunch &a, int cus, hipStream_t stream) {
    const int slots = std::max(1, a.K / 8);
    const void *fn = reinterpret_cast<const void *>(&norm_long_kernel<TYPE>);
    int threads = 1024;
    if (slots <= kMaxChunks) {
        static const void *const fns[2][4] = {
            {reinterpret_cast<const void *>(&norm_rows_kernel<TYPE, 1, false>),
             reinterpret_cast<const void *>(&norm_rows_kernel<TYPE, 2, false>),
             reinterpret_cast<const void *>(&norm_rows_kernel<TYPE, 3, false>),
             reinterpret_cast<const void *>(&norm_rows_kernel<TYPE, 4, false>)},
            {reinterpret_cast<const void *>(&norm_rows_kernel<TYPE, 1, true>),
             reinterpret_cast<const void *>(&norm_rows_kernel<TYPE, 2, true>),
             reinterpret_cast<const void *>(&norm_rows_kernel<TYPE, 3, true>),
             reinterpret_cast<const void *>(&norm_rows_kernel<TYPE, 4, true>)}};
        const int lanes = a.M > cus ? 256 : 1024;
        const int cpl = std::max(std::min(4, (slots + lanes - 1) / lanes), (slots + 1023) / 1024);
        fn = fns[a.K % 8 != 0][cpl - 1];
        threads = ((slots + cpl - 1) / cpl + 63) / 64 * 64;
    }
    NormLaunch l = a;
    void *args[] = {&l};
    return hipLaunchKernel(fn, dim3(unsigned(a.M)), dim3(unsigned(threads)), args, 0, stream);
}

}  // namespace

hipError_t launch_rmsnorm_quant(const NormLaunch &a, int type, int cus, hipStream_t stream) {
    return type == W2A8_F32    ? norm_type<W2A8_F32>(a, cus, stream)
           : type == W2A8_BF16 ? norm_type<W2A8_BF16>(a, cus, stream)
                               : norm_type<W2A8_F16>(a, cus, stream);
}

}  // namespace w2a8
