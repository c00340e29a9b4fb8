// Device helpers of the MX4 product kernels: buffer loads into registers and
// straight into LDS, and the waits that go with them.
//
// The kernels count their loads themselves (the compiler does not tie a read
// of LDS to the load that fills it).  Loads return in the order in which they
// were issued, so "at most N on their way" names the ones that have landed.
#pragma once

#include <type_traits>

#include "mx4.h"

namespace w2a8 {

enum { kMx4Weights = 0, kTernary = 1 };   // KIND of the product kernels

// A buffer resource over `bytes` bytes (reads past them give 0).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t mx4_buffer(const uint8_t *p, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(p), 0,
                                             int(min(bytes, int64_t(0x7FFFFFFF))), 0x00020000);
}

// Loads at lane offset `off` and uniform offset `tile`: 16 or 4 bytes a lane
// straight into LDS (lane l's at dst + 16 l or 4 l), 16 bytes, 4 bytes.  They
// keep their place among the other memory operations.
__device__ __forceinline__ void mx4_load_lds16(__amdgpu_buffer_rsrc_t b, uint8_t *dst, int off,
                                               int tile) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (__attribute__((address_space(3))) void *)dst, 16, off,
                                             tile, 0, 0);
    __asm__ volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void mx4_load_lds4(__amdgpu_buffer_rsrc_t b, uint8_t *dst, int off,
                                              int tile) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (__attribute__((address_space(3))) void *)dst, 4, off,
                                             tile, 0, 0);
    __asm__ volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ v4u mx4_load16(__amdgpu_buffer_rsrc_t b, int off, int tile) {
    const v4u v = __builtin_amdgcn_raw_buffer_load_b128(b, off, tile, 0);
    __asm__ volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    return v;
}
__device__ __forceinline__ uint32_t mx4_load4(__amdgpu_buffer_rsrc_t b, int off, int tile) {
    const uint32_t v = __builtin_amdgcn_raw_buffer_load_b32(b, off, tile, 0);
    __asm__ volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    return v;
}

// Waits until at most N of this wave's loads are on their way.
template <int N>
__device__ __forceinline__ void mx4_wait_loads() {
    static_assert(N < 64, "counter of 6 bits");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (0xF << 8) | (0x7 << 4));
    __asm__ volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}
// This wave's LDS reads (and writes) are done.
__device__ __forceinline__ void mx4_wait_lds() {
    __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
    __asm__ volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}
// All waves are here (what they waited for before is then visible).
__device__ __forceinline__ void mx4_barrier() {
    __asm__ volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    __asm__ volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// A wave's LDS writes are seen by its lanes' reads behind this (LDS keeps a
// wave's order; the compiler has to).
__device__ __forceinline__ void mx4_wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Output tiles of a product, MBLK x NBLK.  Workgroups are dealt to the eight
// dies in turn, so each die is given a run of consecutive units; units walk
// `group` m-blocks, then n, so that what a die works on at a time (32
// compute units) is near square and shares its operands in the die's L2.
// (Groups of 4 against 8 and 32 at 8192 x 13824 x 5120 MX4: 330, 359 and 368
// us with 128 x 256 tiles.)
struct Mx4Grid {
    int MBLK, NBLK, group;
    uint32_t units;
    // False if there are more tiles than a launch numbers (their results
    // would not fit the memory of the device).
    bool set(int M, int N, int BM, int BN) {
        MBLK = int(ceil_div(M, BM));
        NBLK = int(ceil_div(N, BN));
        const int64_t n = int64_t(MBLK) * NBLK;
        units = uint32_t(n);
        group = MBLK < 4 ? MBLK : 4;
        return n < (int64_t(1) << 31) - 16;
    }
};
__device__ __forceinline__ void mx4_unit(const Mx4Grid &gr, uint32_t unit, int *mblk, int *nblk) {
    const uint32_t g0 = unit / (uint32_t(gr.group) * uint32_t(gr.NBLK)) * uint32_t(gr.group);
    const uint32_t gm = min(uint32_t(gr.group), uint32_t(gr.MBLK) - g0);
    const uint32_t in = unit - g0 * uint32_t(gr.NBLK);
    *mblk = int(g0 + in % gm);
    *nblk = int(in / gm);
}

// Result rows in LDS: 16 rows of COLS fp32, in chunks of four columns; with
// SWIZZLE chunk c of row i sits at c ^ (i % 8), otherwise rows are padded by
// one chunk.
template <int COLS, bool SWIZZLE>
__device__ __forceinline__ int mx4_out_at(int row, int chunk) {
    return SWIZZLE ? row * COLS + 4 * (chunk ^ (row & 7)) : row * (COLS + 4) + 4 * chunk;
}

// 16 bytes of a result row; PASS: past the caches.  (Two functions: a template
// argument would drop the pointer's alignment, that of one element.)
template <bool PASS>
__device__ __forceinline__ void mx4_store16(v4f_any *y, v4f v) {
    if constexpr (PASS)
        __builtin_nontemporal_store(v, y);
    else
        *y = v;
}
template <bool PASS>
__device__ __forceinline__ void mx4_store16(v4u_any *y, v4u v) {
    if constexpr (PASS)
        __builtin_nontemporal_store(v, y);
    else
        *y = v;
}

// Stores eight bf16 results of row m from column n where in range.
template <bool PASS>
__device__ __forceinline__ void mx4_store_bf16(const Mx4Launch &a, int m, int n, v4u w) {
    if (m >= a.M || n >= a.N) return;
    uint16_t *y = a.y_bf16 + int64_t(m) * a.N + n;
    if (n + 7 < a.N) {
        mx4_store16<PASS>(reinterpret_cast<v4u_any *>(y), w);
        return;
    }
    for (int e = 0; n + e < a.N; ++e) {
        const uint32_t d = e < 2 ? w[0] : e < 4 ? w[1] : e < 6 ? w[2] : w[3];
        y[e] = uint16_t(d >> (16 * (e & 1)));
    }
}

// Stores 16 result rows of COLS columns to y[mb ..][n0 ..] where in range, 16
// bytes a lane (at any alignment of the rows; single elements where a lane's
// columns pass the row's end).
template <int COLS, bool SWIZZLE, bool PASS>
__device__ __forceinline__ void mx4_store_rows(const Mx4Launch &a, const uint8_t *lds, int mb, int n0,
                                               int lane) {
    const float *rows = reinterpret_cast<const float *>(lds);
    if (a.y_f32) {
        constexpr int kLanes = COLS / 4, kRows = 64 / kLanes;   // lanes of a row, rows at a time
        const int chunk = lane % kLanes, n = n0 + 4 * chunk;
#pragma unroll 2
        for (int row = lane / kLanes; row < 16; row += kRows) {
            const v4f v = *reinterpret_cast<const v4f *>(rows + mx4_out_at<COLS, SWIZZLE>(row, chunk));
            if (mb + row >= a.M || n >= a.N) continue;
            float *y = a.y_f32 + int64_t(mb + row) * a.N + n;
            if (n + 3 < a.N)
                mx4_store16<PASS>(reinterpret_cast<v4f_any *>(y), v);
            else
                for (int e = 0; n + e < a.N; ++e) y[e] = e == 0 ? v[0] : e == 1 ? v[1] : v[2];
        }
    }
    if (a.y_bf16) {
        constexpr int kLanes = COLS / 8, kRows = 64 / kLanes;
        const int chunk = 2 * (lane % kLanes), n = n0 + 4 * chunk;
#pragma unroll 2
        for (int row = lane / kLanes; row < 16; row += kRows) {
            const v4f v = *reinterpret_cast<const v4f *>(rows + mx4_out_at<COLS, SWIZZLE>(row, chunk));
            const v4f u = *reinterpret_cast<const v4f *>(rows + mx4_out_at<COLS, SWIZZLE>(row, chunk + 1));
            mx4_store_bf16<PASS>(a, mb + row, n,
                                 v4u{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(u[0], u[1]),
                                     bf16_pair(u[2], u[3])});
        }
    }
}

}  // namespace w2a8
