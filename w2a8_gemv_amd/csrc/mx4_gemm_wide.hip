// Products of MX4 rows with MX4 weights for the largest grids (prefill of
// thousands of rows) on gfx950: 256 x 256 output tiles, four waves of 128 x
// 128, one workgroup to a compute unit.
//
// The other tiles (mx4_gemm.hip) load a weight byte once for every 128 rows
// or fewer; 8192 x 13824 x 5120 takes them 315 us (128 x 256), and this kernel
// 292 us, 2048 x 5120 x 27648 217 and 161 us.  Where the 292 us go: the loop
// gets through k at 4.9 to 5.1 PFLOP/s (2560 more of k take 113 us, 5120 more
// 235 us), which is 230 us for this k, where the instruction alone takes 160
// (7.2 to 7.4 PFLOP/s on rounded normal values; 9.8 on zeros, where the clock
// stays up).  So some 70 us are the loop's stalls and the idle quarter of the
// last of seven turns of tiles, and some 60 their starts and results, hidden by
// nothing: one workgroup fills the compute unit.  Power costs 65 us of the
// whole: the same product of zeros takes 227.  Keeping workgroups and starting
// the next tile's loads ahead of the results was tried (the registers of both
// do not fit, 350 us), as were results straight from the registers (fp32 324
// against 313 us) and all of a wave's results through LDS at once (no change).
//
//  * Both operands go through LDS (each byte is loaded once per workgroup; a
//    wave's 128 x 128 needs 16 KiB of LDS reads per 64 instructions, half of
//    what the LDS delivers in that time).
//  * A ring of four stages of one k-tile; the barrier of step t says that tile
//    t + 1 has landed, so the operands of the next step's first instructions
//    are read during this one and the pipe does not wait for LDS behind a
//    barrier.
//  * LDS reads and loads are placed one by one between the instructions.
//  * The accumulators (256 registers) live in accumulation registers, so one
//    wave to a SIMD has all it needs.
//  * Results go through LDS, so that stores are whole lines.
//
// Operand, scale and ring layouts are those of mx4_gemm.hip.
#include "mx4.h"
#include "mx4_device.h"

namespace w2a8 {
namespace {

constexpr int kTileM = 256, kTileN = 256;
constexpr int kWaves = 4, kB = 8;                 // blocks of 16 per wave and side
constexpr int kStrips = kTileN / kMxRows;
constexpr int kD = kStrips / kWaves;              // loads of a wave, tile and operand
constexpr int kLoads = 2 * kD, kScaleLoads = 2;
constexpr int kWBase = kTileM * kMxRowTile;       // LDS: activations, weights of a stage ...
constexpr int kStage = 2 * kWBase;
constexpr int kScales = 4 * kStage, kScaleBuf = 2 * 4096;   // ... two buffers of a quad's scales
constexpr int kLds = kScales + 2 * kScaleBuf;
static_assert(kLds <= 160 * 1024, "LDS of a compute unit");
static_assert(kWaves * 16 * 128 * 4 <= kScales, "results pass through the ring");

template <bool PASS>
__global__ __launch_bounds__(64 * kWaves, 1) void mx4_gemm_wide_kernel(Mx4Launch a, Mx4Grid gr) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];
    const int lane = int(threadIdx.x) & 63;
    const int wv = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const int wm = wv >> 1, wn = wv & 1;
    const int r = lane & 15, g = lane >> 4;
    const int last = a.KT - 1;
    const int xrow = a.KT * kMxRowTile, srow = a.KU * 16, wstrip = a.KT * kMxTileBytes;

    // Workgroups are dealt to the eight dies in turn.
    const int64_t id = blockIdx.x + int64_t(blockIdx.y) * gridDim.x;
    const int64_t unit = (id & 7) * ((int64_t(gridDim.x) * gridDim.y) >> 3) + (id >> 3);
    if (unit >= gr.units) return;
    int mblk, nblk;
    mx4_unit(gr, uint32_t(unit), &mblk, &nblk);

    // The operands: a base, the lane's offsets, a tile's.
    const int rows = min(kTileM, a.M - mblk * kTileM);
    const auto xbuf = mx4_buffer(a.xq + int64_t(mblk * kTileM) * xrow, int64_t(rows) * xrow);
    const auto xsbuf = mx4_buffer(a.xs + int64_t(mblk * kTileM) * srow, int64_t(rows) * srow);
    const int s0 = nblk * kStrips;
    const int strips = min(kStrips, (a.N + kMxRows - 1) / kMxRows - s0);
    const auto wbuf = mx4_buffer(a.w + int64_t(s0) * wstrip, int64_t(strips) * wstrip);
    const auto wsbuf = mx4_buffer(a.ws + int64_t(s0) * a.KU * 256, int64_t(strips) * a.KU * 256);
    int xoff[kD], woff[kD];
#pragma unroll
    for (int d = 0; d < kD; ++d) {
        xoff[d] = min(16 * (wv * kD + d) + (lane >> 2), rows - 1) * xrow +
                  16 * ((lane & 3) ^ ((lane >> 3) & 3));
        woff[d] = min(wv * kD + d, strips - 1) * wstrip + 16 * lane;
    }
    // Scales: the 16 bytes of row 64 wv + l; bytes 16 (l % 16) of strip 4 wv + l/16's 256.
    const int xsoff = min(64 * wv + lane, rows - 1) * srow;
    const int wsoff = min(4 * wv + (lane >> 4), strips - 1) * a.KU * 256 + 16 * (lane & 15);
    const int m0 = mblk * kTileM + wm * 128, n0 = nblk * kTileN + wn * 128;

    // Load i of tile t (past the last: of the last) into stage st.
    auto load = [&](int i, int t, int st) __attribute__((always_inline)) {
        const int tc = min(t, last);
        uint8_t *dst = lds + st * kStage;
        if (i < kD)
            mx4_load_lds16(xbuf, dst + (wv * kD + i) * 1024, xoff[i < kD ? i : 0], tc * kMxRowTile);
        else
            mx4_load_lds16(wbuf, dst + kWBase + (wv * kD + i - kD) * 1024, woff[i < kD ? 0 : i - kD],
                           tc * kMxTileBytes);
    };
    auto load_scales = [&](int u, int buf) __attribute__((always_inline)) {
        const int uc = min(u, a.KU - 1);
        uint8_t *dst = lds + kScales + buf * kScaleBuf + wv * 1024;
        mx4_load_lds16(xsbuf, dst, xsoff, uc * 16);
        mx4_load_lds16(wsbuf, dst + 4096, wsoff, uc * 256);
    };

    v4f acc[kB][kB];                  // [activation block][weight block]
    v4u wf[2][kB], x[4];              // weights of this tile and the next; activations ahead
    uint32_t xs[2][kB], ws[2][kB];    // scale words of this quad and the next

    const int xfrag = wm * kB * 1024 + 16 * (4 * r + (g ^ ((r >> 1) & 3)));
    const int wfrag = kWBase + wn * kB * 1024 + 16 * lane;
    auto read_x = [&](int st, int b) __attribute__((always_inline)) {
        x[b & 3] = *reinterpret_cast<const v4u *>(lds + st * kStage + xfrag + b * 1024);
    };
    auto read_w = [&](int st, int i, int b) __attribute__((always_inline)) {
        wf[i][b] = *reinterpret_cast<const v4u *>(lds + st * kStage + wfrag + b * 1024);
    };
    auto read_scales = [&](int buf, int i, int b) __attribute__((always_inline)) {
        const uint8_t *sc = lds + kScales + buf * kScaleBuf;
        xs[i][b] = *reinterpret_cast<const uint32_t *>(sc + (wm * kB + b) * 256 + 16 * r + 4 * g);
        ws[i][b] = *reinterpret_cast<const uint32_t *>(sc + 4096 + (wn * kB + b) * 256 + 4 * lane);
    };

    // One step: tile TT of quad u (its operands' first part is in registers).
    auto tile = [&](auto tt, int u) __attribute__((always_inline)) {
        constexpr int TT = decltype(tt)::value, NEXT = (TT + 1) % 4;
        // Tile t + 1 has landed: issued since are one tile's loads, and before
        // the second and third tile of a quad the next quad's scales.
        mx4_wait_loads<kLoads + (TT == 1 || TT == 2 ? kScaleLoads : 0)>();
        mx4_barrier();
#pragma unroll
        for (int b = 0; b < kB; ++b) {
#pragma unroll
            for (int p = 0; p < 4; ++p) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int j = 2 * p + e;
                    acc[b][j] = mx4_mfma<TT>(wf[TT & 1][j], x[b & 3], acc[b][j], ws[0][j], xs[0][b]);
                }
                __builtin_amdgcn_sched_barrier(0);
                // Between each two: activations two blocks ahead, a load of
                // tile t + 3, the next tile's weights, the next quad's scales.
                if (p == 0) read_x(b + 2 < kB ? TT : NEXT, (b + 2) % kB);
                if (p == 1) load(b, 4 * u + TT + 3, (TT + 3) % 4);
                if (p == 2) read_w(NEXT, NEXT & 1, b);
                if (p == 3 && TT == 3) read_scales((u + 1) & 1, 1, b);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        // (The other buffer was last read in the quad before.)
        if constexpr (TT == 0) load_scales(u + 1, (u + 1) & 1);
        if constexpr (TT == 3) {
#pragma unroll
            for (int b = 0; b < kB; ++b) {
                xs[0][b] = xs[1][b];
                ws[0][b] = ws[1][b];
            }
        }
    };
    static_assert(kLoads == kB, "one load a block");
    // n of quad u's tiles.
    auto quad = [&](int u, int n) __attribute__((always_inline)) {
        tile(std::integral_constant<int, 0>{}, u);
        if (n > 1) tile(std::integral_constant<int, 1>{}, u);
        if (n > 2) tile(std::integral_constant<int, 2>{}, u);
        if (n > 3) tile(std::integral_constant<int, 3>{}, u);
    };

    load_scales(0, 0);
#pragma unroll
    for (int t = 0; t < 3; ++t)
#pragma unroll
        for (int i = 0; i < kLoads; ++i) load(i, t, t);
#pragma unroll
    for (int b = 0; b < kB; ++b)
#pragma unroll
        for (int j = 0; j < kB; ++j) {
            acc[b][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
            __asm__ volatile("" : "+a"(acc[b][j]));   // in accumulation registers
        }
    mx4_wait_loads<2 * kLoads>();                     // the first tile and the scales
    mx4_barrier();
#pragma unroll
    for (int b = 0; b < kB; ++b) read_w(0, 0, b);
#pragma unroll
    for (int b = 0; b < kB; ++b) read_scales(0, 0, b);
    read_x(0, 0);
    read_x(0, 1);
    const int whole = a.KT / 4;
#pragma unroll 1
    for (int u = 0; u < whole; ++u) quad(u, 4);
    if (whole < a.KU) quad(whole, a.KT - 4 * whole);

    // The repeats of the last tile have landed and every wave has read its
    // last operands; the ring is free.
    mx4_wait_loads<0>();
    mx4_wait_lds();
    mx4_barrier();
    // 16 rows of 128 columns at a time; lane (r, g) holds columns 16j + 4g .. of
    // row r.  fp32: chunks of 16 bytes (four columns), chunk c of row i at c ^
    // (i % 8).  bf16 alone: chunks of eight columns.
    uint8_t *out = lds + wv * 16 * 128 * 4;
    const bool only_bf16 = !a.y_f32;
    auto dump = [&](int b) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < kB; ++j) {
            const v4f v = acc[b][j];
            if (only_bf16)
                *reinterpret_cast<v2u *>(out + 256 * r + 16 * ((2 * j + (g >> 1)) ^ (r & 7)) + 8 * (g & 1)) =
                    v2u{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
            else
                *reinterpret_cast<v4f *>(out + 4 * mx4_out_at<128, true>(r, 4 * j + g)) = v;
        }
    };
    auto store = [&](int b) __attribute__((always_inline)) {
        if (only_bf16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = 4 * i + (lane >> 4), c = lane & 15;
                mx4_store_bf16<PASS>(a, m0 + 16 * b + row, n0 + 8 * c,
                                     *reinterpret_cast<const v4u *>(out + 256 * row +
                                                                    16 * (c ^ (row & 7))));
            }
        } else {
            mx4_store_rows<128, true, PASS>(a, out, m0 + 16 * b, n0, lane);
        }
    };
#pragma unroll 1
    for (int b = 0; b < kB; ++b) {
        switch (b) {
        case 0: dump(0); break;
        case 1: dump(1); break;
        case 2: dump(2); break;
        case 3: dump(3); break;
        case 4: dump(4); break;
        case 5: dump(5); break;
        case 6: dump(6); break;
        default: dump(7); break;
        }
        mx4_wave_sync();
        store(b);
        mx4_wave_sync();
    }
}

}  // namespace

hipError_t launch_mx4_gemm_wide(const Mx4Launch &a, bool pass, hipStream_t stream) {
    Mx4Grid gr;
    if (!gr.set(a.M, a.N, kTileM, kTileN)) return hipErrorInvalidValue;
    const int64_t blocks = round_up(int64_t(gr.units), 8);
    const int64_t gx = std::min<int64_t>(blocks, int64_t(1) << 20);
    void *args[] = {const_cast<Mx4Launch *>(&a), &gr};
    const void *kernel = pass ? reinterpret_cast<const void *>(&mx4_gemm_wide_kernel<true>)
                              : reinterpret_cast<const void *>(&mx4_gemm_wide_kernel<false>);
    return hipLaunchKernel(kernel, dim3(unsigned(gx), unsigned(ceil_div(blocks, gx))), dim3(64 * kWaves),
                           args, 0, stream);
}

}  // namespace w2a8
