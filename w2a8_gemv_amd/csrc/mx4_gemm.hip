// Products of MX4 rows for many rows (prefill) on gfx950:
// v_mfma_scale_f32_16x16x128_f8f6f4 tiles, activations through LDS.
//
//   y[m][n] = s_w * sum_b 2^(ex + ew) * sum_{k in b} qx * qw
//
// First operand 16 weight rows x 128 k, second operand 16 activation rows x
// 128 k (lane l: row l % 16, block l / 16 of the tile, 16 bytes).
//
//  * Workgroup = KS groups of WM x WN waves.  Wave (wm, wn) of a group owns
//    MB blocks of 16 activation rows and 64 weight rows (four blocks): every
//    activation operand read from LDS feeds four instructions, every weight
//    operand MB.
//  * MX4 weights go from memory straight into operand registers, three tiles
//    ahead (a tile of a strip is 1 KiB in operand order).
//  * Ternary weights go through LDS, three tiles ahead, because a T32x128
//    slot holds four rows of 16 k: block j of lane r stands for row 4r + j of
//    the wave's 64, so that two 16-byte reads give a lane its words of all
//    four blocks.  Slot kg of row group rg sits at 8 rg + (kg ^ rg % 8).
//  * Activations reach a ring of four LDS stages by direct global->LDS loads,
//    three tiles ahead; 16 bytes of row r, block g sit at slot 4r + (g ^
//    (r / 2 % 4)) of a KiB, so the loads read whole 64-byte rows and eight
//    lanes' operand reads (128 bytes) cover all of 128 bytes' banks.
//  * Scale words (four tiles' bytes) are loaded a group of four tiles ahead,
//    the activations' into LDS by 16 bytes a row, the weights' into
//    registers; the instruction picks the tile's byte.
//  * Per tile: this wave's loads of the tile after it have landed (loads return
//    in order), barrier, then the blocks of instructions; between them, one at
//    a time, the operand reads of the blocks after them (at the end those of
//    the next tile, so that no wave waits for LDS behind the barrier) and the
//    loads of later tiles: issued together, the loads of all waves would hold
//    up every wave's instructions.  The barrier waits for no LDS read: what a
//    stage held has been used before the barrier ahead of its next load.
//  * Ternary words become 4-bit floats between the instructions, one weight
//    block ahead of its use (for all blocks at the start of a tile they kept the
//    matrix pipe waiting: a tile of 64 x 128 over two groups 0.29 us, now
//    0.22, operands in the L2; 1024 x 2560 x 6912 20.2 us, now 18.6).
//  * Tiles that a short last quad lacks are not stepped through (4001 x 13824 x
//    2688 ternary 83.6 us, 92 before).
//  * KS > 1 (grids smaller than the device): the groups take the quads of
//    tiles in turn and add up through LDS at the end, in group order.
//  * Results pass through LDS, 16 rows x 64 columns at a time, so that the
//    stores are whole lines.
//  * Rows past M repeat row M - 1, strips past the matrix its last strip;
//    neither is stored.

#include "mx4.h"
#include "mx4_device.h"

namespace w2a8 {
namespace {

constexpr int kStages = 4;        // tiles in the ring; the unroll of the k loop
constexpr int kNB = 4;            // weight blocks of a wave

template <int KIND, int WM, int WN, int MB, int KS>
struct Tile {
    static constexpr int NW = WM * WN;                 // waves of a group
    static constexpr int BM = WM * MB * 16, BN = WN * kNB * 16;
    // KiB loads of a stage and of a quad's scales, and how many a wave makes
    // (with fewer parts than waves, several waves make the same one).
    static constexpr int per_wave(int parts) { return parts >= NW ? parts / NW : 1; }
    static constexpr bool splits(int parts) { return parts >= NW ? parts % NW == 0 : NW % parts == 0; }
    static constexpr int XPART = BM / 16, WPART = KIND == kTernary ? BN / 32 : 0;
    static constexpr int SPART = BM > 64 ? BM / 64 : 1;
    static_assert(splits(XPART) && splits(SPART) && (KIND != kTernary || splits(WPART)), "uneven");
    static constexpr int XD = per_wave(XPART), SD = per_wave(SPART);
    static constexpr int WD = KIND == kTernary ? per_wave(WPART) : kNB;   // weight loads a tile
    static constexpr int STAGE = (XPART + WPART) * 1024, SBUF = SPART * 1024;
    static constexpr int GROUP = kStages * STAGE + 2 * SBUF;
    static constexpr int RED = (KS - 1) * BM * BN * 4;
    static constexpr int OUTROWS = 16 * 68 * 4, OUT = NW * OUTROWS;   // a wave's result rows
    static constexpr int max3(int a, int b, int c) { return a > b ? (a > c ? a : c) : (b > c ? b : c); }
    static constexpr int LDS = max3(KS * GROUP, RED, OUT);
    static constexpr int THREADS = 64 * NW * KS;
    // Waves per SIMD to leave room for: two workgroups of four waves, or as
    // many as one larger workgroup needs.
    static constexpr int EU = THREADS <= 256 ? 2 : THREADS / 256;
};

template <int KIND, int WM, int WN, int MB, int KS, bool PASS>
__global__ __launch_bounds__(64 * WM * WN * KS, (Tile<KIND, WM, WN, MB, KS>::EU))
    void mx4_gemm_kernel(Mx4Launch a, Mx4Grid gr) {
    using T = Tile<KIND, WM, WN, MB, KS>;
    __shared__ __attribute__((aligned(1024))) uint8_t ring[T::LDS];
    const int lane = int(threadIdx.x) & 63;
    const int wall = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const int grp = wall / T::NW, wv = wall % T::NW;
    const int wm = wv / WN, wn = wv % WN;
    const int r = lane & 15, g = lane >> 4;

    const int64_t blocks = int64_t(gridDim.x) * gridDim.y;   // a multiple of 8
    const int64_t id = blockIdx.x + int64_t(blockIdx.y) * gridDim.x;
    const int64_t unit = (id & 7) * (blocks >> 3) + (id >> 3);
    if (unit >= gr.units) return;
    int mblk, nblk;
    mx4_unit(gr, uint32_t(unit), &mblk, &nblk);
    const int m0 = mblk * T::BM, nb = nblk * T::BN, n0 = nb + wn * 64;
    uint8_t *lds = ring + grp * T::GROUP;

    // Every operand is addressed as a base of the workgroup or wave, an offset
    // of the lane and an offset of the tile (buffer loads: base and tile
    // offset in scalar registers).
    // Direct loads: lane l of part p brings row 16p + l/4, block (l%4) ^ (l/8%4).
    const int xrow = a.KT * kMxRowTile, srow = a.KU * 16;
    const int rows = min(T::BM, a.M - m0);
    const auto xbuf = mx4_buffer(a.xq + int64_t(m0) * xrow, int64_t(rows) * xrow);
    int xoff[T::XD], xpart[T::XD];
#pragma unroll
    for (int d = 0; d < T::XD; ++d) {
        xpart[d] = T::XPART >= T::NW ? wv * T::XD + d : wv % T::XPART;
        xoff[d] = min(16 * xpart[d] + (lane >> 2), rows - 1) * xrow +
                  16 * ((lane & 3) ^ ((lane >> 3) & 3));
    }
    // Weights: a tile of either kind is 1 KiB.  MX4: this wave's four strips,
    // operand order.  Ternary: lane l of part p brings slot (l%8) ^ (l/8) of
    // row group l/8 of the workgroup's strip p.
    constexpr int kRows = KIND == kTernary ? kTileRows : kMxRows;
    const int NS = (a.N + kRows - 1) / kRows;
    const int wstrip = a.KT * 1024;
    const int s0 = min((KIND == kTernary ? nb : n0) / kRows, NS - 1);
    const int strips = min((KIND == kTernary ? T::BN : 64) / kRows, NS - s0);
    const auto wbuf = mx4_buffer(a.w + int64_t(s0) * wstrip, int64_t(strips) * wstrip);
    int woff[T::WD], wpart[T::WD];
#pragma unroll
    for (int d = 0; d < T::WD; ++d) {
        wpart[d] = KIND != kTernary ? d : T::WPART >= T::NW ? wv * T::WD + d : wv % T::WPART;
        woff[d] = min(wpart[d], strips - 1) * wstrip +
                  16 * (KIND == kTernary ? (lane & 56) + ((lane & 7) ^ (lane >> 3)) : lane);
    }
    const auto wsbuf = mx4_buffer(KIND == kTernary ? a.w : a.ws + int64_t(s0) * a.KU * 256,
                              int64_t(strips) * a.KU * 256);
    // Activation scales: lane l of part p brings the 16 bytes of row 64p + l.
    const auto xsbuf = mx4_buffer(a.xs + int64_t(m0) * srow, int64_t(rows) * srow);
    int xsoff[T::SD], spart[T::SD];
#pragma unroll
    for (int d = 0; d < T::SD; ++d) {
        spart[d] = T::SPART >= T::NW ? wv * T::SD + d : wv % T::SPART;
        xsoff[d] = min(64 * spart[d] + lane, rows - 1) * srow;
    }
    const int last = a.KT - 1;

    v4f acc[MB][kNB];
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
        for (int j = 0; j < kNB; ++j) acc[b][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

    v4u w[kStages][kNB];               // MX4: operands of tiles t .. t + 3
    uint32_t ws[kNB], wsn[kNB];        // scales of this quad and the next

    // Load d of tile t's weights (past the last tile: of the last) into
    // register set or stage i, and of its activations into stage i.
    auto load_w = [&](int d, int t, int i) __attribute__((always_inline)) {
        const int tc = min(t, last) * 1024;
        if constexpr (KIND == kTernary)
            mx4_load_lds16(wbuf, lds + i * T::STAGE + (T::XPART + wpart[d]) * 1024, woff[d], tc);
        else
            w[i][d] = mx4_load16(wbuf, woff[d], tc);
    };
    auto load_x = [&](int d, int t, int i) __attribute__((always_inline)) {
        mx4_load_lds16(xbuf, lds + i * T::STAGE + xpart[d] * 1024, xoff[d], min(t, last) * kMxRowTile);
    };
    // Scales of quad u (clamped): the rows' into buffer i, the weights' into s.
    auto scales = [&](int u, int i, uint32_t (&s)[kNB]) {
        const int uc = min(u, a.KU - 1);
#pragma unroll
        for (int d = 0; d < T::SD; ++d)
            mx4_load_lds16(xsbuf, lds + kStages * T::STAGE + i * T::SBUF + spart[d] * 1024, xsoff[d],
                       uc * 16);
        if constexpr (KIND != kTernary) {
#pragma unroll
            for (int j = 0; j < kNB; ++j)
                s[j] = mx4_load4(wsbuf, min(j, strips - 1) * a.KU * 256 + 4 * lane, uc * 256);
        }
    };

    // Operand reads: 16 bytes of row r, block g of a part; ternary: slots 2g
    // and 2g + 1 of row group r (of 8) in the wave's strip r / 8.
    const int xfrag = wm * MB * 1024 + 16 * (4 * r + (g ^ ((r >> 1) & 3)));
    const int wfrag = (T::XPART + 2 * wn + (r >> 3)) * 1024 + 128 * (r & 7);

    // Operands in registers ahead of their instructions.  MX4: kPre activation
    // blocks.  Ternary: all of them, of this tile and the next if MB <= 4, the
    // lane's words of both tiles, and two blocks' weights.
    constexpr int kPre = KIND == kTernary || MB < 4 ? MB : 4, kSets = KIND == kTernary && MB <= 4 ? 2 : 1;
    v4u x[kSets][kPre], half[2][2], wf[2];
    uint32_t xs[MB], xsn[MB];
    auto read_x = [&](int set, int st, int b) __attribute__((always_inline)) {
        x[set][b % kPre] = *reinterpret_cast<const v4u *>(lds + st * T::STAGE + xfrag + b * 1024);
    };
    auto read_half = [&](int set, int st) __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            half[set][h] = *reinterpret_cast<const v4u *>(lds + st * T::STAGE + wfrag +
                                                          16 * ((2 * g + h) ^ (r & 7)));
    };
    auto read_scales = [&](int i, uint32_t (&s)[MB]) __attribute__((always_inline)) {
        const uint8_t *sc = lds + kStages * T::STAGE + i * T::SBUF + wm * MB * 256 + 16 * r + 4 * g;
#pragma unroll
        for (int b = 0; b < MB; ++b) s[b] = *reinterpret_cast<const uint32_t *>(sc + 256 * b);
    };

    // One tile: quad u's tile TT; `next` is the group's quad after u.
    auto tile = [&](auto tt, auto full, int q, int u, int next) __attribute__((always_inline)) {
        constexpr int TT = decltype(tt)::value, NEXT = (TT + 1) % kStages;
        constexpr bool FULL = decltype(full)::value;
        // The loads of the tile after this one have landed.
        if constexpr (KIND == kTernary) {
            // Issued since: those of one tile, and before tiles 1 and 2 the
            // next quad's scales.
            mx4_wait_loads<T::XD + T::WD + (TT == 1 || TT == 2 ? T::SD : 0)>();
        } else {
#pragma unroll
            for (int j = 0; j < kNB; ++j) __asm__ volatile("" ::"v"(w[NEXT][j]));
        }
        // (What a wave has read of the stage that is loaded next, it has used,
        // but for reads past the last tile, whose values nobody uses.)
        mx4_barrier();
        // Loads between the blocks of instructions, three tiles ahead (the
        // weights last: waiting for them covers the activations).
        auto load = [&](int i) __attribute__((always_inline)) {
            const int t = TT < 1 ? 4 * u + 3 : 4 * next + TT - 1;
            if (i < T::XD)
                load_x(i, t, (TT + 3) % kStages);
            else if (i < T::XD + T::WD)
                load_w(i - T::XD, t, (TT + 3) % kStages);
        };
        constexpr int kLoads = T::WD + T::XD, kEach = (kLoads + MB - 1) / MB;
        // (Without other groups, only tiles that exist are stepped through.)
        const bool live = FULL || KS == 1 || 4 * u + TT <= last;
        if constexpr (KIND == kTernary) {
            constexpr int SET = TT & 1, XSET = kSets > 1 ? SET : 0, XNEXT = kSets > 1 ? SET ^ 1 : 0;
            // Weight block j with all activations, and between the
            // instructions the next weight block (of the next tile at last).
#pragma unroll
            for (int j = 0; j < kNB; ++j) {
#pragma unroll
                for (int b = 0; b < MB; ++b) {
                    if (live)
                        acc[b][j] = mx4_mfma<TT>(wf[j & 1], x[XSET][b], acc[b][j], kTernaryScale, xs[b]);
                    __builtin_amdgcn_sched_barrier(0);
                    constexpr int kWords = MB < 4 ? 4 / MB : 1;
#pragma unroll
                    for (int e = b * kWords; e < (b + 1) * kWords; ++e)
                        if (e < 4) {
                            const uint32_t c = j < 3 ? half[SET][e >> 1][j < 3 ? j + 1 : 0]
                                                     : half[SET ^ 1][e >> 1][0];
                            wf[(j + 1) & 1][e] = ternary_word(e & 1 ? c : c << 2);
                        }
                    if (j == (kSets > 1 ? 0 : 3)) read_x(XNEXT, NEXT, b);
                    __builtin_amdgcn_sched_barrier(0);
                }
                if (j == 0) read_half(SET ^ 1, NEXT);
                if (j == 0 && TT == 3) read_scales((q + 1) & 1, xsn);
#pragma unroll
                for (int i = j; i < kLoads; i += 4) load(i);
            }
        } else {
#pragma unroll
            for (int b = 0; b < MB; ++b) {
                if (live) {
#pragma unroll
                    for (int j = 0; j < kNB; ++j)
                        acc[b][j] = mx4_mfma<TT>(w[TT][j], x[0][b % kPre], acc[b][j], ws[j], xs[b]);
                }
                __builtin_amdgcn_sched_barrier(0);
                read_x(0, b + kPre < MB ? TT : NEXT, (b + kPre) % MB);
#pragma unroll
                for (int i = b * kEach; i < (b + 1) * kEach; ++i) load(i);
            }
        }
        // (The other buffer's readers are done; ahead of the loads that the
        // quad's third tile waits for.)
        if constexpr (TT == 0) scales(next, (q + 1) & 1, wsn);
        if constexpr (TT == 3) {
            if constexpr (KIND == kTernary) {
#pragma unroll
                for (int b = 0; b < MB; ++b) xs[b] = xsn[b];
            } else {
                read_scales((q + 1) & 1, xs);
#pragma unroll
                for (int j = 0; j < kNB; ++j) ws[j] = wsn[j];
            }
        }
    };

    // The group's quads: grp, grp + KS, ...; all groups take as many steps.
    scales(grp, 0, ws);
#pragma unroll
    for (int t = 0; t < 3; ++t) {
#pragma unroll
        for (int d = 0; d < T::XD; ++d) load_x(d, 4 * grp + t, t);
#pragma unroll
        for (int d = 0; d < T::WD; ++d) load_w(d, 4 * grp + t, t);
    }
    // The first tile's operands.
    if constexpr (KIND == kTernary) {
        mx4_wait_loads<2 * (T::XD + T::WD)>();
    } else {
#pragma unroll
        for (int j = 0; j < kNB; ++j) __asm__ volatile("" ::"v"(w[0][j]));
    }
    mx4_barrier();
#pragma unroll
    for (int b = 0; b < kPre; ++b) read_x(0, 0, b);
    read_scales(0, xs);
    if constexpr (KIND == kTernary) {
        read_half(0, 0);
        wf[0] = ternary_fp4(half[0][0][0], half[0][1][0]);
    }

    auto quad = [&](auto full, int q) __attribute__((always_inline)) {
        // (All groups take the steps of the first, which has the most tiles.)
        const int u = q * KS + grp, next = u + KS;
        const int n = decltype(full)::value ? 4 : a.KT - 4 * q * KS;
        tile(std::integral_constant<int, 0>{}, full, q, u, next);
        if (n > 1) tile(std::integral_constant<int, 1>{}, full, q, u, next);
        if (n > 2) tile(std::integral_constant<int, 2>{}, full, q, u, next);
        if (n > 3) tile(std::integral_constant<int, 3>{}, full, q, u, next);
    };
    // Rounds of quads that are whole in every group, then the last one.
    const int whole = a.KT / (4 * KS);
#pragma unroll 1
    for (int q = 0; q < whole; ++q) quad(std::true_type{}, q);
    if (4 * whole * KS < a.KT) quad(std::false_type{}, whole);

    // The repeats of the last tile are still on their way into LDS; then every
    // operand has been read.
    mx4_wait_loads<0>();
    __syncthreads();
    if constexpr (KS > 1) {
        v4f *red = reinterpret_cast<v4f *>(ring);
        if (grp > 0) {
#pragma unroll
            for (int b = 0; b < MB; ++b)
#pragma unroll
                for (int j = 0; j < kNB; ++j)
                    red[((((grp - 1) * T::NW + wv) * MB + b) * kNB + j) * 64 + lane] = acc[b][j];
        }
        __syncthreads();
        if (grp == 0) {
#pragma unroll 1
            for (int p = 0; p < KS - 1; ++p)
#pragma unroll
                for (int b = 0; b < MB; ++b)
#pragma unroll
                    for (int j = 0; j < kNB; ++j) {
                        const v4f v = red[(((p * T::NW + wv) * MB + b) * kNB + j) * 64 + lane];
                        acc[b][j] = v4f{acc[b][j][0] + v[0], acc[b][j][1] + v[1],
                                        acc[b][j][2] + v[2], acc[b][j][3] + v[3]};
                    }
        }
        __syncthreads();
        if (grp > 0) return;
    }

    // Lane (r, g) holds row 16b + r and columns 16j + 4g + e (MX4) or 16g +
    // 4e + j (ternary) of the wave's 64.
    uint8_t *out = ring + wv * T::OUTROWS;
    auto dump = [&](int b) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v4f v = acc[b][i];
            if constexpr (KIND == kTernary)
                v = v4f{acc[b][0][i], acc[b][1][i], acc[b][2][i], acc[b][3][i]};
            const int chunk = KIND == kTernary ? 4 * g + i : 4 * i + g;
            *reinterpret_cast<v4f *>(out + 4 * mx4_out_at<64, false>(r, chunk)) =
                KIND == kTernary ? v4f{v[0] * a.sw, v[1] * a.sw, v[2] * a.sw, v[3] * a.sw} : v;
        }
    };
#pragma unroll 1
    for (int b = 0; b < MB; ++b) {
        const int mb = m0 + (wm * MB + b) * 16;
        if (mb >= a.M) break;
        switch (b) {
        case 0: dump(0); break;
        case 1: if (MB > 1) dump(MB > 1 ? 1 : 0); break;
        case 2: if (MB > 2) dump(MB > 2 ? 2 : 0); break;
        case 3: if (MB > 3) dump(MB > 3 ? 3 : 0); break;
        case 4: if (MB > 4) dump(MB > 4 ? 4 : 0); break;
        case 5: if (MB > 5) dump(MB > 5 ? 5 : 0); break;
        case 6: if (MB > 6) dump(MB > 6 ? 6 : 0); break;
        default: if (MB > 7) dump(MB > 7 ? 7 : 0); break;
        }
        mx4_wave_sync();
        mx4_store_rows<64, false, PASS>(a, out, mb, n0, lane);
        mx4_wave_sync();
    }
}

template <int KIND, int WM, int WN, int MB, int KS>
hipError_t gemm_launch(const Mx4Launch &a, bool pass, hipStream_t stream) {
    using T = Tile<KIND, WM, WN, MB, KS>;
    Mx4Grid gr;
    if (!gr.set(a.M, a.N, T::BM, T::BN)) return hipErrorInvalidValue;
    const int64_t blocks = round_up(int64_t(gr.units), 8);
    const int64_t gx = std::min<int64_t>(blocks, int64_t(1) << 20);
    const dim3 grid(unsigned(gx), unsigned(ceil_div(blocks, gx)));
    void *args[] = {const_cast<Mx4Launch *>(&a), &gr};
    // (Where k is split, results always pass: plan_passes.)
    const void *kernel = reinterpret_cast<const void *>(&mx4_gemm_kernel<KIND, WM, WN, MB, KS, true>);
    if constexpr (KS == 1) {
        if (!pass)
            kernel = reinterpret_cast<const void *>(&mx4_gemm_kernel<KIND, WM, WN, MB, KS, false>);
    }
    return hipLaunchKernel(kernel, grid, dim3(T::THREADS), args, 0, stream);
}

// An estimate of what a launch takes in us, from its tiles and the device
// alone: a compute unit takes its workgroups in turns of Q and a last one of m;
// each turn costs E a workgroup (filling, writing results) and per k-tile the
// larger of L (a lone workgroup's latency) and B a workgroup (what the compute
// unit gets through).  All five numbers are fitted (least squares of the
// logarithm) to each tile's times at 150 sizes (M 33 to 4096, N 512 to 55296,
// K 512 to 27648, cold weights, bf16 results), Q as well: it is no occupancy.
// By LDS a compute unit holds one workgroup of 256 x 256, of ternary 16 x 64
// and of 32 x 128, two of ternary 64 x 128, three of MX4 16 x 64, fewer than
// their Q; where L is 0 that changes nothing, at ternary 64 x 128 the estimate
// of a third workgroup is 6% too low, at MX4 16 x 64 that of a fourth 1%.  The
// bytes of results are in it only as far as they go with the tiles.  The choice
// by it is 0.9% (MX4) and 0.4% (ternary) behind the best tile on average, 13%
// at most.  Both sides, us: MX4 512 x 2560 x 6912: 64 x 128 split over two
// groups 14.0, 64 x 256 19.4, 128 x 256 26.1; 512 x 13824 x 2560: 128 x 256
// 18.7, 64 x 256 23.3, 32 x 256 34.3; 64 x 5120 x 27648: 32 x 64 over four
// groups 37.2, 64 x 256 104.  Ternary 512 x 2560 x 6912: 64 x 128 over two
// 12.2, 64 x 256 18.3; 4001 x 13824 x 2560: 128 x 256 73.8, 64 x 256 80.7; 33 x
// 5120 x 27648: 16 x 64 over eight 16.8, 32 x 64 over four 24.4.  (A ring of
// eight stages, six tiles ahead and a barrier for every second tile: 512 x 2560
// x 6912 11.5, but MX4 14.8, and 4001 x 13824 x 2560 104.)
struct Plan {
    int BM, BN, KS, Q;
    float A, E, L, B;
    hipError_t (*launch)(const Mx4Launch &, bool, hipStream_t);
};

float plan_us(const Plan &p, const Mx4Launch &a, int cus) {
    const int64_t units = ceil_div(a.M, p.BM) * ceil_div(a.N, p.BN);
    const int64_t turn = int64_t(cus) * p.Q, full = units / turn;
    const int64_t m = ceil_div(units - full * turn, cus);
    const int round = kMxQuad * p.KS;
    const float tiles = float(a.KT / round * kMxQuad + std::min(a.KT % round, kMxQuad));
    const auto take = [&](float wgs) { return p.E * wgs + tiles * std::max(p.L, p.B * wgs); };
    return p.A + float(full) * take(float(p.Q)) + (m ? take(float(m)) : 0.0f);
}

constexpr Plan kMx4Plans[] = {
    {16, 64, 8, 4, 3.16f, 0.45f, 0.594f, 0.569f, &gemm_launch<kMx4Weights, 1, 1, 1, 8>},
    {32, 64, 4, 4, 3.18f, 0.01f, 0.398f, 0.392f, &gemm_launch<kMx4Weights, 1, 1, 2, 4>},
    {64, 64, 4, 1, 3.29f, 0.77f, 0.543f, 0.0f, &gemm_launch<kMx4Weights, 1, 1, 4, 4>},
    {64, 128, 2, 1, 2.96f, 1.15f, 0.411f, 0.0f, &gemm_launch<kMx4Weights, 1, 2, 4, 2>},
    {32, 256, 1, 4, 3.21f, 0.41f, 0.0f, 0.291f, &gemm_launch<kMx4Weights, 1, 4, 2, 1>},
    {64, 256, 1, 1, 2.57f, 1.40f, 0.337f, 0.0f, &gemm_launch<kMx4Weights, 1, 4, 4, 1>},
    {128, 256, 1, 2, 1.61f, 3.53f, 0.0f, 0.440f, &gemm_launch<kMx4Weights, 1, 4, 8, 1>},
    {256, 256, 1, 2, 0.0f, 10.08f, 0.0f, 0.611f, &launch_mx4_gemm_wide},
};
constexpr Plan kTernaryPlans[] = {
    {16, 64, 8, 2, 1.55f, 1.70f, 0.0f, 0.433f, &gemm_launch<kTernary, 1, 1, 1, 8>},
    {32, 64, 4, 2, 2.24f, 0.87f, 0.362f, 0.261f, &gemm_launch<kTernary, 1, 1, 2, 4>},
    {32, 128, 4, 4, 1.35f, 2.37f, 0.0f, 0.432f, &gemm_launch<kTernary, 1, 2, 2, 4>},
    {64, 128, 2, 3, 2.73f, 1.06f, 0.365f, 0.312f, &gemm_launch<kTernary, 2, 2, 2, 2>},
    {32, 256, 1, 3, 2.60f, 0.75f, 0.276f, 0.167f, &gemm_launch<kTernary, 1, 4, 2, 1>},
    {64, 256, 1, 3, 2.78f, 1.21f, 0.317f, 0.230f, &gemm_launch<kTernary, 1, 4, 4, 1>},
    {128, 256, 1, 2, 2.61f, 2.97f, 0.438f, 0.366f, &gemm_launch<kTernary, 1, 4, 8, 1>},
};

// Whether results pass the caches (non-temporal stores).  That leaves the
// caches to the operands, but where rows of results are no whole lines, the
// parts of a line that two workgroups write no longer meet in them.  Measured
// (MI355X, us, staying and passing): whole lines, 4001 x 13824 x 2560 fp32: MX4
// 123 and 93, ternary 104 and 81.  Parts of lines, 4001 x 13825 fp32, ternary:
// k = 256 54 and 88, 1280 82 and 94, 2560 110 and 105, 5120 165 and 139; MX4
// 256 56 and 80, 2560 133 and 115; 1500 x 13825 bf16, 1920: 31 and 37 ternary;
// small outputs, 1024 x 5121 x 256 fp32: 9.9 and 9.3.
bool results_pass(const Mx4Launch &a) {
    const int64_t bytes = int64_t(a.M) * a.N * ((a.y_f32 ? 4 : 0) + (a.y_bf16 ? 2 : 0));
    const bool lines = a.N % (a.y_bf16 ? 64 : 32) == 0;
    return lines || a.K >= 2048 || bytes < 24 << 20;
}

template <size_t N>
const Plan &best_plan(const Plan (&plans)[N], const Mx4Launch &a, int cus) {
    const Plan *best = plans;
    for (const Plan &p : plans)
        if (plan_us(p, a, cus) < plan_us(*best, a, cus)) best = &p;
    return *best;
}
const Plan &best_plan(const Mx4Launch &a, int cus) {
    return a.ws ? best_plan(kMx4Plans, a, cus) : best_plan(kTernaryPlans, a, cus);
}
// Tiles that split k serve large outputs too, tall ones of few columns; their
// results pass by any sizes.  Measured (MI355X, us, passing and staying, 64 x 128
// over two where results_pass says stay): fp32, MX4: 2217 x 3636 x 919 19.0 and
// 19.6, 72177 x 104 x 1096 23.8 and 24.9; ternary 16.4 and 16.3, 20.4 and 21.5;
// bf16, 38044 x 344 x 985: MX4 23.0 and 25.0, ternary 20.0 and 20.0.
bool plan_passes(const Plan &p, const Mx4Launch &a) { return p.KS > 1 || results_pass(a); }

}  // namespace

Mx4TilePlan mx4_tile_plan(const Mx4Launch &a, int cus) {
    const Plan &p = best_plan(a, cus);
    return {p.BM, p.BN, p.KS, plan_passes(p, a)};
}

hipError_t launch_mx4_gemm(const Mx4Launch &a, int cus, hipStream_t stream) {
    const Plan &p = best_plan(a, cus);
    return p.launch(a, plan_passes(p, a), stream);
}

}  // namespace w2a8
