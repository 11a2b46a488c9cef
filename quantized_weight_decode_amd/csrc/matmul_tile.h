// matmul_tile.h -- e4m3 activations times e4m3 weights on the matrix cores, many
// rows, dense or grouped by expert, with the epilogue: the kernel, which several
// files instantiate (it takes the compiler minutes in one).
#pragma once

#include <type_traits>

#include "qg_device.h"
#include "qg_launch.h"
#include "qg_matmul.h"
#include "qg_tile.h"

namespace qg {

struct TileParams {
    MatmulArgs m;
    const ExpertTile *tiles;             // grouped, else nullptr
    int ntm, ntn, col0;                  // tiles of the launch; its first column of y
    int parts, per;                      // parts of K, of `per` steps (dense)
    float *partial;                      // their sums [parts][halves of W][R][ldp], parts > 1
    int ldp;
    bool wide;                           // y, residual and bias can be taken 16 bytes at a time
};

// A launch of `grid` tiles of a kind (matmul_tile.hip).
hipError_t run_tile_f32(const TileParams &p, bool direct, unsigned grid, hipStream_t st);
hipError_t run_tile_large(const TileParams &p, int kind, unsigned grid, hipStream_t st);
hipError_t run_tile_small(const TileParams &p, int kind, unsigned grid, hipStream_t st);
hipError_t run_tile_square(const TileParams &p, bool direct, unsigned grid, hipStream_t st);

// (each of those files has these for itself)
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int TK = 128;                  // columns per K step: one scale block
constexpr int SG = SCALE_STEPS;          // K steps whose scales are fetched together

// All but the wave's last n loads have arrived, and its LDS reads are done, for every
// wave of the workgroup (n uniform; more than 9: as if 0).
__device__ __forceinline__ void wait_some(int n)
{
#define QG_WAIT(N)                                                                          \
    case N: asm volatile("s_waitcnt vmcnt(" #N ") lgkmcnt(0)\n\ts_barrier" ::: "memory"); break
    switch (n) {
        QG_WAIT(4);
        QG_WAIT(5);
        QG_WAIT(6);
        QG_WAIT(7);
        QG_WAIT(8);
        QG_WAIT(9);
    default: asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); break;
    }
#undef QG_WAIT
}

// finish() for rows whose pieces of eight columns lie on 16 bytes: sums of n rows
// from `own` (rows LDR floats apart; gated: the up sums WC behind the gate's), to
// columns col0 .. col0 + WC - 1 of rows row_of(r) of y.  WC / 8 lanes per row, so
// a lane's columns, and their bias, are the same in all its rows.
template <typename XT, int ACT, bool GATED, int WC, int LDR, typename Row>
__device__ __forceinline__ void finish_rows_act(const LinearArgs &a, int expert, const float *own,
                                                int lane, int n, int col0, Row row_of)
{
    typedef typename XT::raw raw;
    typedef typename Eight<raw>::type piece;
    constexpr int LPR = WC / 8;
    const int oc = GATED ? a.O / 2 : a.O, c = lane % LPR * 8, col = col0 + c;
    if (col >= oc) return;
    float bias[8], ubias[GATED ? 8 : 1];
#pragma unroll
    for (int j = 0; j < 8; j++) bias[j] = 0.0f;
    if (GATED)
#pragma unroll
        for (int j = 0; j < 8; j++) ubias[GATED ? j : 0] = 0.0f;
    if (a.bias) {
        const raw *const b = static_cast<const raw *>(a.bias) + (long long)expert * a.O + col;
        const piece v = *reinterpret_cast<const piece *>(b);
#pragma unroll
        for (int j = 0; j < 8; j++) bias[j] = XT::get(v[j]);
        if (GATED) {
            const piece u = *reinterpret_cast<const piece *>(b + oc);
#pragma unroll
            for (int j = 0; j < 8; j++) ubias[GATED ? j : 0] = XT::get(u[j]);
        }
    }
#pragma unroll 2
    for (int r = lane / LPR; r < n; r += 64 / LPR) {
        const long long row = row_of(r);
        float rs[8];
#pragma unroll
        for (int j = 0; j < 8; j++) rs[j] = 0.0f;
        if (a.residual) {
            const piece v = *reinterpret_cast<const piece *>(
                static_cast<const raw *>(a.residual) + row * a.ldr + col);
#pragma unroll
            for (int j = 0; j < 8; j++) rs[j] = XT::get(v[j]);
        }
        bool bad = false;
        if (a.rows) {
            const int x = a.rows[row];
            bad = x < 0 || x >= a.T;
        }
        const float *const o = own + r * LDR + c;
        piece out;
#pragma unroll
        for (int j = 0; j < 8; j++) {
            float v = activate<ACT>(o[j] + bias[j]);
            if (GATED) v *= o[WC + j] + ubias[GATED ? j : 0];
            out[j] = XT::put(bad ? __builtin_nanf("") : v + rs[j]);
        }
        *reinterpret_cast<piece *>(static_cast<raw *>(a.y) + row * a.ldy + col) = out;
    }
}

template <typename XT, bool GATED, int WC, int LDR, typename Row>
__device__ __forceinline__ void finish_rows(const LinearArgs &a, int expert, const float *own,
                                            int lane, int n, int col0, Row row_of)
{
#define QG_ENDS(ACT) finish_rows_act<XT, ACT, GATED, WC, LDR>(a, expert, own, lane, n, col0, row_of)
    switch (a.act) {
    case QGEMV_ACT_RELU: return QG_ENDS(QGEMV_ACT_RELU);
    case QGEMV_ACT_SILU: return QG_ENDS(QGEMV_ACT_SILU);
    case QGEMV_ACT_GELU: return QG_ENDS(QGEMV_ACT_GELU);
    case QGEMV_ACT_GELU_TANH: return QG_ENDS(QGEMV_ACT_GELU_TANH);
    default: return QG_ENDS(QGEMV_ACT_NONE);
    }
#undef QG_ENDS
}

// Tile kernel.  A workgroup of WW x WT waves makes 16 WT TF rows of y x 16 WW WF
// rows of W (gated: half of them gate rows, half up rows); a wave 16 TF rows of x
// x 16 WF rows of W, its rows of x in fragments of 16 dealt to the waves in turn.
// Both operands come into LDS as they are, a row's 128 bytes of a K step in 16-byte
// chunks, XOR-swizzled by row.
//
// A K step is one scale block: its products are summed from zero and added to the
// total as acc += (xs ws) sum in f32, four FMAs per lane and 16 x 16 block beside the
// next blocks' matrix instructions.  W is the A operand: lane l holds the sums of rows
// 4 (l / 16) + i of W and row l % 16 of x, so that a lane has one scale of x, and W's is
// the same for the wave (ROWS: the up rows of a gated product need not start at a scale
// block, a lane's four rows may lie in two).
//
// EXACT (f32 results): codes unpacked to f16, v_mfma_f32_16x16x32_f16, whose sums are
// f32.  Otherwise (bfloat16 results) v_mfma_f32_16x16x128_f8f6f4, four times the rate.
// Measured, it sums eight consecutive columns after cutting each product to a multiple
// of 2^(e - 13), e the largest exponent of the eight (a product's being the sum of its
// codes', -6 for subnormal codes and zero), and the eights' sums in f32; so does the
// 16x16x32 form of e4m3.  That is at most 2^-9 of what rounding one of its factors to
// e4m3 may have moved the product with that exponent; random normals by random codes
// come out within 5e-5 of their norm, a thirtieth of bfloat16's rounding.  f32 results
// would show it.
//
// DIRECT: rows of both operands on 16 bytes, by memory-to-LDS loads, two or (up to 128
// rows) three stages; the loads of a stage are spread over the first products behind
// the barrier that frees it.  Otherwise through registers and one stage.  RAGGED
// (grouped): fragments of x without rows are neither loaded nor multiplied.
//
// 256 x 256 x 8 waves: a wave reads 12 fragments (24 KB) of LDS for 32 matrix
// instructions of 32 cycles; 128 x 128 of 4 waves, two workgroups per CU, reads 16 KB
// for 16.  4096 x 8192 x 8192 takes 240 us (2290 TFLOP/s) in tiles of 256, 293 of 192,
// 297 of 128 and 317 of 128 x 128; the library's e4m3 product of the size, without
// block scales, 189.  Bound by the matrix cores, LDS reads and the card's power
// together: matrix cores busy 61 % of the cycles at 1.76 GHz (without the LDS loads 66 %
// at 1.96, without the reads either 203 -> 180 us), a tile's start and end 13 us.
// Fragments of W are read three ahead, the sums added three products later, so that
// neither waits; the ends by 16-byte pieces (33 -> 16 us for a tile of two K steps).
template <typename XT, int WF, int TF, int WW, int WT, bool EXACT, bool GATED, bool ROWS,
          bool DIRECT, bool RAGGED>
__global__ __launch_bounds__(WW * WT * 64, 2) void matmul_tile(TileParams p)
{
    constexpr int NT = WW * WT * 64, BW = WW * WF * 16, BT = WT * TF * 16;
    constexpr int PW = BW * 8 / NT, PX = BT * 8 / NT;    // 16-byte chunks per thread
    constexpr int RL = NT / 8;                           // rows of one load of all threads
    // (three where they fit beside the scales; 128 x 128 has two workgroups per CU)
    constexpr bool THREE = !EXACT && BW > 128 && 3 * (BW + BT) * TK + 10240 <= LDS_BUDGET;
    constexpr int STAGES = !DIRECT ? 1 : THREE ? 3 : 2;
    constexpr uint32_t XB = BT * TK, WB = BW * TK, SB = XB + WB;
    constexpr int NX = (BT * SG + NT - 1) / NT;          // scale loads per thread
    constexpr uint32_t XS = NX * NT * 4, SS = XS + WW * WT * 256;
    constexpr int YC = GATED ? BW / 2 : BW;              // columns of y
    constexpr int WC = YC / WW;                          // and per wave
    constexpr int LDR = WF * 16 + 4;                     // epilogue row stride, floats
    constexpr uint32_t LDS = STAGES * SB + 2 * SS, ER = WW * WT * 16 * LDR * 4;
    constexpr int NE = TF * ER <= LDS ? TF : (TF + 1) / 2;
    constexpr uint32_t EB = NE * ER;
    static_assert(PW * NT == BW * 8 && PX * NT == BT * 8, "whole loads");
    static_assert(EB <= LDS_BUDGET, "LDS");
    static_assert(RL % 16 == 0, "a thread's chunk has one place in all its rows");
    __shared__ __align__(16) char smem[LDS > EB ? LDS : EB];

    const LinearArgs &a = p.m.a;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ww = wave % WW, wt = wave / WW;
    const int li = lane & 15, lg = lane >> 4;
    const int oc = GATED ? a.O / 2 : a.O;

    int mt, nt, part = 0;
    ExpertTile t;
    if (p.tiles) {
        // Tiles in the order of experts, an expert's column blocks one after the other
        // with all its rows, dealt to the XCDs in runs of an XCD's CUs (of one row
        // tile where they are few): rows and column blocks that an XCD works on at a
        // time share W and x in its L2.
        const int xcd = blockIdx.x % 8, in = blockIdx.x / 8;
        const int items = min(p.tiles[0].filled, p.ntm) * p.ntn;
        const int run = items >= 1024 ? 32 : min(p.ntn, 32);
        const int item = (in / run * 8 + xcd) * run + in % run;
        if (item >= items) return;
        t = p.tiles[item / p.ntn];
        const int local = item - t.first * p.ntn;
        nt = local / t.count;
        mt = t.first + local - nt * t.count;
        t = p.tiles[mt];
        t.expert = __builtin_amdgcn_readfirstlane(t.expert);
        t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
        t.n = __builtin_amdgcn_readfirstlane(t.n);
        if (t.n <= 0) return;
    } else {
        // consecutive tiles to one XCD, eight row tiles to a column block: the
        // tiles that an XCD works on at a time share rows of both operands
        const int nb = gridDim.x, q8 = nb / 8, r8 = nb % 8;
        const int xcd = blockIdx.x % 8, in = blockIdx.x / 8;
        int b = xcd * q8 + min(xcd, r8) + in;
        part = b / (p.ntm * p.ntn);
        b -= part * p.ntm * p.ntn;
        const int strip = b / (8 * p.ntn), first = strip * 8, h = min(8, p.ntm - first);
        const int i = b - strip * 8 * p.ntn;
        mt = first + i % h;
        nt = i / h;
        t = ExpertTile{0, mt * BT, min(BT, a.R - mt * BT)};
    }

    // A thread loads chunk `ch` of its rows; rows behind the tile or the matrix
    // repeat one that exists, a bad row index reads row 0 and is marked in the end.
    const int row_l = tid >> 3;
    const uint32_t ch = ((tid & 7) ^ swizzle(row_l)) * 16;
    const int c0 = p.col0 + nt * YC;
    const int first_step = RAGGED ? 0 : part * p.per;
    const uint8_t *const wexp =
        a.w + (long long)t.expert * a.w_stride + (long long)first_step * TK;
    // (first row of each half, clamped so that the base is a row)
    const uint8_t *const wbase0 = wexp + (long long)c0 * a.I;
    const uint8_t *const wbase1 = GATED ? wbase0 + (long long)oc * a.I : wbase0;
    const uint8_t *xbase = static_cast<const uint8_t *>(a.x) + (long long)first_step * TK;
    const float *xsbase = p.m.xs + first_step;
    if (!a.rows) {
        xbase += (long long)t.row0 * a.ldx;
        xsbase += (long long)t.row0 * p.m.ldxs;
    }
    uint32_t woff[PW], xsoff[NX];
    uint32_t xoff[DIRECT ? PX : 1];
    const uint8_t *xptr[DIRECT ? 1 : PX];
    auto local_row = [&](int r) {
        r = r < t.n ? r : 0;
        if (!a.rows) return r;
        const int x = a.rows[t.row0 + r];
        return x < 0 || x >= a.T ? 0 : x;
    };
#pragma unroll
    for (int i = 0; i < PW; i++) {
        const int r = row_l + RL * i, half = GATED ? r / (BW / 2) : 0;
        woff[i] = (uint32_t)min(r - half * (BW / 2), oc - 1 - c0) * (uint32_t)a.I + ch;
    }
#pragma unroll
    for (int i = 0; i < PX; i++) {
        const int r = local_row(row_l + RL * i);
        if constexpr (DIRECT) xoff[i] = (uint32_t)r * (uint32_t)a.ldx + ch;
        else xptr[i] = xbase + (long long)r * a.ldx + ch;
    }
#pragma unroll
    for (int i = 0; i < NX; i++) xsoff[i] = (uint32_t)local_row((tid + NT * i) / SG);
    // scales of W: gate (or plain) block, and of a gated product the up rows' two
    const int wr0 = ww * (GATED ? WF / 2 : WF) * 16;     // the wave's first row of each half
    const int blocks = (a.O + 127) / 128;
    const int up0 = oc + c0 + wr0;
    const int sblk[3] = {min((c0 + wr0) / 128, blocks - 1), min(up0 / 128, blocks - 1),
                         min(up0 / 128 + 1, blocks - 1)};
    const float *const sexp = a.scales + (long long)t.expert * a.s_stride + first_step;
    const int seg = min(lane / SG, 2);
    const float *const wsrc =
        sexp + (long long)(seg == 0 ? sblk[0] : seg == 1 ? sblk[1] : sblk[2]) * a.ng;

    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(
        (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)smem);
    const uint32_t ls0 = lds0 + STAGES * SB;
    const int steps = RAGGED ? a.ng : min(p.per, a.ng - first_step);
    const int rem = min(a.I - (first_step + steps - 1) * TK, TK);   // columns of the last step

    // Scales of steps SG g .. SG g + SG - 1 (behind the last: the last again).
    auto load_scales = [&](int g) {
        const uint32_t at = ls0 + (g & 1) * SS;
        const int k = min(g * SG + (lane & (SG - 1)), steps - 1);
#pragma unroll
        for (int i = 0; i < NX; i++)
            load_lds4(xsbase, (xsoff[i] * (uint32_t)p.m.ldxs + (uint32_t)k) * 4,
                      at + (wave * 64 + NT * i) * 4);
        load_lds4(sexp, (uint32_t)((wsrc - sexp) + k) * 4, at + XS + wave * 256);
    };
    f32x4v acc[WF][TF];
#pragma unroll
    for (int m = 0; m < WF; m++)
#pragma unroll
        for (int n = 0; n < TF; n++) acc[m][n] = f32x4v{0.0f, 0.0f, 0.0f, 0.0f};

    // LDS places of the wave's fragments: chunks lg and lg + 4 of row li
    const int ch0 = (lg ^ swizzle(li)) * 16, ch1 = ((lg + 4) ^ swizzle(li)) * 16;
    const int xrow = (wt * 16 + li) * TK;                // fragment n: 16 WT n rows on
    const int wrow0 = XB + (wr0 + li) * TK, wrow1 = wrow0 + (GATED ? BW / 2 * TK : 0);
    // the lane's rows 4 lg + r of up fragment m lie in the second block from here on
    const int edge = (up0 / 128 + 1) * 128 - up0 - 4 * lg;

    // The K loop of a wave with TA fragments of x.
    auto run = [&](auto fragments) {
        constexpr int TA = decltype(fragments)::value, TA1 = TA ? TA : 1;
        // Step s by memory-to-LDS loads.  In a last step of fewer columns the chunks
        // behind them repeat the last one and are cleared before they are read.
        // Loads lo <= i < hi of its PX + PW.
        auto load_part = [&](int s, int lo, int hi) {
            const uint32_t at = lds0 + (uint32_t)(STAGES == 2 ? s & 1 : s % 3) * SB;
            const uint32_t back = s == steps - 1 && rem < TK
                                      ? (ch < (uint32_t)rem ? 0u : ch - (uint32_t)(rem - 16)) : 0u;
            const long long k = (long long)s * TK;
#pragma unroll
            for (int i = 0; i < PX; i++)
                if (i >= lo && i < hi && (!RAGGED || RL * i < t.n))
                    load_lds16(xbase + k, xoff[DIRECT ? i : 0] - back,
                               at + (wave * 64 + NT * i) * 16);
#pragma unroll
            for (int i = 0; i < PW; i++)
                if (PX + i >= lo && PX + i < hi)
                    load_lds16((GATED && i >= PW / 2 ? wbase1 : wbase0) + k, woff[i] - back,
                               at + XB + (wave * 64 + NT * i) * 16);
        };
        auto load_direct = [&](int s) { load_part(s, 0, PX + PW); };
        auto clear_tail = [&](char *at) {
            if (ch >= (uint32_t)rem) {
                const u32x4 zero = {0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < PX + PW; i++)
                    *reinterpret_cast<u32x4 *>(at + (tid + NT * i) * 16) = zero;
            }
        };

        auto multiply = [&](const char *at, const char *sc, int j) {
            float sx[TF], s0[TF], s1[GATED ? TF : 1], s2[ROWS ? TF : 1];
            const float *const sl = reinterpret_cast<const float *>(sc);
            const float *const wl = reinterpret_cast<const float *>(sc + XS + wave * 256);
#pragma unroll
            for (int n = 0; n < TA; n++) sx[n] = sl[((n * WT + wt) * 16 + li) * SG + j];
#pragma unroll
            for (int n = 0; n < TA; n++) {
                s0[n] = sx[n] * wl[j];
                if (GATED) s1[GATED ? n : 0] = sx[n] * wl[SG + j];
                if (ROWS) s2[ROWS ? n : 0] = sx[n] * wl[2 * SG + j];
            }
            i32x8 xf[TF], wf[2];
            auto read = [&](int row) {
                i32x8 v;
                const u32x4 lo = *reinterpret_cast<const u32x4 *>(at + row + ch0);
                const u32x4 hi = *reinterpret_cast<const u32x4 *>(at + row + ch1);
                v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
                v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
                return v;
            };
            auto read_w = [&](int m) {
                return GATED && m >= WF / 2 ? read(wrow1 + (m - WF / 2) * 16 * TK)
                                            : read(wrow0 + m * 16 * TK);
            };
            auto f16s = [&](const i32x8 &v, f16x8 f[4]) {
#pragma unroll
                for (int h = 0; h < 4; h++)
                    f[h] = fp8x8_f16((uint32_t)v[2 * h], (uint32_t)v[2 * h + 1]);
            };
            f16x8 xh[EXACT ? TF : 1][4];
            wf[0] = read_w(0);
#pragma unroll
            for (int n = 0; n < TA; n++) {
                xf[n] = read(xrow + n * WT * 16 * TK);
                if constexpr (EXACT) f16s(xf[n], xh[n]);
            }
            f32x4v g[2][TF];
            auto flush = [&](int m) {
#pragma unroll
                for (int n = 0; n < TA; n++)
#pragma unroll
                    for (int r = 0; r < 4; r++) {
                        float s = s0[n];
                        if (GATED && m >= WF / 2) {
                            s = s1[GATED ? n : 0];
                            if (ROWS && (m - WF / 2) * 16 + r >= edge) s = s2[ROWS ? n : 0];
                        }
                        acc[m][n][r] = fmaf(s, g[m & 1][n][r], acc[m][n][r]);
                    }
            };
#pragma unroll
            for (int m = 0; m < WF; m++) {
                if (m + 1 < WF) wf[(m + 1) & 1] = read_w(m + 1);
                f16x8 wh[4];
                if constexpr (EXACT) f16s(wf[m & 1], wh);
#pragma unroll
                for (int n = 0; n < TA; n++) {
                    f32x4v z = {0.0f, 0.0f, 0.0f, 0.0f};
                    if constexpr (EXACT) {
#pragma unroll
                        for (int h = 0; h < 4; h++)
                            z = __builtin_amdgcn_mfma_f32_16x16x32_f16(wh[h], xh[n][h], z, 0, 0, 0);
                    } else {
                        z = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            wf[m & 1], xf[n], z, 0, 0, 0, 0, 0, 0);
                    }
                    g[m & 1][n] = z;
                }
                if (m > 0) flush(m - 1);
                __builtin_amdgcn_sched_barrier(0);
            }
            flush(WF - 1);
        };

        if constexpr (DIRECT && !EXACT) {
            // A step's loads, fragments and sums overlap with its neighbours': at the last
            // W fragment everything of the step has been read from LDS, so its stage is
            // loaded again, the next one is there, and its first fragments replace the
            // x fragments as their last products start.
            constexpr int AHEAD = WF >= 8 ? 3 : 1, WB2 = AHEAD + 1;
            i32x8 xf[TF], wf[WB2];
            f32x4v g[4];
            float sx[TF], sw[3], s0[TF], s1[GATED ? TF : 1], s2[ROWS ? TF : 1];
            const char *at = smem;
            auto read = [&](int row) {
                i32x8 v;
                const u32x4 lo = *reinterpret_cast<const u32x4 *>(at + row + ch0);
                const u32x4 hi = *reinterpret_cast<const u32x4 *>(at + row + ch1);
                v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
                v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
                return v;
            };
            auto read_w = [&](int m) {
                return GATED && m >= WF / 2 ? read(wrow1 + (m - WF / 2) * 16 * TK)
                                            : read(wrow0 + m * 16 * TK);
            };
            auto read_scales = [&](int s) {
                const char *const sc = smem + STAGES * SB + ((s / SG) & 1) * SS;
                const float *const sl = reinterpret_cast<const float *>(sc) + s % SG;
                const float *const wl =
                    reinterpret_cast<const float *>(sc + XS + wave * 256) + s % SG;
#pragma unroll
                for (int n = 0; n < TA; n++) sx[n] = sl[((n * WT + wt) * 16 + li) * SG];
                sw[0] = wl[0];
                if (GATED) sw[1] = wl[SG];
                if (ROWS) sw[2] = wl[2 * SG];
            };
            // sums of a step's product q = TF m + n, LAG products later
            constexpr int LAG = 3;
            auto flush = [&](int q) {
                const int m = q / TA1, n = q % TA1;
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    float c = s0[n];
                    if (GATED && m >= WF / 2) {
                        c = s1[GATED ? n : 0];
                        if (ROWS && (m - WF / 2) * 16 + r >= edge) c = s2[ROWS ? n : 0];
                    }
                    acc[m][n][r] = fmaf(c, g[q % (LAG + 1)][r], acc[m][n][r]);
                }
                asm volatile("" : "+v"(acc[m][n]));          // (not to be moved past a branch)
            };
            auto scale = [&](int n) {
                s0[n] = sx[n] * sw[0];
                if (GATED) s1[GATED ? n : 0] = sx[n] * sw[1];
                if (ROWS) s2[ROWS ? n : 0] = sx[n] * sw[2];
            };
            static_assert(WF % WB2 == 0 && WF * TA % (LAG + 1) == 0, "buffers alternate");
            __syncthreads();                                 // (earlier loads are done)
            load_scales(0);
            load_direct(0);
            wait_loads<0>();
            if (steps == 1 && rem < TK) {
                clear_tail(smem);
                __syncthreads();
            }
            // the loads of a stage are issued in SLOTS parts, one per W fragment from the
            // one on that frees it, so that the memory pipe takes them without a stall
            constexpr int SLOTS = WF >= 8 ? 4 : 2, PER = (PX + PW + SLOTS - 1) / SLOTS;
#pragma unroll
            for (int i = 1; i + 1 < STAGES; i++)
                if (i < steps) load_direct(i);
            if (STAGES - 1 < steps) {
#pragma unroll
                for (int k = 0; k < AHEAD; k++) load_part(STAGES - 1, k * PER, (k + 1) * PER);
            }
            const int nx = RAGGED ? min((t.n + RL - 1) / RL, PX) : PX;   // loads of x per step
#pragma unroll
            for (int m = 0; m < AHEAD; m++) wf[m] = read_w(m);
#pragma unroll
            for (int n = 0; n < TA; n++) xf[n] = read(xrow + n * WT * 16 * TK);
#pragma unroll
            for (int n = 0; n < TA; n++) {
                s0[n] = 0.0f;
                if (GATED) s1[GATED ? n : 0] = 0.0f;
                if (ROWS) s2[ROWS ? n : 0] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i <= LAG; i++) g[i] = f32x4v{0.0f, 0.0f, 0.0f, 0.0f};
            for (int s = 0; s < steps; s++) {
#pragma unroll
                for (int m = 0; m < WF; m++) {
                    if (m + AHEAD == WF) {
                        // this wave's reads of the stage and its loads of the next are done
                        if constexpr (STAGES == 2) {
                            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
                        } else {
                            // (those of the one after it may be on their way)
                            const int later = s + 2 < steps ? PW + nx + ((s + 2) % SG ? 0 : NX + 1)
                                                            : 0;
                            wait_some(later);
                        }
                        if (s + STAGES < steps && (s + STAGES) % SG == 0)
                            load_scales((s + STAGES) / SG);
                        char *const next = smem + (STAGES == 2 ? (s + 1) & 1 : (s + 1) % 3) * SB;
                        if (s + 2 == steps && rem < TK) {    // uniform over the workgroup
                            clear_tail(next);
                            __syncthreads();
                        }
                        at = next;
                    }
#pragma unroll
                    for (int n = 0; n < TA; n++) {
                        const int q = m * TA + n;
                        __builtin_amdgcn_sched_barrier(0);
                        const f32x4v z = {0.0f, 0.0f, 0.0f, 0.0f};
                        g[q % (LAG + 1)] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            wf[m % WB2], xf[n], z, 0, 0, 0, 0, 0, 0);
                        __builtin_amdgcn_sched_barrier(0);
                        if (n == 0) wf[(m + AHEAD) % WB2] = read_w((m + AHEAD) % WF);
                        if (q == 1) read_scales(s);
                        if (q == LAG) {                      // the last step's sums are done
#pragma unroll
                            for (int i = 0; i < TA; i++) scale(i);
                        }
                        flush(q >= LAG ? q - LAG : WF * TA + q - LAG);
                        if (m + 1 == WF) xf[n] = read(xrow + n * WT * 16 * TK);
                    }
                    const int k = (m + AHEAD) % WF;
                    const int of = m + AHEAD < WF ? s + STAGES - 1 : s + STAGES;
                    if (k < SLOTS && of < steps) load_part(of, k * PER, (k + 1) * PER);
                }
            }
            if constexpr (TA > 0)
#pragma unroll
                for (int q = WF * TA - LAG; q < WF * TA; q++) flush(q);
        } else if constexpr (DIRECT) {
            __syncthreads();                                 // (earlier loads are done)
            load_scales(0);
            load_direct(0);
            for (int s = 0; s < steps; s++) {
                // this step's data is there, and the stage that the last one read is free
                wait_loads<0>();
                if (s + 1 < steps) {
                    if ((s + 1) % SG == 0) load_scales((s + 1) / SG);
                    load_direct(s + 1);
                }
                char *const at = smem + (s & 1) * SB;
                if (s == steps - 1 && rem < TK) {            // uniform over the workgroup
                    clear_tail(at);
                    __syncthreads();
                }
                multiply(at, smem + STAGES * SB + ((s / SG) & 1) * SS, s % SG);
            }
        } else {
            u32x4 xv[PX], wv[PW];
            auto fetch = [&](int s) {
                typedef u32x4 __attribute__((aligned(1))) any;
                const long long k = (long long)s * TK;
                if (s < steps - 1 || rem == TK) {
#pragma unroll
                    for (int i = 0; i < PX; i++)
                        xv[i] = *reinterpret_cast<const any *>(xptr[DIRECT ? 0 : i] + k);
#pragma unroll
                    for (int i = 0; i < PW; i++)
                        wv[i] = *reinterpret_cast<const any *>(
                            (GATED && i >= PW / 2 ? wbase1 : wbase0) + woff[i] + k);
                } else {
                    auto tail = [&](const uint8_t *src) {
                        u32x4 v;
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            uint32_t w = 0;
#pragma unroll
                            for (int b = 0; b < 4; b++)
                                if ((int)ch + 4 * j + b < rem)
                                    w |= (uint32_t)src[4 * j + b] << (8 * b);
                            v[j] = w;
                        }
                        return v;
                    };
#pragma unroll
                    for (int i = 0; i < PX; i++) xv[i] = tail(xptr[DIRECT ? 0 : i] + k);
#pragma unroll
                    for (int i = 0; i < PW; i++)
                        wv[i] = tail((GATED && i >= PW / 2 ? wbase1 : wbase0) + woff[i] + k);
                }
            };
            __syncthreads();
            load_scales(0);
            fetch(0);
            for (int s = 0; s < steps; s++) {
                wait_loads<0>();                         // scales; the last step's reads
#pragma unroll
                for (int i = 0; i < PX; i++)
                    *reinterpret_cast<u32x4 *>(smem + (tid + NT * i) * 16) = xv[i];
#pragma unroll
                for (int i = 0; i < PW; i++)
                    *reinterpret_cast<u32x4 *>(smem + XB + (tid + NT * i) * 16) = wv[i];
                __syncthreads();
                if (s + 1 < steps) {
                    if ((s + 1) % SG == 0) load_scales((s + 1) / SG);
                    fetch(s + 1);
                }
                multiply(smem, smem + STAGES * SB + ((s / SG) & 1) * SS, s % SG);
            }
        }
    };
    if constexpr (RAGGED) {
        // fragments of x that hold rows, dealt to the waves in turn
        const int all = (t.n + 15) / 16;
        switch (__builtin_amdgcn_readfirstlane((all - wt + WT - 1) / WT)) {
        case 0: run(std::integral_constant<int, 0>{}); break;
        case 1: run(std::integral_constant<int, 1>{}); break;
        case 2: run(std::integral_constant<int, TF < 2 ? TF : 2>{}); break;
        case 3: run(std::integral_constant<int, TF < 3 ? TF : 3>{}); break;
        default: run(std::integral_constant<int, TF>{}); break;
        }
    } else {
        run(std::integral_constant<int, TF>{});
    }
    if (!RAGGED && p.parts > 1) {                        // a part's sums
        const int lim = p.ldp, c = c0 + ww * WC + 4 * lg;
#pragma unroll
        for (int n = 0; n < TF; n++) {
            const int r = (n * WT + wt) * 16 + li;
            if (r >= t.n) continue;
#pragma unroll
            for (int m = 0; m < WF; m++) {
                const int half = GATED && m >= WF / 2;
                const int col = c + (half ? m - WF / 2 : m) * 16;
                float *const row = p.partial + ((long long)(part * (GATED ? 2 : 1) + half) * a.R +
                                                t.row0 + r) * lim;
                if (col < lim) *reinterpret_cast<f32x4v *>(row + col) = acc[m][n];
            }
        }
        return;
    }
    __syncthreads();

    // The ends: 16 NE rows at a time through a part of LDS of the wave's own, from
    // which lanes next to each other take pieces of one row.
    float *const own = reinterpret_cast<float *>(smem) + wave * (16 * NE * LDR);
    const int cw = c0 + ww * WC;                         // the wave's first column of y
#pragma unroll
    for (int n0 = 0; n0 < TF; n0 += NE) {
        // fragment n0 + j holds rows first + 16 WT j .. + 15 of the tile
        const int first = (n0 * WT + wt) * 16;
        int rows = 0;
#pragma unroll
        for (int j = 0; j < NE && n0 + j < TF; j++)
            rows += min(max(t.n - first - j * WT * 16, 0), 16);
        if (rows <= 0) break;                            // uniform over the wave
#pragma unroll
        for (int n = n0; n < n0 + NE && n < TF; n++)
#pragma unroll
            for (int m = 0; m < WF; m++)
                *reinterpret_cast<f32x4v *>(own + ((n - n0) * 16 + li) * LDR + m * 16 + 4 * lg) =
                    acc[m][n];
        __builtin_amdgcn_wave_barrier();
        auto row_of = [&](int r) { return t.row0 + first + r / 16 * (WT * 16) + r % 16; };
        if (p.wide) {
            finish_rows<XT, GATED, WC, LDR>(a, t.expert, own, lane, rows, cw, row_of);
        } else {
            finish<XT, 4>(a, t.expert, lane, 64, rows * WC,
                          [&](int i, int &row, int &col, float &v, float &up) {
                              const int r = i / WC, c = i % WC;
                              row = row_of(r);
                              col = cw + c;
                              v = own[r * LDR + c];
                              up = GATED ? own[r * LDR + WC + c] : 0.0f;
                              if (a.rows) {
                                  const int x = a.rows[row];
                                  if (x < 0 || x >= a.T) v = up = __builtin_nanf("");
                              }
                          });
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// GROUPED: plan_tiles gives grouped products this kind, too.
template <typename XT, int WF, int TF, int WW, int WT, bool EXACT, bool DIRECT, bool GROUPED>
hipError_t run_tile(const TileParams &p, unsigned grid, hipStream_t st)
{
    const LinearArgs &a = p.m.a;
    constexpr int NT = WW * WT * 64, WC = WF * 8;        // gated: columns of y per wave
    if (p.tiles && !GROUPED) return hipErrorInvalidValue;
#define QG_RUN1(G, R, N)                                                                    \
    hipLaunchKernelGGL((matmul_tile<XT, WF, TF, WW, WT, EXACT, G, R, DIRECT, N>), dim3(grid), \
                       dim3(NT), 0, st, p)
#define QG_RUN(G, R)                                                                        \
    do {                                                                                    \
        if constexpr (GROUPED)                                                              \
            if (p.tiles) {                                                                  \
                QG_RUN1(G, R, true);                                                        \
                break;                                                                      \
            }                                                                               \
        QG_RUN1(G, R, false);                                                               \
    } while (0)
    if (!a.gated) QG_RUN(false, false);
    else if (a.O / 2 % WC == 0) QG_RUN(true, false);     // a wave's up rows share a scale block
    else QG_RUN(true, true);
#undef QG_RUN
#undef QG_RUN1
    return hipGetLastError();
}

}  // namespace

}  // namespace qg
