// matmul_tile.hip -- e4m3 activations times e4m3 weights on the matrix cores,
// many rows, dense or grouped by expert, with the epilogue.
#include "qg_device.h"
#include "qg_launch.h"
#include "qg_matmul.h"
#include "qg_tile.h"

namespace qg {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int TK = 128;                  // columns per K step: one scale block
constexpr int SG = 4;                    // K steps whose scales are fetched together

struct TileParams {
    MatmulArgs m;
    const RowTile *tiles;                // grouped, else nullptr
    int ntm, ntn;
};

// Tile kernel.  A workgroup of WW x WT waves makes 16 WT TF rows of y x 16 WW WF
// rows of W (gated: half of them gate rows, half up rows); a wave 16 TF rows of x
// x 16 WF rows of W.  Both operands come into LDS as they are, a row's 128 bytes
// of a K step in 16-byte chunks, XOR-swizzled by row.
template <typename XT, int WF, int TF, int WW, int WT, bool EXACT, bool GATED, bool ROWS,
          bool DIRECT>
__global__ __launch_bounds__(WW * WT * 64, WW * WT <= 4 ? 2 : 2) void matmul_tile(TileParams p)
{
    constexpr int NT = WW * WT * 64, BW = WW * WF * 16, BT = WT * TF * 16;
    constexpr int PW = BW * 8 / NT, PX = BT * 8 / NT;    // 16-byte chunks per thread
    constexpr int RL = NT / 8;                           // rows of one load of all threads
    constexpr int STAGES = DIRECT ? 2 : 1;
    constexpr uint32_t XB = BT * TK, WB = BW * TK, SB = XB + WB;
    constexpr int NX = BT * SG / NT;                     // scale loads per thread
    constexpr uint32_t XS = BT * SG * 4, SS = XS + WW * WT * 256;
    constexpr int YC = GATED ? BW / 2 : BW;              // columns of y
    constexpr int WC = YC / WW;                          // and per wave
    constexpr int LDR = WF * 16 + 4;                     // epilogue row stride, floats
    constexpr uint32_t EB = WW * WT * 16 * LDR * 4;
    constexpr uint32_t LDS = STAGES * SB + 2 * SS;
    static_assert(PW * NT == BW * 8 && PX * NT == BT * 8 && NX * NT == BT * SG, "whole loads");
    static_assert(RL % 16 == 0, "a thread's chunk has one place in all its rows");
    __shared__ __align__(16) char smem[LDS > EB ? LDS : EB];

    const LinearArgs &a = p.m.a;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ww = wave % WW, wt = wave / WW;
    const int li = lane & 15, lg = lane >> 4;
    const int oc = GATED ? a.O / 2 : a.O;

    int mt, nt;
    RowTile t;
    if (p.tiles) {
        const int xcd = blockIdx.x % 8, in = blockIdx.x / 8;
        mt = in / p.ntn * 8 + xcd;
        nt = in % p.ntn;
        if (mt >= p.ntm) return;
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
        const int b = xcd * q8 + min(xcd, r8) + in;
        const int strip = b / (8 * p.ntn), first = strip * 8, h = min(8, p.ntm - first);
        const int i = b - strip * 8 * p.ntn;
        mt = first + i % h;
        nt = i / h;
        t = RowTile{0, mt * BT, min(BT, a.R - mt * BT), 0};
    }

    // A thread loads chunk `ch` of its rows; rows behind the tile or the matrix
    // repeat one that exists, a bad row index reads row 0 and is marked in the end.
    const int row_l = tid >> 3;
    const uint32_t ch = ((tid & 7) ^ swizzle(row_l)) * 16;
    const int c0 = nt * YC;
    const uint8_t *const wexp = a.w + (long long)t.expert * a.w_stride;
    // (first row of each half, clamped so that the base is a row)
    const uint8_t *const wbase0 = wexp + (long long)c0 * a.I;
    const uint8_t *const wbase1 = GATED ? wbase0 + (long long)oc * a.I : wbase0;
    const uint8_t *xbase = static_cast<const uint8_t *>(a.x);
    const float *xsbase = p.m.xs;
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
    const float *const sexp = a.scales + (long long)t.expert * a.s_stride;
    const int seg = min(lane / SG, 2);
    const float *const wsrc = sexp + (long long)(seg == 0 ? sblk[0] : seg == 1 ? sblk[1] : sblk[2]) * a.ng;

    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(
        (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)smem);
    const uint32_t ls0 = lds0 + STAGES * SB;
    const int steps = a.ng, rem = a.I - (steps - 1) * TK;    // columns of the last step

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
    // Step s by memory-to-LDS loads.  In a last step of fewer columns the chunks
    // behind them repeat the last one and are cleared before they are read.
    auto load_direct = [&](int s) {
        const uint32_t at = lds0 + (s & 1) * SB;
        const uint32_t back = s == steps - 1 && rem < TK
                                  ? (ch < (uint32_t)rem ? 0u : ch - (uint32_t)(rem - 16)) : 0u;
        const uint8_t *const w0 = wbase0 + (long long)s * TK, *const w1 = wbase1 + (long long)s * TK;
        const uint8_t *const x0 = xbase + (long long)s * TK;
#pragma unroll
        for (int i = 0; i < PX; i++)
            load_lds16(x0, xoff[DIRECT ? i : 0] - back, at + (wave * 64 + NT * i) * 16);
#pragma unroll
        for (int i = 0; i < PW; i++)
            load_lds16(GATED && i >= PW / 2 ? w1 : w0, woff[i] - back,
                       at + XB + (wave * 64 + NT * i) * 16);
    };
    auto clear_tail = [&](char *at) {
        if (ch >= (uint32_t)rem) {
            const u32x4 zero = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < PX + PW; i++)
                *reinterpret_cast<u32x4 *>(at + (tid + NT * i) * 16) = zero;
        }
    };

    f32x4v acc[WF][TF];
#pragma unroll
    for (int m = 0; m < WF; m++)
#pragma unroll
        for (int n = 0; n < TF; n++) acc[m][n] = f32x4v{0.0f, 0.0f, 0.0f, 0.0f};

    // LDS places of the wave's fragments: chunks lg and lg + 4 of row li
    const int ch0 = (lg ^ swizzle(li)) * 16, ch1 = ((lg + 4) ^ swizzle(li)) * 16;
    const int xrow = (wt * TF * 16 + li) * TK;
    const int wrow0 = XB + (wr0 + li) * TK, wrow1 = wrow0 + (GATED ? BW / 2 * TK : 0);
    // the lane's rows 4 lg + r of up fragment m lie in the second block from here on
    const int edge = (up0 / 128 + 1) * 128 - up0 - 4 * lg;

    auto multiply = [&](const char *at, const char *sc, int j) {
        float sx[TF], s0[TF], s1[GATED ? TF : 1], s2[ROWS ? TF : 1];
        const float *const sl = reinterpret_cast<const float *>(sc);
        const float *const wl = reinterpret_cast<const float *>(sc + XS + wave * 256);
#pragma unroll
        for (int n = 0; n < TF; n++) sx[n] = sl[(wt * TF * 16 + n * 16 + li) * SG + j];
#pragma unroll
        for (int n = 0; n < TF; n++) {
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
        for (int n = 0; n < TF; n++) {
            xf[n] = read(xrow + n * 16 * TK);
            if constexpr (EXACT) f16s(xf[n], xh[n]);
        }
        f32x4v g[2][TF];
        auto flush = [&](int m) {
#pragma unroll
            for (int n = 0; n < TF; n++)
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
            for (int n = 0; n < TF; n++) {
                f32x4v z = {0.0f, 0.0f, 0.0f, 0.0f};
                if constexpr (EXACT) {
#pragma unroll
                    for (int h = 0; h < 4; h++)
                        z = __builtin_amdgcn_mfma_f32_16x16x32_f16(wh[h], xh[n][h], z, 0, 0, 0);
                } else {
                    z = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf[m & 1], xf[n], z, 0, 0,
                                                                         0, 0, 0, 0);
                }
                g[m & 1][n] = z;
            }
            if (m > 0) flush(m - 1);
            __builtin_amdgcn_sched_barrier(0);
        }
        flush(WF - 1);
    };

    if constexpr (DIRECT) {
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
                            if ((int)ch + 4 * j + b < rem) w |= (uint32_t)src[4 * j + b] << (8 * b);
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
            wait_loads<0>();                             // scales; the last step's reads are done
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
    __syncthreads();

    // The ends: 16 rows at a time through a part of LDS of the wave's own, from
    // which a lane takes eight columns of a row.
    float *const own = reinterpret_cast<float *>(smem) + wave * 16 * LDR;
    const int cw = c0 + ww * WC;                         // the wave's first column of y
#pragma unroll
    for (int n = 0; n < TF; n++) {
        const int r0 = (wt * TF + n) * 16;
        if (r0 >= t.n) break;                            // uniform over the wave
#pragma unroll
        for (int m = 0; m < WF; m++)
            *reinterpret_cast<f32x4v *>(own + li * LDR + m * 16 + 4 * lg) = acc[m][n];
        __builtin_amdgcn_wave_barrier();
        finish<XT, 4>(a, t.expert, lane, 64, min(16, t.n - r0) * WC,
                      [&](int i, int &row, int &col, float &v, float &up) {
                          const int r = i / WC, c = i % WC;
                          row = t.row0 + r0 + r;
                          col = cw + c;
                          v = own[r * LDR + c];
                          up = GATED ? own[r * LDR + WC + c] : 0.0f;
                          if (a.rows) {
                              const int x = a.rows[row];
                              if (x < 0 || x >= a.T) v = up = __builtin_nanf("");
                          }
                      });
        __builtin_amdgcn_wave_barrier();
    }
}

template <typename XT, int WF, int TF, int WW, int WT, bool EXACT, bool DIRECT>
hipError_t run_tile(const TileParams &p, unsigned grid, hipStream_t st)
{
    const LinearArgs &a = p.m.a;
    constexpr int NT = WW * WT * 64, WC = WF * 8;        // gated: columns of y per wave
#define QG_RUN(G, R)                                                                        \
    hipLaunchKernelGGL((matmul_tile<XT, WF, TF, WW, WT, EXACT, G, R, DIRECT>), dim3(grid),   \
                       dim3(NT), 0, st, p)
    if (!a.gated) QG_RUN(false, false);
    else if (a.O / 2 % WC == 0) QG_RUN(true, false);     // a wave's up rows share a scale block
    else QG_RUN(true, true);
#undef QG_RUN
    return hipGetLastError();
}

}  // namespace

bool matmul_tile_direct(const MatmulArgs &p)
{
    const LinearArgs &a = p.a;
    return a.I % 16 == 0 && (((uintptr_t)a.w | (uintptr_t)a.x | (uintptr_t)a.ldx) & 15) == 0 &&
           (!a.offsets || a.w_stride % 16 == 0);
}

bool matmul_tile_fits(const MatmulArgs &p)
{
    const LinearArgs &a = p.a;
    const long long rows = a.rows ? a.T : 256, most = 1LL << 32;
    return rows * a.ldx < most && rows * p.ldxs * 4 < most &&
           (long long)((a.O + 127) / 128) * a.ng * 4 < most;
}

long long matmul_tile_grid(const MatmulArgs &p, int bm, long long ntm)
{
    const int cols = bm / (p.a.gated ? 2 : 1), oc = p.a.gated ? p.a.O / 2 : p.a.O;
    // grouped row tiles are dealt to the XCDs by eights
    return (p.a.offsets ? (ntm + 7) / 8 * 8 : ntm) * ((oc + cols - 1) / cols);
}

long long matmul_tile_items(const MatmulArgs &p, int bm, long long ntm)
{
    return matmul_tile_grid(p, bm, ntm) * (bm == 256 ? 512 : 256);
}

hipError_t launch_matmul_tile(const MatmulArgs &m, int bm, const RowTile *tiles, int ntm,
                              hipStream_t st)
{
    TileParams p{};
    p.m = m;
    p.tiles = tiles;
    p.ntm = ntm;
    const int cols = bm / (m.a.gated ? 2 : 1), oc = m.a.gated ? m.a.O / 2 : m.a.O;
    p.ntn = (oc + cols - 1) / cols;
    const unsigned grid = (unsigned)matmul_tile_grid(m, bm, ntm);
    const bool direct = matmul_tile_direct(m);
    if (m.a.dtype == QGEMV_F32)
        return direct ? run_tile<F32, 4, 4, 2, 2, true, true>(p, grid, st)
                      : run_tile<F32, 4, 4, 2, 2, true, false>(p, grid, st);
    if (!direct) return run_tile<BF16, 4, 4, 2, 2, false, false>(p, grid, st);
    return bm == 256 ? run_tile<BF16, 8, 4, 2, 4, false, true>(p, grid, st)
                     : run_tile<BF16, 4, 4, 2, 2, false, true>(p, grid, st);
}

}  // namespace qg
