// matmul_stream.hip -- e4m3 activations times e4m3 weights, few rows: the
// weights stream through registers once per row tile.
#include "qg_device.h"
#include "qg_launch.h"
#include "qg_matmul.h"
#include "qg_tile.h"

namespace qg {

namespace {

constexpr int SW = 8;                    // waves of a workgroup, which split K
constexpr int SK = 128;                  // columns per K step: one scale block

// A lane's 32 codes of a row in a K step: 16 from column k, 16 from k + 64.
struct Codes {
    u32x4 v[2];
    // any alignment; the step lies within the row
    template <bool STREAM>
    __device__ __forceinline__ void load(const uint8_t *row, long long k)
    {
#pragma unroll
        for (int h = 0; h < 2; h++) {
            typedef u32x4 __attribute__((aligned(1))) any;
            const any *const p = reinterpret_cast<const any *>(row + k + 64 * h);
            v[h] = STREAM ? __builtin_nontemporal_load(p) : *p;
        }
    }
    // the row's last step: zeros behind its I columns
    __device__ __forceinline__ void load_tail(const uint8_t *row, long long k, int I)
    {
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
            for (int j = 0; j < 4; j++) {
                uint32_t w = 0;
#pragma unroll
                for (int b = 0; b < 4; b++) {
                    const long long c = k + 64 * h + 4 * j + b;
                    if (c < I) w |= (uint32_t)row[c] << (8 * b);
                }
                v[h][j] = w;
            }
    }
    // four fragments of v_mfma_f32_16x16x32_f16; the column order is the same
    // for both operands, so it need not be the rows' own
    __device__ __forceinline__ void f16(f16x8 f[4]) const
    {
#pragma unroll
        for (int h = 0; h < 2; h++) {
            f[2 * h] = fp8x8_f16(v[h].x, v[h].y);
            f[2 * h + 1] = fp8x8_f16(v[h].z, v[h].w);
        }
    }
};

// Stream kernel, every shape, alignment and stride.  A workgroup makes 16 MB
// rows of y x 16 NB rows of W (gated: half of them gate rows, half up rows);
// its 8 waves take the K steps of 128 columns in turn, one step's loads in
// flight during the products of the one before, and join their sums through
// LDS in a fixed order.
// Products are formed as f16 (each code is an f16 number, and a product of two
// has 8 bits) on v_mfma_f32_16x16x32_f16, W as the A operand: lane l holds row
// l % 16 of both, sums of rows 4 (l / 16) + i of W and row l % 16 of x.  A
// scale block's products are summed from zero and added as acc += (xs ws) sum.
// f16's matrix cores sum to f32's precision; those of e4m3 do not (matmul_tile.h),
// and where the weights' bytes bound the product nothing is gained by them.
// Bound by the bytes in flight: 5 x 6144 x 12288 22 us a call for f32 (75 MB, 3.4 TB/s),
// 25 for bf16; 3 x 512 x 256 4.9 us of kernel, its latency.
template <typename XT, int MB, int NB, bool GATED>
__global__ __launch_bounds__(SW * 64, 2) void matmul_stream(MatmulArgs p,
                                                            const ExpertTile *__restrict__ tiles)
{
    constexpr int YC = GATED ? NB * 8 : NB * 16;         // columns of y
    constexpr int LDR = NB * 16 + 4;
    __shared__ __align__(16) float red[SW][MB * 16][LDR];
    const LinearArgs &a = p.a;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int li = lane & 15, lg = lane >> 4;
    const int oc = GATED ? a.O / 2 : a.O;
    const int ntn = (oc + YC - 1) / YC;
    const int o0 = (int)(blockIdx.x % ntn) * YC, mt = (int)(blockIdx.x / ntn);
    ExpertTile t;
    if (tiles) t = tiles[mt];
    else t = ExpertTile{0, mt * (16 * MB), min(16 * MB, a.R - mt * (16 * MB))};
    t.n = __builtin_amdgcn_readfirstlane(t.n);
    t.expert = __builtin_amdgcn_readfirstlane(t.expert);
    if (t.n <= 0) return;                                // uniform over the workgroup

    // Rows behind the tile or the matrix repeat one that exists; a bad row index
    // reads row 0 and is marked in the epilogue.
    const uint8_t *xrow[MB], *wrow[NB];
    const float *xsrow[MB], *wsrow[NB];
    int second[NB];                      // of the lane's rows of W, the first of the next block
#pragma unroll
    for (int m = 0; m < MB; m++) {
        long long r = t.row0 + (m * 16 + li < t.n ? m * 16 + li : 0);
        if (a.rows) {
            const int x = a.rows[r];
            r = x < 0 || x >= a.T ? 0 : x;
        }
        xrow[m] = static_cast<const uint8_t *>(a.x) + r * a.ldx + lg * 16;
        xsrow[m] = p.xs + r * p.ldxs;
    }
    const float *const sbase = a.scales + (long long)t.expert * a.s_stride;
    const int nblk = (a.O + 127) / 128;
#pragma unroll
    for (int n = 0; n < NB; n++) {
        const int half = GATED ? n / (NB / 2) : 0;
        const int c0 = o0 + (GATED ? n % (NB / 2) : n) * 16;
        const int c = c0 + li;
        wrow[n] = a.w + (long long)t.expert * a.w_stride +
                  (long long)((c < oc ? c : oc - 1) + half * oc) * a.I + lg * 16;
        const int r0 = min(c0 + 4 * lg, oc - 1) + half * oc, b0 = r0 / 128;
        wsrow[n] = sbase + (long long)b0 * a.ng;
        second[n] = b0 + 1 < nblk ? (b0 + 1) * 128 - r0 : 4;
    }

    f32x4v acc[MB][NB];
#pragma unroll
    for (int m = 0; m < MB; m++)
#pragma unroll
        for (int n = 0; n < NB; n++) acc[m][n] = f32x4v{0.0f, 0.0f, 0.0f, 0.0f};

    struct Step {
        Codes x[MB], w[NB];
        float xs[MB], ws[NB][GATED ? 2 : 1];
    };
    const int whole = a.I / SK, steps = a.ng;
    auto load = [&](Step &b, int s) {
        const long long k = (long long)s * SK;
        if (s < whole) {                                 // uniform over the wave
#pragma unroll
            for (int n = 0; n < NB; n++) b.w[n].template load<true>(wrow[n], k);
#pragma unroll
            for (int m = 0; m < MB; m++) b.x[m].template load<false>(xrow[m], k);
        } else {
#pragma unroll
            for (int n = 0; n < NB; n++) b.w[n].load_tail(wrow[n], k, a.I - lg * 16);
#pragma unroll
            for (int m = 0; m < MB; m++) b.x[m].load_tail(xrow[m], k, a.I - lg * 16);
        }
#pragma unroll
        for (int n = 0; n < NB; n++) {
            b.ws[n][0] = wsrow[n][s];
            // a gated product's up rows need not start at a block: a lane's four
            // rows may lie in two
            if (GATED) b.ws[n][GATED] = wsrow[n][s + (second[n] < 4 ? a.ng : 0)];
        }
#pragma unroll
        for (int m = 0; m < MB; m++) b.xs[m] = xsrow[m][s];
    };
    auto multiply = [&](const Step &b) {
        f16x8 xf[MB][4];
#pragma unroll
        for (int m = 0; m < MB; m++) b.x[m].f16(xf[m]);
#pragma unroll
        for (int n = 0; n < NB; n++) {
            f16x8 wf[4];
            b.w[n].f16(wf);
#pragma unroll
            for (int m = 0; m < MB; m++) {
                f32x4v g = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int h = 0; h < 4; h++)
                    g = __builtin_amdgcn_mfma_f32_16x16x32_f16(wf[h], xf[m][h], g, 0, 0, 0);
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    const float ws = GATED && r >= second[n] ? b.ws[n][GATED] : b.ws[n][0];
                    acc[m][n][r] = fmaf(b.xs[m] * ws, g[r], acc[m][n][r]);
                }
            }
        }
    };
    Step b0, b1;
    if (wave < steps) load(b0, wave);
    for (int s = wave; s < steps; s += 2 * SW) {
        if (s + SW < steps) load(b1, s + SW);
        multiply(b0);
        if (s + SW >= steps) break;
        if (s + 2 * SW < steps) load(b0, s + 2 * SW);
        multiply(b1);
    }

#pragma unroll
    for (int m = 0; m < MB; m++)
#pragma unroll
        for (int n = 0; n < NB; n++)
            *reinterpret_cast<f32x4v *>(&red[wave][m * 16 + li][n * 16 + 4 * lg]) = acc[m][n];
    __syncthreads();
    finish<XT, 4>(a, t.expert, tid, SW * 64, t.n * YC,
                  [&](int i, int &row, int &col, float &v, float &up) {
                      const int r = i / YC, c = i % YC;
                      row = t.row0 + r;
                      col = o0 + c;
                      v = up = 0.0f;
#pragma unroll
                      for (int w = 0; w < SW; w++) {
                          v += red[w][r][c];
                          if (GATED) up += red[w][r][c + YC];
                      }
                      if (a.rows) {
                          const int x = a.rows[row];
                          if (x < 0 || x >= a.T) v = up = __builtin_nanf("");
                      }
                  });
}

// Blocks of 16 rows of W per workgroup: one where two would leave a CU less than two
// workgroups (gated: a gate and an up block at least).  us, 5 rows: 6144 x 12288 one
// 22.2, two 25.1; 11008 x 4096 15.1 and 22.8; 16384 x 7168 34.4 and 31.4.
int stream_blocks(const MatmulArgs &p, int bm, long long ntm)
{
    const long long wgs = ntm * ((p.a.O + 31) / 32);
    return bm == 16 && !p.a.gated && wgs < 2 * cu_count() ? 1 : 2;
}

template <typename XT, int MB, int NB>
hipError_t run_stream(const MatmulArgs &p, const ExpertTile *tiles, unsigned grid, hipStream_t st)
{
    if constexpr (NB > 1) {
        if (p.a.gated) {
            hipLaunchKernelGGL((matmul_stream<XT, MB, NB, true>), dim3(grid), dim3(SW * 64), 0, st,
                               p, tiles);
            return hipGetLastError();
        }
    }
    hipLaunchKernelGGL((matmul_stream<XT, MB, NB, false>), dim3(grid), dim3(SW * 64), 0, st, p,
                       tiles);
    return hipGetLastError();
}

long long stream_grid(const MatmulArgs &p, int nb, long long ntm)
{
    const int cols = nb * 16 / (p.a.gated ? 2 : 1), oc = p.a.gated ? p.a.O / 2 : p.a.O;
    return ntm * ((oc + cols - 1) / cols);
}

}  // namespace

long long matmul_stream_items(const MatmulArgs &p, int bm, long long ntm)
{
    return stream_grid(p, stream_blocks(p, bm, ntm), ntm) * (SW * 64);
}

hipError_t launch_matmul_stream(const MatmulArgs &p, int bm, const ExpertTile *tiles, int ntm,
                                hipStream_t st)
{
    const int nb = stream_blocks(p, bm, ntm);
    const unsigned grid = (unsigned)stream_grid(p, nb, ntm);
#define QG_STREAM(XT)                                                                       \
    (bm == 16 ? nb == 1 ? run_stream<XT, 1, 1>(p, tiles, grid, st)                          \
                        : run_stream<XT, 1, 2>(p, tiles, grid, st)                          \
     : bm == 32 ? run_stream<XT, 2, 2>(p, tiles, grid, st)                                  \
                : run_stream<XT, 4, 2>(p, tiles, grid, st))
    return p.a.dtype == QGEMV_BF16 ? QG_STREAM(BF16) : QG_STREAM(F32);
#undef QG_STREAM
}

}  // namespace qg
