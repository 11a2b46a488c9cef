// linear.hip -- many-token products with an epilogue, dense or grouped by
// expert: the general kernel, and the choice among kernels.
//
// Y = epilogue(X . W^T), W grouped int4 or fp8-e4m3 with block scales.
#include "qg_device.h"
#include "qg_launch.h"
#include "qg_linear.h"

namespace qg {

namespace {

typedef float f32x4v __attribute__((ext_vector_type(4)));

constexpr int GM = 64;          // rows of y per workgroup tile
constexpr int GN = 64;          // columns of y per workgroup tile
constexpr int GK = 32;          // columns of W per K step
constexpr int GLD = GK + 4;     // LDS row stride in floats

// General kernel: every valid shape, alignment and group size.  W decoded to
// f32 as the definition has it ((q - 8) * s or e4m3 * s, one rounding),
// products and sums in f32 on v_mfma_f32_16x16x4_f32, whose 157 TFLOP/s peak
// bounds it for many rows.  64 x 64 tiles of 4 waves (2 x 2 blocks each); a
// gated product holds the gate's and the up projection's accumulators for the
// same 64 columns of y.  Loads are per element with their column checked, so
// nothing needs alignment or whole K steps.
template <int FMT, typename XT, bool GATED>
__global__ __launch_bounds__(256) void linear_general(LinearArgs a,
                                                      const RowTile *__restrict__ tiles)
{
    typedef typename XT::raw raw;
    constexpr int NW = GATED ? 2 : 1;
    __shared__ __align__(16) float xs[GM * GLD];
    __shared__ __align__(16) float ws[NW][GN * GLD];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave & 1, wn = wave >> 1;
    const int oc = GATED ? a.O / 2 : a.O;                // columns of y
    const int ntn = (oc + GN - 1) / GN;
    const int o0 = (int)(blockIdx.x % ntn) * GN;
    const int mt = (int)(blockIdx.x / ntn);
    RowTile t;
    if (tiles) t = tiles[mt];
    else t = RowTile{0, mt * GM, min(GM, a.R - mt * GM), 0};
    if (t.n <= 0) return;                                // uniform over the workgroup

    f32x4v acc[NW][2][2];
#pragma unroll
    for (int p = 0; p < NW; p++)
#pragma unroll
        for (int i = 0; i < 2; i++)
#pragma unroll
            for (int j = 0; j < 2; j++) acc[p][i][j] = f32x4v{0.0f, 0.0f, 0.0f, 0.0f};

    // thread's staging place: row tid / 4, eight columns from 8 (tid % 4)
    const int sr = tid >> 2, sc = (tid & 3) * 8;
    const bool xok = sr < t.n;
    bool xbad = false;
    long long xrow = t.row0 + (xok ? sr : 0);
    if (a.rows) {
        const int r = a.rows[xrow];
        xbad = r < 0 || r >= a.T;
        xrow = xbad ? 0 : r;
    }
    const raw *xsrc = static_cast<const raw *>(a.x) + (size_t)xrow * a.ldx;
    const bool wok = o0 + sr < oc;
    const int wrow = wok ? o0 + sr : 0;
    const size_t rb = FMT == FMT_I4G ? ((size_t)a.I + 1) / 2 : (size_t)a.I;
    const uint8_t *wsrc = a.w + (size_t)t.expert * a.w_stride;
    const float *ssrc = a.scales + (size_t)t.expert * a.s_stride;

    for (int k0 = 0; k0 < a.I; k0 += GK) {
        float xv[8], wv[NW][8];
        const int k = k0 + sc;
#pragma unroll
        for (int c = 0; c < 8; c++) {
            xv[c] = 0.0f;
            if (xok && k + c < a.I)
                xv[c] = xbad ? __builtin_nanf("") : XT::get(xsrc[k + c]);
        }
#pragma unroll
        for (int p = 0; p < NW; p++) {
            const int row = wrow + p * oc;
            const uint8_t *wp = wsrc + (size_t)row * rb;
            const float *sp = ssrc + (size_t)(FMT == FMT_I4G ? row : row / 128) * a.ng;
#pragma unroll
            for (int c = 0; c < 8; c++) {
                wv[p][c] = 0.0f;
                if (!wok || k + c >= a.I) continue;
                if (FMT == FMT_I4G) {
                    const uint8_t b = wp[(size_t)(k + c) >> 1];
                    const int q = (c & 1) ? b >> 4 : b & 15;
                    wv[p][c] = (float)(q - 8) * sp[(k + c) / a.gs];
                } else {
                    wv[p][c] = fp8pair_lo(wp[k + c]).x * sp[(k + c) / 128];
                }
            }
        }
        if (k0 > 0) __syncthreads();                     // the previous step's reads are done
#pragma unroll
        for (int c = 0; c < 8; c++) xs[sr * GLD + sc + c] = xv[c];
#pragma unroll
        for (int p = 0; p < NW; p++)
#pragma unroll
            for (int c = 0; c < 8; c++) ws[p][sr * GLD + sc + c] = wv[p][c];
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < GK; kk += 4) {
            float av[2], bv[NW][2];
#pragma unroll
            for (int i = 0; i < 2; i++)
                av[i] = xs[(wm * 32 + i * 16 + (lane & 15)) * GLD + kk + (lane >> 4)];
#pragma unroll
            for (int p = 0; p < NW; p++)
#pragma unroll
                for (int j = 0; j < 2; j++)
                    bv[p][j] = ws[p][(wn * 32 + j * 16 + (lane & 15)) * GLD + kk + (lane >> 4)];
#pragma unroll
            for (int p = 0; p < NW; p++)
#pragma unroll
                for (int i = 0; i < 2; i++)
#pragma unroll
                    for (int j = 0; j < 2; j++)
                        acc[p][i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                            av[i], bv[p][j], acc[p][i][j], 0, 0, 0);
        }
    }

    // sums through LDS, 16 rows of each 32 at a time, so that one piece of code
    // ends all outputs
    float *const os = xs;                                // [32][GN + 1]; the gate's up: ws
    static_assert(32 * (GN + 1) <= GM * GLD && GN == GM, "fits the operands' LDS");
#pragma unroll
    for (int i = 0; i < 2; i++) {
        __syncthreads();
#pragma unroll
        for (int p = 0; p < NW; p++)
#pragma unroll
            for (int j = 0; j < 2; j++)
#pragma unroll
                for (int r = 0; r < 4; r++)
                    (p ? ws[0] : os)[(wm * 16 + 4 * (lane >> 4) + r) * (GN + 1) + wn * 32 +
                                     j * 16 + (lane & 15)] = acc[p][i][j][r];
        __syncthreads();
        finish<XT, 4>(a, t.expert, tid, 256, 32 * GN,
                      [&](int k, int &row, int &col, float &v, float &up) {
                          const int m = k / GN, c = k % GN;
                          const int tr = (m >> 4) * 32 + i * 16 + (m & 15);
                          row = t.row0 + tr;
                          col = tr < t.n && o0 + c < oc ? o0 + c : oc;
                          v = os[m * (GN + 1) + c];
                          up = GATED ? ws[0][m * (GN + 1) + c] : 0.0f;
                      });
    }
}

// Row tiles of a grouped product, from the experts' offsets on the device:
// tile i of the list is the i-th block of bm rows, experts in ascending
// order; the rest of the list is empty.  Offsets are clamped to 0..R and a
// negative count counts as none, so that every tile lies within y.  One
// workgroup; each thread takes one expert, then finds its tiles by bisection.
__global__ __launch_bounds__(1024) void plan_tiles(const int32_t *__restrict__ offsets, int E,
                                                   int R, int bm, RowTile *__restrict__ tiles,
                                                   int ntiles)
{
    __shared__ int base[1025];      // first tile of each expert
    __shared__ int start[1024];     // first row
    __shared__ int count[1024];     // rows
    __shared__ int wsum[16];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int lo = 0, n = 0;
    if (tid < E) {
        lo = min(max(offsets[tid], 0), R);
        n = max(min(max(offsets[tid + 1], 0), R) - lo, 0);
    }
    const int mine = (n + bm - 1) / bm;
    int incl = mine;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int v = __shfl_up(incl, d);
        if (lane >= d) incl += v;
    }
    if (lane == 63) wsum[wave] = incl;
    __syncthreads();
    int before = 0;
    for (int i = 0; i < wave; i++) before += wsum[i];
    // overlapping offsets (not allowed) could name more tiles than the list
    // holds; sums of up to 1024 counts of 2^24 / 16 tiles stay below 2^31
    base[tid + 1] = before + incl;
    if (tid == 0) base[0] = 0;
    start[tid] = lo;
    count[tid] = n;
    __syncthreads();
    for (int i = tid; i < ntiles; i += 1024) {
        RowTile t{0, 0, 0, 0};
        if (i < base[1024]) {
            int a = 0, b = 1024;                         // base[a] <= i < base[b]
            while (b - a > 1) {
                const int m = (a + b) / 2;
                if (base[m] <= i) a = m;
                else b = m;
            }
            const int r = (i - base[a]) * bm;
            t = RowTile{a, start[a] + r, min(bm, count[a] - r), 0};
        }
        tiles[i] = t;
    }
}

// tiles that R rows of E experts can need
long long max_tiles(int R, int E, int bm)
{
    return (long long)R / bm + (E < R ? E : R);
}

// Tile of a product: the one whose busiest CU has the least to do, estimated
// as workgroups per CU times the cost of one.  Costs of a workgroup relative
// to 128 x 256, from bf16 int4 at 6144 columns (125 us with one 128 x 256
// tile per CU, 200 with two, 323 with three); f32 counts two planes.  What the
// rule decides, us with the tile chosen and with the next best: 256 x 12288:
// 64 x 256 89, narrow 93, 128 x 256 125; 512 x 12288: 128 x 256 126, 64 x 256
// 139; 512 x 4096 (4096 columns): narrow 49, 32 x 256 53, 128 x 256 95; f32
// 333 x 11008 (4096 columns): 32 x 256 97, 64 x 256 117.  Grouped tiles know
// neither their count (estimated with half a tile per expert) nor their
// filling, and skip what they lack: only the largest of each kind.
void pick_tile(const LinearArgs &a, int oc, int &bm, bool &narrow)
{
    struct Kind {
        int bm;
        bool narrow, grouped;
        double cost;
    };
    static const Kind bf16[] = {{128, false, true, 1.0},
                                {64, false, false, 0.66},
                                {32, false, false, 0.58},
                                {64, true, true, 0.265},
                                {32, true, false, 0.185}};
    static const Kind f32[] = {{64, false, true, 0.93}, {32, false, false, 0.69},
                               {32, true, true, 0.26}};
    const bool half = a.dtype == QGEMV_BF16;
    const Kind *kinds = half ? bf16 : f32;
    const int n = half ? 5 : 3;
    const long long ncu = cu_count();
    double best = -1.0;
    for (int i = 0; i < n; i++) {
        const Kind &k = kinds[i];
        if (a.offsets && !k.grouped) continue;
        const int cols = (k.narrow ? 64 : 256) / (a.gated ? 2 : 1);
        const long long mt = (a.R + k.bm - 1) / k.bm +
                             (a.offsets ? (a.E < a.R ? a.E : a.R) / 2 : 0);
        const long long wgs = mt * ((oc + cols - 1) / cols);
        const double c = (double)((wgs + ncu - 1) / ncu) * k.cost;
        if (best < 0.0 || c < best) {                    // ties: the larger tile
            best = c;
            bm = k.bm;
            narrow = k.narrow;
        }
    }
}

template <int FMT, typename XT>
void run_general(const LinearArgs &a, const RowTile *tiles, unsigned grid, hipStream_t st)
{
    if (a.gated)
        hipLaunchKernelGGL((linear_general<FMT, XT, true>), dim3(grid), dim3(256), 0, st, a, tiles);
    else
        hipLaunchKernelGGL((linear_general<FMT, XT, false>), dim3(grid), dim3(256), 0, st, a,
                           tiles);
}

}  // namespace

size_t linear_workspace(int T, int R, int E, int I, int O, int dtype)
{
    (void)O;
    return (E > 0 ? align256((size_t)max_tiles(R, E, 16) * sizeof(RowTile)) : 0) +
           tile_workspace(T, I, dtype);
}

hipError_t launch_linear(WeightFormat fmt, const LinearArgs &a, void *ws, hipStream_t st)
{
    const int oc = a.gated ? a.O / 2 : a.O;
    const bool fits = tile_fits(fmt, a);
    const int rows = a.offsets ? (a.R + a.E - 1) / a.E : a.R;
    const bool stream = rows <= 16 && stream_fits(fmt, a);
    int bm = GM;
    bool narrow = false;
    if (stream) {
        bm = 16;
    } else if (fits) {
        pick_tile(a, oc, bm, narrow);
    }
    RowTile *tiles = nullptr;
    long long mt = (a.R + bm - 1) / bm;
    if (a.offsets) {
        tiles = static_cast<RowTile *>(ws);
        mt = max_tiles(a.R, a.E, bm);
        hipLaunchKernelGGL(plan_tiles, dim3(1), dim3(1024), 0, st, a.offsets, a.E, a.R, bm, tiles,
                           (int)mt);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        ws = static_cast<char *>(ws) + align256((size_t)max_tiles(a.R, a.E, 16) * sizeof(RowTile));
    }
    if (stream) return launch_stream(fmt, a, tiles, (int)mt, st);
    if (fits) return launch_tile(fmt, a, narrow, bm, tiles, (int)mt, ws, st);
    const long long grid = mt * ((oc + GN - 1) / GN);
    if (grid > 0x7FFFFFFFLL) return hipErrorInvalidValue;
    if (fmt == FMT_I4G) {
        if (a.dtype == QGEMV_BF16) run_general<FMT_I4G, BF16>(a, tiles, (unsigned)grid, st);
        else run_general<FMT_I4G, F32>(a, tiles, (unsigned)grid, st);
    } else {
        if (a.dtype == QGEMV_BF16) run_general<FMT_FP8, BF16>(a, tiles, (unsigned)grid, st);
        else run_general<FMT_FP8, F32>(a, tiles, (unsigned)grid, st);
    }
    return hipGetLastError();
}

}  // namespace qg
