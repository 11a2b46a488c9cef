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

constexpr int GN = 64;          // columns of y per workgroup tile
constexpr int GN_THIN = 16;     // and per thin one
constexpr int GK = 32;          // columns of W per K step
constexpr int GLD = GK + 4;     // LDS row stride in floats
constexpr int GM_FEW = 16;      // rows of y per tile, few rows
constexpr int GM = 64;          // and many

// Eight values of a row of x from column k: one load of any alignment, or, for
// a row's last columns, element by element with zeros behind them.
template <typename XT>
struct X8 {
    typename XT::raw v[8];
    __device__ __forceinline__ void load(const typename XT::raw *row, int k)
    {
        __builtin_memcpy(v, row + k, sizeof(v));
    }
    __device__ __forceinline__ void load_tail(const typename XT::raw *row, int k, int I)
    {
#pragma unroll
        for (int c = 0; c < 8; c++) v[c] = k + c < I ? row[k + c] : typename XT::raw(0);
    }
};

// Eight weights of a row from column k (a multiple of eight), decoded as the
// definition has it.  Group sizes of eight or more have at most two scales
// among them, smaller ones (SMALL, even) one per pair.  The tail's values
// behind the row are finite and meet zeros of x.
template <int FMT, bool SMALL>
struct W8 {
    uint32_t q[2];                       // int4: the first
    float s[4];
    int edge;                            // columns of s[0]
    __device__ __forceinline__ void load_scales(const float *sc, int k, int ng, int gs)
    {
        if (SMALL) {
#pragma unroll
            for (int c = 0; c < 4; c++) s[c] = sc[min((k + 2 * c) / gs, ng - 1)];
        } else {
            const int g = min(k / gs, ng - 1);
            edge = (g + 1) * gs - k;
            s[0] = sc[g];
            s[1] = sc[min(g + 1, ng - 1)];
        }
    }
    __device__ __forceinline__ void load(const uint8_t *row, const float *sc, int k, int ng,
                                         int gs)
    {
        __builtin_memcpy(q, row + (FMT == FMT_I4G ? k / 2 : k), FMT == FMT_I4G ? 4 : 8);
        load_scales(sc, k, ng, gs);
    }
    __device__ __forceinline__ void load_tail(const uint8_t *row, const float *sc, int k, int I,
                                              int ng, int gs)
    {
        q[0] = q[1] = 0;
#pragma unroll
        for (int c = 0; c < 8; c++) {
            if (k + c >= I) continue;
            if (FMT == FMT_I4G) {
                if (c % 2 == 0) q[0] |= (uint32_t)row[(k + c) / 2] << (4 * c);
            } else {
                q[c / 4] |= (uint32_t)row[k + c] << (8 * (c % 4));
            }
        }
        load_scales(sc, k, ng, gs);
    }
    __device__ __forceinline__ void decode(float w[8]) const
    {
        if (FMT == FMT_I4G) {
            float e[4], o[4];
            nib8(q[0], e, o);
#pragma unroll
            for (int c = 0; c < 4; c++) {
                w[2 * c] = e[c] * NIB_XSCALE - 8.0f;
                w[2 * c + 1] = o[c] * NIB_XSCALE - 8.0f;
            }
        } else {
            e4m3x4(q[0], w);
            e4m3x4(q[1], w + 4);
        }
#pragma unroll
        for (int c = 0; c < 8; c++) w[c] *= SMALL ? s[c / 2] : c < edge ? s[0] : s[1];
    }
};

// General kernel: every valid shape, alignment and group size.  W decoded to
// f32 as the definition has it ((q - 8) * s or e4m3 * s, one rounding),
// products and sums in f32 on v_mfma_f32_16x16x4_f32, whose 157 TFLOP/s peak
// bounds it for many rows.  A gated product holds the gate's and the up
// projection's accumulators for the same columns of y.  The global loads of
// the next K step are in flight during the products.
//
// MANY: 64 x 64 tiles of 4 waves (2 x 2 blocks of 16 each), a thread stages
// eight columns of one row of each operand.  FEW: 16 x 64 tiles of 4 waves,
// which take K steps in turn with LDS of their own; their sums are joined in a
// fixed order.  THIN: the same with 16 x 16 tiles of 16 waves, where wider ones
// are too few to cover the latency of their loads.
enum Shape { MANY, FEW, THIN };

template <int FMT, typename XT, bool GATED, Shape SHAPE, bool SMALL>
__global__ __launch_bounds__(SHAPE == THIN ? 1024 : 256) void
linear_general(LinearArgs a, const RowTile *__restrict__ tiles)
{
    typedef typename XT::raw raw;
    constexpr bool SPLIT = SHAPE != MANY;                // K split over the waves
    constexpr int WAVES = SHAPE == THIN ? 16 : 4;
    constexpr int BN = SHAPE == THIN ? GN_THIN : GN;
    constexpr int NW = GATED ? 2 : 1;
    constexpr int BM = SPLIT ? GM_FEW : GM;
    constexpr int MB = SPLIT ? 1 : 2, NB = SPLIT ? BN / 16 : 2;   // blocks of a wave
    constexpr int WR = SPLIT ? BN / 16 : 1;              // rows of W a thread stages
    constexpr int STAGE = (BM + NW * BN) * GLD;          // floats
    constexpr int OLD = BN + 1;                          // epilogue row stride
    constexpr int OUT = (SPLIT ? WAVES * GM_FEW : 32) * OLD * NW;
    constexpr int STAGES = (SPLIT ? WAVES : 1) * STAGE;
    __shared__ __align__(16) float lds[STAGES > OUT ? STAGES : OUT];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = SPLIT ? 0 : wave & 1, wn = SPLIT ? 0 : wave >> 1;
    float *const xs = lds + (SPLIT ? wave * STAGE : 0);
    float *const ws = xs + BM * GLD;
    const int oc = GATED ? a.O / 2 : a.O;                // columns of y
    const int ntn = (oc + BN - 1) / BN;
    const int o0 = (int)(blockIdx.x % ntn) * BN;
    const int mt = (int)(blockIdx.x / ntn);
    RowTile t;
    if (tiles) t = tiles[mt];
    else t = RowTile{0, mt * BM, min(BM, a.R - mt * BM), 0};
    if (t.n <= 0) return;                                // uniform over the workgroup

    f32x4v acc[NW][MB][NB];
#pragma unroll
    for (int p = 0; p < NW; p++)
#pragma unroll
        for (int i = 0; i < MB; i++)
#pragma unroll
            for (int j = 0; j < NB; j++) acc[p][i][j] = f32x4v{0.0f, 0.0f, 0.0f, 0.0f};

    // this thread's staging place: row sr of x, rows sr + 16 i of W, eight
    // columns from sc; rows behind the tile or the matrix repeat the first
    const int u = SPLIT ? lane : tid;
    const int sr = u >> 2, sc = (u & 3) * 8;
    long long xrow = t.row0 + (sr < t.n ? sr : 0);
    if (a.rows) {
        const int r = a.rows[xrow];
        xrow = r < 0 || r >= a.T ? 0 : r;                // marked in the epilogue
    }
    const raw *xsrc = static_cast<const raw *>(a.x) + (size_t)xrow * a.ldx;
    const size_t rb = FMT == FMT_I4G ? ((size_t)a.I + 1) / 2 : (size_t)a.I;
    const uint8_t *wsrc[NW][WR];
    const float *ssrc[NW][WR];
#pragma unroll
    for (int p = 0; p < NW; p++)
#pragma unroll
        for (int i = 0; i < WR; i++) {
            const int c = o0 + sr + 16 * i;
            const int row = (c < oc ? c : 0) + p * oc;
            wsrc[p][i] = a.w + (size_t)t.expert * a.w_stride + (size_t)row * rb;
            ssrc[p][i] = a.scales + (size_t)t.expert * a.s_stride +
                         (size_t)(FMT == FMT_I4G ? row : row / 128) * a.ng;
        }
    const int gs = FMT == FMT_FP8 ? 128 : a.gs;

    X8<XT> xv;
    W8<FMT, SMALL> wv[NW][WR];
    auto load = [&](int k0) {
        const int k = k0 + sc;
        if (k0 + GK <= a.I) {                            // uniform over the wave
            xv.load(xsrc, k);
#pragma unroll
            for (int p = 0; p < NW; p++)
#pragma unroll
                for (int i = 0; i < WR; i++)
                    wv[p][i].load(wsrc[p][i], ssrc[p][i], k, a.ng, gs);
        } else {
            xv.load_tail(xsrc, k, a.I);
#pragma unroll
            for (int p = 0; p < NW; p++)
#pragma unroll
                for (int i = 0; i < WR; i++)
                    wv[p][i].load_tail(wsrc[p][i], ssrc[p][i], k, a.I, a.ng, gs);
        }
    };
    constexpr int STEP = (SPLIT ? WAVES : 1) * GK;
    const int first = SPLIT ? wave * GK : 0;
    if (first < a.I) load(first);
    for (int k0 = first; k0 < a.I; k0 += STEP) {
        if (!SPLIT && k0 > 0) __syncthreads();             // the previous step's reads are done
#pragma unroll
        for (int c = 0; c < 8; c++) xs[sr * GLD + sc + c] = XT::get(xv.v[c]);
#pragma unroll
        for (int p = 0; p < NW; p++)
#pragma unroll
            for (int i = 0; i < WR; i++) {
                float w[8];
                wv[p][i].decode(w);
#pragma unroll
                for (int c = 0; c < 8; c++) ws[(p * BN + sr + 16 * i) * GLD + sc + c] = w[c];
            }
        if (!SPLIT) __syncthreads();
        else __builtin_amdgcn_wave_barrier();            // lanes read each other's values
        if (k0 + STEP < a.I) load(k0 + STEP);
#pragma unroll
        for (int kk = 0; kk < GK; kk += 4) {
            float av[MB], bv[NW][NB];
#pragma unroll
            for (int i = 0; i < MB; i++)
                av[i] = xs[(wm * 32 + i * 16 + (lane & 15)) * GLD + kk + (lane >> 4)];
#pragma unroll
            for (int p = 0; p < NW; p++)
#pragma unroll
                for (int j = 0; j < NB; j++)
                    bv[p][j] =
                        ws[(p * BN + wn * 32 + j * 16 + (lane & 15)) * GLD + kk + (lane >> 4)];
#pragma unroll
            for (int p = 0; p < NW; p++)
#pragma unroll
                for (int i = 0; i < MB; i++)
#pragma unroll
                    for (int j = 0; j < NB; j++)
                        acc[p][i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                            av[i], bv[p][j], acc[p][i][j], 0, 0, 0);
        }
    }

    // sums through LDS (K split: of all waves; else 16 rows of each 32 at a time),
    // so that one piece of code ends all outputs
#pragma unroll
    for (int i = 0; i < MB; i++) {
        __syncthreads();
#pragma unroll
        for (int p = 0; p < NW; p++)
#pragma unroll
            for (int j = 0; j < NB; j++)
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    const int m = (SPLIT ? wave : wm) * 16 + 4 * (lane >> 4) + r;
                    lds[(m * NW + p) * OLD + wn * 32 + j * 16 + (lane & 15)] = acc[p][i][j][r];
                }
        __syncthreads();
        finish<XT, 4>(a, t.expert, tid, WAVES * 64, (SPLIT ? GM_FEW : 32) * BN,
                      [&](int k, int &row, int &col, float &v, float &up) {
                          const int m = k / BN, c = k % BN;
                          const int tr = SPLIT ? m : (m >> 4) * 32 + i * 16 + (m & 15);
                          row = t.row0 + tr;
                          col = tr < t.n && o0 + c < oc ? o0 + c : oc;
                          v = up = 0.0f;
#pragma unroll
                          for (int w = 0; w < (SPLIT ? WAVES : 1); w++) {
                              v += lds[((w * 16 + m) * NW) * OLD + c];
                              if (GATED) up += lds[((w * 16 + m) * NW + 1) * OLD + c];
                          }
                          if (a.rows && col < oc) {
                              const int xi = a.rows[row];
                              if (xi < 0 || xi >= a.T) v = up = __builtin_nanf("");
                          }
                      });
    }
}

// Row tiles of a grouped product, from the experts' offsets on the device:
// first the whole blocks of bm rows, experts in ascending order, then the
// experts' last, shorter blocks, the longest first (in sixteenths of rows), so
// that the short ones fill the end of the launch; the rest of the list is
// empty.  Offsets are clamped to 0..R and a negative count counts as none, so
// that every tile lies within y.  One workgroup, a thread per expert.
__global__ __launch_bounds__(1024) void plan_tiles(const int32_t *__restrict__ offsets, int E,
                                                   int R, int bm, RowTile *__restrict__ tiles,
                                                   int ntiles)
{
    __shared__ int base[1025];      // first whole tile of each expert
    __shared__ int start[1024];     // first row
    __shared__ int wsum[64];        // whole tiles of each wave's experts (16), then the sum before
    __shared__ int wcls[128];       // short tiles by length and wave, then the sum before
    __shared__ int totals[2];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int lo = 0, n = 0;
    if (tid < E) {
        lo = min(max(offsets[tid], 0), R);
        n = max(min(max(offsets[tid + 1], 0), R) - lo, 0);
    }
    const int whole = n / bm, rest = n - whole * bm;
    int incl = whole;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int v = __shfl_up(incl, d);
        if (lane >= d) incl += v;
    }
    if (lane == 63) wsum[wave] = incl;
    // length class of the short tile: 0 the longest, -1 none
    const int cls = rest ? (bm - rest) / 16 : -1;
    int rank = 0;
#pragma unroll
    for (int c = 0; c < 8; c++) {
        const unsigned long long m = __ballot(cls == c);
        if (cls == c) rank = __popcll(m & ((1ull << lane) - 1));
        if (lane == c) wcls[c * 16 + wave] = __popcll(m);
    }
    __syncthreads();
    if (wave < 2) {                                      // exclusive sums, one wave each
        const int w = wave == 0 ? (lane < 16 ? wsum[lane] : 0) : wcls[2 * lane];
        const int w1 = wave == 0 ? 0 : wcls[2 * lane + 1];
        int s = w + w1;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int v = __shfl_up(s, d);
            if (lane >= d) s += v;
        }
        if (lane == 63) totals[wave] = s;
        if (wave == 0) {
            wsum[lane] = s - w;
        } else {
            wcls[2 * lane] = s - w - w1;
            wcls[2 * lane + 1] = s - w1;
        }
    }
    __syncthreads();
    const int before = wsum[wave], total = totals[0], shorts = totals[1];
    // overlapping offsets (not allowed) could name more tiles than the list
    // holds; sums of up to 1024 counts of 2^24 / 16 tiles stay below 2^31
    base[tid + 1] = before + incl;
    if (tid == 0) base[0] = 0;
    start[tid] = lo;
    const int at = cls >= 0 ? wcls[cls * 16 + wave] : 0;
    __syncthreads();
    if (cls >= 0 && total + at + rank < ntiles)
        tiles[total + at + rank] = RowTile{tid, lo + whole * bm, rest, 0};
    for (int i = tid; i < ntiles; i += 1024) {
        if (i >= total && i < total + shorts) continue;
        RowTile t{0, 0, 0, 0};
        if (i < total) {
            int a = 0, b = 1024;                         // base[a] <= i < base[b]
            while (b - a > 1) {
                const int m = (a + b) / 2;
                if (base[m] <= i) a = m;
                else b = m;
            }
            t = RowTile{a, start[a] + (i - base[a]) * bm, bm, 0};
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
// as workgroups per CU times the cost of one, relative to 128 x 256 (a fifth
// more for a tile that has its CU to itself, one wave per SIMD); f32 counts two
// planes.  What the rule decides for int4, us with the tile chosen and with the
// next best: bf16, 6144 deep, 12288 columns: 256 rows: 64 x 256 78, narrow 93;
// 512: 128 x 256 126, 64 x 256 139; 700: 96 x 256 164, 128 x 256 188; 4096
// deep, 4096 columns: 512 rows: narrow 49, 64 x 256 65.  f32, 4096 deep, 11008
// columns: 333 rows: 32 x 256 86, 64 x 256 117.
// Grouped tiles are the largest of each kind, their count estimated with half a
// tile per expert, and a tile skips the rows it lacks: the cost has a fixed part
// and one that goes with the filling.  512 tokens of 8 among 256 experts, 7168 x
// 2048: 128 x 256 618, narrow 760; 200 of 2 among 8, 1024 x 512: narrow 19, 128
// x 256 62.
void pick_tile(const LinearArgs &a, int oc, int &bm, bool &narrow)
{
    struct Kind {
        int bm;
        bool narrow, grouped;
        double cost;
    };
    static const Kind bf16[] = {{128, false, true, 1.0},
                                {96, false, false, 0.83},
                                {64, false, false, 0.66},
                                {64, true, true, 0.235},
                                {32, true, false, 0.16}};
    static const Kind f32[] = {{64, false, true, 0.93}, {32, false, false, 0.69},
                               {32, true, true, 0.21}};
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
        const long long per_cu = (wgs + ncu - 1) / ncu;
        double c = per_cu * k.cost * (per_cu == 1 && !k.narrow ? 1.2 : 1.0);
        if (a.offsets) {
            const double fill = (double)a.R / ((double)mt * k.bm), fixed = k.narrow ? 0.5 : 0.35;
            c *= fixed + (1.0 - fixed) * fill;
        }
        if (best < 0.0 || c < best) {                    // ties: the larger tile
            best = c;
            bm = k.bm;
            narrow = k.narrow;
        }
    }
}

template <int FMT, typename XT>
void run_general(const LinearArgs &a, Shape shape, const RowTile *tiles, unsigned grid,
                 hipStream_t st)
{
#define QG_RUN(G, H, S)                                                                     \
    hipLaunchKernelGGL((linear_general<FMT, XT, G, H, S>), dim3(grid),                      \
                       dim3((H) == THIN ? 1024 : 256), 0, st, a, tiles)
#define QG_RUN_S(S)                                                                         \
    do {                                                                                    \
        if (shape == THIN) {                                                                \
            if (a.gated) QG_RUN(true, THIN, S);                                             \
            else QG_RUN(false, THIN, S);                                                    \
        } else if (shape == FEW) {                                                          \
            if (a.gated) QG_RUN(true, FEW, S);                                              \
            else QG_RUN(false, FEW, S);                                                     \
        } else {                                                                            \
            if (a.gated) QG_RUN(true, MANY, S);                                             \
            else QG_RUN(false, MANY, S);                                                    \
        }                                                                                   \
    } while (0)
    if constexpr (FMT == FMT_I4G) {
        if (a.gs < 8) {
            QG_RUN_S(true);
            return;
        }
    }
    QG_RUN_S(false);
#undef QG_RUN_S
#undef QG_RUN
}

}  // namespace

size_t linear_workspace(int T, int R, int E, int I, int dtype)
{
    const int slice = tile_rows(I);
    const int rows = E > 0 || T < slice ? T : slice;
    return (E > 0 ? align256((size_t)max_tiles(R, E, 16) * sizeof(RowTile)) : 0) +
           (planes_fit(rows, I) ? tile_workspace(rows, I, dtype) : 0);
}

// The kernel of a product, its row tiles and its launch's work items.
struct Choice {
    int stream;                          // rows of the stream kernel's tiles, or 0
    bool fits, narrow;                   // the packed kernels take it
    Shape shape;                         // of the general kernel
    int bm;
    long long mt, items;
};

static Choice choose(WeightFormat fmt, const LinearArgs &a)
{
    Choice c{};
    const int oc = a.gated ? a.O / 2 : a.O;
    c.fits = tile_fits(fmt, a);
    c.stream = stream_rows(fmt, a);
    const int rows = a.offsets ? (a.R + a.E - 1) / a.E : a.R;
    // The general kernel's tiles: 16 rows also where 64-row tiles would give a
    // CU less than two, thin ones where those of 16 x 64 would.  us, bf16 int4:
    // 512 x 3001 x 3001 (376 tiles of 64 rows) 141 in tiles of 16 rows, 160 of
    // 64; 512 x 3001 x 6001 (752) 268 and 205; 2 x 4069 x 2742 (43 tiles of 16 x
    // 64) 45, thin 13; 128 x 3001 x 3001 (376) 56, thin 44; 128 x 3001 x 6001
    // (752) 73, thin 83.
    const long long shorts = a.offsets ? (a.E < a.R ? a.E : a.R) / 2 : 0;
    const long long ntn = (oc + GN - 1) / GN, most = cu_count() * 3 / 2;
    const long long tiles64 = ((a.R + GM - 1) / GM + shorts) * ntn;
    const long long tiles16 = ((a.R + GM_FEW - 1) / GM_FEW + shorts) * ntn;
    c.shape = rows > GM_FEW && tiles64 > most ? MANY : tiles16 > most ? FEW : THIN;
    c.bm = c.shape == MANY ? GM : GM_FEW;
    if (c.stream) c.bm = c.stream;
    else if (c.fits) pick_tile(a, oc, c.bm, c.narrow);
    c.mt = a.offsets ? max_tiles(a.R, a.E, c.bm) : (a.R + c.bm - 1) / c.bm;
    if (c.stream) {
        c.items = stream_items(fmt, a, c.stream, (int)c.mt);
    } else if (c.fits) {
        c.items = tile_items(a, c.narrow, c.bm, (int)c.mt);
    } else {
        const int bn = c.shape == THIN ? GN_THIN : GN;
        c.items = c.mt * ((oc + bn - 1) / bn) * (c.shape == THIN ? 1024 : 256);
    }
    return c;
}

bool linear_launchable(WeightFormat fmt, const LinearArgs &a)
{
    return !a.offsets || choose(fmt, a).items <= MAX_ITEMS;
}

hipError_t launch_linear(WeightFormat fmt, const LinearArgs &args, void *ws, hipStream_t st)
{
    LinearArgs a = args;
    const int oc = a.gated ? a.O / 2 : a.O;
    Choice c;
    if (a.offsets) {
        c = choose(fmt, a);
    } else {
        // slices of rows: a dense product's packed activations must lie within
        // 4 GB, its work items within a launch (128 rows of 2^24 outputs do)
        int slice = tile_rows(a.I);
        for (;; slice = (slice / 2 + 127) / 128 * 128) {
            a.T = a.R = args.R < slice ? args.R : slice;
            c = choose(fmt, a);
            if (c.items <= MAX_ITEMS || slice <= 128) break;
        }
        if (args.R > slice) {
            const size_t el = a.dtype == QGEMV_BF16 ? 2 : 4;
            for (int r = 0; r < args.R; r += slice) {
                a.T = a.R = args.R - r < slice ? args.R - r : slice;
                a.x = static_cast<const char *>(args.x) + (size_t)r * a.ldx * el;
                a.y = static_cast<char *>(args.y) + (size_t)r * a.ldy * el;
                if (args.residual)
                    a.residual = static_cast<const char *>(args.residual) + (size_t)r * a.ldr * el;
                const hipError_t e = launch_linear(fmt, a, ws, st);
                if (e != hipSuccess) return e;
            }
            return hipSuccess;
        }
    }
    if (c.items > MAX_ITEMS) return hipErrorInvalidValue;
    const bool fits = c.fits;
    const int stream = c.stream, bm = c.bm;
    const Shape shape = c.shape;
    const long long mt = c.mt;
    RowTile *tiles = nullptr;
    if (a.offsets) {
        tiles = static_cast<RowTile *>(ws);
        hipLaunchKernelGGL(plan_tiles, dim3(1), dim3(1024), 0, st, a.offsets, a.E, a.R, bm, tiles,
                           (int)mt);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        ws = static_cast<char *>(ws) + align256((size_t)max_tiles(a.R, a.E, 16) * sizeof(RowTile));
    }
    if (stream) return launch_stream(fmt, a, stream, tiles, (int)mt, st);
    if (fits) return launch_tile(fmt, a, c.narrow, bm, tiles, (int)mt, ws, st);
    const int bn = shape == THIN ? GN_THIN : GN;
    const long long grid = mt * ((oc + bn - 1) / bn);
    if (fmt == FMT_I4G) {
        if (a.dtype == QGEMV_BF16) run_general<FMT_I4G, BF16>(a, shape, tiles, (unsigned)grid, st);
        else run_general<FMT_I4G, F32>(a, shape, tiles, (unsigned)grid, st);
    } else {
        if (a.dtype == QGEMV_BF16) run_general<FMT_FP8, BF16>(a, shape, tiles, (unsigned)grid, st);
        else run_general<FMT_FP8, F32>(a, shape, tiles, (unsigned)grid, st);
    }
    return hipGetLastError();
}

}  // namespace qg
