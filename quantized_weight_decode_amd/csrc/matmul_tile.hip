// matmul_tile.hip -- the tile kernel of 8-bit products (matmul_tile.h): which kind of
// tile and how many parts of K a product takes, the launch, and the parts joined.
#include "matmul_tile.h"

namespace qg {

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

namespace {

struct Kind {
    int bt, bw, waves;                   // rows of x, rows of W, waves
    double step, fixed;                  // us per K step and per tile
};
const Kind KINDS[] = {{256, 256, 8, 1.5, 14.0},
                      {192, 256, 8, 1.27, 13.0},
                      {128, 256, 8, 0.97, 12.0},
                      {64, 256, 8, 0.64, 10.0},
                      {128, 128, 4, 1.0, 10.0}};
constexpr int SQUARE = 4;                // the only one for f32, or rows that are not on 16 bytes

// The sums of K's parts joined, in their order, and the ends: a thread has four
// outputs of a row in flight.
template <typename XT, bool GATED>
__global__ __launch_bounds__(256) void join_parts(TileParams p)
{
    const LinearArgs &a = p.m.a;
    const int row_ = blockIdx.y, c0 = p.col0 + blockIdx.x * 1024;
    const long long plane = (long long)a.R * p.ldp;
    const float *const at = p.partial + (long long)row_ * p.ldp;
    auto sums = [&](int i, int &row, int &col, float &v, float &up) {
        row = row_;
        col = c0 + i;
        v = up = 0.0f;
        if (col >= p.ldp) return;
#pragma unroll 4
        for (int k = 0; k < p.parts; k++) {
            v += at[k * (GATED ? 2 : 1) * plane + col];
            if (GATED) up += at[(2 * k + 1) * plane + col];
        }
    };
    finish<XT, 4>(a, 0, threadIdx.x, 256, 1024, sums);
}

}  // namespace

int matmul_tile_rows(int kind) { return KINDS[kind].bt; }

size_t matmul_part_bytes(const MatmulArgs &p, int parts)
{
    const int oc = p.a.gated ? p.a.O / 2 : p.a.O;
    return parts > 1 ? (size_t)parts * (p.a.gated ? 2 : 1) * p.a.R * ((oc + 3) / 4 * 4) * 4 : 0;
}

// Tiles of n columns of y by R rows, and the time of `parts` parts of each, one
// workgroup (of the square kind two) per CU at a time; joining parts costs a launch
// and their sums' way to memory and back.
static long long tiles_of(const MatmulArgs &p, int kind, int n)
{
    const Kind &k = KINDS[kind];
    const int cols = k.bw / (p.a.gated ? 2 : 1);
    return (long long)((p.a.R + k.bt - 1) / k.bt) * ((n + cols - 1) / cols);
}

// The plan of n columns in one launch: the kind, and the parts of K where tiles leave
// CUs without work, for which the busiest CU ends first (1501 x 16384 x 7168, 168
// tiles: 236 us, in three parts 259).
static TilePlan plan_columns(const MatmulArgs &p, bool any, int n, long long ncu)
{
    const LinearArgs &a = p.a;
    TilePlan best{};
    best.us = -1.0;
    for (int i = any ? 0 : SQUARE; i <= SQUARE; i++) {
        const Kind &k = KINDS[i];
        const long long tiles = tiles_of(p, i, n), slots = i == SQUARE ? 2 * ncu : ncu;
        const double c = a.dtype == QGEMV_F32 ? 2 * k.step : k.step;
        for (const int f : {1, 2, 3, 4, 6, 8, 12, 16}) {
            if (f > 1 && (tiles * f > slots || a.R > 4096)) break;
            const int per = ((a.ng + f - 1) / f + SG - 1) / SG * SG;
            if ((a.ng + per - 1) / per != f) continue;
            double us = (double)((tiles * f + slots - 1) / slots) *
                        ((f > 1 ? per : a.ng) * c + k.fixed);
            if (f > 1) us += 5.0 + 8e-6 * f * a.R * (double)a.O / 5.0;
            if (best.us < 0.0 || us < best.us) best = TilePlan{i, f, 0, 0, us};
        }
    }
    return best;
}

// Dense: the faster of one launch and of two, the first with as many columns as give
// every CU the same number of one kind's tiles, the second with the rest, by what suits
// that.  us: 2048 x 6144 x 12288, 384 tiles of 256 x 256 at once 157 (gated 170), 256 of
// them and the rest in tiles of 128 x 256 152 (160).
// Grouped by expert 128 x 256, whose three stages suit experts of few rows, bound by
// their weights' bytes, up to 512 rows per expert.
TilePlan matmul_tile_plan(const MatmulArgs &p, bool direct)
{
    const LinearArgs &a = p.a;
    const bool any = a.dtype == QGEMV_BF16 && direct;
    if (a.offsets) return TilePlan{!any ? SQUARE : a.R / a.E < 512 ? 2 : 0, 1, 0, 0, 0.0};
    const int oc = a.gated ? a.O / 2 : a.O;
    const long long ncu = cu_count();
    TilePlan best = plan_columns(p, any, oc, ncu);
    for (int i = 0; any && i < SQUARE; i++) {
        const Kind &k = KINDS[i];
        const int cols = k.bw / (a.gated ? 2 : 1);
        const long long ntm = (a.R + k.bt - 1) / k.bt, rounds = tiles_of(p, i, oc) / ncu;
        const long long head = rounds * ncu / ntm * cols;
        if (rounds < 1 || head < cols || head >= oc) continue;
        const double us = rounds * (a.ng * k.step + k.fixed) + 7.0;
        if (us >= best.us) continue;
        TilePlan rest = plan_columns(p, any, oc - (int)head, ncu);
        rest.us += us;
        rest.head = (int)head;
        rest.head_kind = i;
        if (rest.us < best.us) best = rest;
    }
    return best;
}

// Workgroups of a launch of n columns, and tiles across them.  Grouped: any number of
// tiles up to ntm may hold rows, and they are dealt to the XCDs in runs of up to 32.
static long long tile_grid(const MatmulArgs &p, int kind, int parts, int n, long long ntm, int &ntn)
{
    const int cols = KINDS[kind].bw / (p.a.gated ? 2 : 1);
    ntn = (n + cols - 1) / cols;
    return p.a.offsets ? (ntm * ntn / 8 + 32) * 8 : ntm * ntn * parts;
}

static long long row_tiles(const MatmulArgs &p, int kind)
{
    return (p.a.R + KINDS[kind].bt - 1) / KINDS[kind].bt;
}

long long matmul_tile_items(const MatmulArgs &p, const TilePlan &plan, long long ntm)
{
    const int oc = p.a.gated ? p.a.O / 2 : p.a.O;
    int ntn;
    const long long n = tile_grid(p, plan.kind, plan.parts, oc - plan.head, ntm, ntn) *
                        KINDS[plan.kind].waves * 64;
    if (!plan.head) return n;
    const long long m =
        tile_grid(p, plan.head_kind, 1, plan.head, row_tiles(p, plan.head_kind), ntn) *
        KINDS[plan.head_kind].waves * 64;
    return n > m ? n : m;
}

// Columns col0 .. col0 + n - 1 of y.
static hipError_t launch_columns(const MatmulArgs &m, int kind, int parts, int col0, int n,
                                 const ExpertTile *tiles, int ntm, void *ws, hipStream_t st)
{
    TileParams p{};
    p.m = m;
    p.tiles = tiles;
    p.ntm = ntm;
    p.col0 = col0;
    const LinearArgs &a = m.a;
    const unsigned grid = (unsigned)tile_grid(m, kind, parts, n, ntm, p.ntn);
    const int oc = a.gated ? a.O / 2 : a.O;
    p.parts = parts;
    p.per = parts > 1 ? ((a.ng + parts - 1) / parts + SG - 1) / SG * SG : a.ng;
    // every part has steps, and a place for its sums
    if ((parts - 1) * (long long)p.per >= a.ng || (parts > 1 && !ws)) return hipErrorInvalidValue;
    p.partial = static_cast<float *>(ws);
    p.ldp = (oc + 3) / 4 * 4;
    const uintptr_t el = a.dtype == QGEMV_BF16 ? 2 : 4;
    p.wide = oc % 8 == 0 && (((uintptr_t)a.y | (uintptr_t)a.residual | (uintptr_t)a.bias |
                              (uintptr_t)a.ldy * el | (uintptr_t)a.ldr * el) & 15) == 0;
    hipError_t e;
    if (a.dtype == QGEMV_F32) e = run_tile_f32(p, matmul_tile_direct(m), grid, st);
    else if (kind == SQUARE) e = run_tile_square(p, matmul_tile_direct(m), grid, st);
    else e = kind < 2 ? run_tile_large(p, kind, grid, st) : run_tile_small(p, kind, grid, st);
    if (e != hipSuccess || parts == 1) return e;
    const dim3 join((n + 1023) / 1024, a.R);
    if (a.dtype == QGEMV_F32) {
        if (a.gated) hipLaunchKernelGGL((join_parts<F32, true>), join, dim3(256), 0, st, p);
        else hipLaunchKernelGGL((join_parts<F32, false>), join, dim3(256), 0, st, p);
    } else {
        if (a.gated) hipLaunchKernelGGL((join_parts<BF16, true>), join, dim3(256), 0, st, p);
        else hipLaunchKernelGGL((join_parts<BF16, false>), join, dim3(256), 0, st, p);
    }
    return hipGetLastError();
}

hipError_t launch_matmul_tile(const MatmulArgs &p, const TilePlan &plan, const ExpertTile *tiles,
                              int ntm, void *ws, hipStream_t st)
{
    const int oc = p.a.gated ? p.a.O / 2 : p.a.O;
    if (plan.head) {
        const hipError_t e = launch_columns(p, plan.head_kind, 1, 0, plan.head, nullptr,
                                            (int)row_tiles(p, plan.head_kind), nullptr, st);
        if (e != hipSuccess) return e;
    }
    return launch_columns(p, plan.kind, plan.parts, plan.head, oc - plan.head, tiles, ntm, ws, st);
}

}  // namespace qg
