// matmul_tile.hip -- the tile kernel of 8-bit products (matmul_tile.h): its launches by
// a plan (qg_matmul_plan.h), and the parts of K joined.
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

size_t matmul_part_bytes(const MatmulArgs &p, int parts)
{
    const int oc = p.a.gated ? p.a.O / 2 : p.a.O;
    return parts > 1 ? (size_t)parts * (p.a.gated ? 2 : 1) * p.a.R * ((oc + 3) / 4 * 4) * 4 : 0;
}

// Workgroups of a launch of n columns, and tiles across them.  Grouped: any number of
// tiles up to ntm may hold rows, and they are dealt to the XCDs in runs of up to 32.
static long long tile_grid(const MatmulArgs &p, int kind, int parts, int n, long long ntm, int &ntn)
{
    const int cols = TILE_KINDS[kind].bw / (p.a.gated ? 2 : 1);
    ntn = (n + cols - 1) / cols;
    return p.a.offsets ? (ntm * ntn / 8 + 32) * 8 : ntm * ntn * parts;
}

static long long row_tiles(const MatmulArgs &p, int kind)
{
    return (p.a.R + TILE_KINDS[kind].bt - 1) / TILE_KINDS[kind].bt;
}

long long matmul_tile_items(const MatmulArgs &p, const TilePlan &plan, long long ntm)
{
    const int oc = p.a.gated ? p.a.O / 2 : p.a.O;
    int ntn;
    const long long n = tile_grid(p, plan.kind, plan.parts, oc - plan.head, ntm, ntn) *
                        TILE_KINDS[plan.kind].waves * 64;
    if (!plan.head) return n;
    const long long m =
        tile_grid(p, plan.head_kind, 1, plan.head, row_tiles(p, plan.head_kind), ntn) *
        TILE_KINDS[plan.head_kind].waves * 64;
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
    p.per = parts > 1 ? steps_per_part(a.ng, parts) : a.ng;
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
