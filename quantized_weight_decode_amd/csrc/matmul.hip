// matmul.hip -- products whose both operands are e4m3, dense or grouped by
// expert: the choice among kernels, and slices of rows.
#include "qg_launch.h"
#include "qg_matmul.h"

namespace qg {

namespace {

// The kernel of a product, its row tiles and its launch's work items.
struct Choice {
    bool tile;
    int bm;
    long long mt, items;
};

Choice choose(const MatmulArgs &p)
{
    Choice c{};
    const LinearArgs &a = p.a;
    const int rows = a.offsets ? (a.R + a.E - 1) / a.E : a.R;
    c.tile = rows > 64 && matmul_tile_fits(p);
    c.bm = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
    if (c.tile) c.bm = 128;
    c.mt = a.offsets ? max_tiles(a.R, a.E, c.bm) : (a.R + c.bm - 1) / c.bm;
    c.items = c.tile ? matmul_tile_items(p, c.bm, c.mt) : matmul_stream_items(p, c.bm, c.mt);
    return c;
}

hipError_t run(const MatmulArgs &p, const Choice &c, const RowTile *tiles, hipStream_t st)
{
    return c.tile ? launch_matmul_tile(p, c.bm, tiles, (int)c.mt, st)
                  : launch_matmul_stream(p, c.bm, tiles, (int)c.mt, st);
}

}  // namespace

size_t matmul_workspace(int R, int E)
{
    return align256((size_t)max_tiles(R, E, 16) * sizeof(RowTile));
}

bool matmul_launchable(const MatmulArgs &p)
{
    return !p.a.offsets || choose(p).items <= MAX_ITEMS;
}

hipError_t launch_matmul(const MatmulArgs &args, void *ws, hipStream_t st)
{
    MatmulArgs p = args;
    LinearArgs &a = p.a;
    if (a.offsets) {
        const Choice c = choose(p);
        if (c.items > MAX_ITEMS) return hipErrorInvalidValue;
        RowTile *const tiles = static_cast<RowTile *>(ws);
        const hipError_t e = launch_plan_tiles(a.offsets, a.E, a.R, c.bm, tiles, (int)c.mt, st);
        if (e != hipSuccess) return e;
        return run(p, c, tiles, st);
    }
    // slices of rows whose work items fit a launch (64 rows of 2^24 outputs do)
    int slice = args.a.R;
    for (;; slice = (slice / 2 + 63) / 64 * 64) {
        a.T = a.R = slice;
        if (slice <= 64 || choose(p).items <= MAX_ITEMS) break;
    }
    const size_t el = a.dtype == QGEMV_BF16 ? 2 : 4;
    for (int r = 0; r < args.a.R; r += slice) {
        a.T = a.R = args.a.R - r < slice ? args.a.R - r : slice;
        a.x = static_cast<const uint8_t *>(args.a.x) + r * a.ldx;
        p.xs = args.xs + r * p.ldxs;
        a.y = static_cast<char *>(args.a.y) + (long long)(r * a.ldy * el);
        if (a.residual)
            a.residual = static_cast<const char *>(args.a.residual) + (long long)(r * a.ldr * el);
        const Choice c = choose(p);
        if (c.items > MAX_ITEMS) return hipErrorInvalidValue;
        const hipError_t e = run(p, c, nullptr, st);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace qg
