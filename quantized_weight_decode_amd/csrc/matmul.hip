// matmul.hip -- products whose both operands are e4m3, dense or grouped by
// expert: the choice among kernels, and slices of rows.
#include "qg_launch.h"
#include "qg_matmul.h"

namespace qg {

namespace {

// Row tiles of a grouped product, from the experts' offsets on the device: each
// expert's rows in blocks of bm, experts in ascending order; the rest of the list
// is empty.  Offsets are clamped to 0..R and a negative count counts as none, so
// that every tile lies within y.  One workgroup, a thread per expert; 5 us, latency.
__global__ __launch_bounds__(1024) void plan_experts(const int32_t *__restrict__ offsets, int E,
                                                     int R, int bm,
                                                     ExpertTile *__restrict__ tiles, int ntiles)
{
    __shared__ int base[1025];           // first tile of each expert
    __shared__ int start[1024], rows[1024];
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
    start[tid] = lo;
    rows[tid] = n;
    __syncthreads();
    // overlapping offsets (not allowed) could name more tiles than the list
    // holds; sums of up to 1024 counts of 2^24 / 16 tiles stay below 2^31
    for (int w = 0; w < wave; w++) incl += wsum[w];
    base[tid + 1] = incl;
    if (tid == 0) base[0] = 0;
    __syncthreads();
    const int filled = min(base[1024], ntiles);
    for (int i = tid; i < ntiles; i += 1024) {
        ExpertTile t{};
        t.filled = filled;
        if (i < filled) {
            int a = 0, b = 1024;                         // base[a] <= i < base[b]
            while (b - a > 1) {
                const int c = (a + b) / 2;
                if (base[c] <= i) a = c;
                else b = c;
            }
            t.expert = a;
            t.first = base[a];
            t.count = min(base[a + 1], ntiles) - base[a];
            t.row0 = start[a] + (i - base[a]) * bm;
            t.n = min(rows[a] - (i - base[a]) * bm, bm);
        }
        tiles[i] = t;
    }
}

// tiles that R rows of E experts can need
long long most_tiles(int R, int E, int bm)
{
    return (long long)R / bm + (E < R ? E : R);
}

// The kernel of a product, its row tiles and its launch's work items.
struct Choice : MatmulPlan {
    long long mt, items;
};

Choice choose(const MatmulArgs &p, bool fits, bool direct)
{
    const LinearArgs &a = p.a;
    Choice c{plan_matmul(sizes_of(p), fits, direct, cu_count()), 0, 0};
    c.mt = a.offsets ? most_tiles(a.R, a.E, c.bm) : (a.R + c.bm - 1) / c.bm;
    c.items = c.tile ? matmul_tile_items(p, c.plan, c.mt)
                     : matmul_stream_items(p, c.bm, c.mt);
    return c;
}

Choice choose(const MatmulArgs &p)
{
    return choose(p, matmul_tile_fits(p), matmul_tile_direct(p));
}

hipError_t run(const MatmulArgs &p, const Choice &c, const ExpertTile *tiles, void *ws,
               hipStream_t st)
{
    return c.tile ? launch_matmul_tile(p, c.plan, tiles, (int)c.mt, ws, st)
                  : launch_matmul_stream(p, c.bm, tiles, (int)c.mt, st);
}

}  // namespace

size_t matmul_workspace(int S, int I, int O, int dtype, int gated)
{
    MatmulArgs p{};
    p.a.T = p.a.R = S;
    p.a.E = 1;
    p.a.I = I;
    p.a.O = O;
    p.a.ng = (I + 127) / 128;
    p.a.dtype = dtype;
    p.a.gated = gated;
    size_t most = 0;
    for (int direct = 0; direct < 2; direct++) {
        const size_t n = matmul_part_bytes(p, choose(p, true, direct).plan.parts);
        most = n > most ? n : most;
    }
    return align256(most);
}

size_t matmul_grouped_workspace(int R, int E)
{
    return align256((size_t)most_tiles(R, E, 16) * sizeof(ExpertTile));
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
        ExpertTile *const tiles = static_cast<ExpertTile *>(ws);
        hipLaunchKernelGGL(plan_experts, dim3(1), dim3(1024), 0, st, a.offsets, a.E, a.R, c.bm,
                           tiles, (int)c.mt);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        return run(p, c, tiles, nullptr, st);
    }
    // slices of rows whose work items fit a launch (64 rows of 2^24 outputs do)
    int slice = args.a.R;
    Choice c;
    for (;; slice = (slice / 2 + 63) / 64 * 64) {
        a.T = a.R = slice;
        c = choose(p);
        if (slice <= 64 || c.items <= MAX_ITEMS) break;
    }
    if (slice == args.a.R)
        return c.items > MAX_ITEMS ? hipErrorInvalidValue : run(p, c, nullptr, ws, st);
    const size_t el = a.dtype == QGEMV_BF16 ? 2 : 4;
    for (int r = 0; r < args.a.R; r += slice) {
        a.T = a.R = args.a.R - r < slice ? args.a.R - r : slice;
        a.x = static_cast<const uint8_t *>(args.a.x) + r * a.ldx;
        p.xs = args.xs + r * p.ldxs;
        a.y = static_cast<char *>(args.a.y) + (long long)(r * a.ldy * el);
        if (args.a.residual)
            a.residual =
                static_cast<const char *>(args.a.residual) + (long long)(r * a.ldr * el);
        c = choose(p);
        if (c.plan.parts > 1) {                          // (the workspace is that of all rows)
            c.plan.parts = 1;
            c.items = matmul_tile_items(p, c.plan, c.mt);
        }
        if (c.items > MAX_ITEMS) return hipErrorInvalidValue;
        const hipError_t e = run(p, c, nullptr, ws, st);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace qg
