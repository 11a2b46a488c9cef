// qg_matmul.h -- launchers of the products whose both operands are e4m3, of
// the quantizer that makes their activations, and of the gradients of routed
// rows.
#pragma once

#include "qg_linear.h"
#include "qg_matmul_plan.h"

namespace qg {

// One product Y = epilogue(X . W^T): a.x holds e4m3 codes [T][a.ldx] (bytes),
// a.dtype is the type of y, bias and residual, a.ng the scales of a row.
struct MatmulArgs {
    LinearArgs a;
    const float *xs;                     // [T][ldxs], a scale per 128 columns
    long long ldxs;
};

inline MatmulSizes sizes_of(const MatmulArgs &p)
{
    const LinearArgs &a = p.a;
    return {a.R, a.offsets ? a.E : 0, a.I, a.O, a.dtype == QGEMV_BF16, a.gated != 0};
}

// One row tile of a grouped product: rows [row0, row0 + n) of y, of one expert,
// whose `count` tiles start at tile `first` of the list.  The list is in the order
// of the experts; its first `filled` tiles hold rows (n > 0).
struct ExpertTile {
    int expert, row0, n, first, count, filled, pad[2];
};

// Workspace bytes: of a dense product (by these sizes and the device's CUs; not
// monotone in S), and of a grouped one (by its sizes only).
size_t matmul_workspace(int S, int I, int O, int dtype, int gated);
size_t matmul_grouped_workspace(int R, int E);
bool matmul_launchable(const MatmulArgs &p);
hipError_t launch_matmul(const MatmulArgs &p, void *ws, hipStream_t st);

// The stream kernel (matmul_stream.hip): row tiles of 16, 32 or 64.
long long matmul_stream_items(const MatmulArgs &p, int bm, long long ntm);
hipError_t launch_matmul_stream(const MatmulArgs &p, int bm, const ExpertTile *tiles, int ntm,
                                hipStream_t st);

// The tile kernel (matmul_tile.hip): whether it takes a product, and by
// memory-to-LDS loads; the bytes of the parts' sums, the work items of the larger
// launch of a plan.
bool matmul_tile_fits(const MatmulArgs &p);
bool matmul_tile_direct(const MatmulArgs &p);
size_t matmul_part_bytes(const MatmulArgs &p, int parts);
long long matmul_tile_items(const MatmulArgs &p, const TilePlan &plan, long long ntm);
hipError_t launch_matmul_tile(const MatmulArgs &p, const TilePlan &plan, const ExpertTile *tiles,
                              int ntm, void *ws, hipStream_t st);

hipError_t launch_fp8_quantize(const void *x, long long ldx, int S, int I, int dtype,
                               uint8_t *codes, long long ldc, float *scales, long long lds,
                               hipStream_t st);

hipError_t launch_moe_dispatch(const void *x, long long ldx, int T, const int32_t *tokens, int R,
                               int I, void *y, long long ldy, int dtype, hipStream_t st);
hipError_t launch_moe_dispatch_grad(const void *dy, long long lddy, int R, const int32_t *pos,
                                    int T, int K, int I, void *dx, long long lddx, int dtype,
                                    hipStream_t st);
hipError_t launch_moe_combine_grad(const void *dy, long long lddy, const void *h, long long ldh,
                                   int R, const int32_t *tokens, const int32_t *pos,
                                   const float *gates, int T, int K, int O, void *dh,
                                   long long lddh, float *dgates, int dtype, hipStream_t st);

}  // namespace qg
