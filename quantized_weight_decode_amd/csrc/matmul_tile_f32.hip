// matmul_tile_f32.hip -- the tile kernel of 8-bit products: f32 results.
#include "matmul_tile.h"

namespace qg {

hipError_t run_tile_f32(const TileParams &p, bool direct, unsigned grid, hipStream_t st)
{
    return direct ? run_tile<F32, 4, 4, 2, 2, true, true, true>(p, grid, st)
                  : run_tile<F32, 4, 4, 2, 2, true, false, true>(p, grid, st);
}

}  // namespace qg
