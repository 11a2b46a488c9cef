// matmul_tile_small.hip -- the tile kernel of 8-bit products: bfloat16, 128 or 64 rows.
#include "matmul_tile.h"

namespace qg {

hipError_t run_tile_small(const TileParams &p, int kind, unsigned grid, hipStream_t st)
{
    return kind == 2 ? run_tile<BF16, 8, 2, 2, 4, false, true, true>(p, grid, st)
                     : run_tile<BF16, 8, 1, 2, 4, false, true, false>(p, grid, st);
}

}  // namespace qg
