// matmul_tile_large.hip -- the tile kernel of 8-bit products: bfloat16, 256 or 192 rows.
#include "matmul_tile.h"

namespace qg {

hipError_t run_tile_large(const TileParams &p, int kind, unsigned grid, hipStream_t st)
{
    return kind == 0 ? run_tile<BF16, 8, 4, 2, 4, false, true, true>(p, grid, st)
                     : run_tile<BF16, 8, 3, 2, 4, false, true, false>(p, grid, st);
}

}  // namespace qg
