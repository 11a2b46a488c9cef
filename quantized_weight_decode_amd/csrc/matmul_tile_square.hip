// matmul_tile_square.hip -- the tile kernel of 8-bit products: bfloat16, 128 x 128.
#include "matmul_tile.h"

namespace qg {

hipError_t run_tile_square(const TileParams &p, bool direct, unsigned grid, hipStream_t st)
{
    return direct ? run_tile<BF16, 4, 4, 2, 2, false, true, false>(p, grid, st)
                  : run_tile<BF16, 4, 4, 2, 2, false, false, true>(p, grid, st);
}

}  // namespace qg
