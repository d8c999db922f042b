// row_tiles.h -- counting the row tiles of ragged groups (device code that the host can check).
#pragma once

namespace mi355gemm {

// Row tiles are counted on the device, some groups at a time, up to `most`, what the
// launch holds for ascending offsets.  Offsets that descend and rise again hold rows more
// than once: their count, times the column tiles, could leave 32 bits and with them the
// ranges of tile_coords.
__host__ __device__ inline int add_row_tiles(int total, unsigned more, int most)
{
    return more >= (unsigned)(most - total) ? most : total + (int)more;
}

}  // namespace mi355gemm
