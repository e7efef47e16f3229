// What the kernels of the 8-bit floating-point product share.
#pragma once

#include "q8.cuh"

namespace smoe {

constexpr int F8_BLOCK = 128;  // columns (and weight rows) of one scale

// The product in row tiles of 128 (f8_rows.cu), from the tile list.
cudaError_t launch_f8_rows(const F8Call &c, const int *ntiles, const Tile *tiles, int max_tiles, cudaStream_t stream);

}  // namespace smoe
