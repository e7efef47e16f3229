// What the kernels of the 8-bit floating-point product share.
#pragma once

#include "q8.cuh"

namespace smoe {

constexpr int F8_BLOCK = 128;  // columns (and weight rows) of one scale

// The product by pairs of CTAs in row tiles of 256 (f8_pair.cu), from the tile list.
cudaError_t launch_f8_pair(const F8Call &c, const int *ntiles, const Tile *tiles, int max_tiles, cudaStream_t stream);

}  // namespace smoe
