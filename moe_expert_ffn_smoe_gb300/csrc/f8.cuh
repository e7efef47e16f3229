// What the kernels of the 8-bit floating-point product share.
#pragma once

#include "q8.cuh"

namespace smoe {

constexpr int F8_BLOCK = 128;  // columns (and weight rows) of one scale

// The arguments of one product (launch_f8), passed on to its kernels.
struct F8Call {
    const uint8_t *xq;
    const float *xs;
    int nsrc;
    const int *order;
    int k;
    const int *offsets;
    int R, n;
    const uint8_t *wq;
    const float *ws;
    int N, K;
    void *y;
    int dtype;
};

// The product on the tensor cores (f8_tc.cu).
size_t f8_tc_workspace(int R, int n);
cudaError_t launch_f8_tc(const F8Call &c, void *workspace, cudaStream_t stream);

// The same by pairs of CTAs in row tiles of 256 (f8_pair.cu), from the tile list.
cudaError_t launch_f8_pair(const F8Call &c, const int *ntiles, const Tile *tiles, int max_tiles, cudaStream_t stream);

}  // namespace smoe
