// What the 8-bit product's kernels share: tiles of one expert's rows, the
// source row of a sorted row, and the stores of the two output types.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"
#include "internal_tokens.h"

namespace smoe {

// At most `rows` consecutive sorted rows of one expert (-1: rows of none).
struct Tile {
    int expert, row0, rows, pad;
};

// Source row of sorted row r (order null: itself), or -1, reported, where
// order points outside the nsrc rows.
__device__ __forceinline__ int source_row(const int *order, int k, int nsrc, int r, unsigned *status)
{
    if (!order) return r;
    const int s = order[r];
    if (s < 0 || s / k >= nsrc) {
        atomicExch(status, kStatusRoute);
        return -1;
    }
    return s / k;
}

__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// Two neighbouring elements, the first at an even index of an aligned row.
__device__ __forceinline__ void put2(float *p, float a, float b) { *reinterpret_cast<float2 *>(p) = make_float2(a, b); }
__device__ __forceinline__ void put2(__nv_bfloat16 *p, float a, float b)
{
    *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(a, b);
}

inline size_t up256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

// Most tiles of up to `step` rows that R rows of n experts (and the rows of
// none) give: every expert that has rows leaves at most one short tile.
inline int most_tiles(int R, int n, int step) { return R / step + (n + 1 < R ? n + 1 : R); }

// The arguments of one product (launch_q8), passed on to its kernels.
struct Q8Call {
    const int8_t *xq;
    const float *xs;
    int nsrc;
    const int *order;
    int k;
    const int *offsets;
    int R, n;
    const int8_t *wq;
    const float *ws;
    int N, K;
    void *y;
    int dtype;
};

// The product on the tensor cores (q8_tc.cu).
size_t q8_tc_workspace(int nsrc, int R, int n, int K);
cudaError_t launch_q8_tc(const Q8Call &c, void *workspace, cudaStream_t stream);

}  // namespace smoe
