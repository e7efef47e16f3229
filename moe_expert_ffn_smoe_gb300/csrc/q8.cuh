// What the kernels of the 8-bit products and quantisers share: tiles of one
// expert's rows, the source row of a sorted row, the stores of the two output
// types, SiLU.
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

// The tile list of a sorted batch, by one CTA of THREADS: every expert's rows cut
// into equal tiles of at most nt rows, multiples of `unit` but for the last.
template <int THREADS>
__device__ __forceinline__ void list_tiles(const int *offsets, int n, int R, int nt, int unit, int max_tiles, int *ntiles,
                                           Tile *tiles, unsigned *status)
{
    __shared__ long long warp_sums[THREADS / 32];
    __shared__ long long run_s;
    const int tid = threadIdx.x;
    const int lane = tid & 31, wi = tid >> 5;
    long long run = 0;  // 64 bits: ranges that overlap (reported) can add up to more than 32
    for (int b = 0; b < n; b += THREADS) {
        const int e = b + tid;
        int lo = 0, hi = 0;
        if (e < n) {
            lo = offsets[e];
            hi = offsets[e + 1];
            if (lo < 0 || hi < lo || hi > R) {
                atomicExch(status, kStatusRoute);
                lo = hi = 0;
            }
        }
        int cnt = (hi - lo + nt - 1) / nt;
        const int step = cnt > 0 ? ((hi - lo + cnt - 1) / cnt + unit - 1) / unit * unit : unit;
        cnt = (hi - lo + step - 1) / step;
        long long inc = cnt;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long o = __shfl_up_sync(FULL_MASK, inc, off);
            if (lane >= off) inc += o;
        }
        if (lane == 31) warp_sums[wi] = inc;
        __syncthreads();
        long long before = run;
        for (int i = 0; i < wi; ++i) before += warp_sums[i];
        if (tid == THREADS - 1) run_s = before + inc;
        const long long t0 = before + inc - cnt;
        for (int i = 0; i < cnt && t0 + i < max_tiles; ++i)
            tiles[t0 + i] = Tile{e, lo + i * step, min(step, hi - lo - i * step), 0};
        __syncthreads();
        run = run_s;
    }
    if (tid == 0) *ntiles = static_cast<int>(min(run, static_cast<long long>(max_tiles)));
}

__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// Two neighbouring elements, the first at an even index of an aligned row.
__device__ __forceinline__ void put2(float *p, float a, float b) { *reinterpret_cast<float2 *>(p) = make_float2(a, b); }
__device__ __forceinline__ void put2(__nv_bfloat16 *p, float a, float b)
{
    *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(a, b);
}

// SiLU, v / (1 + e^-v), as max(v, 0) - |v| e / (1 + e) with e = e^-|v|: e itself
// is never beyond what f32 holds, where SiLU(v) times a large factor may still
// be its row's largest value, and the divisor stays within [1, 2], so that the
// reciprocal instruction alone does (1 unit in the last place; the quantiser is
// bound by instructions, and its step is 2^16 times coarser).  32,768 rows of
// 1536 bf16 52.5 us, as a division of v or v e by 1 + e 60.8.
__device__ __forceinline__ float silu_row(float v)
{
    const float e = expf(-fabsf(v));
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return fmaf(-fabsf(v), e * r, fmaxf(v, 0.f));
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
