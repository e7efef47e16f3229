// 8-bit floating-point (e4m3) rows and weights with a scale for each block of 128:
//   y[r][n] = sum_b xs[src(r)][b] ws[e][n / 128][b] sum_{c in b} xq[src(r)][c] wq[e][n][c]
// over one matrix, or over the experts of a sorted batch.  Here: the products of a
// few rows on the CUDA cores, and the choice of the form.
#include <cuda_fp16.h>

#include "f8.cuh"
#include "smoe.h"

namespace smoe {
namespace {

constexpr int DOT_WARPS = 8;
constexpr int DOT_ROWS = 4;  // activation rows per tile
constexpr int DOT_OUTS = 4;  // weight rows per warp

struct DotArgs {
    const uint8_t *xq;
    const float *xs;
    const int *order, *offsets;  // order null: row r is its own source; offsets null: one matrix
    const uint8_t *wq;
    const float *ws;
    void *y;
    unsigned *status;
    int k, nsrc, N, K, R, n, kb, nb;
};

// Eight e4m3 codes as f32 (every code is an f16 number).
__device__ __forceinline__ void widen8(uint32_t a, uint32_t b, float (&v)[8])
{
    const uint32_t w[2] = {a, b};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)))));
        const float2 f = __half22float2(*reinterpret_cast<__half2 *>(&h));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

// f32 dot products on the CUDA cores: a warp holds four weight rows against up to
// four rows of one expert, 16 columns of each per lane and step (one scale: 16
// divides 128).  A warp walks its groups of four rows as one sequence of steps, the
// weights of the next DEPTH steps in flight across the groups' ends.  blockIdx.x is
// a row of the batch and, of an expert's rows, every DOT_ROWS-th one leads a tile
// (every thread looks at an expert's offsets), so that no list of tiles has to be
// made first.  Bound by streaming the weights: a step is 512 bytes of each of
// four rows and about 200 instructions for one row of activations.
template <typename T>
__global__ void __launch_bounds__(DOT_WARPS * 32, 2) f8_dot(const DotArgs a)
{
    constexpr int DEPTH = 3;
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    int n0 = (blockIdx.y * DOT_WARPS + (threadIdx.x >> 5)) * DOT_OUTS;  // the group being summed
    const int stride = gridDim.y * DOT_WARPS * DOT_OUTS;
    // a prefetch only: the previous kernel may be the one that quantises these weights
    if (!a.offsets && lane < DOT_OUTS && n0 + lane < a.N && a.K > 0)
        prefetch_l2(a.wq + static_cast<size_t>(n0 + lane) * a.K, static_cast<uint32_t>(a.K));
    pdl_wait();
    int expert = 0, row0 = blockIdx.x, rows = 0;
    T *y = static_cast<T *>(a.y);
    if (a.offsets) {
        __shared__ int found[3];
        if (threadIdx.x == 0) found[0] = -1;
        __syncthreads();
        for (int e = threadIdx.x; e < a.n; e += DOT_WARPS * 32) {
            const int lo = a.offsets[e], hi = a.offsets[e + 1];
            if (lo <= row0 && row0 < hi) {  // one expert, unless the list is bad
                found[0] = e;
                found[1] = lo;
                found[2] = hi;
            }
            if (blockIdx.x == 0 && blockIdx.y == 0 && (lo < 0 || hi < lo || hi > a.R)) atomicExch(a.status, kStatusRoute);
        }
        __syncthreads();
        const int first = found[1], end = found[2];
        if (found[0] < 0) {
            if (row0 >= a.offsets[a.n])  // past the last expert's rows: zeros
                for (int i = (blockIdx.y * DOT_WARPS * 32) + threadIdx.x; i < a.N; i += gridDim.y * DOT_WARPS * 32)
                    put(y + static_cast<size_t>(row0) * a.N + i, 0.f);
            return;
        }
        expert = found[0];
        if ((static_cast<unsigned>(row0) - static_cast<unsigned>(first)) % DOT_ROWS) return;
        rows = min(min(end, a.R) - row0, DOT_ROWS);
    } else {
        row0 *= DOT_ROWS;
        rows = min(a.R - row0, DOT_ROWS);
    }
    const uint8_t *w = a.wq + static_cast<size_t>(expert) * a.N * a.K;
    const float *ws = a.ws + static_cast<size_t>(expert) * a.nb * a.kb;
    uint4 wv[DEPTH][DOT_OUTS];
    int fn = n0, fc = lane * 16;  // the next step to fetch
    auto fetch = [&](uint4 (&v)[DOT_OUTS]) {
#pragma unroll
        for (int o = 0; o < DOT_OUTS; ++o)
            v[o] = fn + o < a.N && fc < a.K ? ldg_stream(w + static_cast<size_t>(fn + o) * a.K + fc) : make_uint4(0u, 0u, 0u, 0u);
        fc += 512;
        if (fc - lane * 16 >= a.K) {
            fc = lane * 16;
            fn += stride;
        }
    };
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) fetch(wv[i]);
    int src[DOT_ROWS];
#pragma unroll
    for (int r = 0; r < DOT_ROWS; ++r)
        src[r] = r < rows ? source_row(a.order, a.k, a.nsrc, row0 + r, a.status) : -1;
    float acc[DOT_OUTS][DOT_ROWS];
#pragma unroll
    for (int o = 0; o < DOT_OUTS; ++o)
#pragma unroll
        for (int r = 0; r < DOT_ROWS; ++r) acc[o][r] = 0.f;
    int c = lane * 16;
    while (n0 < a.N) {
#pragma unroll
        for (int i = 0; i < DEPTH; ++i) {
            if (n0 >= a.N) break;
            if (c < a.K) {
                const int b = c >> 7;
                const float wscale = ws[static_cast<size_t>(n0 >> 7) * a.kb + b];  // four rows from a multiple of four: one block
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float wf[DOT_OUTS][8];
#pragma unroll
                    for (int o = 0; o < DOT_OUTS; ++o)
                        widen8(h ? wv[i][o].z : wv[i][o].x, h ? wv[i][o].w : wv[i][o].y, wf[o]);
#pragma unroll
                    for (int r = 0; r < DOT_ROWS; ++r) {
                        if (r >= rows) break;
                        if (src[r] < 0) continue;
                        const uint2 xv = *reinterpret_cast<const uint2 *>(a.xq + static_cast<size_t>(src[r]) * a.K + c + 8 * h);
                        const float f = a.xs[static_cast<size_t>(src[r]) * a.kb + b] * wscale;
                        float x[8];
                        widen8(xv.x, xv.y, x);
#pragma unroll
                        for (int o = 0; o < DOT_OUTS; ++o) {
                            float s = wf[o][0] * x[0];
#pragma unroll
                            for (int j = 1; j < 8; ++j) s = fmaf(wf[o][j], x[j], s);
                            acc[o][r] = fmaf(s, f, acc[o][r]);
                        }
                    }
                }
            }
            fetch(wv[i]);
            c += 512;
            if (c - lane * 16 >= a.K) {  // the group is summed
#pragma unroll
                for (int r = 0; r < DOT_ROWS; ++r) {
                    if (r >= rows) break;
#pragma unroll
                    for (int o = 0; o < DOT_OUTS; ++o) {
                        float sum = acc[o][r];
                        acc[o][r] = 0.f;
#pragma unroll
                        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(FULL_MASK, sum, off);
                        if (lane == o && n0 + o < a.N) put(y + static_cast<size_t>(row0 + r) * a.N + n0 + o, sum);
                    }
                }
                c = lane * 16;
                n0 += stride;
            }
        }
    }
}

}  // namespace

// Where the tensor cores take the product: from three rows on, and from more than
// three for every eight experts.
static bool on_tensor_cores(int R, int n, int K) { return K > 0 && R > 2 && R > 3LL * n / 8; }

size_t f8_workspace(int R, int n) { return f8_tc_workspace(R, n); }

cudaError_t launch_f8(const uint8_t *xq, const float *xs, int nsrc, const int *order, int k, const int *offsets, int R, int n,
                      const uint8_t *wq, const float *ws, int N, int K, void *y, int dtype, void *workspace,
                      cudaStream_t stream)
{
    if (on_tensor_cores(R, n, K))
        return launch_f8_tc(F8Call{xq, xs, nsrc, order, k, offsets, R, n, wq, ws, N, K, y, dtype}, workspace, stream);
    const DeviceInfo *dev = device_info();
    unsigned *status = device_status_word();
    if (!dev || !status) return cudaErrorInvalidDevice;
    const int kb = (K + F8_BLOCK - 1) / F8_BLOCK, nb = (N + F8_BLOCK - 1) / F8_BLOCK;
    const DotArgs a = {xq, xs, order, offsets, wq, ws, y, status, k, nsrc, N, K, R, n, kb, nb};
    // CTAs per tile: eight waves of the device (two CTAs an SM) when every row has
    // an expert of its own
    const int tiles = offsets ? R : (R + DOT_ROWS - 1) / DOT_ROWS;
    const int blocks = (N + DOT_WARPS * DOT_OUTS - 1) / (DOT_WARPS * DOT_OUTS);
    int per_tile = (16 * dev->sm_count + tiles - 1) / tiles;
    if (per_tile > blocks) per_tile = blocks;
    const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(per_tile));
    if (dtype == SMOE_BF16) return launch_pdl(f8_dot<__nv_bfloat16>, grid, dim3(DOT_WARPS * 32), 0, stream, a);
    return launch_pdl(f8_dot<float>, grid, dim3(DOT_WARPS * 32), 0, stream, a);
}

}  // namespace smoe
