// 8-bit weights and activations: the row quantiser and the products
//   y[r][n] = x_scale[src(r)] w_scale[e][n] sum_k xq[src(r)][k] wq[e][n][k]
// over one matrix, or over the experts of a sorted batch (rows
// [offsets[e], offsets[e + 1]) by expert e's matrix, src(r) = order[r] / k).
//
// plan_tiles turns the experts' row counts, which only the device knows,
// into a list of tiles of at most `step` rows of one expert each; rows past
// the last expert's are tiles of expert -1, whose outputs are zeros.
#include "q8.cuh"
#include "rowvec.cuh"
#include "smoe.h"

namespace smoe {
namespace {

// ---------------------------------------------------------------- quantiser

// The VE values at column c of row r: x itself, or silu(gate) * up of a row
// [gate | up] of 2 cols.
template <typename T, int VE, bool ACT>
__device__ __forceinline__ void quant_values(const T *row, int cols, int c, float (&v)[VE])
{
    RowVec<T, VE> a;
    a.load(row + c);
    a.get(v);
    if (ACT) {
        RowVec<T, VE> b;
        float u[VE];
        b.load(row + cols + c);
        b.get(u);
#pragma unroll
        for (int i = 0; i < VE; ++i) v[i] = silu_row(v[i]) * u[i];
    }
}

// Magnitudes as f32 bit patterns: their order is the integers', and a NaN or
// an infinity is above every finite one.
template <int VE>
__device__ __forceinline__ uint32_t magnitude(const float (&v)[VE])
{
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < VE; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    return m;
}

// What a thread keeps of a vector between the two passes over its row: the
// loaded words, or the values of the activation.
template <typename T, int VE, bool ACT>
struct Held {
    float v[VE];
    __device__ __forceinline__ void load(const T *row, int cols, int c) { quant_values<T, VE, ACT>(row, cols, c, v); }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < VE; ++i) v[i] = 0.f;
    }
    __device__ __forceinline__ uint32_t most() const { return magnitude<VE>(v); }
    __device__ __forceinline__ void get(float (&o)[VE]) const
    {
#pragma unroll
        for (int i = 0; i < VE; ++i) o[i] = v[i];
    }
};
template <>
struct Held<__nv_bfloat16, 8, false> {
    RowVec<__nv_bfloat16, 8> r;
    __device__ __forceinline__ void load(const __nv_bfloat16 *row, int, int c) { r.load(row + c); }
    __device__ __forceinline__ void clear() { r.zero(); }
    // the same order holds for bf16's bits, two at a time
    __device__ __forceinline__ uint32_t most() const
    {
        const uint32_t m = __vmaxu2(__vmaxu2(r.raw.x & 0x7fff7fffu, r.raw.y & 0x7fff7fffu),
                                    __vmaxu2(r.raw.z & 0x7fff7fffu, r.raw.w & 0x7fff7fffu));
        return max(m & 0xffff0000u, m << 16);
    }
    __device__ __forceinline__ void get(float (&o)[8]) const { r.get(o); }
};

// The code of a scaled value |p| <= 127.5 in the low byte: adding 1.5 2^23
// rounds p to an integer, ties to even, in the lowest mantissa bits.
__device__ __forceinline__ uint32_t code_bits(float v, float up)
{
    return __float_as_uint(__fadd_rn(__fmul_rn(v, up), 12582912.f));
}

// VE codes (the low bytes of c) as one store.
__device__ __forceinline__ uint32_t pack4(const uint32_t *c)
{
    return __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
}
__device__ __forceinline__ void put_codes(int8_t *q, const uint32_t (&c)[8])
{
    *reinterpret_cast<uint2 *>(q) = make_uint2(pack4(c), pack4(c + 4));
}
__device__ __forceinline__ void put_codes(int8_t *q, const uint32_t (&c)[4]) { *reinterpret_cast<uint32_t *>(q) = pack4(c); }
__device__ __forceinline__ void put_codes(int8_t *q, const uint32_t (&c)[1]) { *q = static_cast<int8_t>(c[0]); }

// Vectors that a thread keeps between the two passes over its row.
template <int VE, bool ACT, int THREADS>
constexpr int held_vectors()
{
    return VE == 1 ? 8 : (THREADS <= 128 && !ACT ? 64 / VE : 32 / VE);
}

// One CTA of THREADS per row: the largest magnitude, then the rounding.  A
// thread keeps its first NV vectors, so that a row of up to NV x THREADS
// vectors is read (and its activation computed) once; what is beyond is read
// again.  Bound by instruction issue: with fewer warps a row, the row's own
// work (reductions, two divisions) is done fewer times, which pays once there
// are rows for the whole device (launch_quantize_rows).
template <typename T, int VE, bool ACT, int THREADS>
__global__ void __launch_bounds__(THREADS) quantize_rows(const T *__restrict__ x, int cols, int8_t *__restrict__ q,
                                                         float *__restrict__ scales)
{
    constexpr int NV = held_vectors<VE, ACT, THREADS>();
    __shared__ uint32_t warp_most[THREADS / 32];
    pdl_launch_dependents();
    pdl_wait();
    const size_t r = blockIdx.x;
    const T *row = x + r * cols * (ACT ? 2 : 1);
    const int c0 = threadIdx.x * VE;
    Held<T, VE, ACT> held[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (c0 + i * THREADS * VE < cols) held[i].load(row, cols, c0 + i * THREADS * VE);
        else held[i].clear();
    }
    uint32_t most = 0u;
#pragma unroll
    for (int i = 0; i < NV; ++i) most = max(most, held[i].most());
    for (int c = c0 + NV * THREADS * VE; c < cols; c += THREADS * VE) {
        float v[VE];
        quant_values<T, VE, ACT>(row, cols, c, v);
        most = max(most, magnitude<VE>(v));
    }
    most = __reduce_max_sync(FULL_MASK, most);
    if ((threadIdx.x & 31) == 0) warp_most[threadIdx.x >> 5] = most;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) most = max(most, warp_most[i]);
    // a row of zeros has scale 0; a row that is not finite scale NaN and
    // codes 0, so that every product of it is NaN
    const bool bad = most >= 0x7f800000u;
    const float top = __uint_as_float(most);
    const float up = bad || most == 0u ? 0.f : __fdiv_rn(127.f, top);
    if (threadIdx.x == 0) scales[r] = bad ? __int_as_float(0x7fffffff) : __fdiv_rn(top, 127.f);
    int8_t *out = q + r * cols;
    if (bad || up == INFINITY) {
        // rare, and kept out of the way of the other rows: 127 / top is beyond
        // f32 below 3.8e-37, where the row is taken 2^64 times
        const float lifted = bad ? 0.f : __fdiv_rn(127.f, top * 0x1p64f);
#pragma unroll 1
        for (int c = threadIdx.x; c < cols; c += THREADS) {
            float v[1];
            quant_values<T, 1, ACT>(row, cols, c, v);
            out[c] = bad ? 0 : static_cast<int8_t>(code_bits(v[0] * 0x1p64f, lifted));
        }
        return;
    }
    auto store = [&](const float (&v)[VE], int c) {
        uint32_t k[VE];
#pragma unroll
        for (int j = 0; j < VE; ++j) k[j] = code_bits(v[j], up);
        put_codes(out + c, k);
    };
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = c0 + i * THREADS * VE;
        if (c >= cols) break;
        float v[VE];
        held[i].get(v);
        store(v, c);
    }
    for (int c = c0 + NV * THREADS * VE; c < cols; c += THREADS * VE) {
        float v[VE];
        quant_values<T, VE, ACT>(row, cols, c, v);
        store(v, c);
    }
}

// ---------------------------------------------------------------- tiles

constexpr int PLAN_THREADS = 1024;

// tiles[0 .. *ntiles): every expert's rows in steps of `step`, then the rows
// past the last expert's.
__global__ void __launch_bounds__(PLAN_THREADS) plan_tiles(const int *__restrict__ offsets, int n, int R, int step,
                                                           int max_tiles, int *__restrict__ ntiles,
                                                           Tile *__restrict__ tiles, unsigned *status)
{
    __shared__ long long warp_sums[PLAN_THREADS / 32];
    __shared__ long long run_s;
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, wi = tid >> 5;
    long long run = 0;  // 64 bits: ranges that overlap (reported) can add up to more than 32
    for (int b = 0; b <= n; b += PLAN_THREADS) {
        const int e = b + tid;
        int lo = 0, hi = 0;
        if (e <= n) {
            lo = offsets[e];
            hi = e < n ? offsets[e + 1] : R;
            if (lo < 0 || hi < lo || hi > R) {
                atomicExch(status, kStatusRoute);
                lo = hi = 0;
            }
        }
        const int cnt = (hi - lo + step - 1) / step;
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
        if (tid == PLAN_THREADS - 1) run_s = before + inc;
        const long long t0 = before + inc - cnt;
        for (int i = 0; i < cnt && t0 + i < max_tiles; ++i)
            tiles[t0 + i] = Tile{e < n ? e : -1, lo + i * step, min(step, hi - lo - i * step), 0};
        __syncthreads();
        run = run_s;
    }
    if (tid == 0) *ntiles = static_cast<int>(min(run, static_cast<long long>(max_tiles)));
}

// ---------------------------------------------------------------- products

constexpr int DOT_WARPS = 8;
constexpr int DOT_ROWS = 8;   // activation rows per tile
constexpr int DOT_OUTS = 4;   // weight rows per warp

struct Q8Args {
    const int8_t *xq;
    const float *xs;
    const int *order;  // null: row r is its own source
    const int8_t *wq;
    const float *ws;
    void *y;
    const int *ntiles;
    const Tile *tiles;
    unsigned *status;
    int k, nsrc, N, K, R;
};

// Integer dot products on the CUDA cores, exact in 32 bits (K <= 32768): a
// warp holds 4 weight rows against the tile's up to 8 activation rows, 16
// columns of each per lane and step.  A warp walks its groups of 4 rows as
// one sequence of steps, the weights of the next DEPTH steps in flight
// across the groups' ends.  Bound by streaming the weights; for one matrix
// (tiles null) the first group's are brought into L2 while the previous
// kernel ends (a prefetch only: that kernel may be the one that quantises
// these weights).
template <typename T>
__global__ void __launch_bounds__(DOT_WARPS * 32, 2) q8_dot(const Q8Args a)
{
    constexpr int DEPTH = 3;
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    int n0 = (blockIdx.y * DOT_WARPS + (threadIdx.x >> 5)) * DOT_OUTS;  // the group being summed
    const int stride = gridDim.y * DOT_WARPS * DOT_OUTS;
    if (!a.tiles && lane < DOT_OUTS && n0 + lane < a.N && a.K > 0)
        prefetch_l2(a.wq + static_cast<size_t>(n0 + lane) * a.K, static_cast<uint32_t>(a.K));
    pdl_wait();
    if (a.tiles && static_cast<int>(blockIdx.x) >= *a.ntiles) return;
    const int row0 = blockIdx.x * DOT_ROWS;
    const Tile tile = a.tiles ? a.tiles[blockIdx.x] : Tile{0, row0, min(DOT_ROWS, a.R - row0), 0};
    T *y = static_cast<T *>(a.y);
    if (tile.expert < 0) {
        for (; n0 < a.N; n0 += stride)
            for (int i = lane; i < tile.rows * DOT_OUTS; i += 32)
                if (n0 + i % DOT_OUTS < a.N)
                    put(y + static_cast<size_t>(tile.row0 + i / DOT_OUTS) * a.N + n0 + i % DOT_OUTS, 0.f);
        return;
    }
    const int8_t *w = a.wq + static_cast<size_t>(tile.expert) * a.N * a.K;
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
        src[r] = r < tile.rows ? source_row(a.order, a.k, a.nsrc, tile.row0 + r, a.status) : -1;
    int acc[DOT_OUTS][DOT_ROWS];
#pragma unroll
    for (int o = 0; o < DOT_OUTS; ++o)
#pragma unroll
        for (int r = 0; r < DOT_ROWS; ++r) acc[o][r] = 0;
    int c = lane * 16;
    while (n0 < a.N) {
#pragma unroll
        for (int i = 0; i < DEPTH; ++i) {
            if (n0 >= a.N) break;
            if (c < a.K) {
#pragma unroll
                for (int r = 0; r < DOT_ROWS; ++r) {
                    if (r >= tile.rows) break;
                    if (src[r] < 0) continue;
                    const uint4 xv = *reinterpret_cast<const uint4 *>(a.xq + static_cast<size_t>(src[r]) * a.K + c);
#pragma unroll
                    for (int o = 0; o < DOT_OUTS; ++o) {
                        acc[o][r] = __dp4a(static_cast<int>(wv[i][o].x), static_cast<int>(xv.x), acc[o][r]);
                        acc[o][r] = __dp4a(static_cast<int>(wv[i][o].y), static_cast<int>(xv.y), acc[o][r]);
                        acc[o][r] = __dp4a(static_cast<int>(wv[i][o].z), static_cast<int>(xv.z), acc[o][r]);
                        acc[o][r] = __dp4a(static_cast<int>(wv[i][o].w), static_cast<int>(xv.w), acc[o][r]);
                    }
                }
            }
            fetch(wv[i]);
            c += 512;
            if (c - lane * 16 >= a.K) {  // the group is summed
#pragma unroll
                for (int r = 0; r < DOT_ROWS; ++r) {
                    if (r >= tile.rows) break;
                    const float xs = src[r] >= 0 ? a.xs[src[r]] : 0.f;
#pragma unroll
                    for (int o = 0; o < DOT_OUTS; ++o) {
                        const int sum = __reduce_add_sync(FULL_MASK, acc[o][r]);
                        acc[o][r] = 0;
                        if (lane == o && n0 + o < a.N)
                            put(y + static_cast<size_t>(tile.row0 + r) * a.N + n0 + o,
                                static_cast<float>(sum) * xs * a.ws[static_cast<size_t>(tile.expert) * a.N + n0 + o]);
                    }
                }
                c = lane * 16;
                n0 += stride;
            }
        }
    }
}

template <typename T, int VE, bool ACT>
cudaError_t quant_t(const void *x, int rows, int cols, int8_t *q, float *scales, cudaStream_t stream)
{
    const DeviceInfo *dev = device_info();
    if (!dev) return cudaErrorInvalidDevice;
    auto go = [&](auto kernel, int threads) {
        return launch_pdl(kernel, dim3(static_cast<unsigned>(rows)), dim3(static_cast<unsigned>(threads)), 0, stream,
                          static_cast<const T *>(x), cols, q, scales);
    };
    // Few rows: eight warps each.  Rows for the whole device: the fewest warps
    // that keep the row between its two passes.  Measured (us, bf16) on 64,
    // 128 and 256 threads: 4096 rows of 4096 7.8 / 7.9 / 10.6, 2000 of 16384
    // 25.0 / 20.0 / 17.3 (one warp is no faster than two: 8000 rows of 512 with
    // the activation 8.7 / 8.6).
    if (rows >= 4 * dev->sm_count) {
        if (cols <= 64 * VE * held_vectors<VE, ACT, 64>()) return go(quantize_rows<T, VE, ACT, 64>, 64);
        if (cols <= 128 * VE * held_vectors<VE, ACT, 128>()) return go(quantize_rows<T, VE, ACT, 128>, 128);
    }
    return go(quantize_rows<T, VE, ACT, 256>, 256);
}

template <typename T, int VE>
cudaError_t quant_a(bool act, const void *x, int rows, int cols, int8_t *q, float *scales, cudaStream_t stream)
{
    return act ? quant_t<T, VE, true>(x, rows, cols, q, scales, stream)
               : quant_t<T, VE, false>(x, rows, cols, q, scales, stream);
}

}  // namespace

cudaError_t launch_quantize_rows(const void *x, int dtype, bool act, int rows, int cols, int8_t *q, float *scales,
                                 cudaStream_t stream)
{
    const bool bf = dtype == SMOE_BF16;
    const size_t pitch = static_cast<size_t>(cols) * (bf ? 2 : 4);
    const bool v = ((reinterpret_cast<uintptr_t>(x) | pitch) & 15u) == 0;
    if (bf)
        return v ? quant_a<__nv_bfloat16, 8>(act, x, rows, cols, q, scales, stream)
                 : quant_a<__nv_bfloat16, 1>(act, x, rows, cols, q, scales, stream);
    return v ? quant_a<float, 4>(act, x, rows, cols, q, scales, stream)
             : quant_a<float, 1>(act, x, rows, cols, q, scales, stream);
}

// Where the tensor cores take the product: from three rows on, and from more
// than three for every eight experts.  Below, the integer dots need no
// preparation.  Measured (us; K = 4096), dots against tensor cores: one matrix
// of 8192, 1 row 7.4 / 13.2, 2 rows 9.9 / 13.5, 4 rows 14.4 / 13.6; of 1536,
// 1 row 6.0 / 8.6, 2 rows 9.1 / 8.6; 128 experts of 1536, 32 rows 38.9 /
// 42.9, 64 rows 62.1 / 58.4.
static bool on_tensor_cores(int R, int n, int K) { return K > 0 && R > 2 && R > 3LL * n / 8; }

// Enough for either form, so that a larger batch never needs less.
size_t q8_workspace(int nsrc, int R, int n, int K)
{
    const size_t dots = up256(16 + static_cast<size_t>(most_tiles(R, n, DOT_ROWS)) * sizeof(Tile));
    const size_t tensor = q8_tc_workspace(nsrc, R, n, K);
    return dots > tensor ? dots : tensor;
}

cudaError_t launch_q8(const int8_t *xq, const float *xs, int nsrc, const int *order, int k, const int *offsets, int R,
                      int n, const int8_t *wq, const float *ws, int N, int K, void *y, int dtype, void *workspace,
                      cudaStream_t stream)
{
    if (on_tensor_cores(R, n, K))
        return launch_q8_tc(Q8Call{xq, xs, nsrc, order, k, offsets, R, n, wq, ws, N, K, y, dtype}, workspace, stream);
    unsigned *status = device_status_word();
    if (!status) return cudaErrorInvalidDevice;
    // one matrix: tiles of consecutive rows, no list needed
    const int max_tiles = offsets ? most_tiles(R, n, DOT_ROWS) : (R + DOT_ROWS - 1) / DOT_ROWS;
    int *ntiles = static_cast<int *>(workspace);
    Tile *tiles = offsets ? reinterpret_cast<Tile *>(static_cast<char *>(workspace) + 16) : nullptr;
    if (offsets) {
        const cudaError_t e = launch_pdl(plan_tiles, dim3(1), dim3(PLAN_THREADS), 0, stream, offsets, n, R, DOT_ROWS,
                                         max_tiles, ntiles, tiles, status);
        if (e != cudaSuccess) return e;
    }
    const Q8Args a = {xq, xs, order, wq, ws, y, ntiles, tiles, status, k, nsrc, N, K, R};
    // CTAs per tile: about eight waves of the device (two CTAs an SM) when
    // every row has an expert of its own (two waves 130 us, four 103, eight
    // 99, sixteen 100 for 128 rows over 128 experts of 1536 x 4096)
    const DeviceInfo *dev = device_info();
    if (!dev) return cudaErrorInvalidDevice;
    const int likely = offsets ? (R < n ? R : n) : max_tiles;
    const int blocks = (N + DOT_WARPS * DOT_OUTS - 1) / (DOT_WARPS * DOT_OUTS);
    int per_tile = (16 * dev->sm_count + likely - 1) / likely;
    if (per_tile > blocks) per_tile = blocks;
    const dim3 grid(static_cast<unsigned>(max_tiles), static_cast<unsigned>(per_tile));
    if (dtype == SMOE_BF16) return launch_pdl(q8_dot<__nv_bfloat16>, grid, dim3(DOT_WARPS * 32), 0, stream, a);
    return launch_pdl(q8_dot<float>, grid, dim3(DOT_WARPS * 32), 0, stream, a);
}

}  // namespace smoe
