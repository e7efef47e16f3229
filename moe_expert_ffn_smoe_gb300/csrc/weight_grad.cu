// The gradient of the experts' weights on a sorted batch, on the tensor cores
// (tcgen05, kind::f16, bf16 operands from shared memory):
//   d_w[e][n][c] = sum over the rows r of expert e of d_ys[r][n] xs[r][c].
//
// The sum runs over rows, so both operands lie in memory with the MMA's M and N along
// the row and its K down the column: they are copied as they are (boxes of 64 columns
// by 64 rows, 128-byte swizzle) and read by the MMA as transposed (MN-major) operands.
// An item is a tile of 256 x 256 of one expert's gradient, by a pair of CTAs
// (cta_group::2), 128 rows of it each; its sum stays in tensor memory (f32, two tiles
// of 256 columns: one is stored while the next is summed) and leaves through shared
// memory by tensor copies, which cut off what lies outside the expert's matrix, or add
// (accumulate).
//
// An expert's rows begin and end anywhere.  The rows of its last, shorter stage come in
// boxes of 32, 16, .. and 1 rows, and copies from past the batch's end, which fill with
// zeros, complete the 16 rows of an MMA: rows of other experts, which may hold a NaN,
// never meet this one's.
//
// Bound by what crosses between L2 and the SMs, whose reads (3.3 GB of them) wait
// behind the writes of d_w: 128 experts, 32,768 rows, 1536 x 4096 in bf16 386 to 396 us (1.6 GB
// written; without the stores 297), with one stage less and two places for the outputs 4%
// more (of few rows 2 to 5% less), with three stages 499.  8 experts of
// 4096 rows each in f32 277 us, 1490 TFLOP/s.  Measured and not kept: two tiles an item
// that share their rows of d_ys (2.5 GB read; both halves of tensor memory are then in
// use, and nothing is summed while the second is stored): 397 and 277; four tiles an
// item with the rows of d_ys kept in shared memory: 458.  Roles (warps): 0-7 store, 8
// issues the MMAs (the even CTA's), 9-12 copy 64 columns each.  Every wait is bounded.
#include <atomic>

#include <cuda_bf16.h>

#include "internal_tokens.h"
#include "smoe.h"
#include "tc_pair.cuh"

namespace smoe {
namespace {

constexpr int MT = 128, NT = 256;  // a CTA's rows of a tile, the tile's columns
constexpr int RT = 64;             // rows of the batch in a stage
constexpr int ST = 6;
constexpr int BOXES = 7;
constexpr uint32_t CHUNK = RT * 128;  // 64 columns of a stage
constexpr uint32_t STAGE = 4 * CHUNK; // two chunks of d_ys, two (the CTA's half) of xs
constexpr int EPI_WARPS = 8, MMA_WARP = 8, LOAD_WARP = 9, LOADERS = 4;
constexpr int WG_THREADS = (LOAD_WARP + LOADERS) * 32;
constexpr uint32_t BOX = 32 * 128;    // 32 rows of 128 bytes on their way out, a warp's
constexpr size_t WG_SMEM = 1024 + ST * STAGE + EPI_WARPS * BOX + 256;

struct alignas(128) GradArgs {
    CUtensorMap dy[BOXES], x[BOXES];  // boxes of 64, 32, .. and 1 rows
    CUtensorMap out;
    const int *offsets;
    unsigned *status;
    int R, n, N, K, mtiles, ntiles;  // tiles of an expert's gradient: 256 rows, 256 columns
    bool accumulate;
};

// Shared-memory descriptor, 128-byte swizzle, MN-major: 64 columns (128 bytes) to a
// chunk, chunks CHUNK bytes apart, eight rows 1024 bytes.
__device__ __forceinline__ uint64_t desc_mn128(uint32_t addr)
{
    return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(CHUNK >> 4) << 16) |
           (static_cast<uint64_t>(1024u >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}

__device__ __forceinline__ void mma_bf16_pair(uint32_t tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

__device__ __forceinline__ void store_box(const CUtensorMap *map, uint32_t src, int x, int y, int z, bool add)
{
    if (add)
        asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                         reinterpret_cast<uint64_t>(map)),
                     "r"(src), "r"(x), "r"(y), "r"(z)
                     : "memory");
    else
        asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                         reinterpret_cast<uint64_t>(map)),
                     "r"(src), "r"(x), "r"(y), "r"(z)
                     : "memory");
}

// Item it's rows (looked up an item ahead: two reads of memory); a range that is none
// counts as empty and is reported.
__device__ __forceinline__ int2 rows_at(const GradArgs &a, int it, int per, int nitems)
{
    if (it >= nitems) return make_int2(0, 0);
    const int e = it / per;
    const int lo = a.offsets[e], hi = a.offsets[e + 1];
    if (lo < 0 || hi < lo || hi > a.R) {
        atomicExch(a.status, kStatusRoute);
        return make_int2(0, 0);
    }
    return make_int2(lo, hi - lo);
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

template <typename T>
__global__ void __launch_bounds__(WG_THREADS, 1) weight_grad(const __grid_constant__ GradArgs a)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const uint32_t out0 = base + ST * STAGE, bars = out0 + EPI_WARPS * BOX;
    const uint32_t full = bars, empty = full + 8 * ST, dfull = empty + 8 * ST, dempty = dfull + 16, tslot = dempty + 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(blockIdx.x & 1u);
    const int first = static_cast<int>(blockIdx.x >> 1), stride = static_cast<int>(gridDim.x >> 1);

    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(full + 8 * i, LOADERS);  // used in the issuing CTA
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(dfull + 8 * i, 1);
            mbar_init(dempty + 8 * i, EPI_WARPS * 2);  // used in the issuing CTA
        }
        fence_mbar_init();
    }
    if (warp == MMA_WARP) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(tslot) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // nothing may reach a CTA whose barriers are not there yet
    tc_fence_after();
    uint32_t tmem;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(tslot));
    if (threadIdx.x == 0) pdl_launch_dependents();
    pdl_wait();

    const int per = a.mtiles * a.ntiles;
    const int nitems = a.n * per;  // at most 2^27
    bool failed = false;

    if (warp >= LOAD_WARP) {
        const int part = warp - LOAD_WARP;  // chunks 0, 1: d_ys; 2, 3: xs
        if (elect_one()) {
            const uint32_t lead = mapa_shared(full, 0);
            const CUtensorMap *map = part < 2 ? a.dy : a.x;
            uint32_t s = 0, p = 1;  // parity of the stage's release one lap ago; none in the first
            bool round0 = true;
            long long steps = 0;
            int2 r, next = rows_at(a, first, per, nitems);
            for (int it = first; it < nitems && !failed; it += stride) {
                const int m = it % per / a.ntiles, c = it % per % a.ntiles;
                r = next;
                next = rows_at(a, it + stride, per, nitems);
                const int col = part < 2 ? (m * 2 + rank) * MT + part * 64 : c * NT + rank * (NT / 2) + (part - 2) * 64;
                for (int t = 0; t < r.y; t += RT) {
                    if (!round0 && !mbar_wait_bounded(empty + 8 * s, p, a.status, 7u)) {
                        failed = true;
                        break;
                    }
                    const int rows = min(RT, r.y - t), used = (rows + 15) & ~15;
                    if (rank == 0) mbar_arrive_expect_tx(full + 8 * s, static_cast<uint32_t>(used) * 256u);
                    const uint32_t dst = base + s * STAGE + part * CHUNK, bar = lead + 8 * s;
                    const int y = r.x + t;
                    if (rows == RT) {
                        tma_load_2d_pair(dst, &map[0], col, y, bar);
                    } else {
                        // the rows by the bits of their number, zeros by those of what is missing
#pragma unroll
                        for (int b = 1; b < BOXES; ++b) {
                            const int size = RT >> b, at = rows & ~(2 * size - 1);
                            if (rows & size) tma_load_2d_pair(dst + at * 128, &map[b], col, y + at, bar);
                        }
#pragma unroll
                        for (int b = BOXES - 4; b < BOXES; ++b) {
                            const int size = RT >> b, missing = used - rows;
                            if (missing & size) tma_load_2d_pair(dst + (used - (missing & ~(size - 1))) * 128, &map[b], col, a.R, bar);
                        }
                    }
                    ++steps;
                    if (++s == ST) {
                        s = 0;
                        p ^= 1u;
                        round0 = false;
                    }
                }
            }
            // the last releases of the stages arrive here from the other CTA's issue
            if (!failed && part == 0)
                for (long long g = steps > ST ? steps - ST : 0; g < steps; ++g)
                    if (!mbar_wait_bounded(empty + 8 * static_cast<uint32_t>(g % ST), static_cast<uint32_t>(g / ST) & 1, a.status, 8u))
                        failed = true;
        }
        failed = __any_sync(FULL_MASK, failed);
    } else if (warp == MMA_WARP) {
        if (rank == 0 && elect_one()) {
            // f32 sums of bf16 products, A and B transposed
            const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) | (static_cast<uint32_t>(NT >> 3) << 17) |
                                   (static_cast<uint32_t>(2 * MT >> 4) << 24);
            uint32_t s = 0, p = 0, d = 0;
            int2 r, next = rows_at(a, first, per, nitems);
            for (int it = first; it < nitems && !failed; it += stride) {
                r = next;
                next = rows_at(a, it + stride, per, nitems);
                if (r.y == 0) continue;
                if (d >= 2 && !wait_pair<2>(dempty + 8 * (d & 1), (d / 2 - 1) & 1, a.status, 4u)) {
                    failed = true;
                    break;
                }
                const uint32_t acc = tmem + (d & 1) * NT;
                for (int t = 0; t < r.y; t += RT) {
                    if (!mbar_test<2>(full + 8 * s, p) && !wait_pair<2>(full + 8 * s, p, a.status, 3u)) {
                        failed = true;
                        break;
                    }
                    tc_fence_after();
                    const int steps = (min(RT, r.y - t) + 15) / 16;
                    const uint64_t ad = desc_mn128(base + s * STAGE), bd = desc_mn128(base + s * STAGE + 2 * CHUNK);
                    for (int kk = 0; kk < steps; ++kk)  // 16 rows are 2048 bytes
                        mma_bf16_pair(acc, ad + kk * 128, bd + kk * 128, idesc, t + kk != 0);
                    mma_commit_pair(empty + 8 * s);
                    if (++s == ST) {
                        s = 0;
                        p ^= 1u;
                    }
                }
                if (!failed) mma_commit_pair(dfull + 8 * (d & 1));
                ++d;
            }
        }
        failed = __any_sync(FULL_MASK, failed);
    } else {
        // warp w: lanes 32 (w % 4) .. + 31 of this CTA's rows, columns 128 (w / 4) .. + 127
        const int q = warp & 3, h = warp >> 2;
        constexpr int COLS = 128 / static_cast<int>(sizeof(T));  // of a box
        const uint32_t lead = mapa_shared(dempty, 0);
        const uint32_t box = out0 + warp * BOX, row = box + static_cast<uint32_t>(lane) * 128u;
        uint32_t d = 0;
        int2 r, next = rows_at(a, first, per, nitems);
        for (int it = first; it < nitems; it += stride) {
            const int e = it / per, m = it % per / a.ntiles, c = it % per % a.ntiles;
            r = next;
            next = rows_at(a, it + stride, per, nitems);
            if (r.y == 0 && a.accumulate) continue;
            if (r.y != 0) {
                if (!__all_sync(FULL_MASK, mbar_wait_bounded(dfull + 8 * (d & 1), (d / 2) & 1, a.status, 6u))) {
                    failed = true;
                    break;
                }
                tc_fence_after();
            }
            const int y = (m * 2 + rank) * MT + q * 32, x0 = c * NT + h * 128;
            const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16) + (d & 1) * NT + h * 128;
            // boxes of the tile that lie in the matrix at all
            const int boxes = y < a.N && x0 < a.K ? min((a.K - x0 + COLS - 1) / COLS, 128 / COLS) : 0;
            if (boxes == 0 && r.y != 0) {
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(lead + 8 * (d & 1));
            }
            for (int j = 0; j < boxes; ++j) {
                float v[COLS];
                if (r.y != 0) {
                    tmem_ld<COLS>(acc + j * COLS, v);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int i = 0; i < COLS; ++i) v[i] = 0.f;
                }
                if (j == boxes - 1 && r.y != 0) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(lead + 8 * (d & 1));
                }
                // the last one stored has been read
                if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t at = row + static_cast<uint32_t>((i ^ (lane & 7)) << 4);
                    if (sizeof(T) == 4) {
                        sts128(at, __float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                               __float_as_uint(v[4 * i + 3]));
                    } else {
                        uint32_t w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int o = (8 * i + 2 * k) % COLS;  // (in bounds for both types)
                            const __nv_bfloat162 t = __floats2bfloat162_rn(v[o], v[o + 1]);
                            w[k] = *reinterpret_cast<const uint32_t *>(&t);
                        }
                        sts128(at, w[0], w[1], w[2], w[3]);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    store_box(&a.out, box, x0 + j * COLS, y, e, a.accumulate);
                    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                }
            }
            if (r.y != 0) ++d;
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    tc_fence_before();
    if (__syncthreads_or(failed)) {
        // a wait gave up: outputs are unspecified, and what this CTA started
        // (at most a ring of copies and MMAs) gets a bounded time to land
        const long long t0 = clock64();
        while (clock64() - t0 < 2000000LL) __nanosleep(1000);
        __syncthreads();
    }
    cluster_sync();  // no CTA leaves while the other's copies or releases may reach it
    if (warp == MMA_WARP) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

bool encode_out(CUtensorMap *map, bool bf, void *p, int n, int N, int K)
{
    EncodeTiled fn = encoder();
    if (!fn) return false;
    const cuuint64_t e = bf ? 2 : 4;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(n)};
    const cuuint64_t strides[2] = {dims[0] * e, dims[0] * dims[1] * e};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / e), 32u, 1u};
    const cuuint32_t estr[3] = {1u, 1u, 1u};
    return fn(map, bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, p, dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T>
cudaError_t launch_t(const GradArgs &a, int sms, cudaStream_t stream)
{
    auto k = weight_grad<T>;
    static_assert(WG_SMEM <= 227 * 1024, "shared memory of a CTA");
    // one size for every launch of this kernel: asked for once per device
    static std::atomic<bool> opted[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!opted[dev].load(std::memory_order_relaxed)) {
        const cudaError_t e = ensure_dynamic_smem(k, WG_SMEM);
        if (e != cudaSuccess) return e;
        opted[dev].store(true, std::memory_order_relaxed);
    }
    long long pairs = sms / 2;
    const int fit = clusters_held<weight_grad<T>>(2, WG_THREADS, WG_SMEM);
    if (fit > 0 && fit < pairs) pairs = fit;
    const long long items = static_cast<long long>(a.n) * a.mtiles * a.ntiles;
    if (items < pairs) pairs = items;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
    cfg.blockDim = dim3(WG_THREADS);
    cfg.dynamicSmemBytes = WG_SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k, a);
}

}  // namespace

cudaError_t launch_weight_grad(const void *d_ys, const void *xs, const int *offsets, int R, int n, int N, int K,
                               bool accumulate, void *d_w, int dtype, cudaStream_t stream)
{
    const DeviceInfo *dev = device_info();
    unsigned *status = device_status_word();
    if (!dev || !status) return cudaErrorInvalidDevice;
    if (R == 0)  // no operand to describe
        return cudaMemsetAsync(d_w, 0, static_cast<size_t>(n) * N * K * (dtype == SMOE_BF16 ? 2 : 4), stream);
    GradArgs a = {};
    for (int i = 0; i < BOXES; ++i) {
        const int rows = RT >> i;
        if (!encode(&a.dy[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, d_ys, N, R, 64, rows) ||
            !encode(&a.x[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, xs, K, R, 64, rows))
            return cudaErrorInvalidValue;
    }
    if (!encode_out(&a.out, dtype == SMOE_BF16, d_w, n, N, K)) return cudaErrorInvalidValue;
    a.offsets = offsets;
    a.status = status;
    a.R = R;
    a.n = n;
    a.N = N;
    a.K = K;
    a.mtiles = (N + 2 * MT - 1) / (2 * MT);
    a.ntiles = (K + NT - 1) / NT;
    a.accumulate = accumulate;
    return dtype == SMOE_BF16 ? launch_t<__nv_bfloat16>(a, dev->sm_count, stream) : launch_t<float>(a, dev->sm_count, stream);
}

}  // namespace smoe
