// The 8-bit floating-point product with a scale for each block of 128, with the rows on
// the MMA's M side, for batches that are bound by the tensor cores (tcgen05,
// kind::f8f6f4, e4m3 operands from shared memory):
//   y[r][n] = sum_b xs[r][b] ws[e][n / 128][b] sum_{c in b} xq[r][c] wq[e][n][c].
//
// The scales change every 128 columns, inside the sum, so each block's products are a
// sum of their own in tensor memory: the MMAs of a block write one accumulator (of
// two), the epilogue warps read it and add it to their registers, times the block's
// scales, while the next block's MMAs run.  The sums of blocks are f32 in registers; a
// block's own is the tensor core's f32.
//
// The rows are the MMA's M side, 128 of them, the weights its N side, 256: a thread of
// the epilogue then holds 128 outputs of one row and of one block of weights, whose
// scale is one number.  With the weights on the M side (as f8_tc.cu has them, whose
// tiles are small) a tile costs its rows only, but every product needs the scale of its
// own column: brought from shared memory beside the MMAs, a block took 1150 clocks
// against the 512 of its MMAs (1999 rows x 8192 x 4096 88 us).  Here a tile of fewer
// than 128 rows costs as much as a full one.
//
// Bound by handing the accumulators over: a block takes 945 clocks (the slope of the time
// over 16 to 64 blocks an item, 1 to 4 items a CTA), since each of the two accumulators
// goes round in some 1900: 1130 from the issue of its MMAs, 512 of them their own, until
// the epilogue sees them, 450 read and added, 350 handed back and issued again (stamps of
// a launch).  An item costs some 8000 clocks more, its stores and the next one's first
// copies: of 32 blocks a fifth of its time.  1999 rows x 8192 x 4096, 3.4 items a CTA run
// as 4, 74.5 us, 1.8 PFLOP/s.
// Pairs of CTAs on 256 rows need two thirds of the copies and took 73 us there, but cost
// 256 rows a tile: through 128 experts, 2047 tokens of 8 221 us against 192, 4096 tokens
// 307 against 291.  Accumulators in halves, barriers tested ahead, 16 epilogue warps and
// spinning waits were no faster.
//
// Persistent: CTAs walk the items (tile of rows, 256 weights).  Roles (warps): 0-7
// epilogue, 8 issues the MMAs, 9 streams the weights, 12-19 the rows, gathered by the
// copies where the batch is sorted by an order.  Every wait is bounded.
#include <atomic>

#include "f8.cuh"
#include "smoe.h"
#include "tc_pair.cuh"

namespace smoe {
namespace {

constexpr int MT = 128, NT = 256;            // rows, weights of a tile
constexpr uint32_t X_BYTES = MT * F8_BLOCK, W_BYTES = NT * F8_BLOCK;  // a block of columns of them
constexpr int ST = 4, D = 2;                 // stages of the operands, accumulators
constexpr int EPI_WARPS = 8, MMA_WARP = 8, W_WARP = 9, X_WARP = 12, X_WARPS = 8;
constexpr int ROWS_THREADS = (X_WARP + X_WARPS) * 32;
constexpr int BOX = 64;                      // rows of one copy (not gathered)
constexpr uint32_t OUT_PITCH = 64 + 16;      // 64 bytes of a row on their way out (rows that begin anywhere)
constexpr size_t rows_smem(bool whole)
{
    return 1024 + ST * (X_BYTES + W_BYTES) + MT * 4 + 256 + (whole ? 0 : EPI_WARPS * 32 * OUT_PITCH);
}

struct alignas(128) RowsArgs {
    CUtensorMap wmap, xmap;
    const float *ws, *xs;  // scales [n x nb x kb], [nsrc x kb]
    void *y;
    const int *ntiles;
    const Tile *tiles;     // null: one matrix, tiles of `step` rows
    const int *order;      // source of every sorted row, times k (gathered), or null
    unsigned *status;
    int R, N, kb, nb, k, nsrc, step, groups;  // groups of 256 weights
};

// Instruction descriptor, kind::f8f6f4: f32 accumulate, A and B e4m3, K-major.
constexpr uint32_t kIdesc = (1u << 4) | (static_cast<uint32_t>(NT >> 3) << 17) | (static_cast<uint32_t>(MT >> 4) << 24);

__device__ __forceinline__ void mma_f8(uint32_t tmem, uint64_t a, uint64_t b, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem),
        "l"(a), "l"(b), "r"(kIdesc), "r"(acc)
        : "memory");
}

// Waits for this thread's loads; what they load goes through it, so that no use
// of it is moved before it.
__device__ __forceinline__ void tmem_loaded(float (&v)[32])
{
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) asm volatile("" : "+f"(v[i]));
}

// a += d f, two at a time.
__device__ __forceinline__ void fma2(float2 &a, float d0, float d1, float f)
{
    asm("{\n\t.reg .b64 d, f, a;\n\tmov.b64 d, {%2, %3};\n\tmov.b64 f, {%4, %4};\n\tmov.b64 a, {%0, %1};\n\t"
        "fma.rn.f32x2 a, d, f, a;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "+f"(a.x), "+f"(a.y)
        : "f"(d0), "f"(d1), "f"(f));
}

__device__ __forceinline__ uint32_t bf16x2(float a, float b)
{
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&p);
}

// 32 neighbouring outputs of a row that begins at a 16-byte boundary, of which the
// first n are there.
__device__ __forceinline__ void store32(float *y, const float2 (&v)[16], int n)
{
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (4 * i < n) *reinterpret_cast<float4 *>(y + 4 * i) = make_float4(v[2 * i].x, v[2 * i].y, v[2 * i + 1].x, v[2 * i + 1].y);
}
__device__ __forceinline__ void store32(__nv_bfloat16 *y, const float2 (&v)[16], int n)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (8 * i < n)
            *reinterpret_cast<uint4 *>(y + 8 * i) = make_uint4(bf16x2(v[4 * i].x, v[4 * i].y), bf16x2(v[4 * i + 1].x, v[4 * i + 1].y),
                                                               bf16x2(v[4 * i + 2].x, v[4 * i + 2].y), bf16x2(v[4 * i + 3].x, v[4 * i + 3].y));
}

// The same of 32 rows, one a lane, that begin anywhere: 64 bytes of each at a time
// through shared memory.  y: the first row's (of `rows`).
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void store32_anywhere(float *y, const float2 (&v)[16], int n, int N, int rows, uint32_t stage)
{
    const uint32_t mine = stage + (threadIdx.x & 31) * OUT_PITCH;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 a = v[8 * h + 2 * i], b = v[8 * h + 2 * i + 1];
            sts128(mine + 16 * i, __float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
        }
        __syncwarp();
        store_staged<32, 16>(stage, OUT_PITCH, y + 16 * h, N, rows, n - 16 * h);
    }
}
__device__ __forceinline__ void store32_anywhere(__nv_bfloat16 *y, const float2 (&v)[16], int n, int N, int rows, uint32_t stage)
{
    const uint32_t mine = stage + (threadIdx.x & 31) * OUT_PITCH;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i)
        sts128(mine + 16 * i, bf16x2(v[4 * i].x, v[4 * i].y), bf16x2(v[4 * i + 1].x, v[4 * i + 1].y),
               bf16x2(v[4 * i + 2].x, v[4 * i + 2].y), bf16x2(v[4 * i + 3].x, v[4 * i + 3].y));
    __syncwarp();
    store_staged<32, 32>(stage, OUT_PITCH, y, N, rows, n);
}

__device__ __forceinline__ Tile tile_at(const RowsArgs &a, int i, int ntiles)
{
    if (i >= ntiles) return Tile{0, 0, 0, 0};
    if (a.tiles) return a.tiles[i];
    return Tile{0, i * a.step, min(a.step, a.R - i * a.step), 0};
}

// WHOLE: every row of y begins at a 16-byte boundary.  (One kernel for both took 81 us
// for 1999 rows x 8192 x 4096 against 74.)
template <typename T, bool WHOLE>
__global__ void __launch_bounds__(ROWS_THREADS, 1) f8_rows(const __grid_constant__ RowsArgs a)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw), base = (raw + 1023u) & ~1023u;
    const uint32_t w0 = base, x0 = w0 + ST * W_BYTES, list0 = x0 + ST * X_BYTES, bars = list0 + MT * 4, out0 = bars + 256;
    const uint32_t full = bars, empty = full + 8 * ST, dfull = empty + 8 * ST, dempty = dfull + 8 * D, tslot = dempty + 8 * D;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int first = static_cast<int>(blockIdx.x), stride = static_cast<int>(gridDim.x);

    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(full + 8 * i, 1 + (a.order ? X_WARPS : 1));  // the loading warps
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < D; ++i) {
            mbar_init(dfull + 8 * i, 1);
            mbar_init(dempty + 8 * i, EPI_WARPS);
        }
        fence_mbar_init();
    }
    if (warp == MMA_WARP) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(tslot) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    uint32_t tmem;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(tslot));
    if (threadIdx.x == 0) pdl_launch_dependents();

    // One matrix: this CTA's first weights are known, and are brought into L2 while
    // the previous kernel ends.  A prefetch only: that kernel may be the one that
    // quantises these weights.
    if (!a.tiles && warp == W_WARP && first < (a.R + a.step - 1) / a.step * a.groups && lane < ST && lane < a.kb)
        tma_prefetch_2d(&a.wmap, lane * F8_BLOCK, first % a.groups * NT);
    pdl_wait();
    const int ntiles = a.tiles ? *a.ntiles : (a.R + a.step - 1) / a.step;
    const long long nitems = static_cast<long long>(ntiles) * a.groups;
    bool failed = false;

    if (warp >= MMA_WARP) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 32;");
        if (warp == W_WARP) {
            if (elect_one()) {
                uint32_t s = 0, p = 1;  // parity of the stage's release one lap ago; none in the first
                bool round0 = true;
                for (long long it = first; it < nitems && !failed; it += stride) {
                    const Tile t = tile_at(a, static_cast<int>(it / a.groups), ntiles);
                    const int row = t.expert * a.N + static_cast<int>(it % a.groups) * NT;
                    for (int c = 0; c < a.kb; ++c) {
                        if (!round0 && !mbar_wait_bounded(empty + 8 * s, p, a.status, 7u)) {
                            failed = true;
                            break;
                        }
                        mbar_arrive_expect_tx(full + 8 * s, W_BYTES);
                        tma_load_2d(w0 + s * W_BYTES, &a.wmap, c * F8_BLOCK, row, full + 8 * s);
                        if (++s == ST) {
                            s = 0;
                            p ^= 1u;
                            round0 = false;
                        }
                    }
                }
            }
            failed = __any_sync(FULL_MASK, failed);
        } else if (warp >= X_WARP && (a.order || warp == X_WARP)) {
            // Gathered: each of the eight warps loads every eighth four rows of every
            // stage (a gather costs its issuer some 100 clocks; four warps: 304 us against
            // 291 for 4096 tokens through 128 experts).
            const int part = warp - X_WARP;
            constexpr int PER = MT / X_WARPS;  // rows of a loading warp, at most
            int *list = reinterpret_cast<int *>(smem_raw + (list0 - raw)) + part * PER;
            uint32_t s = 0, p = 1;
            bool round0 = true;
            for (long long it = first; it < nitems && !failed; it += stride) {
                const Tile t = tile_at(a, static_cast<int>(it / a.groups), ntiles);
                if (a.order) {  // rows past the tile's: any row, their outputs are not stored
                    const int at = 4 * X_WARPS * (lane >> 2) + 4 * part + (lane & 3);
                    __syncwarp();
                    if (lane < PER) list[lane] = at < t.rows ? max(source_row(a.order, a.k, a.nsrc, t.row0 + at, a.status), 0) : 0;
                    __syncwarp();
                }
                if (elect_one()) {
                    const int copies = a.order ? max(0, ((t.rows + 3) / 4 - part + X_WARPS - 1) / X_WARPS) : (t.rows + BOX - 1) / BOX;
                    const uint32_t bytes = static_cast<uint32_t>(copies * (a.order ? 4 : BOX)) * F8_BLOCK;
                    for (int c = 0; c < a.kb; ++c) {
                        if (!round0 && !mbar_wait_bounded(empty + 8 * s, p, a.status, 8u)) {
                            failed = true;
                            break;
                        }
                        const uint32_t dst = x0 + s * X_BYTES, bar = full + 8 * s;
                        mbar_arrive_expect_tx(bar, bytes);
                        if (a.order) {
                            for (int i = 0; i < copies; ++i) {
                                const int4 r = *reinterpret_cast<const int4 *>(list + 4 * i);
                                tma_gather4(dst + static_cast<uint32_t>(4 * (X_WARPS * i + part)) * F8_BLOCK, &a.xmap, c * F8_BLOCK, r, bar);
                            }
                        } else {
                            for (int b = 0; b < copies; ++b)
                                tma_load_2d(dst + static_cast<uint32_t>(b * BOX) * F8_BLOCK, &a.xmap, c * F8_BLOCK, t.row0 + b * BOX, bar);
                        }
                        if (++s == ST) {
                            s = 0;
                            p ^= 1u;
                            round0 = false;
                        }
                    }
                }
                // the elected lane's place in the ring, to all
                const uint32_t from = __ffs(__ballot_sync(FULL_MASK, elect_one())) - 1;
                s = __shfl_sync(FULL_MASK, s, from);
                p = __shfl_sync(FULL_MASK, p, from);
                round0 = __shfl_sync(FULL_MASK, round0, from);
                failed = __shfl_sync(FULL_MASK, failed, from);
            }
        } else if (warp == MMA_WARP) {
            // one thread issues
            if (elect_one()) {
                uint32_t s = 0, p = 0, d = 0, pd = 1;
                bool round0 = true;
                for (long long it = first; it < nitems && !failed; it += stride) {
                    for (int c = 0; c < a.kb; ++c) {
                        // Both barriers looked at together: this thread's own latency counts.
                        // What they hand over is read by the MMAs alone (operands that copies
                        // brought) or is tensor memory, which the tcgen05 fences order.
                        const bool r0 = mbar_test<1>(full + 8 * s, p), r1 = round0 || mbar_test<1>(dempty + 8 * d, pd);
                        if (!(r0 && r1) && !(mbar_wait_bounded(full + 8 * s, p, a.status, 3u) &&
                                             (round0 || mbar_wait_bounded(dempty + 8 * d, pd, a.status, 4u)))) {
                            failed = true;
                            break;
                        }
                        tc_fence_after();
                        const uint64_t xd = desc_sw128(x0 + s * X_BYTES), wd = desc_sw128(w0 + s * W_BYTES);
#pragma unroll
                        for (int kk = 0; kk < F8_BLOCK / 32; ++kk) mma_f8(tmem + d * NT, xd + kk * 2, wd + kk * 2, kk != 0);
                        mma_commit(dfull + 8 * d);
                        mma_commit(empty + 8 * s);
                        if (++s == ST) {
                            s = 0;
                            p ^= 1u;
                        }
                        if (++d == D) {
                            d = 0;
                            pd ^= 1u;
                            round0 = false;
                        }
                    }
                }
            }
            failed = __any_sync(FULL_MASK, failed);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        // warp w: tensor-memory lanes 32 (w % 4) .. + 31 = rows of this CTA's share, the
        // columns of weights 128 (w / 4) .. + 127 of the tile's
        const int q = warp & 3, h = warp >> 2;
        const bool v4 = (a.kb & 3) == 0 && (reinterpret_cast<uintptr_t>(a.xs) & 15u) == 0;
        T *y = static_cast<T *>(a.y);
        const uint32_t mine = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(h * 128);
        uint32_t d = 0, pd = 0;
        for (long long it = first; it < nitems && !failed; it += stride) {
            const Tile t = tile_at(a, static_cast<int>(it / a.groups), ntiles);
            const int nblk = static_cast<int>(it % a.groups) * 2 + h;
            const int r = q * 32 + lane;  // of the tile
            const bool some = q * 32 < t.rows;
            const int src = r < t.rows ? source_row(a.order, a.k, a.nsrc, t.row0 + r, a.status) : -1;
            const float *xs = src >= 0 ? a.xs + static_cast<size_t>(src) * a.kb : nullptr;  // no source: a scale of 0
            const float *ws = a.ws + (static_cast<size_t>(t.expert) * a.nb + min(nblk, a.nb - 1)) * a.kb;
            auto scales4 = [&](int c) {  // the row's, of blocks c .. c + 3, c a multiple of 4
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (!xs || c >= a.kb) return v;
                if (v4) return *reinterpret_cast<const float4 *>(xs + c);
                v.x = xs[c];
                if (c + 1 < a.kb) v.y = xs[c + 1];
                if (c + 2 < a.kb) v.z = xs[c + 2];
                if (c + 3 < a.kb) v.w = xs[c + 3];
                return v;
            };
            float2 acc[4][16];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[j][i] = make_float2(0.f, 0.f);
            float4 xv = make_float4(0.f, 0.f, 0.f, 0.f), next = scales4(0);
            float wl = 0.f;  // the weights' scales, a block a lane
            for (int c = 0; c < a.kb; ++c) {
                if ((c & 31) == 0) wl = c + lane < a.kb ? ws[c + lane] : 0.f;
                if ((c & 3) == 0) {
                    xv = next;
                    next = scales4(c + 4);
                }
                const float f = ((c & 2) ? ((c & 1) ? xv.w : xv.z) : ((c & 1) ? xv.y : xv.x)) * __shfl_sync(FULL_MASK, wl, c & 31);
                if (!__all_sync(FULL_MASK, mbar_test<1>(dfull + 8 * d, pd)) &&
                    !__all_sync(FULL_MASK, mbar_wait_bounded(dfull + 8 * d, pd, a.status, 6u))) {
                    failed = true;
                    break;
                }
                tc_fence_after();
                if (some) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float v[32];
                        tmem_ld32(mine + d * NT + 32 * j, v);
                        tmem_loaded(v);
#pragma unroll
                        for (int i = 0; i < 16; ++i) fma2(acc[j][i], v[2 * i], v[2 * i + 1], f);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(dempty + 8 * d);
                if (++d == D) {
                    d = 0;
                    pd ^= 1u;
                }
            }
            if (failed) break;
            const int n0 = nblk * 128;
            if (WHOLE) {
                T *row = y + static_cast<size_t>(t.row0 + r) * a.N + n0;
                if (r < t.rows) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) store32(row + 32 * j, acc[j], a.N - n0 - 32 * j);
                }
            } else if (some) {
                T *rows = y + static_cast<size_t>(t.row0 + q * 32) * a.N + n0;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    store32_anywhere(rows + 32 * j, acc[j], a.N - n0 - 32 * j, a.N, t.rows - q * 32, out0 + warp * 32 * OUT_PITCH);
            }
        }
    }
    tc_fence_before();
    if (__syncthreads_or(failed)) {
        // a wait gave up: outputs are unspecified, and what this CTA started
        // (at most a ring of copies and MMAs) gets a bounded time to land
        const long long t0 = clock64();
        while (clock64() - t0 < 2000000LL) __nanosleep(1000);
        __syncthreads();
    }
    if (warp == MMA_WARP) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

template <typename T, bool WHOLE>
cudaError_t launch_t(const RowsArgs &a, long long most_items, int sms, cudaStream_t stream)
{
    constexpr size_t smem = rows_smem(WHOLE);
    static_assert(smem <= 227 * 1024, "shared memory of a CTA");
    auto k = f8_rows<T, WHOLE>;
    // one size for every launch of this kernel: asked for once per device
    static std::atomic<bool> opted[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!opted[dev].load(std::memory_order_relaxed)) {
        const cudaError_t e = ensure_dynamic_smem(k, smem);
        if (e != cudaSuccess) return e;
        opted[dev].store(true, std::memory_order_relaxed);
    }
    const long long ctas = most_items < sms ? most_items : sms;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(ROWS_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, a);
}

}  // namespace

cudaError_t launch_f8_rows(const F8Call &c, const int *ntiles, const Tile *tiles, int max_tiles, cudaStream_t stream)
{
    const DeviceInfo *dev = device_info();
    unsigned *status = device_status_word();
    if (!dev || !status) return cudaErrorInvalidDevice;
    RowsArgs a = {};
    if (!encode(&a.wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, c.wq, c.K, static_cast<long long>(c.n) * c.N, F8_BLOCK, NT) ||
        !encode(&a.xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, c.xq, c.K, c.nsrc, F8_BLOCK, c.order ? 1 : BOX))
        return cudaErrorInvalidValue;
    a.ws = c.ws;
    a.xs = c.xs;
    a.order = c.order;
    a.y = c.y;
    a.ntiles = ntiles;
    a.tiles = c.offsets ? tiles : nullptr;
    a.status = status;
    a.R = c.R;
    a.N = c.N;
    a.kb = (c.K + F8_BLOCK - 1) / F8_BLOCK;
    a.nb = (c.N + F8_BLOCK - 1) / F8_BLOCK;
    a.k = c.k;
    a.nsrc = c.nsrc;
    a.groups = (c.N + NT - 1) / NT;
    const int nd = (c.R + MT - 1) / MT;  // equal tiles: an item costs a full one whatever its rows
    a.step = (c.R + nd - 1) / nd;
    const long long most = static_cast<long long>(c.offsets ? max_tiles : nd) * a.groups;
    const int sms = dev->sm_count;
    if (c.dtype == SMOE_BF16)
        return c.N % 8 == 0 ? launch_t<__nv_bfloat16, true>(a, most, sms, stream) : launch_t<__nv_bfloat16, false>(a, most, sms, stream);
    return c.N % 4 == 0 ? launch_t<float, true>(a, most, sms, stream) : launch_t<float, false>(a, most, sms, stream);
}

}  // namespace smoe
