// The 8-bit floating-point product with a scale for each block of 128 on single CTAs,
// for batches that are bound by reading the weights (tcgen05, kind::f8f6f4, e4m3
// operands from shared memory):
//   y[r][n] = sum_b xs[r][b] ws[e][n / 128][b] sum_{c in b} xq[r][c] wq[e][n][c].
// Larger batches go on to f8_rows.cu, after the tile list that is made here.
//
// The scales change every 128 columns, inside the sum, so each block's products are a
// sum of their own in tensor memory: the MMAs of a block write one accumulator (of
// eight), the epilogue warps read it and add it to their registers, times the block's
// scales, while the next blocks' MMAs run.  The sums of blocks are f32 in registers; a
// block's own is the tensor core's f32.
//
// The weights are the MMA's M side (128 rows of one expert: one scale a block), up to
// 64 activation rows its N side, so that a few rows cost a few columns.  The
// accumulator is read in the shape 16x128b, where a thread holds every fourth column of
// four rows: the scales of its columns (the activation rows') are then read from shared
// memory once for four products.
//
// Persistent: CTAs walk the items (tile of rows, 128 weights) with a deep ring of
// weights; few items are split over clusters along the columns, whose CTAs add their
// sums through distributed shared memory.  Roles (warps): 0-7 epilogue, 8 issues the
// MMAs, 9 streams the weights, 10 brings the row scales, 12-15 the rows (gathered by the
// copies where the batch is sorted by an order).  Every wait is bounded.
//
// Bound by reading the weights: 16 tokens through 128 experts of 1536 x 4096, k = 8 78 us
// (6.4 TB/s); one row of 8192 x 4096 9 us, of which a launch that does nothing is 3.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "f8.cuh"
#include "smoe.h"
#include "tc_pair.cuh"

namespace smoe {
namespace {

constexpr int MT = 128;                      // weight rows per CTA tile
constexpr uint32_t W_BYTES = MT * F8_BLOCK;  // a block of columns of them
constexpr int EPI_WARPS = 8, MMA_WARP = 8, W_WARP = 9, S_WARP = 10, X_WARP = 12, X_WARPS = 4;
constexpr int TC_THREADS = (X_WARP + X_WARPS) * 32;
constexpr int SLOTS = 8;                     // blocks whose row scales are on hand
// A warp's place for 8 rows of 32 outputs on their way out: rows of 32 elements
// and 16 bytes (the 16-byte reads of eight lanes then meet no bank twice).
constexpr uint32_t OUT_BYTES = 8 * (32 * 4 + 16);

constexpr int NT = 64, ST = 8, D = 8;        // rows of a tile, stages of the operands, accumulators
constexpr int CB = 32, G = CB / 4;           // columns of an epilogue warp, every fourth a thread
constexpr uint32_t X_BYTES = NT * F8_BLOCK;
constexpr int BOX = 16;                      // rows of one copy (not gathered)
constexpr int OWN_TILES = 288;               // of a list that every CTA makes for itself
constexpr size_t tc_smem(bool own)
{
    return 1024 + ST * (W_BYTES + X_BYTES) + SLOTS * NT * 4 + EPI_WARPS * OUT_BYTES + NT * 4 + 512 + (own ? OWN_TILES * sizeof(Tile) : 0);
}

struct alignas(128) TcArgs {
    CUtensorMap wmap, xmap;
    const float *ws, *xs;  // scales [n x nb x kb], [nsrc x kb]
    void *y;
    const int *ntiles;
    const Tile *tiles;     // the list that f8_prep made; or null
    const int *offsets;    // to make it of here (OWN: at most OWN_TILES); both null: one matrix, tiles of `step` rows
    int n, max_tiles;
    const int *order;      // source of every sorted row, times k (gathered), or null
    unsigned *status;
    int R, N, kb, nb, k, nsrc, step, mtiles;
    int nsplit;            // CTAs that share an item's K range
};

// Instruction descriptor, kind::f8f6f4: f32 accumulate, A and B e4m3, K-major.
__device__ __forceinline__ uint32_t idesc_e4m3(int m, int n)
{
    return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

__device__ __forceinline__ void mma_f8(uint32_t tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// 16 tensor-memory lanes (from that of the address on) by 32 columns: v[2 i] is
// row lane / 4, column 4 i + lane % 4, v[2 i + 1] row lane / 4 + 8 of it.
__device__ __forceinline__ void tmem_ld_16x128(uint32_t at, uint32_t (&v)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.16x128b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
                   "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]),
                   "=r"(v[15])
                 : "r"(at));
}
// Waits for this thread's loads; what they load goes through it, so that no use
// of it is moved before it.
__device__ __forceinline__ void tmem_loaded(uint32_t (&v)[16], uint32_t (&w)[16])
{
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        asm volatile("" : "+r"(v[i]));
        asm volatile("" : "+r"(w[i]));
    }
}

// a += d f, two at a time.
__device__ __forceinline__ void fma2(float2 &a, uint32_t d0, uint32_t d1, float f)
{
    asm("{\n\t.reg .b64 d, f, a;\n\tmov.b64 d, {%2, %3};\n\tmov.b64 f, {%4, %4};\n\tmov.b64 a, {%0, %1};\n\t"
        "fma.rn.f32x2 a, d, f, a;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "+f"(a.x), "+f"(a.y)
        : "r"(d0), "r"(d1), "f"(f));
}

__device__ __forceinline__ float4 lds128f(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void sts32(uint32_t addr, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory"); }
__device__ __forceinline__ void sts_out(uint32_t addr, float v, float *) { sts32(addr, v); }
__device__ __forceinline__ void sts_out(uint32_t addr, float v, __nv_bfloat16 *)
{
    asm volatile("st.shared.b16 [%0], %1;" ::"r"(addr), "h"(__bfloat16_as_ushort(__float2bfloat16_rn(v))) : "memory");
}

// Where row c stands among the scales as they are read: of each 32, every fourth
// one's after one another.
__device__ __forceinline__ int scale_at(int c) { return (c & ~31) + (c & 3) * 8 + (c & 31) / 4; }

__device__ __forceinline__ Tile tile_at(const TcArgs &a, const Tile *tiles, int i, int ntiles)
{
    if (i >= ntiles) return Tile{0, 0, 0, 0};
    if (tiles) return tiles[i];
    return Tile{0, i * a.step, min(a.step, a.R - i * a.step), 0};
}

// Zeros in the rows of y past the last expert's, by thread `at` of `step`: whole 16
// bytes (y begins at such a boundary), and what is before and after them.
__device__ __forceinline__ void zero_tail(void *out, int last, int R, size_t pitch, size_t at, size_t step)
{
    const size_t from = max(0, min(last, R)) * pitch, end = R * pitch;
    const size_t lo = min(end, (from + 15) & ~static_cast<size_t>(15)), hi = max(lo, end & ~static_cast<size_t>(15));
    uint8_t *y = static_cast<uint8_t *>(out);
    for (size_t i = lo + at * 16; i < hi; i += step * 16) *reinterpret_cast<uint4 *>(y + i) = make_uint4(0u, 0u, 0u, 0u);
    if (at < 16) {
        if (from + at < lo) y[from + at] = 0;
        if (hi + at < end) y[hi + at] = 0;
    }
}

// WHOLE: every row of y begins at a 16-byte boundary.  OWN: the tile list is made here
// (its code in every kernel cost a matrix and one row 0.3 us of 9).
template <typename T, bool WHOLE, bool OWN>
__global__ void __launch_bounds__(TC_THREADS, 1) f8_tc(const __grid_constant__ TcArgs a)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t w0 = base, x0 = w0 + ST * W_BYTES, f0 = x0 + ST * X_BYTES, out0 = f0 + SLOTS * NT * 4,
                   list0 = out0 + EPI_WARPS * OUT_BYTES, bars = list0 + NT * 4, own0 = bars + 512;
    const uint32_t full = bars, empty = full + 8 * ST, sfull = empty + 8 * ST, sempty = sfull + 8 * SLOTS,
                   dfull = sempty + 8 * SLOTS, dempty = dfull + 8 * D, tslot = dempty + 8 * D;
    static_assert(16 * (ST + SLOTS + D) + 4 <= 512 && D * NT <= 512, "barriers; tensor memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nsplit = a.nsplit;
    const int krank = nsplit > 1 ? static_cast<int>(blockIdx.x) % nsplit : 0;  // = the rank in the cluster
    const int first = static_cast<int>(blockIdx.x) / nsplit, stride = static_cast<int>(gridDim.x) / nsplit;

    static_assert(ST == SLOTS && ST == D, "a thread for each place of the rings");
    if (threadIdx.x < ST) {
        const uint32_t i = 8 * threadIdx.x;
        mbar_init(full + i, 1 + (a.order ? X_WARPS : 1));  // the loading warps
        mbar_init(empty + i, 1);
        mbar_init(sfull + i, 1);
        mbar_init(sempty + i, EPI_WARPS);
        mbar_init(dfull + i, 1);
        mbar_init(dempty + i, EPI_WARPS);
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

    const int c0 = krank * a.kb / nsplit, c1 = (krank + 1) * a.kb / nsplit;  // this CTA's blocks (columns past K are zeros)
    // One matrix: this CTA's first weights are known, and are brought into L2 while
    // the previous kernel ends.  A prefetch only: that kernel may be the one that
    // quantises these weights.
    if (!OWN && !a.tiles && warp == W_WARP && first < (a.R + a.step - 1) / a.step * a.mtiles && lane < ST && c0 + lane < c1)
        tma_prefetch_2d(&a.wmap, (c0 + lane) * F8_BLOCK, first % a.mtiles * MT);
    pdl_wait();
    const Tile *tiles = a.tiles;
    int ntiles = 0;
    if (OWN) {
        __shared__ int count;
        Tile *own = reinterpret_cast<Tile *>(smem_raw + (own0 - raw));
        list_tiles<TC_THREADS>(a.offsets, a.n, a.R, NT, 16, a.max_tiles, &count, own, a.status);
        zero_tail(a.y, a.offsets[a.n], a.R, static_cast<size_t>(a.N) * sizeof(T),
                  static_cast<size_t>(blockIdx.x) * TC_THREADS + threadIdx.x, static_cast<size_t>(gridDim.x) * TC_THREADS);
        __syncthreads();
        tiles = own;
        ntiles = count;
    } else {
        ntiles = tiles ? *a.ntiles : (a.R + a.step - 1) / a.step;
    }
    const int nitems = ntiles * a.mtiles;  // (below 2^28: y or the weights would not fit the device)
    bool failed = false;

    if (warp >= MMA_WARP) {
        if (warp == W_WARP) {
            if (elect_one()) {
                uint32_t s = 0, p = 1;  // parity of the stage's release one lap ago; none in the first
                bool round0 = true;
                for (int it = first; it < nitems && !failed; it += stride) {
                    const Tile t = tile_at(a, tiles, it / a.mtiles, ntiles);
                    const int row = t.expert * a.N + it % a.mtiles * MT;
                    for (int c = c0; c < c1; ++c) {
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
            // Gathered: each of the four warps loads every fourth four rows of every stage.
            const int part = warp - X_WARP;
            int *list = reinterpret_cast<int *>(smem_raw + (list0 - raw)) + part * (NT / 4);
            uint32_t s = 0, p = 1;
            bool round0 = true;
            for (int it = first; it < nitems && !failed; it += stride) {
                const Tile t = tile_at(a, tiles, it / a.mtiles, ntiles);
                const int cols = mma_cols<1>(t.rows);  // a multiple of 16
                if (a.order) {  // rows past the tile's: any row, their columns are not stored
                    const int at = 16 * (lane >> 2) + 4 * part + (lane & 3);
                    __syncwarp();
                    if (at < NT) list[lane] = at < t.rows ? max(source_row(a.order, a.k, a.nsrc, t.row0 + at, a.status), 0) : 0;
                    __syncwarp();
                }
                if (elect_one()) {
                    const int copies = a.order ? cols / 16 : (cols + BOX - 1) / BOX;
                    const uint32_t bytes = static_cast<uint32_t>(a.order ? cols / 4 : copies * BOX) * F8_BLOCK;
                    for (int c = c0; c < c1; ++c) {
                        if (!round0 && !mbar_wait_bounded(empty + 8 * s, p, a.status, 8u)) {
                            failed = true;
                            break;
                        }
                        const uint32_t dst = x0 + s * X_BYTES, bar = full + 8 * s;
                        mbar_arrive_expect_tx(bar, bytes);
                        if (a.order) {
                            for (int i = 0; i < copies; ++i) {
                                const int4 r = *reinterpret_cast<const int4 *>(list + 4 * i);
                                tma_gather4(dst + static_cast<uint32_t>(16 * i + 4 * part) * F8_BLOCK, &a.xmap, c * F8_BLOCK, r, bar);
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
            if (elect_one()) {  // one thread issues
                uint32_t s = 0, p = 0, d = 0, pd = 1;
                bool round0 = true;
                for (int it = first; it < nitems && !failed; it += stride) {
                    const Tile t = tile_at(a, tiles, it / a.mtiles, ntiles);
                    const uint32_t idesc = idesc_e4m3(MT, mma_cols<1>(t.rows));
                    for (int c = c0; c < c1; ++c) {
                        // both barriers looked at together: this thread's own latency counts
                        const bool r0 = mbar_test<1>(full + 8 * s, p), r1 = round0 || mbar_test<1>(dempty + 8 * d, pd);
                        if (!(r0 && r1) && !(mbar_wait_bounded(full + 8 * s, p, a.status, 3u) &&
                                             (round0 || mbar_wait_bounded(dempty + 8 * d, pd, a.status, 4u)))) {
                            failed = true;
                            break;
                        }
                        tc_fence_after();
                        const uint64_t wd = desc_sw128(w0 + s * W_BYTES), xd = desc_sw128(x0 + s * X_BYTES);
#pragma unroll
                        for (int kk = 0; kk < F8_BLOCK / 32; ++kk)
                            mma_f8(tmem + d * NT, wd + kk * 2, xd + kk * 2, idesc, kk != 0);
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
        } else if (warp == S_WARP) {
            // a lane brings the scales of two rows of the tile, times the weights', four
            // blocks of columns a load
            const bool v4 = (a.kb & 3) == 0 && ((reinterpret_cast<uintptr_t>(a.xs) | reinterpret_cast<uintptr_t>(a.ws)) & 15u) == 0;
            auto scales4 = [&](const float *row, int c, float (&v)[4]) {  // of blocks c .. c + 3, c a multiple of 4
                if (v4) {
                    const float4 f = *reinterpret_cast<const float4 *>(row + c);
                    v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = c + i < a.kb ? row[c + i] : 0.f;
                }
            };
            uint32_t s = 0, p = 1;
            bool round0 = true;
            for (int it = first; it < nitems && !failed; it += stride) {
                const Tile t = tile_at(a, tiles, it / a.mtiles, ntiles);
                const float *ws = a.ws + (static_cast<size_t>(t.expert) * a.nb + it % a.mtiles) * a.kb;
                const float *xs[2];  // null: no source, a scale of 0
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int c = i * 32 + lane;
                    const int src = c < t.rows ? source_row(a.order, a.k, a.nsrc, t.row0 + c, a.status) : -1;
                    xs[i] = src >= 0 ? a.xs + static_cast<size_t>(src) * a.kb : nullptr;
                }
                for (int c4 = c0 & ~3; c4 < c1 && !failed; c4 += 4) {
                    float w[4], x[2][4] = {};
                    scales4(ws, c4, w);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (xs[i]) scales4(xs[i], c4, x[i]);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        if (c4 + q < c0 || c4 + q >= c1) continue;
                        if (!__all_sync(FULL_MASK, round0 || mbar_wait_bounded(sempty + 8 * s, p, a.status, 9u))) {
                            failed = true;
                            break;
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            sts32(f0 + s * (NT * 4) + static_cast<uint32_t>(scale_at(i * 32 + lane)) * 4u, x[i][q] * w[q]);
                        __syncwarp();
                        if (lane == 0) mbar_arrive(sfull + 8 * s);
                        if (++s == SLOTS) {
                            s = 0;
                            p ^= 1u;
                            round0 = false;
                        }
                    }
                }
            }
        }
    } else {
        // warp w: tensor-memory lanes 32 (w % 4) .. + 31 = weight rows, columns
        // 32 (w / 4) .. + 31 = rows of the tile
        const int q = warp & 3, col = (warp >> 2) * CB;
        T *y = static_cast<T *>(a.y);
        const uint32_t mine = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(col);
        uint32_t d = 0, pd = 0, s = 0, p = 0;
        for (int it = first; it < nitems && !failed; it += stride) {
            const Tile t = tile_at(a, tiles, it / a.mtiles, ntiles);
            float2 acc[G][2];  // column 4 g + lane % 4 of rows lane / 4 + 16 i and + 8
#pragma unroll
            for (int g = 0; g < G; ++g) acc[g][0] = acc[g][1] = make_float2(0.f, 0.f);
            for (int c = c0; c < c1; ++c) {
                const bool r0 = mbar_test<1>(sfull + 8 * s, p), r1 = mbar_test<1>(dfull + 8 * d, pd);
                if (!__all_sync(FULL_MASK, r0 && r1) &&
                    !__all_sync(FULL_MASK, mbar_wait_bounded(sfull + 8 * s, p, a.status, 6u) && mbar_wait_bounded(dfull + 8 * d, pd, a.status, 6u))) {
                    failed = true;
                    break;
                }
                tc_fence_after();
                if (col < t.rows) {
                    uint32_t lo[2 * G], hi[2 * G];
                    tmem_ld_16x128(mine + d * NT, lo);
                    tmem_ld_16x128(mine + (16u << 16) + d * NT, hi);
                    const uint32_t fs = f0 + s * (NT * 4) + static_cast<uint32_t>(col + (lane & 3) * G) * 4u;
                    const float4 f0123 = lds128f(fs), f4567 = lds128f(fs + 16u);
                    const float f[G] = {f0123.x, f0123.y, f0123.z, f0123.w, f4567.x, f4567.y, f4567.z, f4567.w};
                    tmem_loaded(lo, hi);
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        fma2(acc[g][0], lo[2 * g], lo[2 * g + 1], f[g]);
                        fma2(acc[g][1], hi[2 * g], hi[2 * g + 1], f[g]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(dempty + 8 * d);
                    mbar_arrive(sempty + 8 * s);
                }
                if (++d == D) {
                    d = 0;
                    pd ^= 1u;
                }
                if (++s == SLOTS) {
                    s = 0;
                    p ^= 1u;
                }
            }
            if (failed) break;
            const int n0 = it % a.mtiles * MT + q * 32;
            if (nsplit > 1) {  // this K range's sums [row][128], for the reduction below
#pragma unroll
                for (int g = 0; g < G; ++g)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int r = col + 4 * g + (lane & 3);
                        const uint32_t to = x0 + static_cast<uint32_t>(r * MT + q * 32 + (lane >> 2) + 16 * i) * 4u;
                        if (r < t.rows) {
                            sts32(to, acc[g][i].x);
                            sts32(to + 32u, acc[g][i].y);
                        }
                    }
                continue;
            }
            // 8 rows at a time through shared memory
            constexpr uint32_t PITCH = 32 * sizeof(T) + 16;
            const uint32_t stage = out0 + warp * OUT_BYTES;
#pragma unroll
            for (int g0 = 0; g0 < G; g0 += 2) {
                const int r0 = col + 4 * g0;
                if (r0 >= t.rows) break;
                __syncwarp();
#pragma unroll
                for (int g = 0; g < 2; ++g)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t to = stage + static_cast<uint32_t>(4 * g + (lane & 3)) * PITCH +
                                            static_cast<uint32_t>((lane >> 2) + 16 * i) * static_cast<uint32_t>(sizeof(T));
                        sts_out(to, acc[g0 + g][i].x, y);
                        sts_out(to + 8 * static_cast<uint32_t>(sizeof(T)), acc[g0 + g][i].y, y);
                    }
                __syncwarp();
                T *to = y + static_cast<size_t>(t.row0 + r0) * a.N + n0;
                if (WHOLE) store_units<uint4, 8, 32>(stage, PITCH, to, a.N, t.rows - r0, a.N - n0);
                else store_staged<8, 32>(stage, PITCH, to, a.N, t.rows - r0, a.N - n0);
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
    if (nsplit > 1) {
        // The cluster is an item's K ranges, each CTA's sums [row][128] in the shared
        // memory of its row stages: every CTA adds every nsplit-th row of all of
        // them, in rank order, and stores it.
        static_assert(NT * MT * 4 <= ST * X_BYTES, "the sums of a tile");
        cluster_sync();
        if (first < nitems) {
            const Tile t = tile_at(a, tiles, first / a.mtiles, ntiles);
            const int nb = (first % a.mtiles) * MT;
            T *y = static_cast<T *>(a.y);
            for (int i = threadIdx.x; i < (t.rows - krank + nsplit - 1) / nsplit * (MT / 4); i += TC_THREADS) {
                const int r = krank + i / (MT / 4) * nsplit, n = nb + i % (MT / 4) * 4;
                const uint32_t at = x0 + static_cast<uint32_t>(r * MT + n - nb) * 4u;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int k = 0; k < nsplit; ++k) {
                    const float4 o = ld_dsmem_f32x4(mapa_shared(at, k));
                    v.x += o.x;
                    v.y += o.y;
                    v.z += o.z;
                    v.w += o.w;
                }
                const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (n + j < a.N) put(y + static_cast<size_t>(t.row0 + r) * a.N + n + j, f[j]);
            }
        }
    }
    if (nsplit > 1) cluster_sync();  // no CTA leaves while another reads its sums
    if (warp == MMA_WARP) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

// ---------------------------------------------------------------- preparation

constexpr int PREP_THREADS = 256;

struct PrepArgs {
    const int *offsets;
    void *y;
    int *ntiles;
    Tile *tiles;
    unsigned *status;
    int R, n, N, nt, unit, max_tiles, elem;  // elem: bytes of an element of y
};

// Block 0: the tile list.  The others: zeros in the rows of y past the last
// expert's.
__global__ void __launch_bounds__(PREP_THREADS) f8_prep(const PrepArgs a)
{
    pdl_launch_dependents();
    pdl_wait();
    if (blockIdx.x == 0) {
        list_tiles<PREP_THREADS>(a.offsets, a.n, a.R, a.nt, a.unit, a.max_tiles, a.ntiles, a.tiles, a.status);
        return;
    }
    zero_tail(a.y, a.offsets[a.n], a.R, static_cast<size_t>(a.N) * a.elem,
              static_cast<size_t>(blockIdx.x - 1) * PREP_THREADS + threadIdx.x, static_cast<size_t>(gridDim.x - 1) * PREP_THREADS);
}

// ---------------------------------------------------------------- host

// Whether f8_rows.cu takes the product, in row tiles of 128 and 256 weights.  An item
// of its takes about twice as long as one of 64 rows and 128 weights (full or not), so
// it does where it needs less than half the rounds over the device, with half a tile an
// expert left over on average.  In us, this form and that, one matrix of 8192 x 4096:
// 128 rows 12.2 and 21.1, 256 rows 20.5 and 21.2, 384 rows 28.7 and 21.6, 1024 rows 61
// and 40; of 1536 x 4096: 1024 rows 19.4 and 21.4, 1999 rows 27.9 and 22.5; 128 experts
// of it, k = 8: 512 tokens 131 and 146, 800 tokens 152 and 150, 2048 tokens 297 and 188.
bool by_rows(int R, int n, bool one, int N, int sms)
{
    const auto rounds = [&](int rows, int cols) {
        const long long tiles = one ? (R + rows - 1) / rows : std::max(std::min(R, n), R / rows + n / 2);
        return (tiles * ((N + cols - 1) / cols) + sms - 1) / sms;
    };
    return rounds(NT, MT) > 2 * rounds(128, 256);
}

template <typename T, bool WHOLE, bool OWN>
cudaError_t launch_t(const TcArgs &args, long long most_items, int sms, cudaStream_t stream)
{
    constexpr size_t smem = tc_smem(OWN);
    static_assert(smem <= 226 * 1024, "shared memory of a CTA, with the list's sums");
    auto k = f8_tc<T, WHOLE, OWN>;
    // one size for every launch of this kernel: asked for once per device
    static std::atomic<bool> opted[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!opted[dev].load(std::memory_order_relaxed)) {
        const cudaError_t e = ensure_dynamic_smem(k, smem);
        if (e != cudaSuccess) return e;
        opted[dev].store(true, std::memory_order_relaxed);
    }
    // Few items: their K ranges are split over clusters of 2, 4 or 8 CTAs, as many as
    // the device holds at once, from 16 blocks on.  1536 x 4096: one row 9.2 -> 5.8 us,
    // 192 rows 10.8 -> 8.3 us; of 8 blocks (1024 x 1024, 128 rows) 5.1 -> 6.4 us: the
    // sum over the cluster costs more than the blocks that it saves.
    int size = 1;
    for (int s = 8; s > 1; s /= 2)
        if (most_items * s <= sms && args.kb >= 16 && most_items <= clusters_held<f8_tc<T, WHOLE, OWN>>(s, TC_THREADS, smem)) {
            size = s;
            break;
        }
    TcArgs a = args;
    a.nsplit = size;
    const long long clusters = most_items < sms / size ? most_items : sms / size;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * size));
    cfg.blockDim = dim3(TC_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(size);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = size > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k, a);
}

}  // namespace

size_t f8_workspace(int R, int n) { return 256 + up256(static_cast<size_t>(most_tiles(R, n, NT)) * sizeof(Tile)); }

cudaError_t launch_f8(const F8Call &c, void *workspace, cudaStream_t stream)
{
    const DeviceInfo *dev = device_info();
    unsigned *status = device_status_word();
    if (!dev || !status) return cudaErrorInvalidDevice;
    if (c.K == 0)  // empty sums
        return cudaMemsetAsync(c.y, 0, static_cast<size_t>(c.R) * c.N * (c.dtype == SMOE_BF16 ? 2 : 4), stream);
    const int mtiles = (c.N + MT - 1) / MT;
    const bool rows = by_rows(c.R, c.n, !c.offsets, c.N, dev->sm_count);
    const int nt = rows ? 128 : NT, max_tiles = most_tiles(c.R, c.n, nt);
    int *ntiles = static_cast<int *>(workspace);
    Tile *tiles = reinterpret_cast<Tile *>(static_cast<char *>(workspace) + 256);
    // A short list is made by every CTA itself, a launch less: 3 tokens through 107 experts
    // of 940 x 1168 7.8 -> 7.0 us, 93 through 106 of 884 x 624 20.7 -> 19.8 us.
    const bool own = c.offsets && !rows && max_tiles <= OWN_TILES;
    if (c.offsets && !own) {
        const PrepArgs p = {c.offsets, c.y, ntiles, tiles, status, c.R, c.n, c.N, nt, 16, max_tiles, c.dtype == SMOE_BF16 ? 2 : 4};
        const cudaError_t e = launch_pdl(f8_prep, dim3(33), dim3(PREP_THREADS), 0, stream, p);
        if (e != cudaSuccess) return e;
    }
    if (rows) return launch_f8_rows(c, ntiles, tiles, max_tiles, stream);

    // one matrix: equal tiles of consecutive rows
    const int nd = (c.R + NT - 1) / NT, step = ((c.R + nd - 1) / nd + 15) / 16 * 16;
    TcArgs a = {};
    if (!encode(&a.wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, c.wq, c.K, static_cast<long long>(c.n) * c.N, F8_BLOCK, MT) ||
        !encode(&a.xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, c.xq, c.K, c.nsrc, F8_BLOCK, c.order ? 1 : BOX))
        return cudaErrorInvalidValue;
    a.ws = c.ws;
    a.xs = c.xs;
    a.order = c.order;
    a.y = c.y;
    a.ntiles = ntiles;
    a.tiles = c.offsets && !own ? tiles : nullptr;
    a.offsets = own ? c.offsets : nullptr;
    a.n = c.n;
    a.max_tiles = max_tiles;
    a.status = status;
    a.R = c.R;
    a.N = c.N;
    a.kb = (c.K + F8_BLOCK - 1) / F8_BLOCK;
    a.nb = (c.N + F8_BLOCK - 1) / F8_BLOCK;
    a.k = c.k;
    a.nsrc = c.nsrc;
    a.step = step;
    a.mtiles = mtiles;
    const long long most = static_cast<long long>(c.offsets ? max_tiles : nd) * mtiles;
    const int sms = dev->sm_count;
    const auto go = [&](auto zero, auto whole) {
        using T = decltype(zero);
        return own ? launch_t<T, whole.value, true>(a, most, sms, stream) : launch_t<T, whole.value, false>(a, most, sms, stream);
    };
    const auto typed = [&](auto zero) {
        return c.N % (16 / static_cast<int>(sizeof(zero))) == 0 ? go(zero, std::true_type{}) : go(zero, std::false_type{});
    };
    return c.dtype == SMOE_BF16 ? typed(__nv_bfloat16{}) : typed(float{});
}

}  // namespace smoe
