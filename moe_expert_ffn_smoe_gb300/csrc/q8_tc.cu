// The 8-bit product on the tensor cores (tcgen05):
//   y[r][n] = x_scale[r] w_scale[e][n] sum_k xq[r][k] wq[e][n][k].
//
// sm_103a has no 8-bit integer form of tcgen05.mma.  An int8 is an exact f16
// (|c| <= 128 < 2^11) and the product of two an exact f32, so kind::f16 with
// f32 accumulation carries the integers: sums are exact below 2^24.  The
// scales, one per row and one per column of y, stay outside the sum.
//
// The weights are the MMA's M side (128 rows of one expert), the activation
// rows its N side, so that any number of rows of an expert (a multiple of 16
// up to the tile's width) costs its own share of tensor-core time.  Weights
// travel as int8 all the way into the SM (half the bytes of their f16 form in
// HBM, L2 and shared memory) and are widened there into tensor memory, where
// the MMA reads its A operand; the activations, reused by every weight tile,
// are widened once by q8_prep into the workspace.
//
// q8_tc is persistent: CTAs, or pairs of them, walk the items (tile of rows,
// weight tiles), accumulators double-buffered so that the store of one item
// runs under the products of the next.  A pair (cta_group::2) multiplies 256
// weight rows at once, each CTA widening its own 128 and holding half of the
// activation rows, so that a row tile crosses from L2 once for 256 weight
// rows and its stages take half the shared memory: twice as many are in
// flight.  Rows of a batch sorted by expert are gathered by the copies
// themselves (gather4): the tokens' widened rows stay in L2, where sorted
// copies of them (k times as many) went out to HBM and back (4096 tokens, k =
// 8, 4096 columns: 50 us and a tenth of the product's time).
// Roles (warps): 0-7 epilogue, 8-23 widen weights (four groups, every
// fourth K tile each), 24 issues the MMAs (of the pair: the even CTA's), 25
// streams the weights, 26-31 the rows.  Every wait is bounded.
#include <cuda_fp16.h>

#include <atomic>

#include "cluster_table.h"
#include "q8.cuh"
#include "smoe.h"
#include "tcgen05.cuh"

namespace smoe {
namespace {

constexpr int KT = 64;                  // columns per K tile
constexpr int MT = 128;                 // weight rows per CTA tile
constexpr uint32_t W_BYTES = MT * 128;  // one weight chunk: 128 rows x 128 columns (two K tiles)
constexpr int EPI_WARPS = 8;
constexpr int CONV_WARP0 = 8, CONV_GROUPS = 4;  // groups of four warps: a row each thread
constexpr int MMA_WARP = CONV_WARP0 + 4 * CONV_GROUPS, W_WARP = MMA_WARP + 1, X_WARP = MMA_WARP + 2, X_PARTS = 3, X_WARPS = 2 * X_PARTS;
constexpr int TC_THREADS = (X_WARP + X_WARPS) * 32;

// Shapes of the two forms: row tile NT, CTAs per tile CL, and the rings of A
// stages (tensor memory, a K tile each), row stages (a CTA's share of the
// rows x two K tiles) and weight chunks (shared memory).
template <int NT>
struct Form;
template <>
struct Form<192> {
    static constexpr int CL = 2, AS = 4, XS = 6, WS = 4;
};
template <>
struct Form<64> {
    static constexpr int CL = 1, AS = 8, XS = 4, WS = 8;
};

template <int NT>
constexpr size_t tc_smem()
{
    using F = Form<NT>;
    return 1024 + static_cast<size_t>(F::WS) * W_BYTES + static_cast<size_t>(F::XS) * (NT / F::CL) * 256 + 512 +
           static_cast<size_t>(X_WARPS) * (NT / F::CL) * 4;
}

struct alignas(128) TcArgs {
    CUtensorMap wmap, xmap;
    const float *ws, *xs;  // w_scales [n x N], x scales in sorted order [R]
    void *y;
    const int *ntiles;
    const Tile *tiles;     // null: one matrix, tiles of `step` rows
    const int *srow;       // source row in xmap of every sorted row (gathered), or null
    unsigned *status;
    int R, N, K, step, mtiles, box;  // box: rows of one copy (not gathered)
    int nsplit;            // CTAs that share an item's K range (single-CTA form)
};

// Four int8 in a word as two f16 pairs: byte b + 128 in the mantissa of
// 1024, minus 1152; every value exact.
__device__ __forceinline__ void s8x4_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    const uint32_t u = w ^ 0x80808080u;
    const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    __half2 ha = __hsub2(*reinterpret_cast<__half2 *>(&a), off), hb = __hsub2(*reinterpret_cast<__half2 *>(&b), off);
    lo = *reinterpret_cast<uint32_t *>(&ha);
    hi = *reinterpret_cast<uint32_t *>(&hb);
}

// Shared-memory matrix descriptor, 128-byte swizzle, K-major: 8-row groups
// 1024 bytes apart, version 1, swizzle mode 2.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr)
{
    return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(1) << 16) |
           (static_cast<uint64_t>(1024u >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
           (static_cast<uint64_t>(2) << 61);
}

// Instruction descriptor, kind::f16: f32 accumulate, A and B f16, K-major.
__device__ __forceinline__ uint32_t idesc_f16(int m, int n)
{
    return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// The pair's form of mma_f16_ta: 256 rows of A, 128 in each CTA's tensor
// memory, B's rows split between the CTAs' shared memory at one address.
__device__ __forceinline__ void mma_f16_ta_pair(uint32_t tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem),
        "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// Arrives on the barrier at this place in both CTAs of the pair.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

// Copies into this CTA that complete on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// Four rows of a tensor map whose box is one row high, one below another.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap *map, int x, const int4 &r, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
        "%5, %6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_gather4_pair(uint32_t dst, const CUtensorMap *map, int x, const int4 &r, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, "
        "{%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w), "r"(bar)
        : "memory");
}

// Arrives on a barrier of either CTA of the cluster (a shared::cluster
// address).  What it hands over is tensor memory, ordered by the tcgen05
// fences and waits around it; a release at cluster scope would also wait for
// this thread's earlier reads and writes elsewhere (1,700 clocks a K tile
// against 500).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// mbar_wait_bounded for barriers that the other CTA's threads arrive on:
// acquires at cluster scope.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, 20000;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}
template <int CL>
__device__ __forceinline__ bool wait_pair(uint32_t bar, uint32_t parity, unsigned *status, unsigned code)
{
    if (CL == 1) return mbar_wait_bounded(bar, parity, status, code);
    if (mbar_try_wait_cluster(bar, parity)) return true;
    const long long t0 = clock64();
    for (uint32_t i = 0; i < (1u << 24); ++i) {
        __nanosleep(64);
        if (mbar_try_wait_cluster(bar, parity)) return true;
        if (clock64() - t0 > 4000000000LL) break;
    }
    atomicExch(status, code);
    return false;
}

// Whether phase `parity` has completed, without waiting.
template <int CL>
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    if (CL > 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(bar), "r"(parity)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(bar), "r"(parity)
            : "memory");
    return done != 0;
}

// Columns of the MMA for a tile of `rows`: a pair's come in 32s.
template <int CL>
__device__ __forceinline__ int mma_cols(int rows)
{
    return (rows + 16 * CL - 1) & ~(16 * CL - 1);
}

__device__ __forceinline__ Tile tile_at(const TcArgs &a, int i, int ntiles)
{
    if (i >= ntiles) return Tile{0, 0, 0, 0};
    if (a.tiles) return a.tiles[i];
    return Tile{0, i * a.step, min(a.step, a.R - i * a.step), 0};
}

template <typename T, int NT>
__global__ void __launch_bounds__(TC_THREADS, 1) q8_tc(const __grid_constant__ TcArgs a)
{
    using F = Form<NT>;
    constexpr int CL = F::CL, AS = F::AS, XS = F::XS, WS = F::WS;
    constexpr int XR = NT / CL;                            // rows of a CTA's share of a tile, at most
    constexpr uint32_t XB = XR * 128u, ACOL0 = 2u * NT;    // XB: one K tile of them; a row stage is two
    static_assert(X_PARTS <= XS, "row stages");
    static_assert(2 * NT + AS * 32 <= 512 && AS % CONV_GROUPS == 0 && WS % (CONV_GROUPS / 2) == 0,
                  "tensor memory; stages of one group of widening warps");
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t w0 = base, x0 = w0 + WS * W_BYTES, list0 = x0 + XS * 2 * XB, bars = list0 + X_WARPS * XR * 4;
    const uint32_t wfull = bars, wempty = wfull + 8 * WS, xfull = wempty + 8 * WS, xempty = xfull + 8 * XS,
                   afull = xempty + 8 * XS, aempty = afull + 8 * AS, dfull = aempty + 8 * AS, dempty = dfull + 16,
                   tslot = dempty + 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = CL > 1 ? static_cast<int>(blockIdx.x % CL) : 0;
    const int nsplit = CL > 1 ? 1 : a.nsplit;
    const int krank = nsplit > 1 ? static_cast<int>(blockIdx.x) % nsplit : 0;  // = the rank in the cluster
    const int first = static_cast<int>(blockIdx.x) / (CL * nsplit), stride = static_cast<int>(gridDim.x) / (CL * nsplit);

    if (threadIdx.x == 0) {
        for (int i = 0; i < WS; ++i) {
            mbar_init(wfull + 8 * i, 1);
            mbar_init(wempty + 8 * i, 8);  // the eight widening warps
        }
        for (int i = 0; i < XS; ++i) {
            mbar_init(xfull + 8 * i, 2);  // the two row-loading warps of the stage; used in the issuing CTA
            mbar_init(xempty + 8 * i, 1);
        }
        for (int i = 0; i < AS; ++i) {
            mbar_init(afull + 8 * i, 4 * CL);  // one group of widening warps of every CTA; used in the issuing CTA
            mbar_init(aempty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(dfull + 8 * i, 1);
            mbar_init(dempty + 8 * i, EPI_WARPS * CL);  // used in the issuing CTA
        }
        fence_mbar_init();
    }
    if (warp == MMA_WARP) {
        if (CL > 1) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(tslot) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(tslot) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    tc_fence_before();
    __syncthreads();
    if (CL > 1) cluster_sync();  // nothing may reach a CTA whose barriers are not there yet
    tc_fence_after();
    uint32_t tmem;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(tslot));
    if (threadIdx.x == 0) pdl_launch_dependents();

    const int nch = (a.K + 127) / 128;  // weight chunks, two K tiles each (columns past K are zeros)
    const int c0 = krank * nch / nsplit, c1 = (krank + 1) * nch / nsplit;  // this CTA's
    const int mgroups = (a.mtiles + CL - 1) / CL;
    // One matrix: this CTA's first weight chunks are known, and are brought
    // into L2 while the previous kernel ends.  A prefetch only: that kernel
    // may be the one that quantises these weights.
    if (!a.tiles && warp == W_WARP && first < (a.R + a.step - 1) / a.step * mgroups && lane < WS && c0 + lane < c1)
        tma_prefetch_2d(&a.wmap, (c0 + lane) * 128, (first % mgroups * CL + rank) * MT);
    pdl_wait();
    const int ntiles = a.tiles ? *a.ntiles : (a.R + a.step - 1) / a.step;
    const long long nitems = static_cast<long long>(ntiles) * mgroups;
    bool failed = false;

    if (warp == W_WARP) {
        if (elect_one()) {
            uint32_t s = 0, p = 1;  // parity of the slot's release one lap ago; none in the first
            bool round0 = true;
            for (long long it = first; it < nitems && !failed; it += stride) {
                const Tile t = tile_at(a, static_cast<int>(it / mgroups), ntiles);
                const int row = t.expert * a.N + (static_cast<int>(it % mgroups) * CL + rank) * MT;
                for (int c = c0; c < c1; ++c) {
                    if (!round0 && !mbar_wait_bounded(wempty + 8 * s, p, a.status, 7u)) {
                        failed = true;
                        break;
                    }
                    mbar_arrive_expect_tx(wfull + 8 * s, W_BYTES);
                    tma_load_2d(w0 + s * W_BYTES, &a.wmap, c * 128, row, wfull + 8 * s);
                    if (++s == WS) {
                        s = 0;
                        p ^= 1u;
                        round0 = false;
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp >= X_WARP) {
        // A stage is two K tiles.  Each of the six warps loads one K tile of
        // every third stage: a copy costs its issuer 50 (a gather) to some
        // hundred clocks beside the other roles, and fewer issuers paced the
        // K loop.  The bytes of both CTAs complete on the issuing CTA's
        // barrier, which alone expects them.
        const uint32_t half = (warp - X_WARP) & 1, part = (warp - X_WARP) >> 1;
        const uint32_t lead = CL > 1 ? mapa_shared(xfull, 0) : xfull;
        int *list = reinterpret_cast<int *>(smem_raw + (list0 - raw)) + (warp - X_WARP) * XR;
        uint32_t s = part, p = 1, due = part;  // due: chunks until this warp's next step
        bool round0 = true;
        for (long long it = first; it < nitems && !failed; it += stride) {
            const Tile t = tile_at(a, static_cast<int>(it / mgroups), ntiles);
            const int share = mma_cols<CL>(t.rows) / CL;  // rows of this CTA's share, a multiple of 16
            const int row0 = t.row0 + rank * share;
            if (a.srow) {  // rows past the tile's: any row, their columns are not stored
                __syncwarp();
                for (int i = lane; i < share; i += 32) list[i] = rank * share + i < t.rows ? a.srow[row0 + i] : 0;
                __syncwarp();
            }
            if (elect_one()) {
                const int copies = (share + a.box - 1) / a.box;
                const uint32_t bytes = static_cast<uint32_t>(a.srow ? share : copies * a.box) * (128u * CL);
                int c = c0 + static_cast<int>(due);
                for (; c < c1; c += X_PARTS) {
                    if (!round0 && !mbar_wait_bounded(xempty + 8 * s, p, a.status, 8u)) {
                        failed = true;
                        break;
                    }
                    if (rank == 0) mbar_arrive_expect_tx(xfull + 8 * s, bytes);
                    const int x = (2 * c + static_cast<int>(half)) * KT;
                    const uint32_t dst = x0 + (2 * s + half) * XB, bar = lead + 8 * s;
                    if (a.srow) {
                        for (int i = 0; i < share; i += 16) {
                            int4 r[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) r[j] = *reinterpret_cast<const int4 *>(list + i + 4 * j);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const uint32_t to = dst + static_cast<uint32_t>(i + 4 * j) * 128u;
                                if (CL > 1) tma_gather4_pair(to, &a.xmap, x, r[j], bar);
                                else tma_gather4(to, &a.xmap, x, r[j], bar);
                            }
                        }
                    } else {
                        for (int b = 0; b < copies; ++b) {
                            const uint32_t to = dst + static_cast<uint32_t>(b * a.box) * 128u;
                            if (CL > 1) tma_load_2d_pair(to, &a.xmap, x, row0 + b * a.box, bar);
                            else tma_load_2d(to, &a.xmap, x, row0 + b * a.box, bar);
                        }
                    }
                    s += X_PARTS;
                    if (s >= XS) {
                        s -= XS;
                        p ^= 1u;
                        round0 = false;
                    }
                }
                due = static_cast<uint32_t>(c - c1);
            }
            // the elected lane's place in the ring, to all
            const uint32_t from = __ffs(__ballot_sync(FULL_MASK, elect_one())) - 1;
            s = __shfl_sync(FULL_MASK, s, from);
            p = __shfl_sync(FULL_MASK, p, from);
            due = __shfl_sync(FULL_MASK, due, from);
            round0 = __shfl_sync(FULL_MASK, round0, from);
            failed = __shfl_sync(FULL_MASK, failed, from);
        }
        // The last releases of the stages arrive here from the other CTA's
        // issue: they must have before this CTA may leave.  The first warp
        // waits for all of them.
        if (CL > 1 && !failed && warp == X_WARP) {
            const long long steps = first < nitems ? (nitems - first + stride - 1) / stride * (c1 - c0) : 0;
            for (long long g = steps > XS ? steps - XS : 0; g < steps; ++g)
                if (!mbar_wait_bounded(xempty + 8 * static_cast<uint32_t>(g % XS), static_cast<uint32_t>(g / XS) & 1,
                                       a.status, 8u))
                    failed = true;
        }
    } else if (warp == MMA_WARP) {
        // one thread issues, of a pair the even CTA's
        if (rank == 0 && elect_one()) {
            uint32_t sa = 0, pa = 0, sx = 0, px = 0, d = 0;
            for (long long it = first; it < nitems && !failed; it += stride, ++d) {
                const Tile t = tile_at(a, static_cast<int>(it / mgroups), ntiles);
                const uint32_t idesc = idesc_f16(MT * CL, mma_cols<CL>(t.rows));
                const uint32_t acc = tmem + (d & 1) * NT;
                if (d >= 2 && !wait_pair<CL>(dempty + 8 * (d & 1), (d / 2 - 1) & 1, a.status, 4u)) failed = true;
                for (int c = c0; c < c1 && !failed; ++c) {
                    // two K tiles at a time, their three barriers looked at
                    // together: this thread's own latency paces the loop
                    // where the tile is narrow
                    const bool rx = mbar_test<CL>(xfull + 8 * sx, px), r0 = mbar_test<CL>(afull + 8 * sa, pa),
                               r1 = mbar_test<CL>(afull + 8 * sa + 8, pa);
                    if (!(rx && r0 && r1) &&
                        !(wait_pair<CL>(xfull + 8 * sx, px, a.status, 3u) && wait_pair<CL>(afull + 8 * sa, pa, a.status, 3u) &&
                          wait_pair<CL>(afull + 8 * sa + 8, pa, a.status, 3u))) {
                        failed = true;
                        break;
                    }
                    tc_fence_after();
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t at = tmem + ACOL0 + (sa + h) * 32;
                        const uint64_t xd = desc_sw128(x0 + (2 * sx + h) * XB);
#pragma unroll
                        for (int kk = 0; kk < KT / 16; ++kk) {
                            if (CL > 1) mma_f16_ta_pair(acc, at + kk * 8, xd + kk * 2, idesc, c - c0 + h + kk != 0);
                            else mma_f16_ta(acc, at + kk * 8, xd + kk * 2, idesc, c - c0 + h + kk != 0);
                        }
                        if (CL > 1) mma_commit_pair(aempty + 8 * (sa + h));
                        else mma_commit(aempty + 8 * (sa + h));
                    }
                    sa += 2;
                    if (sa == AS) {
                        sa = 0;
                        pa ^= 1u;
                    }
                    if (CL > 1) mma_commit_pair(xempty + 8 * sx);
                    else mma_commit(xempty + 8 * sx);
                    if (c == c1 - 1) {
                        if (CL > 1) mma_commit_pair(dfull + 8 * (d & 1));
                        else mma_commit(dfull + 8 * (d & 1));
                    }
                    if (++sx == XS) {
                        sx = 0;
                        px ^= 1u;
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp >= CONV_WARP0 && warp < MMA_WARP) {
        // thread = one weight row; of the K tiles that this CTA streams, one
        // after another over all its items, group grp widens every fourth
        const int ct = threadIdx.x - CONV_WARP0 * 32;
        const uint32_t r = ct & (MT - 1), grp = ct >> 7, half = grp & 1;
        const uint32_t lead = CL > 1 ? mapa_shared(afull, 0) : afull;
        const long long mine = first < nitems ? (nitems - first + stride - 1) / stride : 0;
        const long long chunks = mine * (c1 - c0);
        uint32_t sw = (grp >> 1) % WS, pw = 0, sa = grp % AS, pa = 1;
        bool round0 = true;
        for (long long g = grp >> 1; g < chunks; g += CONV_GROUPS / 2) {
            if (!__all_sync(FULL_MASK, mbar_wait_bounded(wfull + 8 * sw, pw, a.status, 5u))) {
                failed = true;
                break;
            }
            // widened in registers before the stage is waited for: only the
            // store is between its release and its next use
            const uint32_t row = w0 + sw * W_BYTES + r * 128u;
            uint32_t v[2][16];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint4 q = lds128v(row + (((half * 4 + j) ^ (r & 7)) << 4));
                uint32_t *to = &v[j >> 1][8 * (j & 1)];
                s8x4_to_f16(q.x, to[0], to[1]);
                s8x4_to_f16(q.y, to[2], to[3]);
                s8x4_to_f16(q.z, to[4], to[5]);
                s8x4_to_f16(q.w, to[6], to[7]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(wempty + 8 * sw);
            if (!__all_sync(FULL_MASK, round0 || mbar_wait_bounded(aempty + 8 * sa, pa, a.status, 5u))) {
                failed = true;
                break;
            }
            tc_fence_after();
#pragma unroll
            for (int h = 0; h < 2; ++h)
                tmem_st16(tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + ACOL0 + sa * 32 + 16 * h, v[h]);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (CL > 1) mbar_arrive_cluster(lead + 8 * sa);
                else mbar_arrive(afull + 8 * sa);
            }
            sw += CONV_GROUPS / 2;
            if (sw >= WS) {
                sw -= WS;
                pw ^= 1u;
            }
            sa += CONV_GROUPS;
            if (sa >= AS) {
                sa -= AS;
                pa ^= 1u;
                round0 = false;
            }
        }
        // the last releases of this group's stages come from the even CTA
        if (CL > 1 && !failed)
            for (int j = 0; j < AS / CONV_GROUPS; ++j) {
                if (!round0 && !mbar_wait_bounded(aempty + 8 * sa, pa, a.status, 5u)) failed = true;
                sa += CONV_GROUPS;
                if (sa >= AS) {
                    sa -= AS;
                    pa ^= 1u;
                    round0 = false;
                }
            }
    } else if (warp < EPI_WARPS) {
        // warp w: TMEM lanes 32 (w % 4) .. + 31 = weight rows, the 16-column
        // blocks of parity w / 4
        const int q = warp & 3, h = warp >> 2;
        T *y = static_cast<T *>(a.y);
        const uint32_t lead = CL > 1 ? mapa_shared(dempty, 0) : dempty;
        uint32_t d = 0;
        for (long long it = first; it < nitems; it += stride, ++d) {
            const Tile t = tile_at(a, static_cast<int>(it / mgroups), ntiles);
            const int n = (static_cast<int>(it % mgroups) * CL + rank) * MT + q * 32 + lane;
            const bool nok = n < a.N;
            const float ws = nok ? a.ws[static_cast<size_t>(t.expert) * a.N + n] : 0.f;
            // the rows' scales, one lane a row of each 16-row block
            float xv[NT / 32];
#pragma unroll
            for (int j = 0; j < NT / 32; ++j) {
                const int c = h * 16 + j * 32 + (lane & 15);
                xv[j] = c < t.rows ? a.xs[t.row0 + c] : 0.f;
            }
            const bool ok = mbar_wait_bounded(dfull + 8 * (d & 1), (d / 2) & 1, a.status, 6u);
            if (!__all_sync(FULL_MASK, ok)) {
                failed = true;
                break;
            }
            tc_fence_after();
            const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16) + (d & 1) * NT;
#pragma unroll
            for (int j = 0; j < NT / 32; ++j) {
                const int c = h * 16 + j * 32;
                if (c >= t.rows) break;
                float v[16];
                tmem_ld<16>(acc + c, v);
                tmem_wait_ld();
                if (nsplit > 1) {  // this K range's sums, for the reduction below
                    const uint32_t to = x0 + static_cast<uint32_t>(c * MT + q * 32 + lane) * 4u;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        asm volatile("st.shared.f32 [%0], %1;" ::"r"(to + i * MT * 4u), "f"(v[i]) : "memory");
                    continue;
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = v[i] * __shfl_sync(FULL_MASK, xv[j], i) * ws;
                if ((a.N & 1) == 0) {
                    // neighbouring lanes trade every other row, so that each
                    // stores two columns of one row at once
                    const bool odd = lane & 1;
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const float got = __shfl_xor_sync(FULL_MASK, odd ? v[i] : v[i + 1], 1);
                        const int r = c + i + (odd ? 1 : 0);
                        if (nok && r < t.rows)
                            put2(y + static_cast<size_t>(t.row0 + r) * a.N + (n & ~1), odd ? got : v[i], odd ? v[i + 1] : got);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (nok && c + i < t.rows) put(y + static_cast<size_t>(t.row0 + c + i) * a.N + n, v[i]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (CL > 1) mbar_arrive_cluster(lead + 8 * (d & 1));
                else mbar_arrive(dempty + 8 * (d & 1));
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
        // The cluster is an item's K ranges, each CTA's sums [row][128] in
        // the shared memory of its row stages: every CTA adds every nsplit-th
        // row of all of them, in rank order, and stores it.
        static_assert(CL > 1 || NT * MT * 4u <= XS * 2 * XB, "the sums of a tile");
        cluster_sync();
        if (first < nitems) {
            const Tile t = tile_at(a, first / mgroups, ntiles);
            const int nb = (first % mgroups) * MT;
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
                const float xs = a.xs[t.row0 + r];
                const float *ws = a.ws + static_cast<size_t>(t.expert) * a.N;
                const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (n + j < a.N) put(y + static_cast<size_t>(t.row0 + r) * a.N + n + j, f[j] * xs * ws[n + j]);
            }
        }
    }
    if (CL > 1 || nsplit > 1) cluster_sync();  // no CTA leaves while another's copies, releases or reads may reach it
    if (warp == MMA_WARP) {
        tc_fence_after();
        if (CL > 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
        else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

// ---------------------------------------------------------------- preparation

constexpr int PREP_THREADS = 256;

struct PrepArgs {
    const int8_t *xq;
    const float *xs;
    const int *order, *offsets;
    __half *x16;  // [(gathered: nsrc, else R) x K]
    float *xss;   // [R]: the sorted rows' scales
    void *y;
    int *ntiles;
    Tile *tiles;
    unsigned *status;
    int *srow;    // [R]: the sorted rows' sources (gathered), or null
    int nsrc, k, R, n, K, N, nt, unit, max_tiles, zero_bytes;  // unit: MMA columns; zero_bytes: an element of y
};

// Block 0 (with offsets): the tile list, every expert's rows cut into equal
// tiles of at most nt.  The others: the activations widened to f16, the
// sorted rows' sources and scales, and zeros in the rows of y past the last
// expert's.
__global__ void __launch_bounds__(PREP_THREADS) q8_prep(const PrepArgs a)
{
    __shared__ long long warp_sums[PREP_THREADS / 32];
    __shared__ long long run_s;
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x;
    if (a.offsets && blockIdx.x == 0) {
        const int lane = tid & 31, wi = tid >> 5;
        long long run = 0;  // 64 bits: ranges that overlap (reported) can add up to more than 32
        for (int b = 0; b < a.n; b += PREP_THREADS) {
            const int e = b + tid;
            int lo = 0, hi = 0;
            if (e < a.n) {
                lo = a.offsets[e];
                hi = a.offsets[e + 1];
                if (lo < 0 || hi < lo || hi > a.R) {
                    atomicExch(a.status, kStatusRoute);
                    lo = hi = 0;
                }
            }
            int cnt = (hi - lo + a.nt - 1) / a.nt;
            const int step = cnt > 0 ? ((hi - lo + cnt - 1) / cnt + a.unit - 1) / a.unit * a.unit : a.unit;
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
            if (tid == PREP_THREADS - 1) run_s = before + inc;
            const long long t0 = before + inc - cnt;
            for (int i = 0; i < cnt && t0 + i < a.max_tiles; ++i)
                a.tiles[t0 + i] = Tile{e, lo + i * step, min(step, hi - lo - i * step), 0};
            __syncthreads();
            run = run_s;
        }
        if (tid == 0) *a.ntiles = static_cast<int>(min(run, static_cast<long long>(a.max_tiles)));
        return;
    }
    const int b0 = a.offsets ? 1 : 0, blocks = gridDim.x - b0;
    const int last = a.offsets ? max(0, min(a.offsets[a.n], a.R)) : a.R;
    for (int r = (blockIdx.x - b0) * PREP_THREADS + tid; r < a.R; r += blocks * PREP_THREADS) {
        const int src = r < last ? source_row(a.order, a.k, a.nsrc, r, a.status) : -1;
        a.xss[r] = src >= 0 ? a.xs[src] : 0.f;
        if (a.srow) a.srow[r] = max(src, 0);  // none: any row, its scale is 0
    }
    const size_t zero0 = static_cast<size_t>(last) * a.N, zero1 = static_cast<size_t>(a.R) * a.N;
    for (size_t i = zero0 + static_cast<size_t>(blockIdx.x - b0) * PREP_THREADS + tid; i < zero1;
         i += static_cast<size_t>(blocks) * PREP_THREADS) {
        if (a.zero_bytes == 4) static_cast<float *>(a.y)[i] = 0.f;
        else static_cast<uint16_t *>(a.y)[i] = 0;
    }
    // eight columns a thread, so that a warp's stores are whole sectors
    const size_t vecs = static_cast<size_t>(a.srow ? a.nsrc : last) * (a.K / 8);
    const size_t hop = static_cast<size_t>(blocks) * PREP_THREADS;
    for (size_t i = static_cast<size_t>(blockIdx.x - b0) * PREP_THREADS + tid; i < vecs; i += 4 * hop) {
        uint2 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + j * hop < vecs) v[j] = reinterpret_cast<const uint2 *>(a.xq)[i + j * hop];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + j * hop < vecs) {
                uint4 o;
                s8x4_to_f16(v[j].x, o.x, o.y);
                s8x4_to_f16(v[j].y, o.z, o.w);
                reinterpret_cast<uint4 *>(a.x16)[i + j * hop] = o;
            }
    }
}

// ---------------------------------------------------------------- host

bool encode(CUtensorMap *map, CUtensorMapDataType type, int elem, const void *p, long long cols, long long rows, int box_x,
            int box_y)
{
    EncodeTiled fn = encoder();
    if (!fn) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * elem};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_x), static_cast<cuuint32_t>(box_y)};
    const cuuint32_t estr[2] = {1u, 1u};
    return fn(map, type, 2, const_cast<void *>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

// Row tile: 64 (single CTAs, a deep ring of weights) where the product is
// bound by reading the weights or its tiles fit the device at once, 192
// (pairs) beyond.  Measured (us; K = 4096), 64 against 192: one matrix of
// 8192, 128 rows 18.9 / 20.8, 192 rows 29.2 / 24.0; of 1536, 512 rows 18.8 /
// 24.3; 128 experts of 1536, 32 rows each 157 / 170, 64 rows 199 / 186.
int pick_nt(int R, int n, bool one, int mtiles, int sms)
{
    const long long tiles = one ? (R + 63) / 64 : most_tiles(R, n, 64);
    return R <= 48LL * n || tiles * mtiles <= sms ? 64 : 192;
}

// How many tiles one matrix's R rows are cut into for pairs: as many as keep
// waves of `pairs` items on `slots` pairs of SMs shortest.  An item costs its
// rows, but no less than 144 (below, widening the weights paces it), and some
// 16 rows' time of its own.  Against the fewest tiles (us; K = 4096): N =
// 8192, 192 rows 23.9 to 21.4, 512 rows 36.9 to 34.7, 1024 rows 56.0 to 52.2;
// N = 1536, 1536 rows 30.9 to 26.8.
int pair_tiles(int R, int pairs, int slots)
{
    int best = 0;
    long long least = 0;
    for (int nd = (R + 191) / 192; nd <= (R + 95) / 96; ++nd) {
        const int step = ((R + nd - 1) / nd + 31) / 32 * 32;
        const long long waves = (static_cast<long long>((R + step - 1) / step) * pairs + slots - 1) / slots;
        const long long cost = waves * ((step > 144 ? step : 144) + 16);
        if (best == 0 || cost < least) {
            best = nd;
            least = cost;
        }
    }
    return best;
}

struct Layout {
    size_t tiles, xss, srow, x16, total;
};

Layout layout(int nsrc, int R, int n, int K)
{
    Layout l;
    l.tiles = 256;
    l.xss = l.tiles + up256(static_cast<size_t>(most_tiles(R, n, 64)) * sizeof(Tile));
    l.srow = l.xss + up256(static_cast<size_t>(R) * sizeof(float));
    l.x16 = l.srow + up256(static_cast<size_t>(R) * sizeof(int));
    l.total = l.x16 + up256(static_cast<size_t>(nsrc) * K * sizeof(__half));
    return l;
}

// Clusters of `csize` (2, 4 or 8) CTAs of a kernel that the current device
// holds at once (a cluster's CTAs share a GPC, so this may be fewer than its
// SMs divided); 0 if unknown.
template <auto Kernel>
int resident_clusters(int csize, size_t smem)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    return cluster_table<Kernel>().get(dev, csize, [&] {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(csize));
        cfg.blockDim = dim3(TC_THREADS);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(csize);
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, Kernel, &cfg) == cudaSuccess) return n;
        (void)cudaGetLastError();
        return 0;
    });
}

template <typename T, int NT>
cudaError_t launch_tc(const TcArgs &args, long long most_items, int sms, cudaStream_t stream)
{
    using F = Form<NT>;
    constexpr size_t smem = tc_smem<NT>();
    auto k = q8_tc<T, NT>;
    // one size for every launch of this kernel: asked for once per device
    static std::atomic<bool> opted[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!opted[dev].load(std::memory_order_relaxed)) {
        const cudaError_t e = ensure_dynamic_smem(k, smem);
        if (e != cudaSuccess) return e;
        opted[dev].store(true, std::memory_order_relaxed);
    }
    // few items: their K ranges are split over clusters of 2, 4 or 8 CTAs,
    // as many as the device holds at once, each at least two chunks
    int size = F::CL;
    if (F::CL == 1)
        for (int s = 8; s > 1; s /= 2)
            if (most_items * s <= sms && (args.K + 127) / 128 >= 2 * s && most_items <= resident_clusters<q8_tc<T, NT>>(s, smem)) {
                size = s;
                break;
            }
    TcArgs a = args;
    a.nsplit = F::CL > 1 ? 1 : size;
    long long clusters = sms / size;
    if (F::CL > 1) {
        const int fit = resident_clusters<q8_tc<T, NT>>(F::CL, smem);
        if (fit > 0 && fit < clusters) clusters = fit;
    }
    if (most_items < clusters) clusters = most_items;
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

size_t q8_tc_workspace(int nsrc, int R, int n, int K) { return layout(nsrc, R, n, K).total; }

cudaError_t launch_q8_tc(const Q8Call &c, void *workspace, cudaStream_t stream)
{
    const DeviceInfo *dev = device_info();
    unsigned *status = device_status_word();
    if (!dev || !status) return cudaErrorInvalidDevice;
    char *ws = static_cast<char *>(workspace);
    const Layout l = layout(c.nsrc, c.R, c.n, c.K);
    const int mtiles = (c.N + MT - 1) / MT;
    const int nt = pick_nt(c.R, c.n, !c.offsets, mtiles, dev->sm_count), cl = nt == 192 ? Form<192>::CL : Form<64>::CL, unit = 16 * cl;
    const int max_tiles = most_tiles(c.R, c.n, nt);
    int *ntiles = reinterpret_cast<int *>(ws);
    Tile *tiles = reinterpret_cast<Tile *>(ws + l.tiles);
    float *xss = reinterpret_cast<float *>(ws + l.xss);
    int *srow = c.order ? reinterpret_cast<int *>(ws + l.srow) : nullptr;
    __half *x16 = reinterpret_cast<__half *>(ws + l.x16);

    // one matrix: equal tiles of consecutive rows, a CTA's share one copy
    const int nd = nt == 64 ? (c.R + 63) / 64 : pair_tiles(c.R, (mtiles + 1) / 2, dev->sm_count / 2);
    const int step = ((c.R + nd - 1) / nd + unit - 1) / unit * unit;
    TcArgs a = {};
    a.box = c.offsets ? nt / cl / 2 : step / cl;
    if (!encode(&a.wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, c.wq, c.K, static_cast<long long>(c.n) * c.N, 128, MT) ||
        !encode(&a.xmap, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, x16, c.K, srow ? c.nsrc : c.R, KT, srow ? 1 : a.box))
        return cudaErrorInvalidValue;
    const PrepArgs p = {c.xq, c.xs, c.order, c.offsets, x16, xss, c.y, ntiles, tiles, status, srow, c.nsrc, c.k, c.R, c.n,
                        c.K, c.N, nt, unit, max_tiles, c.dtype == SMOE_BF16 ? 2 : 4};
    const long long vecs = static_cast<long long>(srow ? c.nsrc : c.R) * (c.K / 8);
    long long blocks = ((vecs > c.R ? vecs : c.R) + PREP_THREADS - 1) / PREP_THREADS;
    if (blocks > dev->sm_count * 8) blocks = dev->sm_count * 8;
    cudaError_t e = launch_pdl(q8_prep, dim3(static_cast<unsigned>(blocks + (c.offsets ? 1 : 0))), dim3(PREP_THREADS), 0,
                               stream, p);
    if (e != cudaSuccess) return e;
    a.ws = c.ws;
    a.xs = xss;
    a.srow = srow;
    a.y = c.y;
    a.ntiles = ntiles;
    a.tiles = c.offsets ? tiles : nullptr;
    a.status = status;
    a.R = c.R;
    a.N = c.N;
    a.K = c.K;
    a.step = step;
    a.mtiles = mtiles;
    const long long most = static_cast<long long>(c.offsets ? max_tiles : nd) * ((a.mtiles + cl - 1) / cl);
    if (c.dtype == SMOE_BF16)
        return nt == 192 ? launch_tc<__nv_bfloat16, 192>(a, most, dev->sm_count, stream)
                         : launch_tc<__nv_bfloat16, 64>(a, most, dev->sm_count, stream);
    return nt == 192 ? launch_tc<float, 192>(a, most, dev->sm_count, stream)
                     : launch_tc<float, 64>(a, most, dev->sm_count, stream);
}

}  // namespace smoe
