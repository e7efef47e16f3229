// The 8-bit floating-point product with a scale for each block of 128, on the
// tensor cores (tcgen05, kind::f8f6f4, e4m3 operands from shared memory):
//   y[r][n] = sum_b xs[r][b] ws[e][n / 128][b] sum_{c in b} xq[r][c] wq[e][n][c].
//
// The scales change every 128 columns, inside the sum, so each block's products
// are a sum of their own in tensor memory: the MMAs of a block write one
// accumulator (of a ring of them), the epilogue warps read it and add it to their
// registers, times the block's scales, while the next block's MMAs run.  The sums
// of blocks are f32 in registers; a block's own is the tensor core's f32.
//
// The weights are the MMA's M side (128 rows of one expert: one scale a block), the
// activation rows its N side, so that any number of rows of an expert costs its own
// share of tensor-core time.  The accumulator is read in the shape 16x128b, where a
// thread holds every fourth column of four rows: the scales of its columns (the
// activation rows') are then read from shared memory once for four products.  (A row a
// thread, 32x32b, needs a scale for every product, 512 clocks of shared memory a block
// of 256 rows, as long as its MMAs take; 16x256b reads tensor memory at half the rate.)
//
// Persistent: CTAs (row tiles of up to 64: a deep ring of weights, many small
// accumulators) or pairs of them (cta_group::2, up to 256 rows by 256 weight rows)
// walk the items (tile of rows, weight tiles).  Roles (warps): 0-7 epilogue, 8 issues
// the MMAs (of the pair: the even CTA's), 9 streams the weights, 10 brings the row
// scales of the small tiles, 12-15 the rows (gathered by the copies where the batch is
// sorted by an order).  The pairs' row scales are laid out beforehand, in the order in
// which they are read, so that copies bring them: one warp that fetched and stored 256
// of them paced the loop (1999 rows x 8192 x 4096 113 us, without its scales 86).
// Every wait is bounded.
#include <atomic>

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

// Shapes of the two forms: row tile NT, CTAs per tile CL, stages of the operands
// (weights and a CTA's share of the rows), accumulators D, and the columns CB that
// an epilogue warp takes at a time.
template <int NT>
struct Form;
template <>
struct Form<256> {
    static constexpr int CL = 2, ST = 6, D = 2, CB = 32;
};
template <>
struct Form<64> {
    static constexpr int CL = 1, ST = 8, D = 8, CB = 16;
};

template <int NT>
constexpr size_t tc_smem()
{
    using F = Form<NT>;
    return 1024 + static_cast<size_t>(F::ST) * (W_BYTES + NT / F::CL * F8_BLOCK) + static_cast<size_t>(SLOTS) * NT * 4 +
           EPI_WARPS * OUT_BYTES + 512;
}

struct alignas(128) TcArgs {
    CUtensorMap wmap, xmap;
    const float *ws, *xs;  // scales [n x nb x kb]; [nsrc x kb], of the pairs laid out [kb x pitch]
    void *y;
    const int *ntiles;
    const Tile *tiles;     // null: one matrix, tiles of `step` rows
    const int *order;      // source of every sorted row, times k (gathered), or null
    unsigned *status;
    long long pitch;
    int R, N, K, kb, nb, k, nsrc, step, mtiles, box;  // box: rows of one copy (not gathered)
    int nsplit;            // CTAs that share an item's K range (single-CTA form)
};

// Instruction descriptor, kind::f8f6f4: f32 accumulate, A and B e4m3, K-major.
__device__ __forceinline__ uint32_t idesc_e4m3(int m, int n)
{
    return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

template <int CL>
__device__ __forceinline__ void mma_f8(uint32_t tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    if (CL > 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem),
            "l"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem),
            "l"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
}
template <int CL>
__device__ __forceinline__ void commit(uint32_t bar)
{
    if (CL > 1) mma_commit_pair(bar);
    else mma_commit(bar);
}

// 16 tensor-memory lanes (from that of the address on) by 32 or 16 columns: v[2 i] is
// row lane / 4, column 4 i + lane % 4, v[2 i + 1] row lane / 4 + 8 of it.
__device__ __forceinline__ void tmem_ld_16x128(uint32_t at, uint32_t (&v)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.16x128b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
                   "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
                 : "r"(at));
}
__device__ __forceinline__ void tmem_ld_16x128(uint32_t at, uint32_t (&v)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.16x128b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(at));
}
// Waits for this thread's loads; what they load goes through it, so that no use
// of it is moved before it.
template <int N>
__device__ __forceinline__ void tmem_loaded(uint32_t (&v)[N], uint32_t (&w)[N])
{
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < N; ++i) {
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

// Where column c of a group of CB stands among the scales that are read: every
// fourth one's after one another.
template <int CB>
__host__ __device__ __forceinline__ int scale_at(int c)
{
    return (c & 3) * (CB / 4) + c / 4;
}

__device__ __forceinline__ Tile tile_at(const TcArgs &a, int i, int ntiles)
{
    if (i >= ntiles) return Tile{0, 0, 0, 0};
    if (a.tiles) return a.tiles[i];
    return Tile{0, i * a.step, min(a.step, a.R - i * a.step), 0};
}

template <typename T, int NT>
__global__ void __launch_bounds__(TC_THREADS, 1) f8_tc(const __grid_constant__ TcArgs a)
{
    using F = Form<NT>;
    constexpr int CL = F::CL, ST = F::ST, D = F::D, CB = F::CB;
    constexpr int XR = NT / CL;                              // rows of a CTA's share of a tile, at most
    constexpr uint32_t STAGE = W_BYTES + XR * F8_BLOCK;
    constexpr int JB = NT / (2 * CB), G = CB / 4;            // column blocks of an epilogue warp, of four columns each
    constexpr bool LAID = NT == 256;                         // the row scales are laid out
    static_assert(!LAID || (SLOTS >= ST + D && CB == GROUP), "slots that are free with their stage; the order of the scales");
    static_assert(D * NT <= 512, "tensor memory");
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t w0 = base, x0 = w0 + ST * W_BYTES, f0 = base + ST * STAGE, out0 = f0 + SLOTS * NT * 4, bars = out0 + EPI_WARPS * OUT_BYTES;
    const uint32_t full = bars, empty = full + 8 * ST, sfull = empty + 8 * ST, sempty = sfull + 8 * SLOTS,
                   dfull = sempty + 8 * SLOTS, dempty = dfull + 8 * D, tslot = dempty + 8 * D;
    static_assert(16 * (ST + SLOTS + D) + 4 <= 512, "barriers");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = CL > 1 ? static_cast<int>(blockIdx.x % CL) : 0;
    const int nsplit = CL > 1 ? 1 : a.nsplit;
    const int krank = nsplit > 1 ? static_cast<int>(blockIdx.x) % nsplit : 0;  // = the rank in the cluster
    const int first = static_cast<int>(blockIdx.x) / (CL * nsplit), stride = static_cast<int>(gridDim.x) / (CL * nsplit);

    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(full + 8 * i, 1 + (a.order ? X_WARPS : 1));  // the loading warps; used in the issuing CTA
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(sfull + 8 * i, 1);
            mbar_init(sempty + 8 * i, EPI_WARPS);
        }
        for (int i = 0; i < D; ++i) {
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

    const int c0 = krank * a.kb / nsplit, c1 = (krank + 1) * a.kb / nsplit;  // this CTA's blocks (columns past K are zeros)
    const int mgroups = (a.mtiles + CL - 1) / CL;
    // One matrix: this CTA's first weights are known, and are brought into L2 while
    // the previous kernel ends.  A prefetch only: that kernel may be the one that
    // quantises these weights.
    if (!a.tiles && warp == W_WARP && first < (a.R + a.step - 1) / a.step * mgroups && lane < ST && c0 + lane < c1)
        tma_prefetch_2d(&a.wmap, (c0 + lane) * F8_BLOCK, (first % mgroups * CL + rank) * MT);
    pdl_wait();
    const int ntiles = a.tiles ? *a.ntiles : (a.R + a.step - 1) / a.step;
    const long long nitems = static_cast<long long>(ntiles) * mgroups;
    bool failed = false;

    if (warp >= MMA_WARP) {
        if (NT == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == W_WARP) {
            if (elect_one()) {
                const uint32_t lead = CL > 1 ? mapa_shared(full, 0) : full;
                uint32_t s = 0, p = 1, sl = 0;  // p: parity of the stage's release one lap ago; none in the first
                bool round0 = true;
                for (long long it = first; it < nitems && !failed; it += stride) {
                    const Tile t = tile_at(a, static_cast<int>(it / mgroups), ntiles);
                    const int row = t.expert * a.N + (static_cast<int>(it % mgroups) * CL + rank) * MT;
                    for (int c = c0; c < c1; ++c) {
                        if (!round0 && !mbar_wait_bounded(empty + 8 * s, p, a.status, 7u)) {
                            failed = true;
                            break;
                        }
                        if (rank == 0) mbar_arrive_expect_tx(full + 8 * s, W_BYTES * CL);
                        if (CL > 1) tma_load_2d_pair(w0 + s * W_BYTES, &a.wmap, c * F8_BLOCK, row, lead + 8 * s);
                        else tma_load_2d(w0 + s * W_BYTES, &a.wmap, c * F8_BLOCK, row, full + 8 * s);
                        if (LAID) {
                            // The slot is free: its last scales were read before the accumulator of
                            // that block was handed back, which the block D later waited for, and
                            // that block's stage has been released.
                            mbar_arrive_expect_tx(sfull + 8 * sl, NT * 4);
                            bulk_g2s(f0 + sl * (NT * 4), a.xs + c * a.pitch + (a.tiles ? t.laid : t.row0), NT * 4, sfull + 8 * sl);
                            if (++sl == SLOTS) sl = 0;
                        }
                        if (++s == ST) {
                            s = 0;
                            p ^= 1u;
                            round0 = false;
                        }
                    }
                }
                // The last releases of the stages arrive here from the other CTA's
                // issue: they must have before this CTA may leave.
                if (CL > 1 && !failed) {
                    const long long steps = first < nitems ? (nitems - first + stride - 1) / stride * (c1 - c0) : 0;
                    for (long long g = steps > ST ? steps - ST : 0; g < steps; ++g)
                        if (!mbar_wait_bounded(empty + 8 * static_cast<uint32_t>(g % ST), static_cast<uint32_t>(g / ST) & 1,
                                               a.status, 8u))
                            failed = true;
                }
            }
            failed = __any_sync(FULL_MASK, failed);
        } else if (warp >= X_WARP && (a.order || warp == X_WARP)) {
            // Gathered: each of the four warps loads every fourth four rows of every
            // stage (a gather costs its issuer some 50 clocks).  The bytes of both CTAs
            // complete on the issuing CTA's barrier, which alone expects them.
            const int part = warp - X_WARP;
            const uint32_t lead = CL > 1 ? mapa_shared(full, 0) : full;
            uint32_t s = 0, p = 1;
            bool round0 = true;
            for (long long it = first; it < nitems && !failed; it += stride) {
                const Tile t = tile_at(a, static_cast<int>(it / mgroups), ntiles);
                const int share = mma_cols<CL>(t.rows) / CL;  // rows of this CTA's share, a multiple of 16
                const int row0 = t.row0 + rank * share;
                // lane l keeps row 16 (l / 4) + 4 part + l % 4 of the share; rows past
                // the tile's: any row, their columns are not stored
                int mine = 0;
                if (a.order) {
                    const int at = 16 * (lane >> 2) + 4 * part + (lane & 3);
                    if (at < share && rank * share + at < t.rows) mine = max(source_row(a.order, a.k, a.nsrc, row0 + at, a.status), 0);
                }
                const int copies = a.order ? share / 16 : (share + a.box - 1) / a.box;
                const uint32_t bytes = static_cast<uint32_t>(a.order ? share / 4 : copies * a.box) * (F8_BLOCK * CL);
                for (int c = c0; c < c1; ++c) {
                    if (!__all_sync(FULL_MASK, round0 || mbar_wait_bounded(empty + 8 * s, p, a.status, 8u))) {
                        failed = true;
                        break;
                    }
                    const uint32_t dst = x0 + s * (XR * F8_BLOCK), bar = lead + 8 * s;
                    const int x = c * F8_BLOCK;
                    const bool lead_lane = elect_one();
                    if (rank == 0 && lead_lane) mbar_arrive_expect_tx(full + 8 * s, bytes);
                    if (a.order) {
#pragma unroll
                        for (int i = 0; i < XR / 16; ++i) {
                            if (i >= copies) break;
                            int4 r;
                            r.x = __shfl_sync(FULL_MASK, mine, 4 * i);
                            r.y = __shfl_sync(FULL_MASK, mine, 4 * i + 1);
                            r.z = __shfl_sync(FULL_MASK, mine, 4 * i + 2);
                            r.w = __shfl_sync(FULL_MASK, mine, 4 * i + 3);
                            const uint32_t to = dst + static_cast<uint32_t>(16 * i + 4 * part) * F8_BLOCK;
                            if (lead_lane) {
                                if (CL > 1) tma_gather4_pair(to, &a.xmap, x, r, bar);
                                else tma_gather4(to, &a.xmap, x, r, bar);
                            }
                        }
                    } else if (lead_lane) {
                        for (int b = 0; b < copies; ++b) {
                            const uint32_t to = dst + static_cast<uint32_t>(b * a.box) * F8_BLOCK;
                            if (CL > 1) tma_load_2d_pair(to, &a.xmap, x, row0 + b * a.box, bar);
                            else tma_load_2d(to, &a.xmap, x, row0 + b * a.box, bar);
                        }
                    }
                    if (++s == ST) {
                        s = 0;
                        p ^= 1u;
                        round0 = false;
                    }
                }
            }
        } else if (warp == MMA_WARP) {
            // one thread issues, of a pair the even CTA's
            if (rank == 0 && elect_one()) {
                uint32_t s = 0, p = 0, d = 0, pd = 1;
                bool round0 = true;
                for (long long it = first; it < nitems && !failed; it += stride) {
                    const Tile t = tile_at(a, static_cast<int>(it / mgroups), ntiles);
                    const uint32_t idesc = idesc_e4m3(MT * CL, mma_cols<CL>(t.rows));
                    for (int c = c0; c < c1; ++c) {
                        // both barriers looked at together: this thread's own latency counts
                        const bool r0 = mbar_test<CL>(full + 8 * s, p), r1 = round0 || mbar_test<CL>(dempty + 8 * d, pd);
                        if (!(r0 && r1) && !(wait_pair<CL>(full + 8 * s, p, a.status, 3u) &&
                                             (round0 || wait_pair<CL>(dempty + 8 * d, pd, a.status, 4u)))) {
                            failed = true;
                            break;
                        }
                        tc_fence_after();
                        const uint64_t wd = desc_sw128(w0 + s * W_BYTES), xd = desc_sw128(x0 + s * (XR * F8_BLOCK));
#pragma unroll
                        for (int kk = 0; kk < F8_BLOCK / 32; ++kk)
                            mma_f8<CL>(tmem + d * NT, wd + kk * 2, xd + kk * 2, idesc, kk != 0);
                        commit<CL>(dfull + 8 * d);
                        commit<CL>(empty + 8 * s);
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
        } else if (!LAID && warp == S_WARP) {
            // a lane brings the scales of every 32nd row of the tile, times the weights'
            const bool v4 = (a.kb & 3) == 0 && (reinterpret_cast<uintptr_t>(a.xs) & 15u) == 0;
            uint32_t s = 0, p = 1;
            bool round0 = true;
            for (long long it = first; it < nitems && !failed; it += stride) {
                const Tile t = tile_at(a, static_cast<int>(it / mgroups), ntiles);
                const int mt = static_cast<int>(it % mgroups) * CL + rank;
                const float *ws = a.ws + (static_cast<size_t>(t.expert) * a.nb + min(mt, a.nb - 1)) * a.kb;
                int src[NT / 32];
#pragma unroll
                for (int i = 0; i < NT / 32; ++i) {
                    const int c = i * 32 + lane;
                    src[i] = c < t.rows ? source_row(a.order, a.k, a.nsrc, t.row0 + c, a.status) : -1;
                }
                int c = c0;
                while (c < c1 && !failed) {
                    const int n = v4 ? min(4 - (c & 3), c1 - c) : 1;  // blocks of one load
#pragma unroll
                    for (int i0 = 0; i0 < NT / 32; i0 += 4) {
                        float4 v[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (i0 + i < NT / 32 && src[i0 + i < NT / 32 ? i0 + i : 0] >= 0) {
                                const float *x = a.xs + static_cast<size_t>(src[i0 + i < NT / 32 ? i0 + i : 0]) * a.kb;
                                if (v4) v[i] = *reinterpret_cast<const float4 *>(x + (c & ~3));
                                else v[i].x = x[c];
                            }
                        }
                        for (int j = 0; j < n; ++j) {
                            const uint32_t sj = (s + j) % SLOTS;
                            // the slots' releases, once before their first use
                            if (i0 == 0) {
                                const bool lap = s + j >= SLOTS;
                                const bool free = (round0 && !lap) || mbar_wait_bounded(sempty + 8 * sj, lap ? p ^ 1u : p, a.status, 9u);
                                if (!__all_sync(FULL_MASK, free)) {
                                    failed = true;
                                    break;
                                }
                            }
                            const float w = ws[c + j];
                            const int pick = v4 ? (c + j) & 3 : 0;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if (i0 + i >= NT / 32) break;
                                const float f = pick == 0 ? v[i].x : (pick == 1 ? v[i].y : (pick == 2 ? v[i].z : v[i].w));
                                const int at = (i0 + i) * 32 + lane;
                                sts32(f0 + sj * (NT * 4) + static_cast<uint32_t>(at / CB * CB + scale_at<CB>(at % CB)) * 4u, f * w);
                            }
                        }
                        if (failed) break;
                    }
                    __syncwarp();
                    if (!failed)
                        for (int j = 0; j < n; ++j)
                            if (lane == j) mbar_arrive(sfull + 8 * ((s + j) % SLOTS));
                    c += n;
                    s += n;
                    if (s >= SLOTS) {
                        s -= SLOTS;
                        p ^= 1u;
                        round0 = false;
                    }
                }
            }
        }
    } else {
        if (NT == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        // warp w: tensor-memory lanes 32 (w % 4) .. + 31 = weight rows, the blocks of
        // CB columns of parity w / 4
        const int q = warp & 3, h = warp >> 2;
        T *y = static_cast<T *>(a.y);
        const uint32_t lead = CL > 1 ? mapa_shared(dempty, 0) : dempty;
        const uint32_t mine = tmem + (static_cast<uint32_t>(q * 32) << 16);
        uint32_t d = 0, pd = 0, s = 0, p = 0;
        for (long long it = first; it < nitems && !failed; it += stride) {
            const Tile t = tile_at(a, static_cast<int>(it / mgroups), ntiles);
            float2 acc[JB][G][2];  // column 4 g + lane % 4 of rows lane / 4 + 16 i and + 8
#pragma unroll
            for (int j = 0; j < JB; ++j)
#pragma unroll
                for (int g = 0; g < G; ++g) acc[j][g][0] = acc[j][g][1] = make_float2(0.f, 0.f);
            const float *ws = a.ws + (static_cast<size_t>(t.expert) * a.nb + min(static_cast<int>(it % mgroups) * CL + rank, a.nb - 1)) * a.kb;
            float wl = 0.f;  // the weights' scales, a block a lane
            for (int c = c0; c < c1; ++c) {
                if (LAID && ((c - c0) & 31) == 0) wl = c + lane < c1 ? ws[c + lane] : 0.f;
                const bool r0 = mbar_test<1>(sfull + 8 * s, p), r1 = mbar_test<1>(dfull + 8 * d, pd);
                if (!__all_sync(FULL_MASK, r0 && r1) &&
                    !__all_sync(FULL_MASK, mbar_wait_bounded(sfull + 8 * s, p, a.status, 6u) && mbar_wait_bounded(dfull + 8 * d, pd, a.status, 6u))) {
                    failed = true;
                    break;
                }
                tc_fence_after();
                const float w = LAID ? __shfl_sync(FULL_MASK, wl, (c - c0) & 31) : 1.f;
                const uint32_t fs = f0 + s * (NT * 4) + static_cast<uint32_t>((lane & 3) * G) * 4u;
#pragma unroll
                for (int j = 0; j < JB; ++j) {
                    const int at = (2 * j + h) * CB;
                    if (at >= t.rows) break;
                    uint32_t lo[2 * G], hi[2 * G];
                    tmem_ld_16x128(mine + d * NT + at, lo);
                    tmem_ld_16x128(mine + (16u << 16) + d * NT + at, hi);
                    float4 f[G / 4];
#pragma unroll
                    for (int g = 0; g < G / 4; ++g) {
                        f[g] = lds128f(fs + static_cast<uint32_t>(at + 4 * g) * 4u);
                        if (LAID) f[g] = make_float4(f[g].x * w, f[g].y * w, f[g].z * w, f[g].w * w);
                    }
                    tmem_loaded(lo, hi);
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        const float4 v = f[g / 4];
                        const float s1 = (g & 3) == 0 ? v.x : ((g & 3) == 1 ? v.y : ((g & 3) == 2 ? v.z : v.w));
                        fma2(acc[j][g][0], lo[2 * g], lo[2 * g + 1], s1);
                        fma2(acc[j][g][1], hi[2 * g], hi[2 * g + 1], s1);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (CL > 1) mbar_arrive_cluster(lead + 8 * d);
                    else mbar_arrive(dempty + 8 * d);
                    if (!LAID) mbar_arrive(sempty + 8 * s);
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
            const int n0 = (static_cast<int>(it % mgroups) * CL + rank) * MT + q * 32;
            if (nsplit > 1) {  // this K range's sums [row][128], for the reduction below
#pragma unroll
                for (int j = 0; j < JB; ++j)
#pragma unroll
                    for (int g = 0; g < G; ++g)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int r = (2 * j + h) * CB + 4 * g + (lane & 3);
                            const uint32_t to = x0 + static_cast<uint32_t>(r * MT + q * 32 + (lane >> 2) + 16 * i) * 4u;
                            if (r < t.rows) {
                                sts32(to, acc[j][g][i].x);
                                sts32(to + 32u, acc[j][g][i].y);
                            }
                        }
                continue;
            }
            // 8 rows at a time through shared memory, out as 16-byte vectors of a row
            constexpr uint32_t PITCH = 32 * sizeof(T) + 16;
            constexpr int VE = 16 / static_cast<int>(sizeof(T)), LR = 32 / VE;  // lanes of a row
            const uint32_t stage = out0 + warp * OUT_BYTES;
            const bool whole = a.N % VE == 0;
#pragma unroll
            for (int j = 0; j < JB; ++j) {
                if ((2 * j + h) * CB >= t.rows) break;
#pragma unroll
                for (int g0 = 0; g0 < G; g0 += 2) {
                    const int r0 = (2 * j + h) * CB + 4 * g0;
                    if (r0 >= t.rows) break;
                    __syncwarp();
#pragma unroll
                    for (int g = 0; g < 2; ++g)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t to = stage + static_cast<uint32_t>(4 * g + (lane & 3)) * PITCH +
                                                static_cast<uint32_t>((lane >> 2) + 16 * i) * static_cast<uint32_t>(sizeof(T));
                            sts_out(to, acc[j][g0 + g][i].x, y);
                            sts_out(to + 8 * static_cast<uint32_t>(sizeof(T)), acc[j][g0 + g][i].y, y);
                        }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8 * LR / 32; ++i) {
                        const int r = (i * 32 + lane) / LR, n = (lane % LR) * VE;
                        const uint4 v = lds128v(stage + static_cast<uint32_t>(r) * PITCH + static_cast<uint32_t>(lane % LR) * 16u);
                        if (r0 + r >= t.rows || n0 + n >= a.N) continue;
                        T *to = y + static_cast<size_t>(t.row0 + r0 + r) * a.N + n0 + n;
                        if (whole) {
                            *reinterpret_cast<uint4 *>(to) = v;
                        } else {
                            const uint32_t e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int b = 0; b < VE; ++b)
                                if (n0 + n + b < a.N) {
                                    if (sizeof(T) == 4) reinterpret_cast<uint32_t *>(to)[b] = e[b];
                                    else reinterpret_cast<uint16_t *>(to)[b] = static_cast<uint16_t>(e[b / 2] >> (16 * (b & 1)));
                                }
                        }
                    }
                }
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
        static_assert(CL > 1 || NT * MT * 4 <= ST * XR * F8_BLOCK, "the sums of a tile");
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
                const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (n + j < a.N) put(y + static_cast<size_t>(t.row0 + r) * a.N + n + j, f[j]);
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
    const int *offsets;  // null: one matrix
    const int *order;
    const float *xs;
    float *laid;         // null: no scales to lay out
    void *y;
    int *ntiles;
    Tile *tiles;
    unsigned *status;
    long long pitch;
    int R, n, N, nt, unit, max_tiles, elem, kb, k, nsrc;  // elem: bytes of an element of y
};

// Block 0 (with offsets): the tile list.  The others: zeros in the rows of y past the
// last expert's, and the row scales of the pairs, [kb x pitch], every expert's rows from
// laid_row on, those of each 32 in the order in which the epilogue reads them.
__global__ void __launch_bounds__(PREP_THREADS) f8_prep(const PrepArgs a)
{
    pdl_launch_dependents();
    pdl_wait();
    if (a.offsets && blockIdx.x == 0) {
        list_tiles<PREP_THREADS>(a.offsets, a.n, a.R, a.nt, a.unit, a.max_tiles, a.ntiles, a.tiles, a.status);
        return;
    }
    const int b0 = a.offsets ? 1 : 0, blocks = gridDim.x - b0;
    const int last = a.offsets ? max(0, min(a.offsets[a.n], a.R)) : a.R;
    if (a.laid) {
        // a thread takes one row and four blocks of columns
        const int quads = (a.kb + 3) / 4;
        const bool v4 = (a.kb & 3) == 0 && (reinterpret_cast<uintptr_t>(a.xs) & 15u) == 0;
        const int rows = (last + 31) & ~31;  // whole warps: neighbouring lanes, neighbouring rows
        const long long total = static_cast<long long>(rows) * quads;
        for (long long i = static_cast<long long>(blockIdx.x - b0) * PREP_THREADS + threadIdx.x; i < total;
             i += static_cast<long long>(blocks) * PREP_THREADS) {
            const int r = static_cast<int>(i % rows), c = static_cast<int>(i / rows) * 4;
            if (r >= last) continue;
            int at = r;
            if (a.offsets) {  // the last expert whose rows begin at or before this one
                int lo = 0, hi = a.n;
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (a.offsets[mid] <= r) lo = mid;
                    else hi = mid;
                }
                const int first = a.offsets[lo];
                if (first < 0 || first > r) continue;  // no list (reported): its rows are unspecified
                at = laid_row(first, lo) + r - first;
            }
            at = (at & ~(GROUP - 1)) + scale_at<GROUP>(at & (GROUP - 1));
            const int src = source_row(a.order, a.k, a.nsrc, r, a.status);
            const float *x = a.xs + static_cast<size_t>(max(src, 0)) * a.kb;
            float v[4];
            if (v4) {
                const float4 q = *reinterpret_cast<const float4 *>(x + c);
                v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = c + j < a.kb ? x[c + j] : 0.f;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + j < a.kb) a.laid[(c + j) * a.pitch + at] = src < 0 ? 0.f : v[j];
        }
    }
    const size_t end = static_cast<size_t>(a.R) * a.N;
    for (size_t i = static_cast<size_t>(last) * a.N + static_cast<size_t>(blockIdx.x - b0) * PREP_THREADS + threadIdx.x; i < end;
         i += static_cast<size_t>(blocks) * PREP_THREADS) {
        if (a.elem == 4) static_cast<float *>(a.y)[i] = 0.f;
        else static_cast<uint16_t *>(a.y)[i] = 0;
    }
}

// ---------------------------------------------------------------- host

// Row tile: 64 (single CTAs) where the product is bound by reading the weights or
// its tiles fit the device at once, 256 (pairs) beyond.
int pick_nt(int R, int n, bool one, int mtiles, int sms)
{
    const long long tiles = one ? (R + 63) / 64 : most_tiles(R, n, 64);
    return R <= 48LL * n || tiles * mtiles <= sms ? 64 : 256;
}

// How many tiles one matrix's R rows are cut into for pairs: as many as keep
// waves of `pairs` items on `slots` pairs of SMs shortest; an item costs its rows,
// and some 16 rows' time of its own.
int pair_tiles(int R, int pairs, int slots)
{
    int best = 0;
    long long least = 0;
    for (int nd = (R + 255) / 256; nd <= (R + 95) / 96; ++nd) {
        const int step = ((R + nd - 1) / nd + 31) / 32 * 32;
        const long long waves = (static_cast<long long>((R + step - 1) / step) * pairs + slots - 1) / slots;
        const long long cost = waves * (step + 16);
        if (best == 0 || cost < least) {
            best = nd;
            least = cost;
        }
    }
    return best;
}

template <typename T, int NT>
cudaError_t launch_tc(const TcArgs &args, long long most_items, int sms, cudaStream_t stream)
{
    using F = Form<NT>;
    constexpr size_t smem = tc_smem<NT>();
    static_assert(smem <= 227 * 1024, "shared memory of a CTA");
    auto k = f8_tc<T, NT>;
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
    // as many as the device holds at once, each at least two blocks
    int size = F::CL;
    if (F::CL == 1)
        for (int s = 8; s > 1; s /= 2)
            if (most_items * s <= sms && args.kb >= 2 * s && most_items <= clusters_held<f8_tc<T, NT>>(s, TC_THREADS, smem)) {
                size = s;
                break;
            }
    TcArgs a = args;
    a.nsplit = F::CL > 1 ? 1 : size;
    long long clusters = sms / size;
    if (F::CL > 1) {
        const int fit = clusters_held<f8_tc<T, NT>>(F::CL, TC_THREADS, smem);
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

// Laid-out rows: each expert's begin at a multiple of GROUP, and a copy takes a
// whole tile from any of them.
static long long laid_pitch(int R, int n) { return (R + GROUP - 1) / GROUP * GROUP + static_cast<long long>(n) * GROUP + 256; }

// 64 columns of rows' scales at least; all of them only where pairs may take the
// product, which then has rows for the experts' padding.
static size_t tiles_bytes(int R, int n) { return 256 + up256(static_cast<size_t>(most_tiles(R, n, 64)) * sizeof(Tile)); }

size_t f8_tc_workspace(int R, int n, int K)
{
    const size_t laid = R > 48LL * n ? static_cast<size_t>(laid_pitch(R, n)) * ((K + F8_BLOCK - 1) / F8_BLOCK) * sizeof(float) : 0;
    return tiles_bytes(R, n) + up256(laid);
}

cudaError_t launch_f8_tc(const F8Call &c, void *workspace, cudaStream_t stream)
{
    const DeviceInfo *dev = device_info();
    unsigned *status = device_status_word();
    if (!dev || !status) return cudaErrorInvalidDevice;
    const int mtiles = (c.N + MT - 1) / MT, elem = c.dtype == SMOE_BF16 ? 2 : 4;
    const int nt = pick_nt(c.R, c.n, !c.offsets, mtiles, dev->sm_count), cl = nt == 256 ? Form<256>::CL : Form<64>::CL, unit = 16 * cl;
    const int max_tiles = most_tiles(c.R, c.n, nt);
    int *ntiles = static_cast<int *>(workspace);
    Tile *tiles = reinterpret_cast<Tile *>(static_cast<char *>(workspace) + 256);
    float *laid = nt == 256 ? reinterpret_cast<float *>(static_cast<char *>(workspace) + tiles_bytes(c.R, c.n)) : nullptr;

    // one matrix: equal tiles of consecutive rows, a CTA's share one copy
    const int nd = nt == 64 ? (c.R + 63) / 64 : pair_tiles(c.R, (mtiles + 1) / 2, dev->sm_count / 2);
    const int step = ((c.R + nd - 1) / nd + unit - 1) / unit * unit;
    TcArgs a = {};
    a.kb = (c.K + F8_BLOCK - 1) / F8_BLOCK;
    a.pitch = laid_pitch(c.R, c.n);
    a.box = c.offsets ? nt / cl / 2 : step / cl;
    if (!encode(&a.wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, c.wq, c.K, static_cast<long long>(c.n) * c.N, F8_BLOCK, MT) ||
        !encode(&a.xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, c.xq, c.K, c.nsrc, F8_BLOCK, c.order ? 1 : a.box))
        return cudaErrorInvalidValue;
    if (c.offsets || laid) {
        const PrepArgs p = {c.offsets, c.order, c.xs, laid, c.y, ntiles, tiles, status, a.pitch, c.R, c.n, c.N, nt, unit, max_tiles,
                            elem, a.kb, c.k, c.nsrc};
        long long blocks = laid ? (static_cast<long long>(c.R) * ((a.kb + 3) / 4) + PREP_THREADS - 1) / PREP_THREADS : 32;
        if (blocks > 4LL * dev->sm_count) blocks = 4LL * dev->sm_count;
        const cudaError_t e = launch_pdl(f8_prep, dim3(static_cast<unsigned>(blocks + (c.offsets ? 1 : 0))), dim3(PREP_THREADS), 0,
                                         stream, p);
        if (e != cudaSuccess) return e;
    }
    a.ws = c.ws;
    a.xs = laid ? laid : c.xs;
    a.order = c.order;
    a.y = c.y;
    a.ntiles = ntiles;
    a.tiles = c.offsets ? tiles : nullptr;
    a.status = status;
    a.R = c.R;
    a.N = c.N;
    a.K = c.K;
    a.nb = (c.N + F8_BLOCK - 1) / F8_BLOCK;
    a.k = c.k;
    a.nsrc = c.nsrc;
    a.step = step;
    a.mtiles = mtiles;
    const long long most = static_cast<long long>(c.offsets ? max_tiles : nd) * ((a.mtiles + cl - 1) / cl);
    if (c.dtype == SMOE_BF16)
        return nt == 256 ? launch_tc<__nv_bfloat16, 256>(a, most, dev->sm_count, stream)
                         : launch_tc<__nv_bfloat16, 64>(a, most, dev->sm_count, stream);
    return nt == 256 ? launch_tc<float, 256>(a, most, dev->sm_count, stream)
                     : launch_tc<float, 64>(a, most, dev->sm_count, stream);
}

}  // namespace smoe
