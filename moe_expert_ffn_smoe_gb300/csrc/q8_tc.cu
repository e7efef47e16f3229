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
// q8_tc is persistent: clusters walk the items (tile of rows, group of
// weight tiles), accumulators double-buffered so that the store of one item
// runs under the products of the next.  With clusters of two, the two CTAs
// take neighbouring weight tiles of the same rows and each loads half of the
// row tile for both (multicast), which halves the activation traffic from
// L2.  Roles (warps): 0-7 epilogue, 8-15 widen weights (two groups, alternate
// K tiles), 16 issues the MMAs, 17 streams the weights, 18 and 19
// the rows.
// Every wait is bounded.
#include <cuda_fp16.h>

#include <atomic>

#include "q8.cuh"
#include "smoe.h"
#include "tcgen05.cuh"

namespace smoe {
namespace {

constexpr int KT = 64;                  // columns per K tile
constexpr int MT = 128;                 // weight rows per CTA tile
constexpr uint32_t W_BYTES = MT * 128;  // one weight chunk: 128 rows x 128 columns (two K tiles)
constexpr int EPI_WARPS = 8;
constexpr int CONV_WARP0 = 8;
constexpr int MMA_WARP = 16, W_WARP = 17, X_WARP = 18;
constexpr int TC_THREADS = 20 * 32;

// Shapes of the two forms: row tile NT, cluster CL, the rings of A stages
// (tensor memory), row stages and weight chunks (shared memory), and the rows
// of one tensor copy of activations (a copy costs its issuer about 100 clocks
// whatever its size: 16-row boxes made the issuing warp pace the K loop).
template <int NT>
struct Form;
template <>
struct Form<192> {
    static constexpr int CL = 2, AS = 4, XS = 6, WS = 4, BOX = 48;
};
template <>
struct Form<64> {
    static constexpr int CL = 1, AS = 8, XS = 8, WS = 8, BOX = 16;
};

template <int NT>
constexpr size_t tc_smem()
{
    using F = Form<NT>;
    return 1024 + static_cast<size_t>(F::WS) * W_BYTES + static_cast<size_t>(F::XS) * NT * 128 + 512;
}

struct alignas(128) TcArgs {
    CUtensorMap wmap, xmap;
    const float *ws, *xs;  // w_scales [n x N], x scales in sorted order [R]
    void *y;
    const int *ntiles;
    const Tile *tiles;     // null: one matrix, tiles of `step` rows
    unsigned *status;
    int R, N, K, step, mtiles;
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
__device__ __forceinline__ uint32_t idesc_f16(int n)
{
    return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(MT >> 4) << 24);
}

// 2-D tensor copy of one box into the same place of every CTA of `mask`,
// completing on the barrier at the same place.
__device__ __forceinline__ void tma_load_2d_mc(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar,
                                               uint16_t mask)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.multicast::cluster [%0], [%1, {%2, "
        "%3}], [%4], %5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "h"(mask)
        : "memory");
}

__device__ __forceinline__ void mma_commit_mc(uint32_t bar, uint16_t mask)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                     bar),
                 "h"(mask)
                 : "memory");
}

// Whether phase `parity` of an mbarrier has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
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
    constexpr uint32_t XB = NT * 128u, ACOL0 = 2u * NT;
    static_assert(2 * NT + AS * 32 <= 512 && AS % 2 == 0 && XS % 2 == 0, "tensor memory; two issuers");
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t w0 = base, x0 = w0 + WS * W_BYTES, bars = x0 + XS * XB;
    const uint32_t wfull = bars, wempty = wfull + 8 * WS, xfull = wempty + 8 * WS, xempty = xfull + 8 * XS,
                   afull = xempty + 8 * XS, aempty = afull + 8 * AS, dfull = aempty + 8 * AS, dempty = dfull + 16,
                   tslot = dempty + 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = CL > 1 ? static_cast<int>(blockIdx.x % CL) : 0;
    const int first = static_cast<int>(blockIdx.x / CL), stride = static_cast<int>(gridDim.x / CL);

    if (threadIdx.x == 0) {
        for (int i = 0; i < WS; ++i) {
            mbar_init(wfull + 8 * i, 1);
            mbar_init(wempty + 8 * i, 8);  // the eight widening warps
        }
        for (int i = 0; i < XS; ++i) {
            mbar_init(xfull + 8 * i, 1);
            mbar_init(xempty + 8 * i, CL);  // every CTA that the stage's boxes go to
        }
        for (int i = 0; i < AS; ++i) {
            mbar_init(afull + 8 * i, 4);  // one group of widening warps
            mbar_init(aempty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
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
    if (CL > 1) cluster_sync();  // no copy may reach a CTA whose barriers are not there yet
    __syncthreads();
    tc_fence_after();
    uint32_t tmem;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(tslot));
    if (threadIdx.x == 0) pdl_launch_dependents();

    const int nch = (a.K + 127) / 128;  // weight chunks, two K tiles each (columns past K are zeros)
    const int nkt = 2 * nch;
    const int mgroups = (a.mtiles + CL - 1) / CL;
    // the tile list comes from the previous kernel; without one the weights,
    // which no kernel of this call writes, are asked for at once
    if (a.tiles || warp != W_WARP) pdl_wait();
    const int ntiles = a.tiles ? *a.ntiles : (a.R + a.step - 1) / a.step;
    const long long nitems = static_cast<long long>(ntiles) * mgroups;
    bool failed = false;

    if (warp == W_WARP) {
        if (elect_one()) {
            uint32_t s = 0, p = 1;  // parity of the release before this round; none waited for in the first
            bool round0 = true;
            for (long long it = first; it < nitems && !failed; it += stride) {
                const Tile t = tile_at(a, static_cast<int>(it / mgroups), ntiles);
                const int row = t.expert * a.N + (static_cast<int>(it % mgroups) * CL + rank) * MT;
                for (int c = 0; c < nch; ++c) {
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
    } else if (warp == X_WARP || warp == X_WARP + 1) {
        // the two warps take alternate K tiles: a tensor copy costs its
        // issuer 100 to 200 clocks, and one issuer paced the K loop
        if (elect_one()) {
            uint32_t s = warp - X_WARP, p = 1;
            bool round0 = true;
            for (long long it = first; it < nitems && !failed; it += stride) {
                const Tile t = tile_at(a, static_cast<int>(it / mgroups), ntiles);
                const int boxes = (t.rows + F::BOX - 1) / F::BOX;
                for (int kt = warp - X_WARP; kt < nkt; kt += 2) {
                    if (!round0 && !mbar_wait_bounded(xempty + 8 * s, p, a.status, 8u)) {
                        failed = true;
                        break;
                    }
                    mbar_arrive_expect_tx(xfull + 8 * s, static_cast<uint32_t>(boxes) * (F::BOX * 128u));
                    for (int b = rank; b < boxes; b += CL) {
                        const uint32_t dst = x0 + s * XB + static_cast<uint32_t>(b) * (F::BOX * 128u);
                        if (CL > 1)
                            tma_load_2d_mc(dst, &a.xmap, kt * KT, t.row0 + b * F::BOX, xfull + 8 * s, (1u << CL) - 1);
                        else tma_load_2d(dst, &a.xmap, kt * KT, t.row0 + b * F::BOX, xfull + 8 * s);
                    }
                    s += 2;
                    if (s >= XS) {
                        s -= XS;
                        p ^= 1u;
                        round0 = false;
                    }
                }
            }
            // the other CTA's last releases of this warp's stages arrive
            // here: they must have before this CTA may leave
            if (CL > 1 && !failed) {
                for (int j = 0; j < XS / 2; ++j) {
                    if (!round0 && !mbar_wait_bounded(xempty + 8 * s, p, a.status, 8u)) failed = true;
                    s += 2;
                    if (s >= XS) {
                        s -= XS;
                        p ^= 1u;
                        round0 = false;
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp == MMA_WARP) {
        // one thread issues; it looks at both barriers of a stage before it
        // waits for either, so that two stages that are ready cost one look
        if (elect_one()) {
            uint32_t sa = 0, pa = 0, sx = 0, px = 0, d = 0;
            for (long long it = first; it < nitems && !failed; it += stride, ++d) {
                const Tile t = tile_at(a, static_cast<int>(it / mgroups), ntiles);
                const uint32_t idesc = idesc_f16((t.rows + 15) & ~15);
                const uint32_t acc = tmem + (d & 1) * NT;
                if (d >= 2 && !mbar_wait_bounded(dempty + 8 * (d & 1), (d / 2 - 1) & 1, a.status, 4u)) failed = true;
                for (int kt = 0; kt < nkt && !failed; ++kt) {
                    const bool rx = mbar_test(xfull + 8 * sx, px), ra = mbar_test(afull + 8 * sa, pa);
                    if (!(rx && ra) && !(mbar_wait_bounded(xfull + 8 * sx, px, a.status, 3u) &&
                                         mbar_wait_bounded(afull + 8 * sa, pa, a.status, 3u))) {
                        failed = true;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t at = tmem + ACOL0 + sa * 32;
                    const uint64_t xd = desc_sw128(x0 + sx * XB);
#pragma unroll
                    for (int kk = 0; kk < KT / 16; ++kk)
                        mma_f16_ta(acc, at + kk * 8, xd + kk * 2, idesc, kt + kk != 0);
                    mma_commit(aempty + 8 * sa);
                    if (CL > 1) mma_commit_mc(xempty + 8 * sx, (1u << CL) - 1);
                    else mma_commit(xempty + 8 * sx);
                    if (kt == nkt - 1) mma_commit(dfull + 8 * (d & 1));
                    if (++sa == AS) {
                        sa = 0;
                        pa ^= 1u;
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
        // thread = one weight row; group grp widens the K tiles 2 c + grp
        const int ct = threadIdx.x - CONV_WARP0 * 32;
        const uint32_t r = ct & (MT - 1), grp = ct >> 7;
        uint32_t g = 0;
        for (long long it = first; it < nitems && !failed; it += stride) {
            for (int c = 0; c < nch; ++c, ++g) {
                const uint32_t sw = g % WS, ga = 2 * g + grp, sa = ga % AS;
                const bool ok = mbar_wait_bounded(wfull + 8 * sw, (g / WS) & 1, a.status, 5u) &&
                                (ga < AS || mbar_wait_bounded(aempty + 8 * sa, (ga / AS - 1) & 1, a.status, 5u));
                if (!__all_sync(FULL_MASK, ok)) {
                    failed = true;
                    break;
                }
                tc_fence_after();
                const uint32_t row = w0 + sw * W_BYTES + r * 128u;
                uint4 w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = lds128v(row + (((grp * 4 + j) ^ (r & 7)) << 4));
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t v[16];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint4 q = w[2 * h + j];
                        s8x4_to_f16(q.x, v[8 * j], v[8 * j + 1]);
                        s8x4_to_f16(q.y, v[8 * j + 2], v[8 * j + 3]);
                        s8x4_to_f16(q.z, v[8 * j + 4], v[8 * j + 5]);
                        s8x4_to_f16(q.w, v[8 * j + 6], v[8 * j + 7]);
                    }
                    tmem_st16(tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + ACOL0 + sa * 32 + 16 * h, v);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(wempty + 8 * sw);
                    mbar_arrive(afull + 8 * sa);
                }
            }
        }
    } else if (warp < EPI_WARPS) {
        // warp w: TMEM lanes 32 (w % 4) .. + 31 = weight rows, the 16-column
        // blocks of parity w / 4
        const int q = warp & 3, h = warp >> 2;
        T *y = static_cast<T *>(a.y);
        uint32_t d = 0;
        for (long long it = first; it < nitems; it += stride, ++d) {
            const Tile t = tile_at(a, static_cast<int>(it / mgroups), ntiles);
            const int n = (static_cast<int>(it % mgroups) * CL + rank) * MT + q * 32 + lane;
            const bool nok = n < a.N;
            const float ws = nok ? a.ws[static_cast<size_t>(t.expert) * a.N + n] : 0.f;
            const bool ok = mbar_wait_bounded(dfull + 8 * (d & 1), (d / 2) & 1, a.status, 6u);
            if (!__all_sync(FULL_MASK, ok)) {
                failed = true;
                break;
            }
            tc_fence_after();
            const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16) + (d & 1) * NT;
            for (int c = h * 16; c < t.rows; c += 32) {
                float v[16];
                tmem_ld<16>(acc + c, v);
                const float xl = (lane & 15) < t.rows - c ? a.xs[t.row0 + c + (lane & 15)] : 0.f;
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float xi = __shfl_sync(FULL_MASK, xl, i);
                    if (nok && c + i < t.rows) put(y + static_cast<size_t>(t.row0 + c + i) * a.N + n, v[i] * xi * ws);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(dempty + 8 * (d & 1));
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
    if (CL > 1) cluster_sync();  // no CTA leaves while the other's copies or releases may reach it
    if (warp == MMA_WARP) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

// ---------------------------------------------------------------- preparation

constexpr int PREP_THREADS = 256;

struct PrepArgs {
    const int8_t *xq;
    const float *xs;
    const int *order, *offsets;
    __half *x16;  // [R x K]
    float *xss;   // [R]
    void *y;
    int *ntiles;
    Tile *tiles;
    unsigned *status;
    int nsrc, k, R, n, K, N, nt, max_tiles, zero_bytes;  // zero_bytes: bytes of one element of y
};

// Block 0 (with offsets): the tile list, every expert's rows cut into equal
// tiles of at most nt.  The others: the rows in sorted order, widened to
// f16, with their scales; rows past the last expert's get zeros in y.
__global__ void __launch_bounds__(PREP_THREADS) q8_prep(const PrepArgs a)
{
    __shared__ int warp_sums[PREP_THREADS / 32];
    __shared__ int run_s;
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x;
    if (a.offsets && blockIdx.x == 0) {
        const int lane = tid & 31, wi = tid >> 5;
        int run = 0;
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
            const int step = cnt > 0 ? ((hi - lo + cnt - 1) / cnt + 15) & ~15 : 16;
            cnt = (hi - lo + step - 1) / step;
            int inc = cnt;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int o = __shfl_up_sync(FULL_MASK, inc, off);
                if (lane >= off) inc += o;
            }
            if (lane == 31) warp_sums[wi] = inc;
            __syncthreads();
            int before = run;
            for (int i = 0; i < wi; ++i) before += warp_sums[i];
            if (tid == PREP_THREADS - 1) run_s = before + inc;
            const int t0 = before + inc - cnt;
            for (int i = 0; i < cnt && t0 + i < a.max_tiles; ++i)
                a.tiles[t0 + i] = Tile{e, lo + i * step, min(step, hi - lo - i * step), 0};
            __syncthreads();
            run = run_s;
        }
        if (tid == 0) *a.ntiles = min(run, a.max_tiles);
        return;
    }
    const int b0 = a.offsets ? 1 : 0;
    const int last = a.offsets ? max(0, min(a.offsets[a.n], a.R)) : a.R;
    for (int r = blockIdx.x - b0; r < a.R; r += gridDim.x - b0) {
        if (r >= last) {  // no expert: zeros
            const size_t n = static_cast<size_t>(a.N);
            for (size_t i = tid; i < n; i += PREP_THREADS) {
                if (a.zero_bytes == 4) static_cast<float *>(a.y)[r * n + i] = 0.f;
                else static_cast<uint16_t *>(a.y)[r * n + i] = 0;
            }
        }
        const int src = r < last ? source_row(a.order, a.k, a.nsrc, r, a.status) : -1;
        if (tid == 0) a.xss[r] = src >= 0 ? a.xs[src] : 0.f;
        __half *out = a.x16 + static_cast<size_t>(r) * a.K;
        for (int c = tid * 16; c < a.K; c += PREP_THREADS * 16) {
            uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
            if (src >= 0) {
                const uint4 v = *reinterpret_cast<const uint4 *>(a.xq + static_cast<size_t>(src) * a.K + c);
                s8x4_to_f16(v.x, lo.x, lo.y);
                s8x4_to_f16(v.y, lo.z, lo.w);
                s8x4_to_f16(v.z, hi.x, hi.y);
                s8x4_to_f16(v.w, hi.z, hi.w);
            }
            reinterpret_cast<uint4 *>(out + c)[0] = lo;
            reinterpret_cast<uint4 *>(out + c)[1] = hi;
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

// Row tile: 192 where the experts have more than a small tile of rows on
// average, 64 (single CTAs, a deep ring of weights) where the product is
// bound by reading the weights.
int pick_nt(int R, int n) { return R > 64LL * n ? 192 : 64; }

struct Layout {
    size_t tiles, xss, x16, total;
};

Layout layout(int R, int n, int K)
{
    Layout l;
    l.tiles = 256;
    l.xss = l.tiles + up256(static_cast<size_t>(most_tiles(R, n, 64)) * sizeof(Tile));
    l.x16 = l.xss + up256(static_cast<size_t>(R) * sizeof(float));
    l.total = l.x16 + up256(static_cast<size_t>(R) * K * sizeof(__half));
    return l;
}

// Clusters of a kernel that the current device holds at once (a cluster's
// CTAs share a GPC, so this may be fewer than its SMs divided), looked up
// once per kernel type and device; 0 if unknown.
template <typename K>
int resident_clusters(K kernel, int csize, size_t smem)
{
    static std::atomic<int> cache[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int n = cache[dev].load(std::memory_order_relaxed);
    if (n != 0) return n > 0 ? n : 0;
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
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
        (void)cudaGetLastError();
        n = -1;
    }
    cache[dev].store(n, std::memory_order_relaxed);
    return n > 0 ? n : 0;
}

template <typename T, int NT>
cudaError_t launch_tc(const TcArgs &a, long long most_items, int sms, cudaStream_t stream)
{
    using F = Form<NT>;
    constexpr size_t smem = tc_smem<NT>();
    auto k = q8_tc<T, NT>;
    cudaError_t e = ensure_dynamic_smem(k, smem);
    if (e != cudaSuccess) return e;
    long long clusters = sms / F::CL;
    if (F::CL > 1) {
        const int fit = resident_clusters(k, F::CL, smem);
        if (fit > 0 && fit < clusters) clusters = fit;
    }
    if (most_items < clusters) clusters = most_items;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * F::CL));
    cfg.blockDim = dim3(TC_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = F::CL;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = F::CL > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k, a);
}

}  // namespace

size_t q8_tc_workspace(int R, int n, int K) { return layout(R, n, K).total; }

cudaError_t launch_q8_tc(const Q8Call &c, void *workspace, cudaStream_t stream)
{
    const DeviceInfo *dev = device_info();
    unsigned *status = device_status_word();
    if (!dev || !status) return cudaErrorInvalidDevice;
    char *ws = static_cast<char *>(workspace);
    const Layout l = layout(c.R, c.n, c.K);
    const int nt = pick_nt(c.R, c.n);
    const int max_tiles = most_tiles(c.R, c.n, nt);
    int *ntiles = reinterpret_cast<int *>(ws);
    Tile *tiles = reinterpret_cast<Tile *>(ws + l.tiles);
    float *xss = reinterpret_cast<float *>(ws + l.xss);
    __half *x16 = reinterpret_cast<__half *>(ws + l.x16);

    TcArgs a = {};
    if (!encode(&a.wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, c.wq, c.K, static_cast<long long>(c.n) * c.N, 128, MT) ||
        !encode(&a.xmap, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, x16, c.K, c.R, KT, nt == 192 ? Form<192>::BOX : Form<64>::BOX))
        return cudaErrorInvalidValue;
    const PrepArgs p = {c.xq, c.xs, c.order, c.offsets, x16, xss, c.y, ntiles, tiles, status, c.nsrc, c.k, c.R, c.n, c.K,
                        c.N, nt, max_tiles, c.dtype == SMOE_BF16 ? 2 : 4};
    const int rows_blocks = c.R < dev->sm_count * 8 ? c.R : dev->sm_count * 8;
    cudaError_t e = launch_pdl(q8_prep, dim3(static_cast<unsigned>(rows_blocks + (c.offsets ? 1 : 0))), dim3(PREP_THREADS), 0,
                               stream, p);
    if (e != cudaSuccess) return e;
    a.ws = c.ws;
    a.xs = xss;
    a.y = c.y;
    a.ntiles = ntiles;
    a.tiles = c.offsets ? tiles : nullptr;
    a.status = status;
    a.R = c.R;
    a.N = c.N;
    a.K = c.K;
    const int nd = (c.R + nt - 1) / nt;
    a.step = ((c.R + nd - 1) / nd + 15) & ~15;
    a.mtiles = (c.N + MT - 1) / MT;
    const int cl = nt == 192 ? 2 : 1;
    const long long most = static_cast<long long>(c.offsets ? max_tiles : nd) * ((a.mtiles + cl - 1) / cl);
    if (c.dtype == SMOE_BF16)
        return nt == 192 ? launch_tc<__nv_bfloat16, 192>(a, most, dev->sm_count, stream)
                         : launch_tc<__nv_bfloat16, 64>(a, most, dev->sm_count, stream);
    return nt == 192 ? launch_tc<float, 192>(a, most, dev->sm_count, stream)
                     : launch_tc<float, 64>(a, most, dev->sm_count, stream);
}

}  // namespace smoe
