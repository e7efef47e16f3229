// Many tokens between the router and the experts: the top-k selection of
// every row of logits, the stable sort of the tokens' slots by expert with
// the gather of their rows, the weighted sum of the experts' rows back into
// token order, and the gradients of all three.
//
// A slot a = t k + s is the s-th selection of token t.  The sort gives every
// slot a row: rows [offsets[e], offsets[e + 1]) belong to expert e, in slot
// order; slots without an expert take the rows past offsets[E] and their
// place is written as -1 - row.
#include "common.cuh"
#include "internal_tokens.h"
#include "rowvec.cuh"
#include "smoe.h"

namespace smoe {
namespace {

constexpr uint32_t kKeyNegInf = 0x007FFFFFu;  // value_key(-inf)

// Order-preserving 32-bit key of a logit: larger = ranks first, NaN below
// every number (1), 0 = retired.  -0 ranks with +0 (v + 0).
__device__ __forceinline__ uint32_t value_key(float v)
{
    const uint32_t u = __float_as_uint(v + 0.f);
    const uint32_t key = u ^ (static_cast<uint32_t>(static_cast<int>(u) >> 31) | 0x80000000u);
    return v != v ? 1u : key;
}

__device__ __forceinline__ float value_of_key(uint32_t u)
{
    if (u <= 1u) return __int_as_float(0x7fffffff);
    return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}

// Softmax over the k selected values of one row, by one warp: lane l holds
// ranks l and l + 32 (keys ka, kb; indices ea, eb).  A selected -inf is a
// masked expert: index -1, weight 0, and a row of nothing else is all that.
__device__ __forceinline__ void write_row(uint32_t ka, uint32_t kb, int ea, int eb, int k, int *__restrict__ idx,
                                          float *__restrict__ w)
{
    const int lane = threadIdx.x & 31;
    const float v0 = value_of_key(__shfl_sync(FULL_MASK, ka, 0));
    const bool ha = lane < k && ka != kKeyNegInf, hb = lane + 32 < k && kb != kKeyNegInf;
    const float xa = ha ? expf(value_of_key(ka) - v0) : 0.f;
    const float xb = k > 32 && hb ? expf(value_of_key(kb) - v0) : 0.f;
    float sum = xa + xb;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(FULL_MASK, sum, off);
    if (lane < k) {
        idx[lane] = ha ? ea : -1;
        w[lane] = ha ? xa / sum : 0.f;
    }
    if (lane + 32 < k) {
        idx[lane + 32] = hb ? eb : -1;
        w[lane + 32] = hb ? xb / sum : 0.f;
    }
}

constexpr int TOPK_WARPS = 8;

// k rounds of a warp-wide maximum over V keys per lane (expert i 32 + lane);
// among equal values the lowest expert wins.  Lane l ends with ranks l and
// l + 32.  Any k, any ties.
template <int V>
__device__ __forceinline__ void select_by_rounds(uint32_t (&key)[V], int k, uint32_t &ka, uint32_t &kb, int &ea, int &eb)
{
    const int lane = threadIdx.x & 31;
    for (int r = 0; r < k; ++r) {
        uint32_t best = key[0];
        int bi = 0;
#pragma unroll
        for (int i = 1; i < V; ++i)
            if (key[i] > best) {
                best = key[i];
                bi = i;
            }
        const uint32_t top = __reduce_max_sync(FULL_MASK, best);
        const unsigned e = __reduce_min_sync(FULL_MASK, best == top ? static_cast<unsigned>(bi * 32 + lane) : 0xFFFFFFFFu);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (e == static_cast<unsigned>(i * 32 + lane)) key[i] = 0u;  // retired
        if ((r & 31) == lane) {
            if (r < 32) {
                ka = top;
                ea = static_cast<int>(e);
            } else {
                kb = top;
                eb = static_cast<int>(e);
            }
        }
    }
}

// The filter of a row for k <= FILTER_K: the k-th largest of the lanes' maxima
// is a lower bound of the k-th largest logit; the few logits not below it (k
// and one or two more, as a rule) are gathered one to a lane in expert order,
// where counting the larger ones gives each its rank.  Against k rounds over
// the whole row (us, 32,768 rows): 128 experts, k = 8 11.8 / 17.5, k = 16 16.2 /
// 29.6; 512 experts, k = 8 21.3 / 46.6.
constexpr int FILTER_K = 16;

// The bound from every lane's maximum `most`; first: the row's largest key.
__device__ __forceinline__ uint32_t filter_bound(uint32_t most, int k, uint32_t &first)
{
    first = __reduce_max_sync(FULL_MASK, most);
    uint32_t bound = first;
    if (most == first) most = 0u;
#pragma unroll 4
    for (int r = 1; r < k; ++r) {
        const uint32_t top = __reduce_max_sync(FULL_MASK, most);
        if (top != 0u) bound = top;  // 0: every lane's maximum is among them
        if (most == top) most = 0u;
    }
    return bound;
}

// The filter's candidates of one row: keys in expert order, then zeros.
struct Candidates {
    uint32_t key[32];
    uint16_t expert[32];
};

// One step of the gathering: this lane's key (expert e) joins if `in`.
__device__ __forceinline__ void gather_candidate(Candidates &c, bool in, uint32_t key, int e, int &count)
{
    const uint32_t m = __ballot_sync(FULL_MASK, in);
    const int at = count + __popc(m & ((1u << (threadIdx.x & 31)) - 1u));
    if (in && at < 32) {
        c.key[at] = key;
        c.expert[at] = static_cast<uint16_t>(e);
    }
    count += __popc(m);
}

// Ranks and weighs `count` <= 32 candidates and writes the row's k selected.
__device__ __forceinline__ void write_candidates(const Candidates &cand, int count, uint32_t first, int k,
                                                 int *__restrict__ idx, float *__restrict__ w)
{
    const int lane = threadIdx.x & 31;
    __syncwarp();
    // the larger ones, and of the equal ones those before it (in expert order)
    const uint32_t mine = cand.key[lane];
    int rank = 0;
    for (int c = 0; c < count; c += 4) {
        const uint4 o = *reinterpret_cast<const uint4 *>(&cand.key[c]);
        rank += o.x >= mine + (c >= lane ? 1u : 0u);
        rank += o.y >= mine + (c + 1 >= lane ? 1u : 0u);
        rank += o.z >= mine + (c + 2 >= lane ? 1u : 0u);
        rank += o.w >= mine + (c + 3 >= lane ? 1u : 0u);
    }
    const bool sel = lane < count && rank < k, there = sel && mine != kKeyNegInf;
    const float x = there ? expf(value_of_key(mine) - value_of_key(first)) : 0.f;
    float sum = x;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(FULL_MASK, sum, off);
    if (sel) {
        idx[rank] = there ? static_cast<int>(cand.expert[lane]) : -1;
        w[rank] = there ? x / sum : 0.f;
    }
}

// A row whose k selected are all masked experts.  That no logit beats -inf does
// not say so: a NaN ranks below it, and is selected where fewer than k are -inf.
__device__ __forceinline__ void write_masked(int k, int *__restrict__ idx, float *__restrict__ w)
{
    for (int r = threadIdx.x & 31; r < k; r += 32) {
        idx[r] = -1;
        w[r] = 0.f;
    }
}

// n <= 32 V: one warp per row, V logits per lane; the filter up to k = FILTER_K,
// rounds above it or where more than 32 candidates are left (ties).  Bound by
// instruction issue (32,768 rows of 128, k = 8: 340 a row).
template <int V>
__global__ void __launch_bounds__(TOPK_WARPS * 32) topk_rows_warp(const float *__restrict__ logits, int T, int n, int ld,
                                                                  int k, int *__restrict__ idx, float *__restrict__ w)
{
    __shared__ __align__(16) Candidates cands[TOPK_WARPS];
    const int wi = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x * TOPK_WARPS + wi;
    pdl_launch_dependents();
    pdl_wait();
    if (t >= T) return;
    const float *row = logits + static_cast<size_t>(t) * ld;
    idx += static_cast<size_t>(t) * k;
    w += static_cast<size_t>(t) * k;
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = i * 32 + lane < n ? value_key(row[i * 32 + lane]) : 0u;
    if (k <= FILTER_K) {
        uint32_t most = key[0], first;
#pragma unroll
        for (int i = 1; i < V; ++i) most = max(most, key[i]);
        const uint32_t bound = filter_bound(most, k, first);
        if (first == kKeyNegInf) {
            int masked = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) masked += key[i] == kKeyNegInf;
            if (__reduce_add_sync(FULL_MASK, masked) >= k) {
                write_masked(k, idx, w);
                return;
            }
        }
        Candidates &c = cands[wi];
        c.key[lane] = 0u;
        __syncwarp();
        int count = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) gather_candidate(c, key[i] >= bound, key[i], i * 32 + lane, count);
        if (count <= 32) {
            write_candidates(c, count, first, k, idx, w);
            return;
        }
    }
    uint32_t ka = 0u, kb = 0u;
    int ea = -1, eb = -1;
    select_by_rounds<V>(key, k, ka, kb, ea, eb);
    write_row(ka, kb, ea, eb, k, idx, w);
}

// n <= LONG_EXPERTS, k <= FILTER_K: the same filter over two passes of the row,
// the second out of the cache; where more than 32 candidates are left (ties), k
// passes that each find the next one in order.  Against one CTA per row
// (topk_rows_block; us, k = 8): 1 row of 520 3.3 / 4.8, 1 of 1024 4.3 / 4.3,
// 3000 of 1024 6.7 / 24.5, 32,768 of 520 34.8 / 216; but 1 of 8192 19.4 / 7.2.
constexpr int LONG_EXPERTS = 2048;

__global__ void __launch_bounds__(TOPK_WARPS * 32) topk_rows_long(const float *__restrict__ logits, int T, int n, int ld,
                                                                  int k, int *__restrict__ idx, float *__restrict__ w)
{
    __shared__ __align__(16) Candidates cands[TOPK_WARPS];
    const int wi = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x * (blockDim.x >> 5) + wi;
    pdl_launch_dependents();
    pdl_wait();
    if (t >= T) return;
    const float *row = logits + static_cast<size_t>(t) * ld;
    idx += static_cast<size_t>(t) * k;
    w += static_cast<size_t>(t) * k;
    // eight loads in flight at a time
    uint32_t most = 0u, first;
    float v[8];
    auto fetch = [&](int e0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = e0 + i * 32 + lane < n ? row[e0 + i * 32 + lane] : 0.f;
    };
    for (int e0 = 0; e0 < n; e0 += 256) {
        fetch(e0);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (e0 + i * 32 + lane < n) most = max(most, value_key(v[i]));
    }
    const uint32_t bound = filter_bound(most, k, first);
    if (first == kKeyNegInf) {
        int masked = 0;
        for (int e0 = 0; e0 < n && masked < k; e0 += 32)
            masked += __popc(__ballot_sync(FULL_MASK, e0 + lane < n && value_key(row[e0 + lane]) == kKeyNegInf));
        if (masked >= k) {
            write_masked(k, idx, w);
            return;
        }
    }
    Candidates &c = cands[wi];
    c.key[lane] = 0u;
    __syncwarp();
    int count = 0;
    for (int e0 = 0; e0 < n; e0 += 256) {
        fetch(e0);
        uint32_t key[8], in = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            key[i] = e0 + i * 32 + lane < n ? value_key(v[i]) : 0u;
            in |= static_cast<uint32_t>(key[i] >= bound) << i;
        }
        const uint32_t any = __reduce_or_sync(FULL_MASK, in);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (any >> i & 1u) gather_candidate(c, in >> i & 1u, key[i], e0 + i * 32 + lane, count);
    }
    if (count <= 32) {
        write_candidates(c, count, first, k, idx, w);
        return;
    }
    uint32_t ka = 0u, last = 0xFFFFFFFFu;
    int ea = -1, last_e = -1;
    for (int r = 0; r < k; ++r) {
        uint32_t best = 0u, be = 0xFFFFFFFFu;
        for (int e = lane; e < n; e += 32) {
            const uint32_t key = value_key(row[e]);
            if ((key < last || (key == last && e > last_e)) && key > best) {
                best = key;
                be = static_cast<uint32_t>(e);
            }
        }
        last = __reduce_max_sync(FULL_MASK, best);
        last_e = static_cast<int>(__reduce_min_sync(FULL_MASK, best == last ? be : 0xFFFFFFFFu));
        if (lane == r) {
            ka = last;
            ea = last_e;
        }
    }
    write_row(ka, 0u, ea, -1, k, idx, w);
}

constexpr int TOPK_BLOCK = 256;

// Any n and k: one CTA per row, k rounds over the keys in shared memory.
__global__ void __launch_bounds__(TOPK_BLOCK) topk_rows_block(const float *__restrict__ logits, int n, int ld, int k,
                                                              int *__restrict__ idx, float *__restrict__ w)
{
    extern __shared__ uint32_t keys[];  // [n]
    __shared__ unsigned long long warp_best[TOPK_BLOCK / 32];
    __shared__ uint32_t sel_k[SMOE_MAX_TOP_K];
    __shared__ int sel_e[SMOE_MAX_TOP_K];
    const int tid = threadIdx.x;
    pdl_launch_dependents();
    pdl_wait();
    const size_t t = blockIdx.x;
    const float *row = logits + t * ld;
    for (int e = tid; e < n; e += TOPK_BLOCK) keys[e] = value_key(row[e]);
    __syncthreads();
    for (int r = 0; r < k; ++r) {
        unsigned long long best = 0;
        for (int e = tid; e < n; e += TOPK_BLOCK) {
            const unsigned long long c =
                (static_cast<unsigned long long>(keys[e]) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(e));
            best = c > best ? c : best;
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            const unsigned long long o = __shfl_xor_sync(FULL_MASK, best, off);
            best = o > best ? o : best;
        }
        if ((tid & 31) == 0) warp_best[tid >> 5] = best;
        __syncthreads();
        if (tid == 0) {
            for (int i = 1; i < TOPK_BLOCK / 32; ++i) best = warp_best[i] > best ? warp_best[i] : best;
            const int e = static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(best));
            sel_k[r] = static_cast<uint32_t>(best >> 32);
            sel_e[r] = e;
            keys[e] = 0u;  // retired
        }
        __syncthreads();
    }
    if (tid < 32) {
        const uint32_t ka = tid < k ? sel_k[tid] : 0u, kb = tid + 32 < k ? sel_k[tid + 32] : 0u;
        const int ea = tid < k ? sel_e[tid] : -1, eb = tid + 32 < k ? sel_e[tid + 32] : -1;
        write_row(ka, kb, ea, eb, k, idx + t * k, w + t * k);
    }
}

constexpr int GRAD_ROWS = 2;  // rows per warp, whose loads are in flight together

// dl[idx[r]] = w[r] (dw[r] - sum_q w[q] dw[q]), every other logit's gradient
// is 0.  A warp writes its rows' zeros while their few inputs are on their
// way, then the selected ones.
__global__ void __launch_bounds__(TOPK_WARPS * 32) topk_rows_grad(const int *__restrict__ idx, const float *__restrict__ w,
                                                                  const float *__restrict__ dw, int T, int n, int k,
                                                                  float *__restrict__ dl)
{
    const int t0 = (blockIdx.x * TOPK_WARPS + (threadIdx.x >> 5)) * GRAD_ROWS;
    const int lane = threadIdx.x & 31;
    pdl_launch_dependents();
    pdl_wait();
    if (t0 >= T) return;
    int e[GRAD_ROWS][2];
    float wr[GRAD_ROWS][2], g[GRAD_ROWS][2];
#pragma unroll
    for (int i = 0; i < GRAD_ROWS; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const bool in = t0 + i < T && lane + 32 * h < k;
            const size_t a = static_cast<size_t>(t0 + i) * k + lane + 32 * h;
            e[i][h] = in ? idx[a] : -1;
            wr[i][h] = in ? w[a] : 0.f;
            g[i][h] = in ? dw[a] : 0.f;
        }
    float *row = dl + static_cast<size_t>(t0) * n;
    const int words = min(GRAD_ROWS, T - t0) * n;
    if ((n & 3) == 0) {
        for (int c = lane; c < (words >> 2); c += 32) reinterpret_cast<float4 *>(row)[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    } else {
        for (int c = lane; c < words; c += 32) row[c] = 0.f;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < GRAD_ROWS; ++i) {
        // a slot without an expert has no weight, and its gradient is nothing
        float c = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (e[i][h] >= 0 && e[i][h] < n) c = fmaf(wr[i][h], g[i][h], c);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) c += __shfl_xor_sync(FULL_MASK, c, off);
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (e[i][h] >= 0 && e[i][h] < n) row[static_cast<size_t>(i) * n + e[i][h]] = wr[i][h] * (g[i][h] - c);
    }
}

// ---------------------------------------------------------------- the sort

constexpr int SORT_THREADS = 256;  // = slots per chunk

// An index outside [0, n) goes to the bucket n: no expert.
__device__ __forceinline__ int bucket(int e, int n) { return e >= 0 && e < n ? e : n; }

// hist[c][e] = slots of chunk c in bucket e <= n.
__global__ void __launch_bounds__(SORT_THREADS) sort_hist(const int *__restrict__ top_idx, int R, int n,
                                                          int *__restrict__ hist)
{
    extern __shared__ int cnt[];  // [n + 1]
    pdl_launch_dependents();
    for (int e = threadIdx.x; e <= n; e += SORT_THREADS) cnt[e] = 0;
    __syncthreads();
    pdl_wait();
    const long long a = static_cast<long long>(blockIdx.x) * SORT_THREADS + threadIdx.x;
    if (a < R) atomicAdd(&cnt[bucket(top_idx[a], n)], 1);
    __syncthreads();
    int *h = hist + static_cast<size_t>(blockIdx.x) * (n + 1);
    for (int e = threadIdx.x; e <= n; e += SORT_THREADS) h[e] = cnt[e];
}

// hist[c][e] becomes the sum over earlier chunks, total[e] the sum over all.
// A CTA takes 32 buckets; its 32 warps take equal runs of chunks.
__global__ void __launch_bounds__(1024) sort_scan(int *__restrict__ hist, int *__restrict__ total, int nchunks, int n)
{
    __shared__ int part[32][33];
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, wi = threadIdx.x >> 5;
    const int e = blockIdx.x * 32 + lane;
    const int per = (nchunks + 31) / 32;
    const int c0 = min(nchunks, wi * per), c1 = min(nchunks, c0 + per);
    int sum = 0;
    if (e <= n)
        for (int c = c0; c < c1; ++c) sum += hist[static_cast<size_t>(c) * (n + 1) + e];
    part[wi][lane] = sum;
    __syncthreads();
    int before = 0;
    for (int i = 0; i < wi; ++i) before += part[i][lane];
    if (e <= n) {
        for (int c = c0; c < c1; ++c) {
            int *h = hist + static_cast<size_t>(c) * (n + 1) + e;
            const int v = *h;
            *h = before;
            before += v;
        }
        if (wi == 31) total[e] = before;
    }
}

// Exclusive prefix sum of v over the block's threads (blockDim.x <= 1024).
__device__ __forceinline__ int block_exclusive(int v, int *warp_sums)
{
    const int lane = threadIdx.x & 31, wi = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(FULL_MASK, inc, off);
        if (lane >= off) inc += o;
    }
    if (lane == 31) warp_sums[wi] = inc;
    __syncthreads();
    int before = 0;
    for (int i = 0; i < wi; ++i) before += warp_sums[i];
    __syncthreads();
    return before + inc - v;
}

// Row of every slot: the bucket's first row, the bucket's slots in earlier
// chunks, and the equal slots before it in its own chunk.
__global__ void __launch_bounds__(SORT_THREADS) sort_place(const int *__restrict__ top_idx, int R, int n,
                                                           const int *__restrict__ hist, const int *__restrict__ total,
                                                           int *__restrict__ offsets, int *__restrict__ order,
                                                           int *__restrict__ place)
{
    extern __shared__ int first[];  // [n + 1]
    __shared__ __align__(16) int mine[SORT_THREADS];
    __shared__ int warp_sums[SORT_THREADS / 32];
    const int tid = threadIdx.x;
    pdl_launch_dependents();
    pdl_wait();
    const long long a = static_cast<long long>(blockIdx.x) * SORT_THREADS + tid;
    const int e = a < R ? bucket(top_idx[a], n) : n + 1;
    mine[tid] = e;
    int run = 0;
    for (int b = 0; b <= n; b += SORT_THREADS) {
        const int v = b + tid <= n ? total[b + tid] : 0;
        const int ex = run + block_exclusive(v, warp_sums);
        if (b + tid <= n) first[b + tid] = ex;
        if (tid == SORT_THREADS - 1) warp_sums[0] = ex + v;
        __syncthreads();
        run = warp_sums[0];
        __syncthreads();
    }
    if (blockIdx.x == 0)
        for (int i = tid; i <= n; i += SORT_THREADS) offsets[i] = first[i];
    if (a >= R) return;
    int rank = 0;
    for (int i = 0; i < (tid >> 2); ++i) {
        const int4 o = reinterpret_cast<const int4 *>(mine)[i];
        rank += (o.x == e) + (o.y == e) + (o.z == e) + (o.w == e);
    }
    for (int i = tid & ~3; i < tid; ++i) rank += mine[i] == e;
    const int row = first[e] + hist[static_cast<size_t>(blockIdx.x) * (n + 1) + e] + rank;
    order[row] = static_cast<int>(a);
    place[a] = e < n ? row : -1 - row;
}

// ---------------------------------------------------------------- small sorts

constexpr int SMALL_THREADS = 256;

constexpr int ODD_COLS = 256;  // columns that a warp takes at a time of rows that no 16-byte vector fits

// This CTA's share (blockIdx.y of gridDim.y) of nt tokens' rows, each copied to
// the rows of its k slots; a slot without an expert gets zeros.  The tokens'
// vectors are one sequence over the threads, so that short rows fill them.
template <typename T, int VE>
__device__ __forceinline__ void copy_rows(const T *__restrict__ x, const int *rows, int nt, int k, int d, T *__restrict__ xs)
{
    if constexpr (VE == 1) {
        // rows that no vector fits: a warp takes 256 columns, eight a lane
        const int lane = threadIdx.x & 31, blocks = (d + ODD_COLS - 1) / ODD_COLS;
        const int warps = SMALL_THREADS / 32;
        for (int i = blockIdx.y * warps + (threadIdx.x >> 5); i < nt * blocks; i += gridDim.y * warps) {
            const int j = i / blocks, c0 = (i - j * blocks) * ODD_COLS + lane;
            RowVec<T, 1> v[ODD_COLS / 32], z;
            z.zero();
#pragma unroll
            for (int u = 0; u < ODD_COLS / 32; ++u)
                if (c0 + 32 * u < d) v[u].load(x + static_cast<size_t>(j) * d + c0 + 32 * u);
            for (int s = 0; s < k; ++s) {
                const int p = rows[j * k + s];
                T *to = xs + static_cast<size_t>(p >= 0 ? p : -1 - p) * d + c0;
#pragma unroll
                for (int u = 0; u < ODD_COLS / 32; ++u)
                    if (c0 + 32 * u < d) (p >= 0 ? v[u] : z).store(to + 32 * u);
            }
        }
    } else {
        const int nvec = d / VE;
        for (int i = blockIdx.y * SMALL_THREADS + threadIdx.x; i < nt * nvec; i += gridDim.y * SMALL_THREADS) {
            const int j = nt > 1 ? i / nvec : 0, c = (i - j * nvec) * VE;
            RowVec<T, VE> v, z;
            v.load(x + static_cast<size_t>(j) * d + c);
            z.zero();
            for (int s = 0; s < k; ++s) {
                const int p = rows[j * k + s];
                if (p >= 0) v.store(xs + static_cast<size_t>(p) * d + c);
                else z.store(xs + static_cast<size_t>(-1 - p) * d + c);
            }
        }
    }
}

// The whole dispatch of a small batch in one launch: every CTA finds the
// rows of its own token's slots by counting, over all R slots, those that
// sort before them, then copies its share of the token's row; one CTA more
// counts the buckets and writes the offsets.  R^2 / 32 warp steps in all.
// Against the two launches of the middle form (us, rows of 512 bytes, 128
// experts): 256 slots 2.1 / 4.2, 1024 slots 3.3 / 4.3, 2048 slots 5.2 / 4.3.
constexpr int SMALL_SLOTS = 1536;

template <typename T, int VE>
__global__ void __launch_bounds__(SMALL_THREADS) dispatch_small(const int *__restrict__ top_idx, int tokens, int tpc, int k, int n,
                                                                const T *__restrict__ x, int d, int *__restrict__ offsets,
                                                                int *__restrict__ order, int *__restrict__ place,
                                                                T *__restrict__ xs)
{
    extern __shared__ int cnt[];  // [n + 1]; the gathering CTAs use [0, tpc k) for their rows
    __shared__ int warp_sums[SMALL_THREADS / 32];
    const int tid = threadIdx.x, lane = tid & 31;
    const int R = tokens * k;
    pdl_launch_dependents();
    if (blockIdx.x == gridDim.x - 1) {
        if (blockIdx.y != 0) return;
        for (int e = tid; e <= n; e += SMALL_THREADS) cnt[e] = 0;
        __syncthreads();
        pdl_wait();
        for (int a = tid; a < R; a += SMALL_THREADS) atomicAdd(&cnt[bucket(top_idx[a], n)], 1);
        __syncthreads();
        int run = 0;
        for (int b = 0; b <= n; b += SMALL_THREADS) {
            const int v = b + tid <= n ? cnt[b + tid] : 0;
            const int ex = run + block_exclusive(v, warp_sums);
            if (b + tid <= n) offsets[b + tid] = ex;
            if (tid == SMALL_THREADS - 1) warp_sums[0] = ex + v;
            __syncthreads();
            run = warp_sums[0];
            __syncthreads();
        }
        return;
    }
    pdl_wait();
    const int t0 = blockIdx.x * tpc, nt = min(tpc, tokens - t0);
    for (int s = tid >> 5; s < nt * k; s += SMALL_THREADS / 32) {
        const int a = t0 * k + s;
        const int e = bucket(top_idx[a], n);
        int before = 0;
        for (int b = lane; b < R; b += 32) {
            const int o = bucket(top_idx[b], n);
            before += o < e || (o == e && b < a);
        }
        const int row = __reduce_add_sync(FULL_MASK, before);
        if (lane == 0) {
            cnt[s] = e < n ? row : -1 - row;
            if (blockIdx.y == 0) {
                order[row] = a;
                place[a] = e < n ? row : -1 - row;
            }
        }
    }
    if (!xs) return;
    __syncthreads();
    copy_rows<T, VE>(x + static_cast<size_t>(t0) * d, cnt, nt, k, d, xs);
}

// ---------------------------------------------------------------- middle sorts

// Between the one-launch dispatch and the four launches of a large one: with
// few chunks a slot's row needs no scan of its own.  sort_below leaves, for
// every chunk c and bucket e, how many of the chunk's slots are in buckets
// below e (cum[e][c]); the row of a slot of bucket e in chunk c is then
//   sum over all c' of cum[e][c'] + sum over c' < c of (cum[e + 1][c'] -
//   cum[e][c']) + the equal slots before it in its chunk,
// two short rows that the slot's warp reads in a step or four.  Against the
// four launches (us, as above): 8000 slots 5.4 / 8.5, 24,000 slots 9.7 / 12.0,
// 32,768 slots 12.1 / 12.2.
constexpr int MIDDLE_CHUNKS = 128;

constexpr int MIDDLE_SMALL_CHUNK = 256, MIDDLE_LARGE_CHUNK = 1024;

// One CTA per chunk, one thread per slot.
__global__ void __launch_bounds__(MIDDLE_LARGE_CHUNK) sort_below(const int *__restrict__ top_idx, int R, int n, int nchunks,
                                                                 int *__restrict__ cum)
{
    extern __shared__ int cnt[];  // [n + 1]
    __shared__ int warp_sums[MIDDLE_LARGE_CHUNK / 32];
    pdl_launch_dependents();
    const int tid = threadIdx.x, threads = blockDim.x;
    for (int e = tid; e <= n; e += threads) cnt[e] = 0;
    __syncthreads();
    pdl_wait();
    const int a = blockIdx.x * threads + tid;
    if (a < R) atomicAdd(&cnt[bucket(top_idx[a], n)], 1);
    __syncthreads();
    int run = 0;
    for (int b = 0; b <= n; b += threads) {
        const int v = b + tid <= n ? cnt[b + tid] : 0;
        const int ex = run + block_exclusive(v, warp_sums);
        if (b + tid <= n) cum[static_cast<size_t>(b + tid) * nchunks + blockIdx.x] = ex;
        if (tid == threads - 1) warp_sums[0] = ex + v;
        __syncthreads();
        run = warp_sums[0];
        __syncthreads();
    }
    if (tid == 0) cum[static_cast<size_t>(n + 1) * nchunks + blockIdx.x] = run;
}

// The first CTAs: tpc tokens' rows found as above and the tokens' rows copied to
// them; the CTAs behind: the offsets, a warp each.
template <typename T, int VE>
__global__ void __launch_bounds__(SMALL_THREADS) dispatch_middle(const int *__restrict__ top_idx, int tokens, int tpc, int k, int n,
                                                                 int nchunks, int chunk, const int *__restrict__ cum,
                                                                 const T *__restrict__ x, int d, int *__restrict__ offsets,
                                                                 int *__restrict__ order, int *__restrict__ place,
                                                                 T *__restrict__ xs)
{
    __shared__ int rows[SMOE_MAX_TOP_K];
    const int tid = threadIdx.x, lane = tid & 31;
    pdl_launch_dependents();
    pdl_wait();
    const int ctas = (tokens + tpc - 1) / tpc;
    if (static_cast<int>(blockIdx.x) >= ctas) {
        const int e = (blockIdx.x - ctas) * (SMALL_THREADS / 32) + (tid >> 5);
        if (e > n || blockIdx.y != 0) return;
        int first = 0;
        for (int c = lane; c < nchunks; c += 32) first += cum[static_cast<size_t>(e) * nchunks + c];
        first = __reduce_add_sync(FULL_MASK, first);
        if (lane == 0) offsets[e] = first;
        return;
    }
    const int t0 = blockIdx.x * tpc, nt = min(tpc, tokens - t0);
    for (int s = tid >> 5; s < nt * k; s += SMALL_THREADS / 32) {
        const int a = t0 * k + s;
        const int e = bucket(top_idx[a], n), mine = a / chunk;
        const int *lo = cum + static_cast<size_t>(e) * nchunks, *hi = lo + nchunks;
        int before = 0;
        for (int c = lane; c < nchunks; c += 32) before += c < mine ? hi[c] : lo[c];
        for (int b = mine * chunk + lane; b < a; b += 32) before += bucket(top_idx[b], n) == e;
        const int row = __reduce_add_sync(FULL_MASK, before);
        if (lane == 0) {
            rows[s] = e < n ? row : -1 - row;
            if (blockIdx.y == 0) {
                order[row] = a;
                place[a] = e < n ? row : -1 - row;
            }
        }
    }
    if (!xs) return;
    __syncthreads();
    copy_rows<T, VE>(x + static_cast<size_t>(t0) * d, rows, nt, k, d, xs);
}

// ---------------------------------------------------------------- rows

constexpr int ROW_THREADS = 256;

// A place read from device memory, checked: the row (>= 0) of a slot with an
// expert, or -1.  A row outside [0, R) is reported and treated as none.
__device__ __forceinline__ int checked_place(int p, int R, unsigned *status)
{
    if (p >= R || p < -R) {
        atomicExch(status, kStatusRoute);
        return -1;
    }
    return p;
}

// xs[place[t, s]] = x[t]; the rows of slots without an expert are zeros.  A
// CTA takes tpc tokens and a column block: x is read once and written k
// times.  Bound by HBM writes (16,400 tokens of 8 KB, k = 8: 190 us, 95% of the
// copy rate).
template <typename T, int VE>
__global__ void __launch_bounds__(ROW_THREADS) gather_rows(const T *__restrict__ x, const int *__restrict__ place,
                                                           int tokens, int tpc, int k, int d, T *__restrict__ xs)
{
    static_assert(ROW_THREADS == SMALL_THREADS, "copy_rows");
    pdl_launch_dependents();
    pdl_wait();
    const int t0 = blockIdx.x * tpc;
    copy_rows<T, VE>(x + static_cast<size_t>(t0) * d, place + static_cast<size_t>(t0) * k, min(tpc, tokens - t0), k, d, xs);
}

// out[t] = sum over s, in order, of w[t, s] ys[place[t, s]] (w null: of the
// rows themselves), f32 sums.  A thread takes a vector of a token's row, four
// slots' loads in flight; a CTA tpc tokens and a column block.  Bound by HBM
// reads (4099 tokens of 16 KB, k = 8, one slot in twenty without an expert: 88.7
// us, 98% of the copy rate).
template <typename T, int VE>
__global__ void __launch_bounds__(ROW_THREADS) sum_rows(const T *__restrict__ ys, const int *__restrict__ place,
                                                        const float *__restrict__ w, int tokens, int tpc, int k, int d,
                                                        T *__restrict__ out, unsigned *status)
{
    pdl_launch_dependents();
    pdl_wait();
    const int t0 = blockIdx.x * tpc, nt = min(tpc, tokens - t0), R = tokens * k;
    if constexpr (VE == 1) {
        // rows that no vector fits: a warp takes 256 columns, eight a lane, so
        // that a slot's place and weight are read once for eight (511 columns
        // of bf16, 4001 tokens, k = 8: 20.1 us with one a lane, 15.5 so; 512
        // columns in vectors 8.2)
        const int lane = threadIdx.x & 31, blocks = (d + ODD_COLS - 1) / ODD_COLS, warps = ROW_THREADS / 32;
        for (int i = blockIdx.y * warps + (threadIdx.x >> 5); i < nt * blocks; i += gridDim.y * warps) {
            const int j = i / blocks, c0 = (i - j * blocks) * ODD_COLS + lane;
            const size_t t = t0 + j;
            float acc[ODD_COLS / 32];
#pragma unroll
            for (int u = 0; u < ODD_COLS / 32; ++u) acc[u] = 0.f;
#pragma unroll 2
            for (int s = 0; s < k; ++s) {
                const int p = checked_place(place[t * k + s], R, status);
                if (p < 0) continue;
                const float ws = w ? w[t * k + s] : 1.f;
                const T *y = ys + static_cast<size_t>(p) * d + c0;
                RowVec<T, 1> v[ODD_COLS / 32];
#pragma unroll
                for (int u = 0; u < ODD_COLS / 32; ++u)
                    if (c0 + 32 * u < d) v[u].load(y + 32 * u);
#pragma unroll
                for (int u = 0; u < ODD_COLS / 32; ++u)
                    if (c0 + 32 * u < d) {
                        float f[1];
                        v[u].get(f);
                        acc[u] = fmaf(ws, f[0], acc[u]);
                    }
            }
#pragma unroll
            for (int u = 0; u < ODD_COLS / 32; ++u)
                if (c0 + 32 * u < d) {
                    const float f[1] = {acc[u]};
                    RowVec<T, 1> o;
                    o.set(f);
                    o.store(out + t * d + c0 + 32 * u);
                }
        }
    } else {
        const int nvec = d / VE;
        for (int i = blockIdx.y * ROW_THREADS + threadIdx.x; i < nt * nvec; i += gridDim.y * ROW_THREADS) {
            const int j = nt > 1 ? i / nvec : 0, c = (i - j * nvec) * VE;
            const size_t t = t0 + j;
            float acc[VE];
#pragma unroll
            for (int v = 0; v < VE; ++v) acc[v] = 0.f;
            for (int s0 = 0; s0 < k; s0 += 4) {
                int p[4];
                float ws[4];
                RowVec<T, VE> y[4];
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    p[s] = s0 + s < k ? checked_place(place[t * k + s0 + s], R, status) : -1;
                    ws[s] = w && s0 + s < k ? w[t * k + s0 + s] : 1.f;
                }
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    if (p[s] >= 0) y[s].load(ys + static_cast<size_t>(p[s]) * d + c);
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    if (p[s] >= 0) {
                        float f[VE];
                        y[s].get(f);
#pragma unroll
                        for (int v = 0; v < VE; ++v) acc[v] = fmaf(ws[s], f[v], acc[v]);
                    }
            }
            RowVec<T, VE> o;
            o.set(acc);
            o.store(out + t * d + c);
        }
    }
}

// d_ys[place[t, s]] = w[t, s] d_out[t] (zeros in the rows of slots without an
// expert) and d_w[t, s] = <d_out[t], ys[place[t, s]]>: one warp per slot.
template <typename T, int VE>
__global__ void __launch_bounds__(ROW_THREADS) combine_grad(const T *__restrict__ d_out, const T *__restrict__ ys,
                                                            const int *__restrict__ place, const float *__restrict__ w,
                                                            int R, int k, int d, T *__restrict__ d_ys,
                                                            float *__restrict__ d_w, unsigned *status)
{
    pdl_launch_dependents();
    pdl_wait();
    const size_t t = blockIdx.x;
    const int lane = threadIdx.x & 31;
    const T *g = d_out + t * d;
    for (int s = threadIdx.x >> 5; s < k; s += ROW_THREADS / 32) {
        const int raw = place[t * k + s];
        const int p = checked_place(raw, R, status);
        if (p < 0) {
            if (raw < 0 && raw >= -R) {
                RowVec<T, VE> z;
                z.zero();
                for (int c = lane * VE; c < d; c += 32 * VE) z.store(d_ys + static_cast<size_t>(-1 - raw) * d + c);
            }
            if (lane == 0) d_w[t * k + s] = 0.f;
            continue;
        }
        const float ws = w[t * k + s];
        float dot = 0.f;
        constexpr int U = VE > 1 ? 2 : (sizeof(T) == 4 ? 4 : 1);  // vectors of each row in flight (as measured)
        for (int c0 = lane * VE; c0 < d; c0 += U * 32 * VE) {
            RowVec<T, VE> gv[U], yv[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c0 + u * 32 * VE < d) {
                    gv[u].load(g + c0 + u * 32 * VE);
                    yv[u].load(ys + static_cast<size_t>(p) * d + c0 + u * 32 * VE);
                }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c0 + u * 32 * VE < d) {
                    float gf[VE], yf[VE];
                    gv[u].get(gf);
                    yv[u].get(yf);
#pragma unroll
                    for (int i = 0; i < VE; ++i) {
                        dot = fmaf(gf[i], yf[i], dot);
                        gf[i] *= ws;
                    }
                    gv[u].set(gf);
                    gv[u].store(d_ys + static_cast<size_t>(p) * d + c0 + u * 32 * VE);
                }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(FULL_MASK, dot, off);
        if (lane == 0) d_w[t * k + s] = dot;
    }
}

__global__ void __launch_bounds__(ROW_THREADS) zero_words(int *__restrict__ p, int n)
{
    pdl_launch_dependents();
    pdl_wait();
    const int i = blockIdx.x * ROW_THREADS + threadIdx.x;
    if (i < n) p[i] = 0;
}

bool vec16(const void *p, size_t row_bytes)
{
    return ((reinterpret_cast<uintptr_t>(p) | row_bytes) & 15u) == 0;
}

}  // namespace

cudaError_t launch_topk_rows(const float *logits, int T, int n, int ld, int k, int *idx, float *w, cudaStream_t stream)
{
    const dim3 grid(static_cast<unsigned>((T + TOPK_WARPS - 1) / TOPK_WARPS)), block(TOPK_WARPS * 32);
    if (n <= 64) return launch_pdl(topk_rows_warp<2>, grid, block, 0, stream, logits, T, n, ld, k, idx, w);
    if (n <= 128) return launch_pdl(topk_rows_warp<4>, grid, block, 0, stream, logits, T, n, ld, k, idx, w);
    if (n <= 256) return launch_pdl(topk_rows_warp<8>, grid, block, 0, stream, logits, T, n, ld, k, idx, w);
    if (n <= 512) return launch_pdl(topk_rows_warp<16>, grid, block, 0, stream, logits, T, n, ld, k, idx, w);
    if (k <= FILTER_K && n <= LONG_EXPERTS) {
        const int warps = T <= 1024 ? 1 : TOPK_WARPS;  // few rows: an SM each
        return launch_pdl(topk_rows_long, dim3(static_cast<unsigned>((T + warps - 1) / warps)),
                          dim3(static_cast<unsigned>(warps * 32)), 0, stream, logits, T, n, ld, k, idx, w);
    }
    const size_t smem = static_cast<size_t>(n) * sizeof(uint32_t);
    return launch_pdl(topk_rows_block, dim3(static_cast<unsigned>(T)), dim3(TOPK_BLOCK), smem, stream, logits, n, ld, k,
                      idx, w);
}

cudaError_t launch_topk_rows_grad(const int *idx, const float *w, const float *dw, int T, int n, int k, float *dl,
                                  cudaStream_t stream)
{
    constexpr int rows = TOPK_WARPS * GRAD_ROWS;
    return launch_pdl(topk_rows_grad, dim3(static_cast<unsigned>((T + rows - 1) / rows)),
                      dim3(TOPK_WARPS * 32), 0, stream, idx, w, dw, T, n, k, dl);
}

cudaError_t launch_zero_words(int *p, int n, cudaStream_t stream)
{
    return launch_pdl(zero_words, dim3(static_cast<unsigned>((n + ROW_THREADS - 1) / ROW_THREADS)), dim3(ROW_THREADS), 0,
                      stream, p, n);
}

size_t dispatch_workspace(int T, int k, int n)
{
    const size_t R = static_cast<size_t>(T) * k;
    const size_t chunks = (R + SORT_THREADS - 1) / SORT_THREADS;
    return ((chunks + 1) * (static_cast<size_t>(n) + 2) * sizeof(int) + 255) & ~static_cast<size_t>(255);
}

namespace {

cudaError_t launch_sort_tokens(const int *top_idx, int R, int n, int *offsets, int *order, int *place, void *workspace,
                               cudaStream_t stream)
{
    const int chunks = (R + SORT_THREADS - 1) / SORT_THREADS;
    int *hist = static_cast<int *>(workspace);
    int *total = hist + static_cast<size_t>(chunks) * (n + 1);
    const size_t smem = (static_cast<size_t>(n) + 1) * sizeof(int);
    cudaError_t e = launch_pdl(sort_hist, dim3(static_cast<unsigned>(chunks)), dim3(SORT_THREADS), smem, stream, top_idx,
                               R, n, hist);
    if (e != cudaSuccess) return e;
    e = launch_pdl(sort_scan, dim3(static_cast<unsigned>((n + 32) / 32)), dim3(1024), 0, stream, hist, total, chunks, n);
    if (e != cudaSuccess) return e;
    return launch_pdl(sort_place, dim3(static_cast<unsigned>(chunks)), dim3(SORT_THREADS), smem, stream, top_idx, R, n,
                      hist, total, offsets, order, place);
}

// Tokens per CTA: as many as their rows' vectors take to fill its threads (or,
// where a warp looks for each slot's row, as their slots take to fill its
// warps), while that leaves four CTAs an SM.
int tokens_per_cta(int tokens, int k, int threads, bool search)
{
    const DeviceInfo *dev = device_info();
    const int sms = dev ? dev->sm_count : 152;
    int tpc = threads > 0 && threads < ROW_THREADS ? ROW_THREADS / threads : 1;
    if (search && tpc < (SMALL_THREADS / 32) / k) tpc = (SMALL_THREADS / 32) / k;
    if (tpc > SMOE_MAX_TOP_K / k) tpc = SMOE_MAX_TOP_K / k;
    while (tpc > 1 && tokens / tpc < 4 * sms) tpc /= 2;
    return tpc;
}

// Threads that a row takes: one a vector, or a warp for ODD_COLS columns.
template <int VE>
int row_threads(int d)
{
    return VE == 1 ? (d + ODD_COLS - 1) / ODD_COLS * 32 : d / VE;
}

// (CTAs of tpc tokens, column blocks).  Every column block looks for its slots'
// rows again, so there are only as many as make eight CTAs an SM.
template <typename T, int VE>
dim3 row_grid(int tokens, int tpc, int d, bool search)
{
    long long cols = (static_cast<long long>(tpc) * row_threads<VE>(d) + ROW_THREADS - 1) / ROW_THREADS;
    const int x = (tokens + tpc - 1) / tpc;
    if (search) {
        const DeviceInfo *dev = device_info();
        const int want = (8 * (dev ? dev->sm_count : 152) + x - 1) / x;
        if (cols > want) cols = want;
    }
    return dim3(static_cast<unsigned>(x), static_cast<unsigned>(cols < 1 ? 1 : (cols < 64 ? cols : 64)));
}

template <typename T, int VE>
cudaError_t gather_t(const void *x, const int *place, int tokens, int k, int d, void *xs, cudaStream_t stream)
{
    const int tpc = tokens_per_cta(tokens, k, row_threads<VE>(d), false);
    return launch_pdl(gather_rows<T, VE>, row_grid<T, VE>(tokens, tpc, d, false), dim3(ROW_THREADS), 0, stream,
                      static_cast<const T *>(x), place, tokens, tpc, k, d, static_cast<T *>(xs));
}

template <typename T, int VE>
cudaError_t sum_t(const void *ys, const int *place, const float *w, int tokens, int k, int d, void *out, unsigned *status,
                  cudaStream_t stream)
{
    const int tpc = tokens_per_cta(tokens, 1, row_threads<VE>(d), false);
    return launch_pdl(sum_rows<T, VE>, row_grid<T, VE>(tokens, tpc, d, false), dim3(ROW_THREADS), 0, stream,
                      static_cast<const T *>(ys), place, w, tokens, tpc, k, d, static_cast<T *>(out), status);
}

template <typename T, int VE>
cudaError_t grad_t(const void *d_out, const void *ys, const int *place, const float *w, int tokens, int k, int d,
                   void *d_ys, float *d_w, unsigned *status, cudaStream_t stream)
{
    return launch_pdl(combine_grad<T, VE>, dim3(static_cast<unsigned>(tokens)), dim3(ROW_THREADS), 0, stream,
                      static_cast<const T *>(d_out), static_cast<const T *>(ys), place, w, tokens * k, k, d,
                      static_cast<T *>(d_ys), d_w, status);
}

template <typename T, int VE>
cudaError_t small_t(const int *top_idx, int tokens, int k, int n, const void *x, int d, int *offsets, int *order,
                    int *place, void *xs, cudaStream_t stream)
{
    const int tpc = tokens_per_cta(tokens, k, xs ? row_threads<VE>(d) : 0, true);
    dim3 grid = row_grid<T, VE>(tokens, tpc, xs ? d : 0, true);
    grid.x += 1;
    const size_t words = static_cast<size_t>(n) + 1 > SMOE_MAX_TOP_K ? static_cast<size_t>(n) + 1 : SMOE_MAX_TOP_K;
    return launch_pdl(dispatch_small<T, VE>, grid, dim3(SMALL_THREADS), words * sizeof(int), stream, top_idx, tokens, tpc, k, n,
                      static_cast<const T *>(x), d, offsets, order, place, static_cast<T *>(xs));
}

}  // namespace

namespace {

template <typename T, int VE>
cudaError_t middle_t(const int *top_idx, int tokens, int k, int n, int nchunks, int chunk, const int *cum, const void *x, int d,
                     int *offsets, int *order, int *place, void *xs, cudaStream_t stream)
{
    const int tpc = tokens_per_cta(tokens, k, xs ? row_threads<VE>(d) : 0, true);
    dim3 grid = row_grid<T, VE>(tokens, tpc, xs ? d : 0, true);
    grid.x += static_cast<unsigned>((n + SMALL_THREADS / 32) / (SMALL_THREADS / 32));
    return launch_pdl(dispatch_middle<T, VE>, grid, dim3(SMALL_THREADS), 0, stream, top_idx, tokens, tpc, k, n, nchunks, chunk,
                      cum, static_cast<const T *>(x), d, offsets, order, place, static_cast<T *>(xs));
}

}  // namespace

cudaError_t launch_dispatch(const int *top_idx, int tokens, int k, int n, const void *x, int dtype, int d, int *offsets,
                            int *order, int *place, void *xs, void *workspace, cudaStream_t stream)
{
    const size_t pitch = static_cast<size_t>(d) * (dtype == SMOE_BF16 ? 2 : 4);
    const bool v = vec16(x, pitch) && vec16(xs, pitch);
    const int R = tokens * k;
    if (R <= SMALL_SLOTS) {
        if (dtype == SMOE_BF16)
            return v ? small_t<__nv_bfloat16, 8>(top_idx, tokens, k, n, x, d, offsets, order, place, xs, stream)
                     : small_t<__nv_bfloat16, 1>(top_idx, tokens, k, n, x, d, offsets, order, place, xs, stream);
        return v ? small_t<float, 4>(top_idx, tokens, k, n, x, d, offsets, order, place, xs, stream)
                 : small_t<float, 1>(top_idx, tokens, k, n, x, d, offsets, order, place, xs, stream);
    }
    // larger chunks, whose search takes longer, where a token's k rows take
    // longer still to copy
    const bool wide = xs && static_cast<size_t>(k) * pitch >= 32768u;
    const int chunk = R <= MIDDLE_CHUNKS * MIDDLE_SMALL_CHUNK || !wide ? MIDDLE_SMALL_CHUNK : MIDDLE_LARGE_CHUNK;
    const int chunks = (R + chunk - 1) / chunk;
    if (chunks <= MIDDLE_CHUNKS) {
        int *cum = static_cast<int *>(workspace);
        const size_t smem = (static_cast<size_t>(n) + 1) * sizeof(int);
        const cudaError_t e = launch_pdl(sort_below, dim3(static_cast<unsigned>(chunks)), dim3(static_cast<unsigned>(chunk)),
                                         smem, stream, top_idx, R, n, chunks, cum);
        if (e != cudaSuccess) return e;
        auto go = [&](auto run) { return run(top_idx, tokens, k, n, chunks, chunk, cum, x, d, offsets, order, place, xs, stream); };
        if (dtype == SMOE_BF16) return v ? go(middle_t<__nv_bfloat16, 8>) : go(middle_t<__nv_bfloat16, 1>);
        return v ? go(middle_t<float, 4>) : go(middle_t<float, 1>);
    }
    const cudaError_t e = launch_sort_tokens(top_idx, R, n, offsets, order, place, workspace, stream);
    if (e != cudaSuccess || !xs) return e;
    if (dtype == SMOE_BF16)
        return v ? gather_t<__nv_bfloat16, 8>(x, place, tokens, k, d, xs, stream)
                 : gather_t<__nv_bfloat16, 1>(x, place, tokens, k, d, xs, stream);
    return v ? gather_t<float, 4>(x, place, tokens, k, d, xs, stream)
             : gather_t<float, 1>(x, place, tokens, k, d, xs, stream);
}

cudaError_t launch_sum_tokens(const void *ys, int dtype, const int *place, const float *w, int tokens, int k, int d,
                              void *out, cudaStream_t stream)
{
    unsigned *status = device_status_word();
    if (!status) return cudaErrorInvalidDevice;
    const size_t pitch = static_cast<size_t>(d) * (dtype == SMOE_BF16 ? 2 : 4);
    const bool v = vec16(ys, pitch) && vec16(out, pitch);
    if (dtype == SMOE_BF16)
        return v ? sum_t<__nv_bfloat16, 8>(ys, place, w, tokens, k, d, out, status, stream)
                 : sum_t<__nv_bfloat16, 1>(ys, place, w, tokens, k, d, out, status, stream);
    return v ? sum_t<float, 4>(ys, place, w, tokens, k, d, out, status, stream)
             : sum_t<float, 1>(ys, place, w, tokens, k, d, out, status, stream);
}

cudaError_t launch_combine_tokens_grad(const void *d_out, const void *ys, int dtype, const int *place, const float *w,
                                       int tokens, int k, int d, void *d_ys, float *d_w, cudaStream_t stream)
{
    unsigned *status = device_status_word();
    if (!status) return cudaErrorInvalidDevice;
    const size_t pitch = static_cast<size_t>(d) * (dtype == SMOE_BF16 ? 2 : 4);
    const bool v = vec16(d_out, pitch) && vec16(ys, pitch) && vec16(d_ys, pitch);
    if (dtype == SMOE_BF16)
        return v ? grad_t<__nv_bfloat16, 8>(d_out, ys, place, w, tokens, k, d, d_ys, d_w, status, stream)
                 : grad_t<__nv_bfloat16, 1>(d_out, ys, place, w, tokens, k, d, d_ys, d_w, status, stream);
    return v ? grad_t<float, 4>(d_out, ys, place, w, tokens, k, d, d_ys, d_w, status, stream)
             : grad_t<float, 1>(d_out, ys, place, w, tokens, k, d, d_ys, d_w, status, stream);
}

}  // namespace smoe
