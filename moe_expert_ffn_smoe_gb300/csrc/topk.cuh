// What the selections of the k largest of a row share: order-preserving keys, the
// filter that leaves a warp a few candidates, rounds over a whole row.
#pragma once

#include "common.cuh"

namespace smoe {

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

// A row whose k selected are all masked experts.  That no logit beats -inf does
// not say so: a NaN ranks below it, and is selected where fewer than k are -inf.
__device__ __forceinline__ void write_masked(int k, int *__restrict__ idx, float *__restrict__ w)
{
    for (int r = threadIdx.x & 31; r < k; r += 32) {
        idx[r] = -1;
        w[r] = 0.f;
    }
}

}  // namespace smoe
