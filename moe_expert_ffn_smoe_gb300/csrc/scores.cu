// Routing by scores: softmax or sigmoid scores of every row of logits, a bias
// that moves the choice alone, groups of experts, the k best of the best groups,
// and their weights; and the gradient of the weights to the logits.
//
//   s_i = 1 / (1 + e^-l_i)   or   e^(l_i - max) / sum over the row
//   c_i = s_i + b_i                      (what the choice goes by)
//   w_r = scale s_r / sum over the chosen   or   scale s_r
//
// The choice is the one that the real numbers c_i make.  Where no bias is added that
// is the order of the logits, but for groups that count two scores.  Elsewhere c_i
// is taken in f32 with a bound of its error, and what lies closer than the bounds
// (a row in some thousands) is decided by the same values in 64 bits: of the
// candidates alone, one a lane, or, where the border between groups is in doubt,
// of the whole row.  64-bit arithmetic runs at a 64th of the f32 rate here: all
// scores in it took 30 times as long as the rest.
#include "common.cuh"
#include "internal_tokens.h"
#include "smoe.h"
#include "topk.cuh"

namespace smoe {
namespace {

constexpr int ROW_WARPS = 4, GRAD_WARPS = 8;  // rows of a CTA

// What the choice goes by.
enum class By { Logit, Sigmoid, Softmax };

struct RouteArgs {
    const float *logits, *bias;  // bias null: none
    int *idx;
    float *w;
    int T, n, ld, k, groups, top_groups, best;
    int size;        // experts of a group
    int shift;       // 2^shift lanes look at a group: lanes g 2^shift .. at group g
    unsigned magic;  // ceil(2^20 / size): e magic >> 20 = e / size for e < 1024
    float scale;
    bool softmax, norm;
    bool wide;       // logits and bias begin at 16-byte boundaries, in every row
};

// Which expert a lane's i-th value is.  NEAR: a lane holds V neighbours, so that a
// group is some lanes' own; otherwise every 32nd, so that few experts are spread
// over all lanes.
template <int V, bool NEAR>
__device__ __forceinline__ int expert_at(int i)
{
    const int lane = threadIdx.x & 31;
    return NEAR ? lane * V + i : i * 32 + lane;
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL_MASK, v, off));
    return v;
}
// The largest of values that are not negative: their bits are ordered as they are.
__device__ __forceinline__ float warp_max_positive(float v)
{
    return __uint_as_float(__reduce_max_sync(FULL_MASK, __float_as_uint(v)));
}
__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(FULL_MASK, v, off);
    return v;
}

// value_key of what is no NaN.
__device__ __forceinline__ uint32_t number_key(float v)
{
    const uint32_t u = __float_as_uint(v + 0.f);
    return u ^ (static_cast<uint32_t>(static_cast<int>(u) >> 31) | 0x80000000u);
}

__device__ __forceinline__ float rcp_approx(float v)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// A row's constants: its largest logit and what e^(l - m) is multiplied by
// (softmax), and the row itself.
struct Row {
    const float *l, *b;
    float m, inv;
    int n, V;
};

// c of logit l and bias b, and a bound of its error.  Sigmoid: __expf is off by 2 +
// 1.173 |l| units of 2^-23 at most, the sum and the reciprocal instruction by one
// each.  Softmax: l - m is rounded (2^-24 of its size, in the exponent), the row's
// sum has V + 5 additions after terms as exact; the rounding of s + b is 2^-24 of c.
// Below the normal numbers the instructions flush.
template <By BY>
__device__ __forceinline__ float choice(const Row &r, float l, float b, float &err)
{
    float s, rel;
    if (BY == By::Sigmoid) {
        s = rcp_approx(1.0f + __expf(-l));
        rel = fmaf(fabsf(l), 1.25f * 0x1p-23f, 0x1p-21f);
    } else {
        s = expf(l - r.m) * r.inv;
        rel = (fabsf(l - r.m) + static_cast<float>(r.V + 32)) * 0x1p-24f;
    }
    const float c = s + b;
    err = fmaf(s, rel, fmaf(fabsf(c), 0x1p-23f, 1e-37f));
    return c;
}

// The same in 64 bits; inv64: 1 / the row's sum (softmax).
template <By BY>
__device__ __forceinline__ double choice64(const Row &r, int e, double inv64)
{
    const double l = r.l[e], b = r.b ? r.b[e] : 0.f;
    return (BY == By::Sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - r.m) * inv64) + b;
}

__device__ __forceinline__ bool is_off(const Row &r, int e)
{
    return r.l[e] == -INFINITY || (r.b && r.b[e] == -INFINITY);
}

template <By BY>
__device__ __noinline__ double inverse_sum64(const Row r)
{
    if (BY != By::Softmax) return 0.0;
    double sum = 0.0;
    for (int e = threadIdx.x & 31; e < r.n; e += 32) sum += exp(static_cast<double>(r.l[e]) - r.m);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(FULL_MASK, sum, off);
    return 1.0 / sum;
}

// Whether all experts of the row that are on have one logit and one bias: then sums
// of as many scores are equal, and no 64-bit look is needed (a router whose weights
// are still zero).
__device__ __noinline__ bool all_alike(const Row r)
{
    float lo = INFINITY, hi = -INFINITY, blo = INFINITY, bhi = -INFINITY;
    for (int e = threadIdx.x & 31; e < r.n; e += 32)
        if (!is_off(r, e)) {
            lo = fminf(lo, r.l[e]);
            hi = fmaxf(hi, r.l[e]);
            blo = fminf(blo, r.b ? r.b[e] : 0.f);
            bhi = fmaxf(bhi, r.b ? r.b[e] : 0.f);
        }
    return -warp_max(-lo) == warp_max(hi) && -warp_max(-blo) == warp_max(bhi);
}

// The groups that lanes hold: every lane of a group the same.
struct Groups {
    float value, err;  // what the group counts (-inf: no expert on), a bound of its error
    bool taken;
    uint32_t low, high;  // keys of the least that one taken may count, of the most that one left out may
};

__device__ __forceinline__ void take_groups(Groups &q, const RouteArgs &a)
{
    const int lane = threadIdx.x & 31, P = 1 << a.shift, g = lane >> a.shift, in = lane & (P - 1);
    // each of a group's lanes looks at every P-th other group
    int before = 0;
    for (int h = in; h - in < a.groups; h += P) {
        const float o = __shfl_sync(FULL_MASK, q.value, h << a.shift);  // (the lanes wrap round past the last group)
        before += h < a.groups && (o > q.value || (o == q.value && h < g));
    }
    for (int off = P >> 1; off > 0; off >>= 1) before += __shfl_xor_sync(FULL_MASK, before, off);
    const bool on = g < a.groups && q.value > -INFINITY;
    q.taken = on && before < a.top_groups;
    q.low = __reduce_min_sync(FULL_MASK, q.taken ? number_key(q.value - q.err) : 0xFFFFFFFFu);
    q.high = __reduce_max_sync(FULL_MASK, on && !q.taken ? number_key(q.value + q.err) : 0u);
}

// Whether this lane's group is taken, where the border between the groups lies within
// the bounds (high >= low): those that the bounds leave on one side of it stay there
// (one taken that counts more than any left out may has less than top_groups before
// it; one left out that counts less than any taken has as many), the others are
// ordered by 64 bits.  least: what one of the best of this lane's group counts at
// least.  v: the row's c (expert_at), err: their bound.  32,768 rows by groups in us,
// against scores of the whole row in 64 bits: 512 experts 59 / 69, 128 experts 27 / 30.
template <By BY, int V, bool NEAR>
__device__ __noinline__ bool take_groups64(const Row r, const RouteArgs &a, const Groups q, const float (&v)[V], float least,
                                           float err, Candidates &c)
{
    const int lane = threadIdx.x & 31, g = lane >> a.shift;
    const bool first = (lane & ((1 << a.shift) - 1)) == 0;
    const bool open = g < a.groups && q.value > -INFINITY &&
                      (q.taken ? number_key(q.value - q.err) <= q.high : number_key(q.value + q.err) >= q.low);
    const uint32_t opens = __ballot_sync(FULL_MASK, open);
    const int places = a.top_groups - __popc(__ballot_sync(FULL_MASK, q.taken && !open && first));
    const double inv64 = inverse_sum64<BY>(r);
    double b1 = -INFINITY, b2 = -INFINITY;
    int count = 0;
    const auto weigh = [&] {  // the gathered experts' c, one a lane, into their groups' two best
        __syncwarp();
        const int e = lane < count ? c.expert[lane] : -1;
        const double c64 = e >= 0 ? choice64<BY>(r, e, inv64) : 0.0;
        for (int o = 0; o < count; ++o) {
            const double t = __shfl_sync(FULL_MASK, c64, o);
            const int of = static_cast<int>((static_cast<unsigned>(c.expert[o]) * a.magic) >> 20);
            if (of == g) {
                b2 = fmax(b2, fmin(b1, t));
                b1 = fmax(b1, t);
            }
        }
        __syncwarp();
        count = 0;
    };
#pragma unroll 1
    for (int i = 0; i < V; ++i) {
        float mine = -INFINITY;
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (j == i) mine = v[j];
        const int e = expert_at<V, NEAR>(i);
        const int at = (static_cast<int>((static_cast<unsigned>(e) * a.magic) >> 20) << a.shift) & 31;  // a lane of its group
        const float floor = __shfl_sync(FULL_MASK, least, at) - 2.f * err;
        const bool in = e < a.n && (opens >> at & 1u) && mine > -INFINITY && mine >= floor;
        if (count + __popc(__ballot_sync(FULL_MASK, in)) > 32) weigh();
        gather_candidate(c, in, 0u, e, count);
    }
    weigh();
    const double value = b1 + (a.best == 2 && b2 > -INFINITY ? b2 : 0.0);
    int before = 0;
    for (int h = 0; h < a.groups; ++h) {
        const double o = __shfl_sync(FULL_MASK, value, h << a.shift);
        before += (opens >> (h << a.shift) & 1u) && (o > value || (o == value && h < g));
    }
    return open ? before < places : q.taken;
}

// The next of the row in the order of the real c, among those not yet taken
// (key > kKeyNegInf): the largest in f32, unless others lie within the bound
// `err` of it that are not its equals.
template <By BY, int V, bool NEAR>
__device__ __noinline__ int next_in_doubt(const uint32_t (&key)[V], const Row r, float top, float err, double inv64)
{
    double best = -INFINITY;
    int be = 0x7fffffff;
#pragma unroll 1
    for (int j = 0; j < V; ++j) {
        const int e = expert_at<V, NEAR>(j);
        uint32_t mine = 0u;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i == j) mine = key[i];
        if (mine <= kKeyNegInf || value_of_key(mine) < top - 2.f * err) continue;
        const double c = choice64<BY>(r, e, inv64);
        if (c > best) {
            best = c;
            be = e;
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const double o = __shfl_xor_sync(FULL_MASK, best, off);
        const int oe = __shfl_xor_sync(FULL_MASK, be, off);
        if (o > best || (o == best && oe < be)) {
            best = o;
            be = oe;
        }
    }
    return be;
}

// k rounds over the row by c, for rows that the filter leaves with more than a
// warp's candidates, and for k > FILTER_K.  Lane l ends with ranks l and l + 32
// (-1: none left).
template <By BY, int V, bool NEAR>
__device__ __forceinline__ void choose_by_rounds(uint32_t (&key)[V], const Row &r, int k, float err, int &ea, int &eb)
{
    const int lane = threadIdx.x & 31;
    double inv64 = 0.0;
    bool summed = false;
    for (int q = 0; q < k; ++q) {
        uint32_t best = 0u;
        int bi = 0;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (key[i] > best) {
                best = key[i];
                bi = i;
            }
        const uint32_t top = __reduce_max_sync(FULL_MASK, best);
        if (top <= kKeyNegInf) return;
        int e = static_cast<int>(
            __reduce_min_sync(FULL_MASK, best == top ? static_cast<unsigned>(expert_at<V, NEAR>(bi)) : 0xFFFFFFFFu));
        const float ct = value_of_key(top), lt = r.l[e], bt = r.b ? r.b[e] : 0.f;
        bool doubt = false;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int o = expert_at<V, NEAR>(i);
            if (key[i] > kKeyNegInf && o != e && value_of_key(key[i]) >= ct - 2.f * err)
                doubt |= r.l[o] != lt || (r.b && r.b[o] != bt);
        }
        if (__any_sync(FULL_MASK, doubt)) {
            if (!summed) inv64 = inverse_sum64<BY>(r);
            summed = true;
            e = next_in_doubt<BY, V, NEAR>(key, r, ct, err, inv64);
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (e == expert_at<V, NEAR>(i)) key[i] = 0u;
        if (q == lane) ea = e;
        if (q == lane + 32) eb = e;
    }
}

// Score of a chosen logit v (of softmax less the row's largest), times e^-m where
// the weights are renormalised: with m the largest of the chosen, or 0 if that is
// less, small scores keep the digits that they would lose on their own.
__device__ __forceinline__ float chosen_score(const RouteArgs &a, const Row &r, float v, float m)
{
    if (a.softmax) return expf(v - m) * r.inv;
    return v > 0.f || !a.norm ? rcp_approx(1.f + expf(-v)) : expf(v - m) * rcp_approx(1.f + expf(v));
}

// Weights of the experts that this warp's lanes hold (ea and eb; -1: none), at
// the ranks ra and rb.
__device__ __forceinline__ void write_weights(const RouteArgs &a, const Row &r, int ea, int eb, int ra, int rb, int *idx, float *w)
{
    const float la = ea >= 0 ? r.l[ea] - (a.softmax ? r.m : 0.f) : -INFINITY;
    const float lb = eb >= 0 ? r.l[eb] - (a.softmax ? r.m : 0.f) : -INFINITY;
    const float m = a.norm ? fminf(value_of_key(__reduce_max_sync(FULL_MASK, value_key(fmaxf(la, lb)))), 0.f) : 0.f;
    const float sa = ea >= 0 ? chosen_score(a, r, la, m) : 0.f;
    float sb = 0.f;
    if (a.k > 32 && eb >= 0) sb = chosen_score(a, r, lb, m);
    // (the sum is never small: of a sigmoid at least a half, of a softmax 2^-11; the
    // scale over it may be beyond f32 where no weight is)
    const float over = a.norm ? rcp_approx(warp_sum(sa + sb)) : 1.f;
    if (ra >= 0 && ra < a.k) {
        idx[ra] = ea;
        w[ra] = ea >= 0 ? sa * over * a.scale : 0.f;
    }
    if (rb >= 0 && rb < a.k) {
        idx[rb] = eb;
        w[rb] = eb >= 0 ? sb * over * a.scale : 0.f;
    }
}

// A row's values (which: expert_at); fill: past the last.
template <int V, bool NEAR>
__device__ __forceinline__ void load_row(const float *p, int n, bool wide, float fill, float (&v)[V])
{
    if (NEAR && wide) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 u = *reinterpret_cast<const float4 *>(p + expert_at<V, NEAR>(i));
            v[i] = u.x, v[i + 1] = u.y, v[i + 2] = u.z, v[i + 3] = u.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = expert_at<V, NEAR>(i);
            v[i] = NEAR || e < n ? p[e] : fill;
        }
    }
}

// What a warp has in shared memory.
template <int V, bool NEAR>
struct WarpRoom {
    alignas(16) Candidates cands;
    float sorted[32];
    float row[NEAR ? 1 : 32 * V];
};

// One row: its logits and the biases of this lane's experts.  BIAS: there are some, and
// the choice among the experts goes by c, not by the logits.  (As a question to the
// arguments: 28.3 us against 27.7 for 32,768 rows by groups.)
template <By BY, bool BIAS, int V, bool NEAR>
__device__ __forceinline__ void route_row(const RouteArgs &a, int t, const float (&l)[V], const float (&b)[V],
                                          WarpRoom<V, NEAR> &room)
{
    const int lane = threadIdx.x & 31;
    Row r = {a.logits + static_cast<size_t>(t) * a.ld, a.bias, 0.f, 0.f, a.n, V};
    int *idx = a.idx + static_cast<size_t>(t) * a.k;
    float *w = a.w + static_cast<size_t>(t) * a.k;
    bool bad = false;
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        bad |= l[i] != l[i];
        top = fmaxf(top, l[i]);
    }
    if (a.softmax) bad |= top == INFINITY;
    if (a.softmax) {
        r.m = value_of_key(__reduce_max_sync(FULL_MASK, value_key(top)));
        if (r.m > -INFINITY && (BY == By::Softmax || !a.norm)) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) sum += expf(l[i] - r.m);
            r.inv = 1.f / warp_sum(sum);
        } else {
            r.inv = 1.f;  // weights that are renormalised need no sum
        }
    }
    // what the choice goes by; off: -inf
    float v[V];
    float err = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        v[i] = l[i];
        if (BY != By::Logit) {
            float d;
            const float c = choice<BY>(r, l[i], b[i], d);
            const bool on = l[i] != -INFINITY && b[i] != -INFINITY;
            v[i] = on ? c : -INFINITY;
            err = fmaxf(err, on ? d : 0.f);
            bad |= on && !(c < INFINITY);  // a bias that is no number
        }
    }
    if (__any_sync(FULL_MASK, bad)) {
        // no order and no weights: NaN for k experts, so that the token's output is NaN
        for (int q = lane; q < a.k; q += 32) {
            idx[q] = q;
            w[q] = __int_as_float(0x7fffffff);
        }
        return;
    }
    if (BY != By::Logit) err = warp_max_positive(err);

    if (NEAR || a.groups > 1) {
        const int P = 1 << a.shift, g = lane >> a.shift;
        float b1 = -INFINITY, b2 = -INFINITY;
        if (NEAR) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                b2 = fmaxf(b2, fminf(b1, v[i]));
                b1 = fmaxf(b1, v[i]);
            }
        } else {
            float *c = room.row;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i * 32 + lane < a.n) c[i * 32 + lane] = v[i];
            __syncwarp();
            if (g < a.groups)
                for (int e = g * a.size + (lane & (P - 1)); e < (g + 1) * a.size; e += P) {
                    b2 = fmaxf(b2, fminf(b1, c[e]));
                    b1 = fmaxf(b1, c[e]);
                }
        }
        for (int off = P >> 1; off > 0; off >>= 1) {
            const float o1 = __shfl_xor_sync(FULL_MASK, b1, off), o2 = __shfl_xor_sync(FULL_MASK, b2, off);
            b2 = fmaxf(fminf(b1, o1), fmaxf(b2, o2));
            b1 = fmaxf(b1, o1);
        }
        const bool two = a.best == 2 && b2 > -INFINITY;
        float value = b1 + (two ? b2 : 0.f);
        Groups q = {value, BY == By::Logit ? 0.f : fmaf(fabsf(value), 0x1p-23f, 2.f * err)};
        if (BY != By::Logit && two && fabsf(value) == INFINITY)  // two biases that leave f32 (a mask of its lowest value)
            q = {value = copysignf(0x1.fffffep127f, value), INFINITY};
        take_groups(q, a);
        if (BY != By::Logit && q.high >= q.low) {
            // groups of one expert that is on and groups of more differ however alike those are
            const bool on = g < a.groups && value > -INFINITY;
            const bool even = a.best == 1 || !__any_sync(FULL_MASK, on && two) || !__any_sync(FULL_MASK, on && !two);
            if (!even || !all_alike(r)) q.taken = take_groups64<BY, V, NEAR>(r, a, q, v, two ? b2 : b1, err, room.cands);
        }
        const uint32_t taken = NEAR ? 0u : __ballot_sync(FULL_MASK, q.taken);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int of = static_cast<int>((static_cast<unsigned>(i * 32 + lane) * a.magic) >> 20) << a.shift;
            if (NEAR ? !q.taken : i * 32 + lane < a.n && !(taken >> of & 1u)) v[i] = -INFINITY;
        }
        if (BY != By::Logit && !BIAS) {
            // the scores' order is the logits', which have digits where scores have none left
            float again[V];
            load_row<V, NEAR>(r.l, a.n, a.wide, -INFINITY, again);
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = v[i] > -INFINITY ? again[i] : v[i];
            err = 0.f;
        }
    }
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = NEAR || i * 32 + lane < a.n ? number_key(v[i]) : 0u;

    if (a.k <= FILTER_K) {
        uint32_t most = key[0], first;
#pragma unroll
        for (int i = 1; i < V; ++i) most = max(most, key[i]);
        uint32_t bound = filter_bound(most, a.k, first);
        if (first <= kKeyNegInf) {
            write_masked(a.k, idx, w);
            return;
        }
        // what may be among the k best: within the bounds of the bound
        if (BIAS && bound > kKeyNegInf) bound = value_key(value_of_key(bound) - 2.f * err);
        bound = max(bound, kKeyNegInf + 1u);
        Candidates &c = room.cands;
        c.key[lane] = 0u;
        __syncwarp();
        int count = 0;
        if (NEAR) {  // in expert order: after those of the lanes before
#pragma unroll
            for (int i = 0; i < V; ++i) count += key[i] >= bound;
            int at = count;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int o = __shfl_up_sync(FULL_MASK, at, off);
                if (lane >= off) at += o;
            }
            const int all = __shfl_sync(FULL_MASK, at, 31);
            at -= count;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (key[i] >= bound) {
                    if (at < 32) {
                        c.key[at] = key[i];
                        c.expert[at] = static_cast<uint16_t>(lane * V + i);
                    }
                    ++at;
                }
            count = all;
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) gather_candidate(c, key[i] >= bound, key[i], i * 32 + lane, count);
        }
        __syncwarp();
        if (count <= 32) {
            const int e = lane < count ? c.expert[lane] : -1;
            const uint32_t mine = c.key[lane];
            // the larger ones, and of the equal ones those before it (in expert order)
            int rank = 0;
            for (int o = 0; o < count; o += 4) {
                const uint4 u = *reinterpret_cast<const uint4 *>(&c.key[o]);
                if (!BIAS) {
                    rank += u.x >= mine + (o >= lane ? 1u : 0u);
                    rank += u.y >= mine + (o + 1 >= lane ? 1u : 0u);
                    rank += u.z >= mine + (o + 2 >= lane ? 1u : 0u);
                    rank += u.w >= mine + (o + 3 >= lane ? 1u : 0u);
                } else {  // (equal ones are in doubt, below)
                    rank += (u.x > mine) + (u.y > mine) + (u.z > mine) + (u.w > mine);
                }
            }
            if (BIAS) {
                // One bound for all: two that it does not separate make neighbours that it does
                // not.  Equal ones leave the ranks after the first empty (infinite).
                float *by_rank = room.sorted;
                by_rank[lane] = INFINITY;
                __syncwarp();
                if (lane < count) by_rank[rank] = value_of_key(mine);
                __syncwarp();
                const bool doubt = lane < a.k && lane + 1 < count && by_rank[lane] - by_rank[lane + 1] <= 2.f * err;
                if (__any_sync(FULL_MASK, doubt)) {
                    const double inv64 = inverse_sum64<BY>(r);
                    const double c64 = e >= 0 ? choice64<BY>(r, e, inv64) : -INFINITY;
                    rank = 0;
                    for (int o = 0; o < count; ++o) {
                        const double v = __shfl_sync(FULL_MASK, c64, o);
                        rank += v > c64 || (v == c64 && o < lane);
                    }
                }
            }
            // ranks past the candidates: none left
            const bool sel = lane < count && rank < a.k;
            write_weights(a, r, sel ? e : -1, -1, sel ? rank : (lane >= count ? lane : -1), -1, idx, w);
            return;
        }
    }
    int ea = -1, eb = -1;
    choose_by_rounds<BY, V, NEAR>(key, r, a.k, err, ea, eb);
    write_weights(a, r, ea, eb, lane, lane + 32, idx, w);
}

// A warp per row, n <= 32 V; NEAR: n == 32 V, in groups of whole lanes.  Bound by
// instruction issue and the gaps that 30 warps an SM leave: 32,768 rows of 128 experts in
// 8 groups of which 4 stay, k = 8 24.6 us (8 warps a CTA 27; 690 instructions a row),
// where reading and writing takes 2.8; CTAs that walk the rows, the next one's logits
// loaded ahead, 29 us: the registers cost the warps that would have filled the gaps.
template <By BY, bool BIAS, int V, bool NEAR>
__global__ void __launch_bounds__(ROW_WARPS * 32) route_rows_warp(const RouteArgs a)
{
    __shared__ WarpRoom<V, NEAR> rooms[ROW_WARPS];
    const int wi = threadIdx.x >> 5, t = blockIdx.x * ROW_WARPS + wi;
    pdl_launch_dependents();
    pdl_wait();
    if (t >= a.T) return;
    float l[V], b[V];
#pragma unroll
    for (int i = 0; i < V; ++i) b[i] = 0.f;
    load_row<V, NEAR>(a.logits + static_cast<size_t>(t) * a.ld, a.n, a.wide, -INFINITY, l);
    if (BIAS) load_row<V, NEAR>(a.bias, a.n, a.wide, 0.f, b);
    route_row<BY, BIAS, V, NEAR>(a, t, l, b, rooms[wi]);
}

// ---------------------------------------------------------------- gradient

struct RouteGradArgs {
    const float *logits;
    const int *idx;
    const float *w, *dw;
    float *dl;
    int T, n, ld, k;
    float scale;
    bool softmax, norm;
};

// With g_r = w_r (dw_r - sum_q w_q dw_q / scale) where the weights are
// renormalised, w_r dw_r where not:
//   sigmoid            dl_r = g_r (1 - s_r)
//   softmax, norm      dl_r = g_r
//   softmax            dl_j = (g_r of the slot of j) - s_j sum_r g_r, for every j
// A warp per row, which makes the row in shared memory and writes it once.  Bound
// by writing the gradients (and, for the last form, reading the logits) and by
// instruction issue: 16,383 rows of 128 experts, softmax of all, with the selection
// before it 13.7 us (2.7 of them for the bytes).
template <int V, bool WIDE>  // WIDE: k > 32, lane l holds the slots l and l + 32
__global__ void __launch_bounds__(GRAD_WARPS * 32) route_rows_grad(const RouteGradArgs a)
{
    constexpr int H = WIDE ? 2 : 1;
    __shared__ alignas(16) float rows[GRAD_WARPS][32 * V];  // (written out in 16 bytes a lane)
    const int wi = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x * GRAD_WARPS + wi;
    pdl_launch_dependents();
    pdl_wait();
    if (t >= a.T) return;
    const float *l = a.logits + static_cast<size_t>(t) * a.ld;
    const bool dense = a.softmax && !a.norm;
    float p[V];
    if (dense) {
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = i * 32 + lane < a.n ? l[i * 32 + lane] : -INFINITY;
    }
    int e[H];
    float w[H], g[H], dot = 0.f, sum = 0.f;
#pragma unroll
    for (int h = 0; h < H; ++h) {
        const bool in = lane + 32 * h < a.k;
        const size_t at = static_cast<size_t>(t) * a.k + lane + 32 * h;
        e[h] = in ? a.idx[at] : -1;
        w[h] = in ? a.w[at] : 0.f;
        g[h] = in ? a.dw[at] : 0.f;
        if (e[h] < 0 || e[h] >= a.n) e[h] = -1;  // no expert: counts for nothing
        // (weights over the scale are at most 1: a sum of the weights' own could leave f32)
        if (e[h] >= 0) dot = fmaf(a.norm ? w[h] / a.scale : w[h], g[h], dot);
    }
    if (dense) {
        float top = p[0];
#pragma unroll
        for (int i = 1; i < V; ++i) top = fmaxf(top, p[i]);
        top = value_of_key(__reduce_max_sync(FULL_MASK, value_key(top)));
        const float m = top > -INFINITY ? top : 0.f;  // a row of nothing else: scores of 0
#pragma unroll
        for (int i = 0; i < V; ++i) {
            p[i] = expf(p[i] - m);
            sum += p[i];
        }
        sum = warp_sum(sum);
    }
    dot = warp_sum(dot);
    // slots of one expert (a selection has none twice, a caller's list may)?
    float *row = rows[wi];
    bool twice = false;
    if (!WIDE) {
        if (e[0] >= 0) reinterpret_cast<int *>(row)[e[0]] = lane;
        __syncwarp();
        twice = e[0] >= 0 && reinterpret_cast<const int *>(row)[e[0]] != lane;
        twice = __any_sync(FULL_MASK, twice);
    }
    const float mean = a.norm ? dot : 0.f;
#pragma unroll
    for (int h = 0; h < H; ++h) {
        g[h] = w[h] * (g[h] - mean);
        if (!a.softmax && e[h] >= 0) g[h] *= rcp_approx(1.f + expf(l[e[h]]));  // 1 - s = 1 / (1 + e^l)
    }
    if (dense) {
        const float inv = sum > 0.f || sum != sum ? -dot / sum : 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) row[i * 32 + lane] = p[i] * inv;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) row[i * 32 + lane] = 0.f;
    }
    __syncwarp();
    if (!WIDE && !twice) {
        if (e[0] >= 0) row[e[0]] += g[0];
    } else {  // in slot order
#pragma unroll
        for (int h = 0; h < H; ++h)
            for (int q = 0; q < 32; ++q) {
                if (q == lane && e[h] >= 0) row[e[h]] += g[h];
                __syncwarp();
            }
    }
    __syncwarp();
    float *dl = a.dl + static_cast<size_t>(t) * a.n;
    if ((a.n & 3) == 0) {
        for (int c = lane; c < (a.n >> 2); c += 32)
            reinterpret_cast<float4 *>(dl)[c] = reinterpret_cast<const float4 *>(row)[c];
    } else {
        for (int c = lane; c < a.n; c += 32) dl[c] = row[c];
    }
}

template <bool WIDE>
cudaError_t grad_wide(const RouteGradArgs &a, cudaStream_t stream)
{
    const dim3 grid(static_cast<unsigned>((a.T + GRAD_WARPS - 1) / GRAD_WARPS)), block(GRAD_WARPS * 32);
    if (a.n <= 128) return launch_pdl(route_rows_grad<4, WIDE>, grid, block, 0, stream, a);
    if (a.n <= 256) return launch_pdl(route_rows_grad<8, WIDE>, grid, block, 0, stream, a);
    if (a.n <= 512) return launch_pdl(route_rows_grad<16, WIDE>, grid, block, 0, stream, a);
    return launch_pdl(route_rows_grad<32, WIDE>, grid, block, 0, stream, a);
}

template <By BY, bool BIAS, int V>
cudaError_t route_wide(const RouteArgs &a, bool near, cudaStream_t stream)
{
    const dim3 grid(static_cast<unsigned>((a.T + ROW_WARPS - 1) / ROW_WARPS)), block(ROW_WARPS * 32);
    return near ? launch_pdl(route_rows_warp<BY, BIAS, V, true>, grid, block, 0, stream, a)
                : launch_pdl(route_rows_warp<BY, BIAS, V, false>, grid, block, 0, stream, a);
}

template <By BY, bool BIAS>
cudaError_t route_by(RouteArgs a, cudaStream_t stream)
{
    const int V = a.n <= 128 ? 4 : a.n <= 256 ? 8 : a.n <= 512 ? 16 : 32;
    // Neighbours to a lane where groups are whole lanes and those that stay fill twice k
    // lanes (with fewer, too many of their experts would be candidates), or leave a warp
    // no more than its 32.  Against every 32nd, in us: 32,768 rows of 128 experts, 4 of 8
    // groups stay, k = 8 27.4 / 31.7; k = 16 (which this leaves out) 69 / 38; 3 stay, k = 16
    // 81 / 39; 512 experts, k = 8 66 / 80.
    const int stay = a.top_groups * a.size;
    const bool near = a.groups > 1 && a.n == 32 * V && a.size % V == 0 && (a.size / V & (a.size / V - 1)) == 0 &&
                      (stay >= 2 * a.k * V || stay <= 32);
    int lanes = near ? a.size / V : 32 / a.groups;  // the largest power of two that leaves every group its lanes
    for (a.shift = 0; lanes > 1; lanes /= 2) ++a.shift;
    if (V == 4) return route_wide<BY, BIAS, 4>(a, near, stream);
    if (V == 8) return route_wide<BY, BIAS, 8>(a, near, stream);
    if (V == 16) return route_wide<BY, BIAS, 16>(a, near, stream);
    return route_wide<BY, BIAS, 32>(a, near, stream);
}

}  // namespace

cudaError_t launch_route_rows(const float *logits, int T, int n, int ld, const float *bias, bool softmax, int groups,
                              int top_groups, int best, int k, bool norm, float scale, int *idx, float *w,
                              cudaStream_t stream)
{
    const int size = n / groups;
    if (groups > 1 && top_groups >= groups) groups = top_groups = 1;  // all of them
    const RouteArgs a = {logits, bias, idx, w, T, n, ld, k, groups, top_groups, best, size, 0,
                         static_cast<unsigned>(((1 << 20) + size - 1) / size), scale, softmax, norm,
                         ld % 4 == 0 && reinterpret_cast<uintptr_t>(logits) % 16 == 0 && reinterpret_cast<uintptr_t>(bias) % 16 == 0};
    if (!bias && (groups == 1 || best == 1)) return route_by<By::Logit, false>(a, stream);
    if (!bias) return softmax ? route_by<By::Softmax, false>(a, stream) : route_by<By::Sigmoid, false>(a, stream);
    return softmax ? route_by<By::Softmax, true>(a, stream) : route_by<By::Sigmoid, true>(a, stream);
}

cudaError_t launch_route_rows_grad(const float *logits, int T, int n, int ld, bool softmax, int k, bool norm, float scale,
                                   const int *idx, const float *w, const float *dw, float *dl, cudaStream_t stream)
{
    const RouteGradArgs a = {logits, idx, w, dw, dl, T, n, ld, k, scale, softmax, norm};
    return k > 32 ? grad_wide<true>(a, stream) : grad_wide<false>(a, stream);
}

}  // namespace smoe
