// The extern "C" entry points declared in include/smoe.h: argument checks
// on the host, then the kernel launches.  Nothing here allocates memory.
#include <mutex>

#include "internal_tokens.h"
#include "smoe.h"

namespace smoe {

const DeviceInfo *device_info()
{
    constexpr int kMaxDevices = 64;
    static DeviceInfo cache[kMaxDevices];
    static bool ready[kMaxDevices] = {};
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
    std::lock_guard<std::mutex> lock(mu);
    if (!ready[dev]) {
        DeviceInfo d = {};
        d.device = dev;
        if (cudaDeviceGetAttribute(&d.sm_count, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return nullptr;
        if (cudaDeviceGetAttribute(&d.max_smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) !=
            cudaSuccess)
            return nullptr;
        cache[dev] = d;
        ready[dev] = true;
    }
    return &cache[dev];
}

}  // namespace smoe

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Span {
    const void *p;
    size_t bytes;
};

bool overlap(Span a, Span b)
{
    if (a.bytes == 0 || b.bytes == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

// True if any output span overlaps any input span or another output span.
bool any_alias(const Span *outs, int nout, const Span *ins, int nin)
{
    for (int i = 0; i < nout; ++i) {
        for (int j = 0; j < nin; ++j)
            if (overlap(outs[i], ins[j])) return true;
        for (int j = i + 1; j < nout; ++j)
            if (overlap(outs[i], outs[j])) return true;
    }
    return false;
}

int to_status(cudaError_t e) { return e == cudaSuccess ? SMOE_OK : SMOE_ERR_LAUNCH; }

// Layout contract of a packed [rows x cols] matrix ("Layout assumptions the
// kernels rely on"): cols % 32 (Q4) / % 64 (Q2), group a positive multiple of
// the same unit dividing cols, cols <= SMOE_MAX_COLS.
int check_q_shape(int bits, int rows, int cols, int group)
{
    if (rows < 0 || cols < 0) return SMOE_ERR_SHAPE;
    if (cols > SMOE_MAX_COLS) return SMOE_ERR_SHAPE;
    const int unit = bits == 4 ? 32 : 64;
    if (cols % unit != 0) return SMOE_ERR_SHAPE;
    if (group <= 0 || group % unit != 0) return SMOE_ERR_SHAPE;
    if (cols > 0 && cols % group != 0) return SMOE_ERR_SHAPE;
    return SMOE_OK;
}

size_t q_bytes(int bits, int rows, int cols)
{
    return static_cast<size_t>(rows) * static_cast<size_t>(cols) * bits / 8;
}

size_t scale_bytes(int rows, int cols, int group)
{
    return static_cast<size_t>(rows) * static_cast<size_t>(cols / group) * sizeof(float);
}

int gate_up_impl(int bits, const uint8_t *gc, const float *gs, const uint8_t *uc, const float *us,
                 const float *x, float *hidden, int d_ff, int d_model, int group, void *stream)
{
    int st = check_q_shape(bits, d_ff, d_model, group);
    if (st != SMOE_OK) return st;
    if (d_ff == 0) return SMOE_OK;
    if (!hidden) return SMOE_ERR_NULL;
    if (!aligned16(hidden)) return SMOE_ERR_ALIGN;
    if (d_model > 0) {
        if (!gc || !gs || !uc || !us || !x) return SMOE_ERR_NULL;
        if (!aligned16(gc) || !aligned16(uc) || !aligned16(gs) || !aligned16(us) || !aligned16(x))
            return SMOE_ERR_ALIGN;
    }
    const Span out[1] = {{hidden, static_cast<size_t>(d_ff) * sizeof(float)}};
    const Span in[5] = {{gc, q_bytes(bits, d_ff, d_model)},
                        {gs, scale_bytes(d_ff, d_model, group)},
                        {uc, q_bytes(bits, d_ff, d_model)},
                        {us, scale_bytes(d_ff, d_model, group)},
                        {x, static_cast<size_t>(d_model) * sizeof(float)}};
    if (any_alias(out, 1, in, 5)) return SMOE_ERR_ALIAS;
    const uint8_t *codes[2] = {gc, uc};
    const float *scales[2] = {gs, us};
    return to_status(smoe::launch_qgemv(bits, 2, codes, scales, x, hidden, d_ff, d_model, group,
                                        static_cast<cudaStream_t>(stream)));
}

int down_impl(int bits, const uint8_t *dc, const float *ds, const float *hidden, float *out,
              int d_model, int d_ff, int group, void *stream)
{
    int st = check_q_shape(bits, d_model, d_ff, group);
    if (st != SMOE_OK) return st;
    if (d_model == 0) return SMOE_OK;
    if (!out) return SMOE_ERR_NULL;
    if (!aligned16(out)) return SMOE_ERR_ALIGN;
    if (d_ff > 0) {
        if (!dc || !ds || !hidden) return SMOE_ERR_NULL;
        if (!aligned16(dc) || !aligned16(ds) || !aligned16(hidden)) return SMOE_ERR_ALIGN;
    }
    const Span o[1] = {{out, static_cast<size_t>(d_model) * sizeof(float)}};
    const Span in[3] = {{dc, q_bytes(bits, d_model, d_ff)},
                        {ds, scale_bytes(d_model, d_ff, group)},
                        {hidden, static_cast<size_t>(d_ff) * sizeof(float)}};
    if (any_alias(o, 1, in, 3)) return SMOE_ERR_ALIAS;
    const uint8_t *codes[2] = {dc, dc};
    const float *scales[2] = {ds, ds};
    return to_status(smoe::launch_qgemv(bits, 1, codes, scales, hidden, out, d_model, d_ff, group,
                                        static_cast<cudaStream_t>(stream)));
}

constexpr int kExpertsPerLaunch = 64;

int launch_grouped(int bits, int nmat, int n, const uint8_t *const *c0, const float *const *s0,
                   const uint8_t *const *c1, const float *const *s1, const float *x, float *y, int units, int K,
                   int group, cudaStream_t s);

// Grouped calls: per-expert checks, then launches of up to 64 experts each
// (experts of one launch share the grid; a shape the grouped kernel does not
// take is run expert by expert with the single-expert launcher).
int experts_impl(int bits, int nmat, int n, const uint8_t *const *c0, const float *const *s0,
                 const uint8_t *const *c1, const float *const *s1, const float *x, float *y, int units, int K,
                 int group, void *stream)
{
    if (n < 0) return SMOE_ERR_SHAPE;
    int st = check_q_shape(bits, units, K, group);
    if (st != SMOE_OK) return st;
    if (n == 0 || units == 0) return SMOE_OK;
    if (!c0 || !s0 || (nmat == 2 && (!c1 || !s1))) return SMOE_ERR_NULL;
    if (!y) return SMOE_ERR_NULL;
    if (!aligned16(y)) return SMOE_ERR_ALIGN;
    // x: one shared vector for gate/up, one row per expert for down
    const size_t x_bytes = static_cast<size_t>(K) * sizeof(float) * (nmat == 2 ? 1 : static_cast<size_t>(n));
    const Span out = {y, static_cast<size_t>(n) * static_cast<size_t>(units) * sizeof(float)};
    if (K > 0) {
        if (!x) return SMOE_ERR_NULL;
        if (!aligned16(x)) return SMOE_ERR_ALIGN;
        if (overlap(out, Span{x, x_bytes})) return SMOE_ERR_ALIAS;
        for (int e = 0; e < n; ++e) {
            const uint8_t *cs[2] = {c0[e], nmat == 2 ? c1[e] : c0[e]};
            const float *ss[2] = {s0[e], nmat == 2 ? s1[e] : s0[e]};
            for (int m = 0; m < nmat; ++m) {
                if (!cs[m] || !ss[m]) return SMOE_ERR_NULL;
                if (!aligned16(cs[m]) || !aligned16(ss[m])) return SMOE_ERR_ALIGN;
                if (overlap(out, Span{cs[m], q_bytes(bits, units, K)}) ||
                    overlap(out, Span{ss[m], scale_bytes(units, K, group)}))
                    return SMOE_ERR_ALIAS;
            }
        }
    }
    return launch_grouped(bits, nmat, n, c0, s0, c1, s1, x, y, units, K, group, static_cast<cudaStream_t>(stream));
}

// The launches of a grouped call whose arguments have been checked.
int launch_grouped(int bits, int nmat, int n, const uint8_t *const *c0, const float *const *s0,
                   const uint8_t *const *c1, const float *const *s1, const float *x, float *y, int units, int K,
                   int group, cudaStream_t s)
{
    if (n == 0 || units == 0) return SMOE_OK;
    const float *xs[kExpertsPerLaunch];
    float *ys[kExpertsPerLaunch];
    for (int e0 = 0; e0 < n; e0 += kExpertsPerLaunch) {
        const int cnt = (n - e0) < kExpertsPerLaunch ? (n - e0) : kExpertsPerLaunch;
        for (int i = 0; i < cnt; ++i) {
            xs[i] = nmat == 2 ? x : (x ? x + static_cast<size_t>(e0 + i) * K : nullptr);
            ys[i] = y + static_cast<size_t>(e0 + i) * units;
        }
        bool unsupported = true;
        cudaError_t err = cudaSuccess;
        if (K > 0)
            err = smoe::launch_qgemv_experts(bits, nmat, cnt, c0 + e0, nmat == 2 ? c1 + e0 : c0 + e0, s0 + e0,
                                             nmat == 2 ? s1 + e0 : s0 + e0, xs, ys, units, K, group, s,
                                             &unsupported);
        if (err != cudaSuccess) return SMOE_ERR_LAUNCH;
        if (unsupported) {
            for (int i = 0; i < cnt; ++i) {
                const uint8_t *codes[2] = {c0[e0 + i], nmat == 2 ? c1[e0 + i] : c0[e0 + i]};
                const float *scales[2] = {s0[e0 + i], nmat == 2 ? s1[e0 + i] : s0[e0 + i]};
                err = smoe::launch_qgemv(bits, nmat, codes, scales, xs[i], ys[i], units, K, group, s);
                if (err != cudaSuccess) return SMOE_ERR_LAUNCH;
            }
        }
    }
    return SMOE_OK;
}

size_t ffn_workspace_bytes(int n, int d_ff)
{
    if (d_ff < 0) return static_cast<size_t>(-1);
    if (n <= 0) return 0;
    const size_t e = static_cast<size_t>(n < kExpertsPerLaunch ? n : kExpertsPerLaunch);
    const size_t b = SMOE_FFN_SYNC_BYTES + e * static_cast<size_t>(d_ff) * sizeof(float);
    return (b + 255u) & ~static_cast<size_t>(255u);
}

// smoe_experts_ffn_q4/q2: checks, then per 64 experts the one-launch
// kernel, or gate/up into the workspace followed by down.
int experts_ffn_impl(int bits, int n, const uint8_t *const *gc, const float *const *gs, const uint8_t *const *uc,
                     const float *const *us, const uint8_t *const *dc, const float *const *ds, const float *x,
                     float *out, int d_model, int d_ff, int group, void *workspace, size_t ws_bytes, void *stream)
{
    if (n < 0) return SMOE_ERR_SHAPE;
    int st = check_q_shape(bits, d_ff, d_model, group);
    if (st != SMOE_OK) return st;
    st = check_q_shape(bits, d_model, d_ff, group);
    if (st != SMOE_OK) return st;
    if (n == 0 || d_model == 0) return SMOE_OK;
    if (!gc || !gs || !uc || !us || !dc || !ds || !x || !out) return SMOE_ERR_NULL;
    if (!aligned16(x) || !aligned16(out)) return SMOE_ERR_ALIGN;
    const size_t need = ffn_workspace_bytes(n, d_ff);
    if (!workspace || ws_bytes < need) return SMOE_ERR_WORKSPACE;
    if (!aligned16(workspace)) return SMOE_ERR_ALIGN;
    const Span o = {out, static_cast<size_t>(n) * static_cast<size_t>(d_model) * sizeof(float)};
    const Span w = {workspace, need};
    const Span xi = {x, static_cast<size_t>(d_model) * sizeof(float)};
    if (overlap(o, xi) || overlap(o, w) || overlap(w, xi)) return SMOE_ERR_ALIAS;
    for (int e = 0; e < n; ++e) {
        const void *ptrs[6] = {gc[e], gs[e], uc[e], us[e], dc[e], ds[e]};
        for (const void *p : ptrs) {
            if (!p) return SMOE_ERR_NULL;
            if (!aligned16(p)) return SMOE_ERR_ALIGN;
        }
        const Span ins[6] = {{gc[e], q_bytes(bits, d_ff, d_model)}, {gs[e], scale_bytes(d_ff, d_model, group)},
                             {uc[e], q_bytes(bits, d_ff, d_model)}, {us[e], scale_bytes(d_ff, d_model, group)},
                             {dc[e], q_bytes(bits, d_model, d_ff)}, {ds[e], scale_bytes(d_model, d_ff, group)}};
        for (const Span &in : ins)
            if (overlap(o, in) || overlap(w, in)) return SMOE_ERR_ALIAS;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    unsigned *sync = static_cast<unsigned *>(workspace);
    float *hidden = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + SMOE_FFN_SYNC_BYTES);
    for (int e0 = 0; e0 < n; e0 += kExpertsPerLaunch) {
        const int cnt = (n - e0) < kExpertsPerLaunch ? (n - e0) : kExpertsPerLaunch;
        float *o0 = out + static_cast<size_t>(e0) * d_model;
        bool unsupported = true;
        cudaError_t err = cudaSuccess;
        if (d_ff > 0)
            err = smoe::launch_expert_ffn(bits, cnt, gc + e0, gs + e0, uc + e0, us + e0, dc + e0, ds + e0, x,
                                          hidden, o0, sync, d_model, d_ff, group, s, &unsupported);
        if (err != cudaSuccess) return SMOE_ERR_LAUNCH;
        if (unsupported) {
            st = launch_grouped(bits, 2, cnt, gc + e0, gs + e0, uc + e0, us + e0, x, hidden, d_ff, d_model, group,
                                s);
            if (st != SMOE_OK) return st;
            st = launch_grouped(bits, 1, cnt, dc + e0, ds + e0, nullptr, nullptr, hidden, o0, d_model, d_ff, group,
                                s);
            if (st != SMOE_OK) return st;
        }
    }
    return SMOE_OK;
}

// ffn_batch_q4/q2: checks, then the token-batch launches.
int ffn_batch_impl(int bits, const uint8_t *gate_codes, const float *gate_scales, const uint8_t *up_codes,
                 const float *up_scales, const uint8_t *down_codes, const float *down_scales,
                 const float *X, float *Y, int T, int d_model, int d_ff, int group,
                 void *workspace, size_t workspace_bytes, void *stream)
{
    if (T < 0) return SMOE_ERR_SHAPE;
    int st = check_q_shape(bits, d_ff, d_model, group);
    if (st != SMOE_OK) return st;
    st = check_q_shape(bits, d_model, d_ff, group);
    if (st != SMOE_OK) return st;
    if (T == 0 || d_model == 0) return SMOE_OK;
    if (!X || !Y) return SMOE_ERR_NULL;
    if (!aligned16(X) || !aligned16(Y)) return SMOE_ERR_ALIGN;
    if (d_ff > 0) {
        if (!gate_codes || !gate_scales || !up_codes || !up_scales || !down_codes || !down_scales)
            return SMOE_ERR_NULL;
        if (!aligned16(gate_codes) || !aligned16(gate_scales) || !aligned16(up_codes) ||
            !aligned16(up_scales) || !aligned16(down_codes) || !aligned16(down_scales))
            return SMOE_ERR_ALIGN;
    }
    const size_t need = smoe::ffn_batch_workspace(T, d_model, d_ff, group);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return SMOE_ERR_WORKSPACE;
        if (!aligned16(workspace)) return SMOE_ERR_ALIGN;
    }
    const size_t xy = static_cast<size_t>(T) * static_cast<size_t>(d_model) * sizeof(float);
    const Span outs[2] = {{Y, xy}, {workspace, need}};
    const Span ins[7] = {{gate_codes, q_bytes(bits, d_ff, d_model)},
                         {gate_scales, scale_bytes(d_ff, d_model, group)},
                         {up_codes, q_bytes(bits, d_ff, d_model)},
                         {up_scales, scale_bytes(d_ff, d_model, group)},
                         {down_codes, q_bytes(bits, d_model, d_ff)},
                         {down_scales, scale_bytes(d_model, d_ff, group)},
                         {X, xy}};
    if (any_alias(outs, 2, ins, 7)) return SMOE_ERR_ALIAS;
    const uint8_t *gu_codes[2] = {gate_codes, up_codes};
    const float *gu_scales[2] = {gate_scales, up_scales};
    return to_status(smoe::launch_ffn_batch(bits, gu_codes, gu_scales, down_codes, down_scales, X, Y, T,
                                            d_model, d_ff, group, workspace,
                                            static_cast<cudaStream_t>(stream)));
}

// smoe_experts_ffn_batch_q4/q2: per-expert checks, then the grouped
// token-batch launches.
int experts_batch_impl(int bits, int n, const uint8_t *const *gc, const float *const *gs,
                       const uint8_t *const *uc, const float *const *us, const uint8_t *const *dc,
                       const float *const *ds, const float *const *X, float *const *Y, const int *T, int d_model,
                       int d_ff, int group, void *workspace, size_t ws_bytes, void *stream)
{
    if (n < 0) return SMOE_ERR_SHAPE;
    int st = check_q_shape(bits, d_ff, d_model, group);
    if (st != SMOE_OK) return st;
    st = check_q_shape(bits, d_model, d_ff, group);
    if (st != SMOE_OK) return st;
    if (n == 0 || d_model == 0) return SMOE_OK;
    if (!T) return SMOE_ERR_NULL;
    bool any = false;
    for (int e = 0; e < n; ++e) {
        if (T[e] < 0) return SMOE_ERR_SHAPE;
        any = any || T[e] > 0;
    }
    if (!any) return SMOE_OK;
    if (!gc || !gs || !uc || !us || !dc || !ds || !X || !Y) return SMOE_ERR_NULL;
    const size_t need = smoe::ffn_batch_workspace_experts(n, T, d_model, d_ff, group);
    if (need > 0) {
        if (!workspace || ws_bytes < need) return SMOE_ERR_WORKSPACE;
        if (!aligned16(workspace)) return SMOE_ERR_ALIGN;
    }
    const Span w = {workspace, need};
    for (int e = 0; e < n; ++e) {
        if (T[e] == 0) continue;
        const void *ptrs[8] = {gc[e], gs[e], uc[e], us[e], dc[e], ds[e], X[e], Y[e]};
        for (const void *p : ptrs) {
            if (!p) return SMOE_ERR_NULL;
            if (!aligned16(p)) return SMOE_ERR_ALIGN;
        }
    }
    // every output against every input, the workspace and the other outputs
    for (int e = 0; e < n; ++e) {
        if (T[e] == 0) continue;
        const Span o = {Y[e], static_cast<size_t>(T[e]) * static_cast<size_t>(d_model) * sizeof(float)};
        if (need > 0 && overlap(o, w)) return SMOE_ERR_ALIAS;
        for (int f = 0; f < n; ++f) {
            if (T[f] == 0) continue;
            const Span ins[7] = {{gc[f], q_bytes(bits, d_ff, d_model)}, {gs[f], scale_bytes(d_ff, d_model, group)},
                                 {uc[f], q_bytes(bits, d_ff, d_model)}, {us[f], scale_bytes(d_ff, d_model, group)},
                                 {dc[f], q_bytes(bits, d_model, d_ff)}, {ds[f], scale_bytes(d_model, d_ff, group)},
                                 {X[f], static_cast<size_t>(T[f]) * static_cast<size_t>(d_model) * sizeof(float)}};
            for (const Span &in : ins)
                if (overlap(o, in) || (need > 0 && overlap(w, in))) return SMOE_ERR_ALIAS;
            if (f > e && overlap(o, Span{Y[f], static_cast<size_t>(T[f]) * static_cast<size_t>(d_model) *
                                                   sizeof(float)}))
                return SMOE_ERR_ALIAS;
        }
    }
    return to_status(smoe::launch_ffn_batch_experts(bits, n, gc, gs, uc, us, dc, ds, X, Y, T, d_model, d_ff, group,
                                                    workspace, static_cast<cudaStream_t>(stream)));
}

// Routed FFN: hidden[k x d_ff] in the workspace, out[k x d_model].
size_t routed_hidden_bytes(int k, int d_ff)
{
    const size_t b = static_cast<size_t>(k) * static_cast<size_t>(d_ff) * sizeof(float);
    return (b + 255u) & ~static_cast<size_t>(255u);
}

int experts_ffn_routed_impl(int bits, int n_experts, int k, const uint8_t *const *gc, const float *const *gs,
                            const uint8_t *const *uc, const float *const *us, const uint8_t *const *dc,
                            const float *const *ds, const int *top_idx, const float *x, float *out, int d_model,
                            int d_ff, int group, void *workspace, size_t workspace_bytes, void *stream)
{
    if (n_experts < 0 || k < 0 || k > SMOE_MAX_ROUTED_SLOTS) return SMOE_ERR_SHAPE;
    int st = check_q_shape(bits, d_ff, d_model, group);
    if (st != SMOE_OK) return st;
    st = check_q_shape(bits, d_model, d_ff, group);
    if (st != SMOE_OK) return st;
    // rows the bulk-copy decode kernels take: whole multiples of 8 chunks of
    // 16 bytes, at most 8192 columns (their staging then always fits)
    const int unit = bits == 4 ? 256 : 512;
    if (d_model % unit || d_ff % unit || d_model > 8192 || d_ff > 8192) return SMOE_ERR_SHAPE;
    if (k == 0 || d_model == 0) return SMOE_OK;
    if (n_experts == 0) return SMOE_ERR_SHAPE;  // no index could be valid
    if (!out || !top_idx) return SMOE_ERR_NULL;
    if (!aligned16(out) || (reinterpret_cast<uintptr_t>(top_idx) & 3u)) return SMOE_ERR_ALIGN;
    const size_t out_bytes = static_cast<size_t>(k) * static_cast<size_t>(d_model) * sizeof(float);
    const Span idx_span = {top_idx, static_cast<size_t>(k) * sizeof(int)};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (d_ff == 0) {
        // every output is an empty sum
        if (overlap(Span{out, out_bytes}, idx_span)) return SMOE_ERR_ALIAS;
        return to_status(cudaMemsetAsync(out, 0, out_bytes, s));
    }
    if (!gc || !gs || !uc || !us || !dc || !ds || !x) return SMOE_ERR_NULL;
    const void *tabs[6] = {gc, gs, uc, us, dc, ds};
    for (const void *t : tabs)
        if (reinterpret_cast<uintptr_t>(t) & 7u) return SMOE_ERR_ALIGN;
    if (!aligned16(x)) return SMOE_ERR_ALIGN;
    const size_t need = routed_hidden_bytes(k, d_ff);
    if (!workspace || workspace_bytes < need) return SMOE_ERR_WORKSPACE;
    if (!aligned16(workspace)) return SMOE_ERR_ALIGN;
    const size_t tab_bytes = static_cast<size_t>(n_experts) * sizeof(void *);
    const Span outs[2] = {{out, out_bytes}, {workspace, need}};
    const Span ins[8] = {{x, static_cast<size_t>(d_model) * sizeof(float)}, idx_span,
                         {gc, tab_bytes}, {gs, tab_bytes}, {uc, tab_bytes}, {us, tab_bytes},
                         {dc, tab_bytes}, {ds, tab_bytes}};
    if (any_alias(outs, 2, ins, 8)) return SMOE_ERR_ALIAS;
    float *hidden = static_cast<float *>(workspace);
    const float *xs[SMOE_MAX_ROUTED_SLOTS];
    float *ys[SMOE_MAX_ROUTED_SLOTS];
    for (int e = 0; e < k; ++e) {
        xs[e] = x;
        ys[e] = hidden + static_cast<size_t>(e) * d_ff;
    }
    bool unsupported = true;
    cudaError_t err = smoe::launch_qgemv_routed(bits, 2, k, gc, uc, gs, us, top_idx, n_experts, xs, ys, d_ff,
                                                d_model, group, s, &unsupported);
    if (unsupported) return SMOE_ERR_SHAPE;
    if (err != cudaSuccess) return SMOE_ERR_LAUNCH;
    for (int e = 0; e < k; ++e) {
        xs[e] = hidden + static_cast<size_t>(e) * d_ff;
        ys[e] = out + static_cast<size_t>(e) * d_model;
    }
    err = smoe::launch_qgemv_routed(bits, 1, k, dc, dc, ds, ds, top_idx, n_experts, xs, ys, d_model, d_ff, group,
                                    s, &unsupported);
    if (unsupported) return SMOE_ERR_SHAPE;
    return to_status(err);
}

}  // namespace

extern "C" {

size_t smoe_experts_ffn_workspace_bytes(int n_experts, int d_ff) { return ffn_workspace_bytes(n_experts, d_ff); }

int smoe_experts_ffn_q4(int n_experts, const uint8_t *const *gate_codes, const float *const *gate_scales,
                        const uint8_t *const *up_codes, const float *const *up_scales,
                        const uint8_t *const *down_codes, const float *const *down_scales, const float *x,
                        float *out, int d_model, int d_ff, int group, void *workspace, size_t workspace_bytes,
                        void *stream)
{
    return experts_ffn_impl(4, n_experts, gate_codes, gate_scales, up_codes, up_scales, down_codes, down_scales,
                            x, out, d_model, d_ff, group, workspace, workspace_bytes, stream);
}

int smoe_experts_ffn_q2(int n_experts, const uint8_t *const *gate_codes, const float *const *gate_scales,
                        const uint8_t *const *up_codes, const float *const *up_scales,
                        const uint8_t *const *down_codes, const float *const *down_scales, const float *x,
                        float *out, int d_model, int d_ff, int group, void *workspace, size_t workspace_bytes,
                        void *stream)
{
    return experts_ffn_impl(2, n_experts, gate_codes, gate_scales, up_codes, up_scales, down_codes, down_scales,
                            x, out, d_model, d_ff, group, workspace, workspace_bytes, stream);
}

int smoe_experts_gate_up_q4(int n_experts, const uint8_t *const *gate_codes, const float *const *gate_scales,
                            const uint8_t *const *up_codes, const float *const *up_scales, const float *x,
                            float *hidden, int d_ff, int d_model, int group, void *stream)
{
    return experts_impl(4, 2, n_experts, gate_codes, gate_scales, up_codes, up_scales, x, hidden, d_ff,
                        d_model, group, stream);
}

int smoe_experts_gate_up_q2(int n_experts, const uint8_t *const *gate_codes, const float *const *gate_scales,
                            const uint8_t *const *up_codes, const float *const *up_scales, const float *x,
                            float *hidden, int d_ff, int d_model, int group, void *stream)
{
    return experts_impl(2, 2, n_experts, gate_codes, gate_scales, up_codes, up_scales, x, hidden, d_ff,
                        d_model, group, stream);
}

int smoe_experts_down_q4(int n_experts, const uint8_t *const *down_codes, const float *const *down_scales,
                         const float *hidden, float *out, int d_model, int d_ff, int group, void *stream)
{
    return experts_impl(4, 1, n_experts, down_codes, down_scales, nullptr, nullptr, hidden, out, d_model,
                        d_ff, group, stream);
}

int smoe_experts_down_q2(int n_experts, const uint8_t *const *down_codes, const float *const *down_scales,
                         const float *hidden, float *out, int d_model, int d_ff, int group, void *stream)
{
    return experts_impl(2, 1, n_experts, down_codes, down_scales, nullptr, nullptr, hidden, out, d_model,
                        d_ff, group, stream);
}

int smoe_abi_version(void) { return SMOE_ABI_VERSION; }

const char *smoe_status_string(int status)
{
    switch (status) {
    case SMOE_OK: return "ok";
    case SMOE_ERR_NULL: return "a required pointer is NULL";
    case SMOE_ERR_ALIGN: return "a pointer is not 16-byte aligned";
    case SMOE_ERR_SHAPE: return "sizes break the layout contract or the limits";
    case SMOE_ERR_WORKSPACE: return "workspace missing or too small";
    case SMOE_ERR_LAUNCH: return "CUDA launch or device query failed";
    case SMOE_ERR_TIMEOUT: return "a device-side bounded wait gave up";
    case SMOE_ERR_ALIAS: return "an output overlaps an input or another output";
    case SMOE_ERR_MEMORY: return "a buffer is not accessible from the device";
    case SMOE_ERR_ROUTE: return "a device-side expert index or table entry was invalid";
    default: return "unknown status";
    }
}

int smoe_gate_up_q4(const uint8_t *gate_codes, const float *gate_scales, const uint8_t *up_codes,
                    const float *up_scales, const float *x, float *hidden, int d_ff, int d_model,
                    int group, void *stream)
{
    return gate_up_impl(4, gate_codes, gate_scales, up_codes, up_scales, x, hidden, d_ff, d_model,
                        group, stream);
}

int smoe_gate_up_q2(const uint8_t *gate_codes, const float *gate_scales, const uint8_t *up_codes,
                    const float *up_scales, const float *x, float *hidden, int d_ff, int d_model,
                    int group, void *stream)
{
    return gate_up_impl(2, gate_codes, gate_scales, up_codes, up_scales, x, hidden, d_ff, d_model,
                        group, stream);
}

int smoe_down_q4(const uint8_t *down_codes, const float *down_scales, const float *hidden,
                 float *out, int d_model, int d_ff, int group, void *stream)
{
    return down_impl(4, down_codes, down_scales, hidden, out, d_model, d_ff, group, stream);
}

int smoe_down_q2(const uint8_t *down_codes, const float *down_scales, const float *hidden,
                 float *out, int d_model, int d_ff, int group, void *stream)
{
    return down_impl(2, down_codes, down_scales, hidden, out, d_model, d_ff, group, stream);
}

int matvec_bf16(const uint16_t *w, const float *x, float *y, int rows, int cols, void *stream)
{
    if (rows < 0 || cols < 0 || cols > SMOE_MAX_COLS || cols % 8 != 0) return SMOE_ERR_SHAPE;
    if (rows == 0) return SMOE_OK;
    if (!y) return SMOE_ERR_NULL;
    if (!aligned16(y)) return SMOE_ERR_ALIGN;
    if (cols > 0) {
        if (!w || !x) return SMOE_ERR_NULL;
        if (!aligned16(w) || !aligned16(x)) return SMOE_ERR_ALIGN;
    }
    const Span o[1] = {{y, static_cast<size_t>(rows) * sizeof(float)}};
    const Span in[2] = {{w, static_cast<size_t>(rows) * static_cast<size_t>(cols) * 2},
                        {x, static_cast<size_t>(cols) * sizeof(float)}};
    if (any_alias(o, 1, in, 2)) return SMOE_ERR_ALIAS;
    return to_status(smoe::launch_bf16_gemv(w, x, y, rows, cols, static_cast<cudaStream_t>(stream)));
}

int matvec_bf16_batch(int n, const uint16_t *const *w, const float *const *x, float *const *y,
                      const int *rows, const int *cols, void *stream)
{
    if (n < 0) return SMOE_ERR_SHAPE;
    if (n == 0) return SMOE_OK;
    if (!w || !x || !y || !rows || !cols) return SMOE_ERR_NULL;
    for (int i = 0; i < n; ++i) {
        if (rows[i] < 0 || cols[i] < 0 || cols[i] > SMOE_MAX_COLS || cols[i] % 8 != 0) return SMOE_ERR_SHAPE;
        if (rows[i] == 0) continue;
        if (!y[i]) return SMOE_ERR_NULL;
        if (!aligned16(y[i])) return SMOE_ERR_ALIGN;
        if (cols[i] > 0) {
            if (!w[i] || !x[i]) return SMOE_ERR_NULL;
            if (!aligned16(w[i]) || !aligned16(x[i])) return SMOE_ERR_ALIGN;
        }
    }
    // every output against every input and every other output
    for (int i = 0; i < n; ++i) {
        if (rows[i] == 0) continue;
        const Span o = {y[i], static_cast<size_t>(rows[i]) * sizeof(float)};
        for (int j = 0; j < n; ++j) {
            if (rows[j] == 0) continue;
            if (j > i && overlap(o, Span{y[j], static_cast<size_t>(rows[j]) * sizeof(float)})) return SMOE_ERR_ALIAS;
            if (cols[j] == 0) continue;
            if (overlap(o, Span{w[j], static_cast<size_t>(rows[j]) * static_cast<size_t>(cols[j]) * 2}) ||
                overlap(o, Span{x[j], static_cast<size_t>(cols[j]) * sizeof(float)}))
                return SMOE_ERR_ALIAS;
        }
    }
    return to_status(smoe::launch_bf16_gemv_batch(n, w, x, y, rows, cols, static_cast<cudaStream_t>(stream)));
}

size_t smoe_ffn_batch_workspace_bytes(int T, int d_model, int d_ff, int group)
{
    if (check_q_shape(4, d_ff, d_model, group) != SMOE_OK ||
        check_q_shape(4, d_model, d_ff, group) != SMOE_OK)
        return static_cast<size_t>(-1);
    if (T <= 0) return 0;
    return smoe::ffn_batch_workspace(T, d_model, d_ff, group);
}

int ffn_batch_q4(const uint8_t *gate_codes, const float *gate_scales, const uint8_t *up_codes,
                 const float *up_scales, const uint8_t *down_codes, const float *down_scales,
                 const float *X, float *Y, int T, int d_model, int d_ff, int group,
                 void *workspace, size_t workspace_bytes, void *stream)
{
    return ffn_batch_impl(4, gate_codes, gate_scales, up_codes, up_scales, down_codes, down_scales, X, Y, T,
                          d_model, d_ff, group, workspace, workspace_bytes, stream);
}

int ffn_batch_q2(const uint8_t *gate_codes, const float *gate_scales, const uint8_t *up_codes,
                 const float *up_scales, const uint8_t *down_codes, const float *down_scales,
                 const float *X, float *Y, int T, int d_model, int d_ff, int group,
                 void *workspace, size_t workspace_bytes, void *stream)
{
    return ffn_batch_impl(2, gate_codes, gate_scales, up_codes, up_scales, down_codes, down_scales, X, Y, T,
                          d_model, d_ff, group, workspace, workspace_bytes, stream);
}

size_t smoe_experts_ffn_batch_workspace_bytes(int n_experts, const int *T, int d_model, int d_ff, int group)
{
    if (n_experts <= 0) return 0;
    if (!T) return static_cast<size_t>(-1);
    // the Q4 layout rules (Q2's are stricter: a Q2 shape passes them too)
    if (check_q_shape(4, d_ff, d_model, group) != SMOE_OK || check_q_shape(4, d_model, d_ff, group) != SMOE_OK)
        return static_cast<size_t>(-1);
    for (int e = 0; e < n_experts; ++e)
        if (T[e] < 0) return static_cast<size_t>(-1);
    return smoe::ffn_batch_workspace_experts(n_experts, T, d_model, d_ff, group);
}

int smoe_experts_ffn_batch_q4(int n_experts, const uint8_t *const *gate_codes, const float *const *gate_scales,
                              const uint8_t *const *up_codes, const float *const *up_scales,
                              const uint8_t *const *down_codes, const float *const *down_scales,
                              const float *const *X, float *const *Y, const int *T, int d_model, int d_ff,
                              int group, void *workspace, size_t workspace_bytes, void *stream)
{
    return experts_batch_impl(4, n_experts, gate_codes, gate_scales, up_codes, up_scales, down_codes, down_scales,
                              X, Y, T, d_model, d_ff, group, workspace, workspace_bytes, stream);
}

int smoe_experts_ffn_batch_q2(int n_experts, const uint8_t *const *gate_codes, const float *const *gate_scales,
                              const uint8_t *const *up_codes, const float *const *up_scales,
                              const uint8_t *const *down_codes, const float *const *down_scales,
                              const float *const *X, float *const *Y, const int *T, int d_model, int d_ff,
                              int group, void *workspace, size_t workspace_bytes, void *stream)
{
    return experts_batch_impl(2, n_experts, gate_codes, gate_scales, up_codes, up_scales, down_codes, down_scales,
                              X, Y, T, d_model, d_ff, group, workspace, workspace_bytes, stream);
}

size_t smoe_experts_ffn_routed_workspace_bytes(int k, int d_ff)
{
    if (k < 0 || k > SMOE_MAX_ROUTED_SLOTS || d_ff < 0) return static_cast<size_t>(-1);
    return routed_hidden_bytes(k, d_ff);
}

int smoe_experts_ffn_routed_q4(int n_experts, int k, const uint8_t *const *gate_codes,
                               const float *const *gate_scales, const uint8_t *const *up_codes,
                               const float *const *up_scales, const uint8_t *const *down_codes,
                               const float *const *down_scales, const int *top_idx, const float *x, float *out,
                               int d_model, int d_ff, int group, void *workspace, size_t workspace_bytes,
                               void *stream)
{
    return experts_ffn_routed_impl(4, n_experts, k, gate_codes, gate_scales, up_codes, up_scales, down_codes,
                                   down_scales, top_idx, x, out, d_model, d_ff, group, workspace, workspace_bytes,
                                   stream);
}

int smoe_experts_ffn_routed_q2(int n_experts, int k, const uint8_t *const *gate_codes,
                               const float *const *gate_scales, const uint8_t *const *up_codes,
                               const float *const *up_scales, const uint8_t *const *down_codes,
                               const float *const *down_scales, const int *top_idx, const float *x, float *out,
                               int d_model, int d_ff, int group, void *workspace, size_t workspace_bytes,
                               void *stream)
{
    return experts_ffn_routed_impl(2, n_experts, k, gate_codes, gate_scales, up_codes, up_scales, down_codes,
                                   down_scales, top_idx, x, out, d_model, d_ff, group, workspace, workspace_bytes,
                                   stream);
}

int smoe_route_topk_bf16(const uint16_t *gate_w, const float *x, int n_experts, int d_model, int k, float *logits,
                         int *top_idx, float *top_w, void *stream)
{
    if (n_experts < 1 || n_experts > SMOE_MAX_ROUTE_EXPERTS) return SMOE_ERR_SHAPE;
    if (k < 1 || k > n_experts || k > SMOE_MAX_TOP_K) return SMOE_ERR_SHAPE;
    if (d_model < 0 || d_model > SMOE_MAX_COLS || d_model % 8 != 0) return SMOE_ERR_SHAPE;
    if (!logits || !top_idx || !top_w) return SMOE_ERR_NULL;
    if (d_model > 0 && (!gate_w || !x)) return SMOE_ERR_NULL;
    if (!aligned16(logits) || (d_model > 0 && (!aligned16(gate_w) || !aligned16(x)))) return SMOE_ERR_ALIGN;
    if ((reinterpret_cast<uintptr_t>(top_idx) & 3u) || (reinterpret_cast<uintptr_t>(top_w) & 3u))
        return SMOE_ERR_ALIGN;
    const Span outs[3] = {{logits, static_cast<size_t>(n_experts) * sizeof(float)},
                          {top_idx, static_cast<size_t>(k) * sizeof(int)},
                          {top_w, static_cast<size_t>(k) * sizeof(float)}};
    const Span ins[2] = {{gate_w, static_cast<size_t>(n_experts) * static_cast<size_t>(d_model) * 2},
                         {x, static_cast<size_t>(d_model) * sizeof(float)}};
    if (any_alias(outs, 3, ins, d_model > 0 ? 2 : 0)) return SMOE_ERR_ALIAS;
    return to_status(smoe::launch_route(gate_w, x, n_experts, d_model, k, logits, top_idx, top_w,
                                        static_cast<cudaStream_t>(stream)));
}

int smoe_combine(int k, const float *expert_out, const float *top_w, float *out, int d_model, void *stream)
{
    if (k < 0 || d_model < 0) return SMOE_ERR_SHAPE;
    if (d_model == 0) return SMOE_OK;
    if (!out || (k > 0 && (!expert_out || !top_w))) return SMOE_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(out) & 3u) || (k > 0 && ((reinterpret_cast<uintptr_t>(expert_out) & 3u) ||
                                                             (reinterpret_cast<uintptr_t>(top_w) & 3u))))
        return SMOE_ERR_ALIGN;
    const Span o[1] = {{out, static_cast<size_t>(d_model) * sizeof(float)}};
    const Span ins[2] = {{expert_out, static_cast<size_t>(k) * static_cast<size_t>(d_model) * sizeof(float)},
                         {top_w, static_cast<size_t>(k) * sizeof(float)}};
    if (any_alias(o, 1, ins, k > 0 ? 2 : 0)) return SMOE_ERR_ALIAS;
    return to_status(smoe::launch_combine(k, expert_out, top_w, out, d_model, static_cast<cudaStream_t>(stream)));
}

// ---- many tokens

static bool aligned_to(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

static size_t elem_bytes(int dtype) { return dtype == SMOE_BF16 ? 2u : 4u; }

// Sizes shared by the calls over T tokens' k slots: T k slots are counted in
// 32 bits.
static int check_slots(int n_tokens, int k)
{
    if (n_tokens < 0 || k < 1 || k > SMOE_MAX_TOP_K) return SMOE_ERR_SHAPE;
    if (static_cast<long long>(n_tokens) * k > SMOE_MAX_SLOTS) return SMOE_ERR_SHAPE;
    return SMOE_OK;
}

static int check_rows(int dtype, int d_model)
{
    if (dtype != SMOE_F32 && dtype != SMOE_BF16) return SMOE_ERR_SHAPE;
    return d_model < 0 || d_model > SMOE_MAX_SLOTS ? SMOE_ERR_SHAPE : SMOE_OK;
}

int smoe_topk_rows(const float *logits, int n_tokens, int n_experts, int ld, int k, int *top_idx, float *top_w,
                   void *stream)
{
    const int st = check_slots(n_tokens, k);
    if (st != SMOE_OK) return st;
    if (n_experts < 1 || n_experts > SMOE_MAX_ROUTE_EXPERTS || k > n_experts || ld < n_experts) return SMOE_ERR_SHAPE;
    if (n_tokens == 0) return SMOE_OK;
    if (!logits || !top_idx || !top_w) return SMOE_ERR_NULL;
    if (!aligned_to(logits, 4) || !aligned_to(top_idx, 4) || !aligned_to(top_w, 4)) return SMOE_ERR_ALIGN;
    const size_t slots = static_cast<size_t>(n_tokens) * k;
    const Span outs[2] = {{top_idx, slots * sizeof(int)}, {top_w, slots * sizeof(float)}};
    const Span ins[1] = {
        {logits, (static_cast<size_t>(n_tokens - 1) * ld + static_cast<size_t>(n_experts)) * sizeof(float)}};
    if (any_alias(outs, 2, ins, 1)) return SMOE_ERR_ALIAS;
    return to_status(smoe::launch_topk_rows(logits, n_tokens, n_experts, ld, k, top_idx, top_w,
                                            static_cast<cudaStream_t>(stream)));
}

int smoe_topk_rows_backward(const int *top_idx, const float *top_w, const float *d_top_w, int n_tokens, int n_experts,
                            int k, float *d_logits, void *stream)
{
    const int st = check_slots(n_tokens, k);
    if (st != SMOE_OK) return st;
    if (n_experts < 1 || n_experts > SMOE_MAX_ROUTE_EXPERTS || k > n_experts) return SMOE_ERR_SHAPE;
    if (n_tokens == 0) return SMOE_OK;
    if (!top_idx || !top_w || !d_top_w || !d_logits) return SMOE_ERR_NULL;
    if (!aligned_to(top_idx, 4) || !aligned_to(top_w, 4) || !aligned_to(d_top_w, 4) || !aligned16(d_logits))
        return SMOE_ERR_ALIGN;
    const size_t slots = static_cast<size_t>(n_tokens) * k;
    const Span outs[1] = {{d_logits, static_cast<size_t>(n_tokens) * n_experts * sizeof(float)}};
    const Span ins[3] = {{top_idx, slots * sizeof(int)}, {top_w, slots * sizeof(float)}, {d_top_w, slots * sizeof(float)}};
    if (any_alias(outs, 1, ins, 3)) return SMOE_ERR_ALIAS;
    return to_status(smoe::launch_topk_rows_grad(top_idx, top_w, d_top_w, n_tokens, n_experts, k, d_logits,
                                                 static_cast<cudaStream_t>(stream)));
}

size_t smoe_dispatch_workspace_bytes(int n_tokens, int k, int n_experts)
{
    if (check_slots(n_tokens, k) != SMOE_OK || n_experts < 1 || n_experts > SMOE_MAX_ROUTE_EXPERTS)
        return static_cast<size_t>(-1);
    return n_tokens == 0 ? 0 : smoe::dispatch_workspace(n_tokens, k, n_experts);
}

int smoe_dispatch_tokens(const int *top_idx, int n_tokens, int k, int n_experts, const void *x, int dtype, int d_model,
                         int *offsets, int *order, int *place, void *xs, void *workspace, size_t workspace_bytes,
                         void *stream)
{
    int st = check_slots(n_tokens, k);
    if (st == SMOE_OK) st = check_rows(dtype, d_model);
    if (st != SMOE_OK) return st;
    if (n_experts < 1 || n_experts > SMOE_MAX_ROUTE_EXPERTS) return SMOE_ERR_SHAPE;
    if (!offsets) return SMOE_ERR_NULL;
    if (!aligned_to(offsets, 4)) return SMOE_ERR_ALIGN;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (n_tokens == 0) return to_status(smoe::launch_zero_words(offsets, n_experts + 1, s));
    if (!top_idx || !order || !place) return SMOE_ERR_NULL;
    const bool rows = (x || xs) && d_model > 0;
    if (rows && (!x || !xs)) return SMOE_ERR_NULL;
    const size_t e = elem_bytes(dtype);
    if (!aligned_to(top_idx, 4) || !aligned_to(order, 4) || !aligned_to(place, 4)) return SMOE_ERR_ALIGN;
    if (rows && (!aligned_to(x, e) || !aligned_to(xs, e))) return SMOE_ERR_ALIGN;
    const size_t need = smoe::dispatch_workspace(n_tokens, k, n_experts);
    if (!workspace || workspace_bytes < need) return SMOE_ERR_WORKSPACE;
    if (!aligned16(workspace)) return SMOE_ERR_ALIGN;
    const size_t slots = static_cast<size_t>(n_tokens) * k;
    const Span outs[5] = {{offsets, (static_cast<size_t>(n_experts) + 1) * sizeof(int)},
                          {order, slots * sizeof(int)},
                          {place, slots * sizeof(int)},
                          {workspace, need},
                          {xs, rows ? slots * d_model * e : 0}};
    const Span ins[2] = {{top_idx, slots * sizeof(int)}, {x, rows ? static_cast<size_t>(n_tokens) * d_model * e : 0}};
    if (any_alias(outs, 5, ins, 2)) return SMOE_ERR_ALIAS;
    return to_status(smoe::launch_dispatch(top_idx, n_tokens, k, n_experts, rows ? x : nullptr, dtype, d_model, offsets,
                                           order, place, rows ? xs : nullptr, workspace, s));
}

// out[t] = sum over s of w[t, s] rows[place[t, s]], w null: of the rows.
static int sum_impl(const void *rows, int dtype, const int *place, const float *w, bool weighted, int n_tokens, int k,
                    int d_model, void *out, void *stream)
{
    int st = check_slots(n_tokens, k);
    if (st == SMOE_OK) st = check_rows(dtype, d_model);
    if (st != SMOE_OK) return st;
    if (n_tokens == 0 || d_model == 0) return SMOE_OK;
    if (!rows || !place || !out || (weighted && !w)) return SMOE_ERR_NULL;
    const size_t e = elem_bytes(dtype), slots = static_cast<size_t>(n_tokens) * k;
    if (!aligned_to(rows, e) || !aligned_to(out, e) || !aligned_to(place, 4) || (weighted && !aligned_to(w, 4)))
        return SMOE_ERR_ALIGN;
    const Span outs[1] = {{out, static_cast<size_t>(n_tokens) * d_model * e}};
    const Span ins[3] = {{rows, slots * d_model * e}, {place, slots * sizeof(int)}, {w, weighted ? slots * sizeof(float) : 0}};
    if (any_alias(outs, 1, ins, 3)) return SMOE_ERR_ALIAS;
    return to_status(smoe::launch_sum_tokens(rows, dtype, place, weighted ? w : nullptr, n_tokens, k, d_model, out,
                                             static_cast<cudaStream_t>(stream)));
}

int smoe_dispatch_tokens_backward(const void *d_xs, int dtype, const int *place, int n_tokens, int k, int d_model,
                                  void *d_x, void *stream)
{
    return sum_impl(d_xs, dtype, place, nullptr, false, n_tokens, k, d_model, d_x, stream);
}

int smoe_combine_tokens(const void *ys, int dtype, const int *place, const float *top_w, int n_tokens, int k, int d_model,
                        void *out, void *stream)
{
    return sum_impl(ys, dtype, place, top_w, true, n_tokens, k, d_model, out, stream);
}

int smoe_combine_tokens_backward(const void *d_out, const void *ys, int dtype, const int *place, const float *top_w,
                                 int n_tokens, int k, int d_model, void *d_ys, float *d_top_w, void *stream)
{
    int st = check_slots(n_tokens, k);
    if (st == SMOE_OK) st = check_rows(dtype, d_model);
    if (st != SMOE_OK) return st;
    if (n_tokens == 0) return SMOE_OK;
    if (!place || !top_w || !d_top_w || (d_model > 0 && (!d_out || !ys || !d_ys))) return SMOE_ERR_NULL;
    const size_t e = elem_bytes(dtype), slots = static_cast<size_t>(n_tokens) * k;
    if (!aligned_to(place, 4) || !aligned_to(top_w, 4) || !aligned_to(d_top_w, 4)) return SMOE_ERR_ALIGN;
    if (d_model > 0 && (!aligned_to(d_out, e) || !aligned_to(ys, e) || !aligned_to(d_ys, e))) return SMOE_ERR_ALIGN;
    const Span outs[2] = {{d_ys, slots * d_model * e}, {d_top_w, slots * sizeof(float)}};
    const Span ins[4] = {{d_out, static_cast<size_t>(n_tokens) * d_model * e},
                         {ys, slots * d_model * e},
                         {place, slots * sizeof(int)},
                         {top_w, slots * sizeof(float)}};
    if (any_alias(outs, 2, ins, 4)) return SMOE_ERR_ALIAS;
    return to_status(smoe::launch_combine_tokens_grad(d_out, ys, dtype, place, top_w, n_tokens, k, d_model, d_ys, d_top_w,
                                                      static_cast<cudaStream_t>(stream)));
}

// ---- 8-bit weights and activations

int smoe_quantize_rows_q8(const void *x, int dtype, int act, int rows, int cols, int8_t *q, float *scales, void *stream)
{
    const int st = check_rows(dtype, cols);
    if (st != SMOE_OK) return st;
    if (rows < 0 || cols > SMOE_MAX_COLS || (act != SMOE_Q8_PLAIN && act != SMOE_Q8_SILU_MUL)) return SMOE_ERR_SHAPE;
    if (rows == 0) return SMOE_OK;
    if (!scales || (cols > 0 && (!x || !q))) return SMOE_ERR_NULL;
    const size_t e = elem_bytes(dtype), n = static_cast<size_t>(rows) * cols;
    if (!aligned_to(scales, 4) || (cols > 0 && (!aligned_to(x, e) || !aligned16(q)))) return SMOE_ERR_ALIGN;
    const Span outs[2] = {{q, n}, {scales, static_cast<size_t>(rows) * sizeof(float)}};
    const Span ins[1] = {{x, n * e * (act == SMOE_Q8_SILU_MUL ? 2 : 1)}};
    if (any_alias(outs, 2, ins, 1)) return SMOE_ERR_ALIAS;
    return to_status(smoe::launch_quantize_rows(x, dtype, act == SMOE_Q8_SILU_MUL, rows, cols, q, scales,
                                                static_cast<cudaStream_t>(stream)));
}

// Sizes of an 8-bit product: rows of whole 16-byte vectors, with source rows to
// come from; the weights' rows are counted in 32 bits.
static int check_q8(int n_src, int n_rows, int n_experts, int n_out, int n_in)
{
    if (n_src < 0 || (n_src == 0 && n_rows > 0)) return SMOE_ERR_SHAPE;
    if (n_rows < 0 || n_rows > SMOE_MAX_SLOTS || n_out < 0 || n_in < 0) return SMOE_ERR_SHAPE;
    if (n_experts < 1 || n_experts > SMOE_MAX_ROUTE_EXPERTS) return SMOE_ERR_SHAPE;
    if (n_in % 16 != 0 || n_in > SMOE_MAX_COLS) return SMOE_ERR_SHAPE;
    if (static_cast<long long>(n_experts) * n_out > SMOE_MAX_SLOTS) return SMOE_ERR_SHAPE;
    return SMOE_OK;
}

size_t smoe_experts_matmul_q8_workspace_bytes(int n_src, int n_rows, int n_experts, int n_out, int n_in)
{
    if (check_q8(n_src, n_rows, n_experts, n_out, n_in) != SMOE_OK) return static_cast<size_t>(-1);
    return n_rows == 0 || n_out == 0 ? 0 : smoe::q8_workspace(n_src, n_rows, n_experts, n_in);
}

size_t smoe_matmul_q8_workspace_bytes(int n_rows, int n_out, int n_in)
{
    return smoe_experts_matmul_q8_workspace_bytes(n_rows, n_rows, 1, n_out, n_in);
}

static int q8_impl(const int8_t *xq, const float *x_scales, int n_src, const int *order, int k, const int *offsets,
                   bool sorted, int n_rows, int n_experts, const int8_t *wq, const float *w_scales, int n_out, int n_in,
                   void *y, int dtype, void *workspace, size_t workspace_bytes, void *stream)
{
    int st = check_q8(n_src, n_rows, n_experts, n_out, n_in);
    if (st == SMOE_OK) st = check_rows(dtype, 0);
    if (st != SMOE_OK) return st;
    if (order ? (k < 1 || k > SMOE_MAX_TOP_K) : n_src < n_rows) return SMOE_ERR_SHAPE;
    if (n_rows == 0 || n_out == 0) return SMOE_OK;
    if (!x_scales || !w_scales || !y || (sorted && !offsets) || (n_in > 0 && (!xq || !wq))) return SMOE_ERR_NULL;
    const size_t e = elem_bytes(dtype);
    if (!aligned_to(x_scales, 4) || !aligned16(w_scales) || !aligned16(y) || (order && !aligned_to(order, 4)) ||
        (sorted && !aligned_to(offsets, 4)) || (n_in > 0 && (!aligned16(xq) || !aligned16(wq))))
        return SMOE_ERR_ALIGN;
    const size_t need = smoe::q8_workspace(n_src, n_rows, n_experts, n_in);
    if (!workspace || workspace_bytes < need) return SMOE_ERR_WORKSPACE;
    if (!aligned16(workspace)) return SMOE_ERR_ALIGN;
    const size_t wrows = static_cast<size_t>(n_experts) * n_out;
    const Span outs[2] = {{y, static_cast<size_t>(n_rows) * n_out * e}, {workspace, need}};
    const Span ins[6] = {{xq, static_cast<size_t>(n_src) * n_in},
                         {x_scales, static_cast<size_t>(n_src) * sizeof(float)},
                         {wq, wrows * n_in},
                         {w_scales, wrows * sizeof(float)},
                         {order, order ? static_cast<size_t>(n_rows) * sizeof(int) : 0},
                         {offsets, sorted ? (static_cast<size_t>(n_experts) + 1) * sizeof(int) : 0}};
    if (any_alias(outs, 2, ins, 6)) return SMOE_ERR_ALIAS;
    return to_status(smoe::launch_q8(xq, x_scales, n_src, order, k, sorted ? offsets : nullptr, n_rows, n_experts, wq,
                                     w_scales, n_out, n_in, y, dtype, workspace, static_cast<cudaStream_t>(stream)));
}

int smoe_matmul_q8(const int8_t *xq, const float *x_scales, int n_rows, const int8_t *wq, const float *w_scales, int n_out,
                   int n_in, void *y, int dtype, void *workspace, size_t workspace_bytes, void *stream)
{
    return q8_impl(xq, x_scales, n_rows, nullptr, 1, nullptr, false, n_rows, 1, wq, w_scales, n_out, n_in, y, dtype,
                   workspace, workspace_bytes, stream);
}

int smoe_experts_matmul_q8(const int8_t *xq, const float *x_scales, int n_src, const int *order, int k,
                           const int *offsets, int n_rows, int n_experts, const int8_t *wq, const float *w_scales,
                           int n_out, int n_in, void *y, int dtype, void *workspace, size_t workspace_bytes, void *stream)
{
    return q8_impl(xq, x_scales, n_src, order, k, offsets, true, n_rows, n_experts, wq, w_scales, n_out, n_in, y, dtype,
                   workspace, workspace_bytes, stream);
}

int smoe_copy(void *dst, const void *src, size_t bytes, void *stream)
{
    if (bytes == 0) return SMOE_OK;
    if (!dst || !src) return SMOE_ERR_NULL;
    if (((reinterpret_cast<uintptr_t>(dst) | reinterpret_cast<uintptr_t>(src) | bytes) & 15u) != 0)
        return SMOE_ERR_ALIGN;
    if (overlap(Span{dst, bytes}, Span{src, bytes})) return SMOE_ERR_ALIAS;
    void *d = smoe::device_address(dst);
    const void *s = smoe::device_address(src);
    if (!d || !s) return SMOE_ERR_MEMORY;
    return to_status(smoe::launch_copy16(d, s, bytes, static_cast<cudaStream_t>(stream)));
}

int smoe_selftest_bounded_wait(int kind, void *stream)
{
    if (kind != 0 && kind != 1) return SMOE_ERR_SHAPE;
    return to_status(smoe::launch_bounded_wait_selftest(kind, static_cast<cudaStream_t>(stream)));
}

int smoe_last_device_status(void *stream)
{
    unsigned v = 0;
    if (smoe::read_and_clear_device_status(static_cast<cudaStream_t>(stream), &v) != cudaSuccess)
        return SMOE_ERR_LAUNCH;
    if (v == smoe::kStatusRoute) return SMOE_ERR_ROUTE;
    return v ? SMOE_ERR_TIMEOUT : SMOE_OK;
}

}  // extern "C"
