// Quantisers to 8-bit floating point (e4m3) with one f32 scale for each block of
// 128: rows in blocks of 1 x 128 (activations and their gradients), matrices in
// blocks of 128 x 128 (weights), the latter in both directions.
//
//   top = max |v| of the block,  scale = top / 448,  code = e4m3(v (448 / top))
//
// each f32 operation rounded once, the code to nearest, ties to even: the codes of
// a block are the same on any machine, and after the activation wherever expf is the
// same.  448 / top is beyond f32 below 1.4e-36:
// there top and v are taken 2^64 times.  A block of zeros has scale 0 and codes that
// keep their sign; one that holds a NaN or an infinity has scale NaN and codes 0, so
// that every product of it is NaN.
#include "q8.cuh"
#include "rowvec.cuh"
#include "smoe.h"

namespace smoe {
namespace {

constexpr float F8_MAX = 448.f;

// Two e4m3 codes, lo in the low byte; ties to even, largest finite beyond it.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) { return e4m3x2(a, b) | e4m3x2(c, d) << 16; }

// What a block's values are multiplied by, and its scale, from the bits of its
// largest magnitude.  lift: the values are to be taken 2^64 times first.
struct BlockScale {
    float up, scale;
    bool lift;
};
__device__ __forceinline__ BlockScale block_scale(uint32_t most)
{
    const float top = __uint_as_float(most);
    BlockScale s = {0.f, 0.f, false};
    if (most >= 0x7f800000u) {
        s.scale = __int_as_float(0x7fffffff);
    } else if (most != 0u) {
        s.scale = __fdiv_rn(top, F8_MAX);
        s.up = __fdiv_rn(F8_MAX, top);
        if (s.up == INFINITY) {
            s.lift = true;
            s.up = __fdiv_rn(F8_MAX, top * 0x1p64f);
        }
    }
    return s;
}
// Two f32 operations in one instruction, each rounded as it is alone.
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
        "mul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "+f"(a.x), "+f"(a.y)
        : "f"(b.x), "f"(b.y));
    return a;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\tmov.b64 c, {%4, %5};\n\t"
        "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "+f"(a.x), "+f"(a.y)
        : "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return a;
}

// The codes of four values (lifted already).
__device__ __forceinline__ uint32_t codes4(const float *v, float up)
{
    const float2 u = make_float2(up, up), a = mul2(make_float2(v[0], v[1]), u), b = mul2(make_float2(v[2], v[3]), u);
    return e4m3x4(a.x, a.y, b.x, b.y);
}

// SiLU by the steps g / (1 + e^-g), each rounded once.  The quotient is the reciprocal
// instruction's, corrected once by its remainder (Markstein 1990): off by 1.5 2^-46 of
// itself before it is rounded, so that one in two million may be rounded to the other
// side.  The exponential is beyond what the instruction takes from g = -87.3 on: at and
// below SILU_FAR the division is taken, and g e^g where e^-g leaves f32.  32,768 rows of
// 1536 in bf16: 44.5 us, by divisions throughout 67.
constexpr float SILU_FAR = -64.f;
__device__ __forceinline__ float2 silu2(float a, float b)  // both above SILU_FAR
{
    const auto rcp = [](float d) {
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
        return r;
    };
    const float2 g = make_float2(a, b), minus = make_float2(-1.f, -1.f);
    const float2 nd = fma2(make_float2(expf(-a), expf(-b)), minus, minus);  // -(1 + e^-g)
    const float2 r = make_float2(rcp(-nd.x), rcp(-nd.y)), q = mul2(g, r);
    return fma2(fma2(q, nd, g), r, q);
}
__device__ __forceinline__ float silu_far(float g) { return g <= -88.f ? g * expf(g) : __fdiv_rn(g, 1.f + expf(-g)); }

constexpr int RUN = 16;           // columns of a thread: 8 threads a block
constexpr int ROWS_THREADS = 128;

// The 16 values at column c of a row (zeros past cols).  VEC: 16-byte vectors that
// lie within the row or past it.
template <typename T, bool VEC>
__device__ __forceinline__ void load_run(const T *row, int c, int cols, float (&v)[RUN])
{
    constexpr int VE = VEC ? 16 / static_cast<int>(sizeof(T)) : 1;
    RowVec<T, VE> x[RUN / VE];
#pragma unroll
    for (int i = 0; i < RUN / VE; ++i) {
        if (c + i * VE < cols) x[i].load(row + c + i * VE);
        else x[i].zero();
    }
#pragma unroll
    for (int i = 0; i < RUN / VE; ++i) {
        float t[VE];
        x[i].get(t);
#pragma unroll
        for (int j = 0; j < VE; ++j) v[i * VE + j] = t[j];
    }
}

// Eight threads a block of 128 columns, 16 each, a warp four blocks.  HBM-bound, with 76% of
// the issue slots taken where the activation is: 32,768 rows of 1536 in bf16 (253 MB)
// 44.5 us, 5.7 TB/s (40 registers, for more warps, 44.4).  Rows that no vector fits, with
// the activation, have the registers of seven CTAs an SM (left to itself the compiler
// spills at 64): 8191 rows of 1001 in f32 37.1 us against 38.1, in bf16 26.4 against 27.3.
template <typename T, bool VEC, bool ACT>
__global__ void __launch_bounds__(ROWS_THREADS, ACT && !VEC ? 7 : 0) quantize_rows_f8(const T *__restrict__ x, long long blocks, int nkb,
                                                                 unsigned long long magic, int cols, uint8_t *__restrict__ q,
                                                                 float *__restrict__ scales)
{
    pdl_launch_dependents();
    pdl_wait();
    const long long b = static_cast<long long>(blockIdx.x) * (ROWS_THREADS / 8) + (threadIdx.x >> 3);
    const bool in = b < blocks;
    // b / nkb: magic = ceil(2^56 / nkb), exact for b nkb < 2^56
    const long long r = in ? static_cast<long long>(__umul64hi(static_cast<unsigned long long>(b) << 8, magic)) : 0;
    const int c = static_cast<int>(b - r * nkb) * 128 + (threadIdx.x & 7) * RUN;
    const T *row = x + r * cols * (ACT ? 2 : 1);
    float v[RUN];
    load_run<T, VEC>(row, c, in ? cols : 0, v);
    if (ACT) {
        float u[RUN];
        load_run<T, VEC>(row + cols, c, in ? cols : 0, u);
        float low = v[0];
#pragma unroll
        for (int i = 1; i < RUN; ++i) low = fminf(low, v[i]);
        if (low > SILU_FAR) {
#pragma unroll
            for (int i = 0; i < RUN; i += 2) {
                const float2 t = mul2(silu2(v[i], v[i + 1]), make_float2(u[i], u[i + 1]));
                v[i] = t.x;
                v[i + 1] = t.y;
            }
        } else {  // (read again: holding both rows for this costs the other way its warps, 46 us)
#pragma unroll 1
            for (int h = 0; h < RUN; ++h) {
                const float t = c + h < cols ? silu_far(static_cast<float>(row[c + h])) * static_cast<float>(row[cols + c + h]) : 0.f;
#pragma unroll
                for (int i = 0; i < RUN; ++i)
                    if (i == h) v[i] = t;
            }
        }
    }
    float top = 0.f;  // NaN where one is
#pragma unroll
    for (int i = 0; i < RUN; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(fabsf(v[i])));
    uint32_t most = __float_as_uint(top);
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) most = max(most, __shfl_xor_sync(FULL_MASK, most, off));
    if (!in) return;
    const BlockScale s = block_scale(most);
    if ((threadIdx.x & 7) == 0) scales[b] = s.scale;
    uint32_t k[RUN / 4];
    if (s.scale != s.scale) {
#pragma unroll
        for (int i = 0; i < RUN / 4; ++i) k[i] = 0u;
    } else {
        if (s.lift) {  // (a select at each value: 2 of its 28 instructions)
#pragma unroll
            for (int i = 0; i < RUN; ++i) v[i] *= 0x1p64f;
        }
#pragma unroll
        for (int i = 0; i < RUN / 4; ++i) k[i] = codes4(v + 4 * i, s.up);
    }
    uint8_t *out = q + r * cols + c;
    if ((cols & 15) == 0) {
        if (c < cols) *reinterpret_cast<uint4 *>(out) = make_uint4(k[0], k[1], k[2], k[3]);
    } else if ((cols & 3) == 0) {
#pragma unroll
        for (int i = 0; i < RUN / 4; ++i)
            if (c + 4 * i < cols) reinterpret_cast<uint32_t *>(out)[i] = k[i];
    } else {
#pragma unroll
        for (int i = 0; i < RUN; ++i)
            if (c + i < cols) out[i] = static_cast<uint8_t>(k[i / 4] >> (8 * (i & 3)));
    }
}

// ---------------------------------------------------------------- weights

constexpr int MAT_THREADS = 256;  // 8 warps of 16 rows, a lane four columns

struct BlocksArgs {
    const void *w;
    uint8_t *q, *qt;         // qt null: one direction
    float *scales, *scales_t;
    int rows, cols, rb, cb;  // blocks along each
};

// One CTA a block: its 64 values a thread stay in registers between the maximum
// and the codes; the transposed codes go through shared memory, four rows of a
// column to a word (row 4 i + j of the block lies in slot 32 j + i, 33 words
// apart: no bank is asked twice).  HBM-bound: 16 matrices of 1536 x 4096 in f32 with both
// directions (604 MB) 96 us, 6.3 TB/s.
template <typename T, bool VEC>
__global__ void __launch_bounds__(MAT_THREADS) quantize_blocks_f8(const BlocksArgs a)
{
    __shared__ uint32_t tile[128 * 33];
    __shared__ uint32_t warp_most[MAT_THREADS / 32];
    pdl_launch_dependents();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned per = static_cast<unsigned>(a.rb) * static_cast<unsigned>(a.cb);
    const unsigned mat = blockIdx.x / per, at = blockIdx.x % per;
    const int rb = static_cast<int>(at / a.cb), cb = static_cast<int>(at % a.cb);
    const size_t elems = static_cast<size_t>(a.rows) * a.cols;
    const T *w = static_cast<const T *>(a.w) + mat * elems;
    const int r0 = rb * 128 + warp * 16, c0 = cb * 128 + lane * 4;
    float v[16][4];
    uint32_t most = 0u;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const T *p = w + static_cast<size_t>(r0 + i) * a.cols + c0;
        const bool in = r0 + i < a.rows;
        if (VEC) {  // four columns: 16 or 8 bytes
            if (in && c0 < a.cols) {
                if (sizeof(T) == 4) {
                    const float4 t = *reinterpret_cast<const float4 *>(p);
                    v[i][0] = t.x; v[i][1] = t.y; v[i][2] = t.z; v[i][3] = t.w;
                } else {
                    const uint2 t = *reinterpret_cast<const uint2 *>(p);
                    v[i][0] = __uint_as_float(t.x << 16); v[i][1] = __uint_as_float(t.x & 0xffff0000u);
                    v[i][2] = __uint_as_float(t.y << 16); v[i][3] = __uint_as_float(t.y & 0xffff0000u);
                }
            } else {
                v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0.f;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i][j] = in && c0 + j < a.cols ? static_cast<float>(p[j]) : 0.f;
        }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) most = max(most, __float_as_uint(v[i][j]) & 0x7fffffffu);
    most = __reduce_max_sync(FULL_MASK, most);
    if (lane == 0) warp_most[warp] = most;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MAT_THREADS / 32; ++i) most = max(most, warp_most[i]);
    const BlockScale s = block_scale(most);
    if (threadIdx.x == 0) {
        a.scales[(static_cast<size_t>(mat) * a.rb + rb) * a.cb + cb] = s.scale;
        if (a.qt) a.scales_t[(static_cast<size_t>(mat) * a.cb + cb) * a.rb + rb] = s.scale;
    }
    uint8_t *q = a.q + mat * elems;
    if (s.lift) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i][j] *= 0x1p64f;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const uint32_t k = s.scale != s.scale ? 0u : codes4(v[i], s.up);
        const int r = warp * 16 + i;
        tile[((r & 3) * 32 + (r >> 2)) * 33 + lane] = k;
        if (r0 + i >= a.rows) continue;
        uint8_t *out = q + static_cast<size_t>(r0 + i) * a.cols + c0;
        if ((a.cols & 3) == 0) {
            if (c0 < a.cols) *reinterpret_cast<uint32_t *>(out) = k;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c0 + j < a.cols) out[j] = static_cast<uint8_t>(k >> (8 * j));
        }
    }
    if (!a.qt) return;
    __syncthreads();
    // a lane takes rows 4 lane .. + 3 of the block, a warp 16 columns
    uint8_t *qt = a.qt + mat * elems;
    const int tr = rb * 128 + lane * 4;
#pragma unroll
    for (int c4 = 0; c4 < 4; ++c4) {
        uint32_t k[4], o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) k[j] = tile[(j * 32 + lane) * 33 + warp * 4 + c4];
        const uint32_t a01 = __byte_perm(k[0], k[1], 0x5140), b01 = __byte_perm(k[0], k[1], 0x7362);
        const uint32_t a23 = __byte_perm(k[2], k[3], 0x5140), b23 = __byte_perm(k[2], k[3], 0x7362);
        o[0] = __byte_perm(a01, a23, 0x5410);
        o[1] = __byte_perm(a01, a23, 0x7632);
        o[2] = __byte_perm(b01, b23, 0x5410);
        o[3] = __byte_perm(b01, b23, 0x7632);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = cb * 128 + warp * 16 + c4 * 4 + j;
            if (c >= a.cols) continue;
            uint8_t *out = qt + static_cast<size_t>(c) * a.rows + tr;
            if ((a.rows & 3) == 0) {
                if (tr < a.rows) *reinterpret_cast<uint32_t *>(out) = o[j];
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (tr + i < a.rows) out[i] = static_cast<uint8_t>(o[j] >> (8 * i));
            }
        }
    }
}

template <typename T>
cudaError_t rows_t(const void *x, bool act, int rows, int cols, uint8_t *q, float *scales, cudaStream_t stream)
{
    const int nkb = (cols + 127) / 128;
    const long long blocks = static_cast<long long>(rows) * nkb;
    const unsigned long long magic = ((1ull << 56) + nkb - 1) / nkb;
    const size_t pitch = static_cast<size_t>(cols) * sizeof(T);
    const bool vec = ((reinterpret_cast<uintptr_t>(x) | pitch) & 15u) == 0;
    auto go = [&](auto kernel) {
        return launch_pdl(kernel, dim3(static_cast<unsigned>((blocks + ROWS_THREADS / 8 - 1) / (ROWS_THREADS / 8))),
                          dim3(ROWS_THREADS), 0, stream, static_cast<const T *>(x), blocks, nkb, magic, cols, q, scales);
    };
    if (act) return vec ? go(quantize_rows_f8<T, true, true>) : go(quantize_rows_f8<T, false, true>);
    return vec ? go(quantize_rows_f8<T, true, false>) : go(quantize_rows_f8<T, false, false>);
}

template <typename T>
cudaError_t blocks_t(const BlocksArgs &a, int n, cudaStream_t stream)
{
    const bool vec = (a.cols & 3) == 0 && (reinterpret_cast<uintptr_t>(a.w) & (4 * sizeof(T) - 1)) == 0;
    const dim3 grid(static_cast<unsigned>(static_cast<long long>(n) * a.rb * a.cb));
    return vec ? launch_pdl(quantize_blocks_f8<T, true>, grid, dim3(MAT_THREADS), 0, stream, a)
               : launch_pdl(quantize_blocks_f8<T, false>, grid, dim3(MAT_THREADS), 0, stream, a);
}

}  // namespace

cudaError_t launch_quantize_rows_f8(const void *x, int dtype, bool act, int rows, int cols, uint8_t *q, float *scales,
                                    cudaStream_t stream)
{
    return dtype == SMOE_BF16 ? rows_t<__nv_bfloat16>(x, act, rows, cols, q, scales, stream)
                              : rows_t<float>(x, act, rows, cols, q, scales, stream);
}

cudaError_t launch_quantize_blocks_f8(const void *w, int dtype, int n, int rows, int cols, uint8_t *q, float *scales,
                                      uint8_t *qt, float *scales_t, cudaStream_t stream)
{
    const BlocksArgs a = {w, q, qt, scales, scales_t, rows, cols, (rows + 127) / 128, (cols + 127) / 128};
    return dtype == SMOE_BF16 ? blocks_t<__nv_bfloat16>(a, n, stream) : blocks_t<float>(a, n, stream);
}

}  // namespace smoe
