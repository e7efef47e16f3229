// Rows of f32 or bf16 elements as 16-byte vectors or single elements,
// widened to f32 for arithmetic and rounded once when stored.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace smoe {

// VE elements of type T as one aligned load: a 16-byte vector, or (VE == 1)
// an element, for rows whose pitch or base is not a multiple of 16 bytes.
template <typename T, int VE>
struct RowVec;

template <>
struct RowVec<float, 4> {
    uint4 raw;
    __device__ __forceinline__ void get(float (&v)[4]) const
    {
        v[0] = __uint_as_float(raw.x); v[1] = __uint_as_float(raw.y);
        v[2] = __uint_as_float(raw.z); v[3] = __uint_as_float(raw.w);
    }
    __device__ __forceinline__ void set(const float (&v)[4])
    {
        raw = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
    __device__ __forceinline__ void load(const float *p) { raw = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void store(float *p) const { *reinterpret_cast<uint4 *>(p) = raw; }
    __device__ __forceinline__ void zero() { raw = make_uint4(0u, 0u, 0u, 0u); }
};

template <>
struct RowVec<float, 1> {
    float raw;
    __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = raw; }
    __device__ __forceinline__ void set(const float (&v)[1]) { raw = v[0]; }
    __device__ __forceinline__ void load(const float *p) { raw = *p; }
    __device__ __forceinline__ void store(float *p) const { *p = raw; }
    __device__ __forceinline__ void zero() { raw = 0.f; }
};

// bf16 to f32 is a shift; f32 to bf16 rounds to nearest even.
template <>
struct RowVec<__nv_bfloat16, 8> {
    uint4 raw;
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ void set(const float (&v)[8])
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = static_cast<uint32_t>(__bfloat16_as_ushort(p.x)) |
                   (static_cast<uint32_t>(__bfloat16_as_ushort(p.y)) << 16);
        }
        raw = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { raw = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void store(__nv_bfloat16 *p) const { *reinterpret_cast<uint4 *>(p) = raw; }
    __device__ __forceinline__ void zero() { raw = make_uint4(0u, 0u, 0u, 0u); }
};

template <>
struct RowVec<__nv_bfloat16, 1> {
    __nv_bfloat16 raw;
    __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = __bfloat162float(raw); }
    __device__ __forceinline__ void set(const float (&v)[1]) { raw = __float2bfloat16_rn(v[0]); }
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { raw = *p; }
    __device__ __forceinline__ void store(__nv_bfloat16 *p) const { *p = raw; }
    __device__ __forceinline__ void zero() { raw = __ushort_as_bfloat16(0); }
};

}  // namespace smoe
