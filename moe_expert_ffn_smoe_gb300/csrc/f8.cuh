// What the kernels of the 8-bit floating-point product share.
#pragma once

#include "q8.cuh"
#include "tcgen05.cuh"

namespace smoe {

constexpr int F8_BLOCK = 128;  // columns (and weight rows) of one scale

__device__ __forceinline__ void lds_unit(uint4 &v, uint32_t addr) { v = lds128v(addr); }
__device__ __forceinline__ void lds_unit(uint2 &v, uint32_t addr)
{
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
}
__device__ __forceinline__ void lds_unit(uint32_t &v, uint32_t addr)
{
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
}
__device__ __forceinline__ void lds_unit(uint16_t &v, uint32_t addr)
{
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
}

// A warp's ROWS x COLS outputs, staged in rows `pitch` bytes apart, to y (rows of N
// elements), of which `rows` and `cols` are there: neighbouring lanes store neighbouring
// units, the largest that every row of y is a multiple of (units of an element by the
// lanes that hold 16 bytes took 24 us for 275 tokens through 99 experts of 1332 x 208).
template <typename U, int ROWS, int COLS, typename T>
__device__ __forceinline__ void store_units(uint32_t stage, uint32_t pitch, T *y, int N, int rows, int cols)
{
    constexpr int VE = sizeof(U) / sizeof(T), PER = COLS / VE;
    const int lane = threadIdx.x & 31;
#pragma unroll(ROWS > 8 ? 1 : 8)
    for (int i = 0; i < ROWS * PER / 32; ++i) {
        const int r = (i * 32 + lane) / PER, c = (i * 32 + lane) % PER * VE;
        U v;
        lds_unit(v, stage + static_cast<uint32_t>(r) * pitch + static_cast<uint32_t>(c) * static_cast<uint32_t>(sizeof(T)));
        if (r < rows && c < cols) *reinterpret_cast<U *>(y + static_cast<size_t>(r) * N + c) = v;
    }
}
template <int ROWS, int COLS, typename T>
__device__ __forceinline__ void store_staged(uint32_t stage, uint32_t pitch, T *y, int N, int rows, int cols)
{
    const uint32_t low = static_cast<uint32_t>(N) * static_cast<uint32_t>(sizeof(T));
    if ((low & 15u) == 0) store_units<uint4, ROWS, COLS>(stage, pitch, y, N, rows, cols);
    else if ((low & 7u) == 0) store_units<uint2, ROWS, COLS>(stage, pitch, y, N, rows, cols);
    else if (sizeof(T) == 4 || (low & 3u) == 0) store_units<uint32_t, ROWS, COLS>(stage, pitch, y, N, rows, cols);
    else if constexpr (sizeof(T) == 2) store_units<uint16_t, ROWS, COLS>(stage, pitch, y, N, rows, cols);
}

// The product in row tiles of 128 (f8_rows.cu), from the tile list.
cudaError_t launch_f8_rows(const F8Call &c, const int *ntiles, const Tile *tiles, int max_tiles, cudaStream_t stream);

}  // namespace smoe
