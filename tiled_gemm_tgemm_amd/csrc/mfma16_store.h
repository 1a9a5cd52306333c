// How a tile's rows leave the registers (mfma16.h).
#pragma once

#include "mfma16.h"

namespace tgemm {
namespace m16 {

// A row's adjacent columns that a lane holds.
template <class Tile>
constexpr int kHeld = 4 * Tile::FN;

__device__ __forceinline__ uint32_t pack(__bf16 a, __bf16 b)
{
    return (uint32_t)__builtin_bit_cast(uint16_t, a) | (uint32_t)__builtin_bit_cast(uint16_t, b) << 16;
}
__device__ __forceinline__ uint32_t pack(_Float16 a, _Float16 b)
{
    return (uint32_t)__builtin_bit_cast(uint16_t, a) | (uint32_t)__builtin_bit_cast(uint16_t, b) << 16;
}

// Device memory takes 16-byte stores at any address.
typedef uint32_t u32x4_anywhere __attribute__((ext_vector_type(4), aligned(2)));
typedef f32x4 f32x4_anywhere __attribute__((aligned(4)));

// N (a multiple of 8) adjacent values as 16-bit numbers.
template <class E, int N>
__device__ __forceinline__ void store_packed(E *to, const float (&v)[N])
{
#pragma unroll
    for (int q = 0; q < N / 8; ++q) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = pack((E)v[8 * q + 2 * e], (E)v[8 * q + 2 * e + 1]);
        reinterpret_cast<u32x4_anywhere *>(to)[q] = u32x4_anywhere{w[0], w[1], w[2], w[3]};
    }
}

// N adjacent values of a row of the result, `left` of them inside it.
template <class T, int N>
__device__ __forceinline__ void store_row(T *to, const float (&v)[N], int left)
{
    if (left >= N) {
        if constexpr (sizeof(T) == 2) {
            store_packed<T, N>(to, v);
        } else {
#pragma unroll
            for (int q = 0; q < N / 4; ++q) {
                f32x4 w;
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = v[4 * q + e];
                reinterpret_cast<f32x4_anywhere *>(to)[q] = w;
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (e < left) to[e] = (T)v[e];
    }
}

// The four lanes that share a row (16 apart) exchange their four times four
// columns, so that what they store at once lies side by side: lane q's v[j]
// becomes lane j's v[q].
__device__ __forceinline__ void turn(f32x4 (&v)[4])
{
    auto word = [](float f) { return __builtin_bit_cast(uint32_t, f); };
    auto value = [](uint32_t w) { return __builtin_bit_cast(float, w); };
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {  // lanes 2, 3 of one and 0, 1 of the other
            const auto r = __builtin_amdgcn_permlane32_swap(word(v[j][e]), word(v[j + 2][e]), false, false);
            v[j][e] = value(r[0]);
            v[j + 2][e] = value(r[1]);
        }
#pragma unroll
        for (int j = 0; j < 4; j += 2) {  // lanes 1, 3 of one and 0, 2 of the other
            const auto r = __builtin_amdgcn_permlane16_swap(word(v[j][e]), word(v[j + 1][e]), false, false);
            v[j][e] = value(r[0]);
            v[j + 1][e] = value(r[1]);
        }
    }
}

}  // namespace m16
}  // namespace tgemm
