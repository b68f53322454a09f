// Device helpers of the 8-bit kernels.
#pragma once

#include "../../include/ternary.h"
#include <type_traits>

#include "common.h"

namespace ternary {

typedef unsigned int u32x4_v __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2_v __attribute__((ext_vector_type(2)));

constexpr float kE4m3Max = 448.f;

// The element at p of a ternary_dtype.
template <int DT>
__device__ __forceinline__ float load_elem(const void *p, int64_t i)
{
    if constexpr (DT == TERNARY_FP32)
        return static_cast<const float *>(p)[i];
    else if constexpr (DT == TERNARY_FP16)
        return f16_bits_to_f32(static_cast<const uint16_t *>(p)[i]);
    else
        return __builtin_bit_cast(float, (uint32_t)static_cast<const uint16_t *>(p)[i] << 16);
}

template <int DT>
__device__ __forceinline__ void store_elem(void *p, int64_t i, float v)
{
    if constexpr (DT == TERNARY_FP32)
        static_cast<float *>(p)[i] = v;
    else
        static_cast<uint16_t *>(p)[i] = round_out<DT == TERNARY_FP16>(v);
}

// Eight consecutive elements from a 16-byte aligned address.
template <int DT>
__device__ __forceinline__ void load8(const void *p, int64_t i, float v[8])
{
    if constexpr (DT == TERNARY_FP32) {
        const float4 a = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
        const float4 b = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i + 4);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const u32x4_v d = *reinterpret_cast<const u32x4_v *>(static_cast<const uint16_t *>(p) + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (DT == TERNARY_FP16) {
                v[2 * j] = f16_bits_to_f32((uint16_t)d[j]);
                v[2 * j + 1] = f16_bits_to_f32((uint16_t)(d[j] >> 16));
            } else {
                v[2 * j] = __builtin_bit_cast(float, d[j] << 16);
                v[2 * j + 1] = __builtin_bit_cast(float, d[j] & 0xffff0000u);
            }
        }
    }
}

// Four consecutive outputs, rounded, to an address aligned to four elements.
template <int DT>
__device__ __forceinline__ void store4(void *p, int64_t i, f32x4_t v)
{
    if constexpr (DT == TERNARY_FP32) {
        *reinterpret_cast<f32x4_t *>(static_cast<float *>(p) + i) = v;
    } else {
        constexpr bool H = DT == TERNARY_FP16;
        const u32x2_v d = {(uint32_t)round_out<H>(v[0]) | (uint32_t)round_out<H>(v[1]) << 16,
                           (uint32_t)round_out<H>(v[2]) | (uint32_t)round_out<H>(v[3]) << 16};
        *reinterpret_cast<u32x2_v *>(static_cast<uint16_t *>(p) + i) = d;
    }
}

// Runs f(integral_constant<dtype>) for a ternary_dtype.
template <class F>
inline auto with_dtype(int dtype, F f)
{
    if (dtype == TERNARY_BF16)
        return f(std::integral_constant<int, TERNARY_BF16>());
    if (dtype == TERNARY_FP16)
        return f(std::integral_constant<int, TERNARY_FP16>());
    return f(std::integral_constant<int, TERNARY_FP32>());
}

}  // namespace ternary
