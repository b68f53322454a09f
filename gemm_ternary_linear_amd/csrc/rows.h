// Pieces of eight elements of a row, of any alignment: device helpers.
#pragma once

#include "fp8_common.h"

namespace ternary {

typedef unsigned int u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef unsigned int u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

// Eight elements as they lie: 16 bytes, or 32 of fp32.
template <int DT>
struct Raw {
    u32x4_v d[DT == TERNARY_FP32 ? 2 : 1];
};

// The piece of eight elements at element i of p, `n` of which belong to the row (none if n <= 0); the others are 0.
// WIDE: pieces are 16-byte aligned and rows hold whole ones.  STREAM: what is read or written once of a large array, past
// the caches (wide pieces only).
template <int DT, bool WIDE, bool STREAM = false>
__device__ __forceinline__ Raw<DT> load_piece(const void *p, int64_t i, int n)
{
    Raw<DT> r;
    if (n >= 8) {
        if constexpr (DT == TERNARY_FP32) {
            const float *f = static_cast<const float *>(p) + i;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if constexpr (WIDE && STREAM)
                    r.d[h] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_v *>(f + 4 * h));
                else if constexpr (WIDE)
                    r.d[h] = *reinterpret_cast<const u32x4_v *>(f + 4 * h);
                else
                    r.d[h] = *reinterpret_cast<const u32x4_a4 *>(f + 4 * h);
        } else {
            const uint16_t *f = static_cast<const uint16_t *>(p) + i;
            if constexpr (WIDE && STREAM)
                r.d[0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_v *>(f));
            else if constexpr (WIDE)
                r.d[0] = *reinterpret_cast<const u32x4_v *>(f);
            else
                r.d[0] = *reinterpret_cast<const u32x4_a2 *>(f);
        }
    } else {
        r = Raw<DT>{};
        if constexpr (WIDE) {
        } else if constexpr (DT == TERNARY_FP32) {
#pragma unroll
            for (int k = 0; k < 7; ++k)
                if (k < n)
                    r.d[k / 4][k % 4] = static_cast<const uint32_t *>(p)[i + k];
        } else {
#pragma unroll
            for (int k = 0; k < 7; ++k)
                if (k < n)
                    r.d[0][k / 2] |= (uint32_t)static_cast<const uint16_t *>(p)[i + k] << (k % 2 * 16);
        }
    }
    return r;
}

template <int DT, bool WIDE, bool STREAM = false>
__device__ __forceinline__ void store_piece(void *p, int64_t i, int n, const Raw<DT> &r)
{
    if (n >= 8) {
        if constexpr (DT == TERNARY_FP32) {
            float *f = static_cast<float *>(p) + i;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if constexpr (WIDE && STREAM)
                    __builtin_nontemporal_store(r.d[h], reinterpret_cast<u32x4_v *>(f + 4 * h));
                else if constexpr (WIDE)
                    *reinterpret_cast<u32x4_v *>(f + 4 * h) = r.d[h];
                else
                    *reinterpret_cast<u32x4_a4 *>(f + 4 * h) = r.d[h];
        } else {
            uint16_t *f = static_cast<uint16_t *>(p) + i;
            if constexpr (WIDE && STREAM)
                __builtin_nontemporal_store(r.d[0], reinterpret_cast<u32x4_v *>(f));
            else if constexpr (WIDE)
                *reinterpret_cast<u32x4_v *>(f) = r.d[0];
            else
                *reinterpret_cast<u32x4_a2 *>(f) = r.d[0];
        }
    } else {
        if constexpr (WIDE) {
        } else if constexpr (DT == TERNARY_FP32) {
#pragma unroll
            for (int k = 0; k < 7; ++k)
                if (k < n)
                    static_cast<uint32_t *>(p)[i + k] = r.d[k / 4][k % 4];
        } else {
#pragma unroll
            for (int k = 0; k < 7; ++k)
                if (k < n)
                    static_cast<uint16_t *>(p)[i + k] = (uint16_t)(r.d[0][k / 2] >> (k % 2 * 16));
        }
    }
}

template <int DT>
__device__ __forceinline__ void widen_piece(const Raw<DT> &r, float v[8])
{
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if constexpr (DT == TERNARY_FP32)
            v[k] = __builtin_bit_cast(float, (uint32_t)r.d[k / 4][k % 4]);
        else if constexpr (DT == TERNARY_FP16)
            v[k] = f16_bits_to_f32((uint16_t)(r.d[0][k / 2] >> (k % 2 * 16)));
        else
            v[k] = __builtin_bit_cast(float, k % 2 ? r.d[0][k / 2] & 0xffff0000u : r.d[0][k / 2] << 16);
}

template <int DT>
__device__ __forceinline__ Raw<DT> round_piece(const float v[8])
{
    Raw<DT> r;
    if constexpr (DT == TERNARY_FP32) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            r.d[k / 4][k % 4] = __builtin_bit_cast(uint32_t, v[k]);
    } else {
        constexpr bool H = DT == TERNARY_FP16;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            r.d[0][k] = (uint32_t)round_out<H>(v[2 * k]) | (uint32_t)round_out<H>(v[2 * k + 1]) << 16;
    }
    return r;
}

}  // namespace ternary
