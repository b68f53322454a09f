// e4m3 codes and block scales of a matrix, on gfx950.
//
// Per block of 128 values (of one row, or of 128 rows): s = max|v| / 448 in
// fp32, q = v / s rounded to fp32, then to the nearest e4m3 (the hardware
// conversion, ties to even).  The codes are rounded against the stored s, as
// ternary_quantize rounds against its stored scale; the quotient is the rounded
// one, because a product with a rounded 1/s would move values off the ties that a
// 16-bit v often hits exactly.  v is x, or for SwiGLU
// silu(gate) * up in fp32.
//
// HBM-bound: e bytes read (2 e for SwiGLU) and one written per value.  A row
// block is 16 lanes of 8 values (one 16-byte load each for 16-bit types), its
// maximum a butterfly over those lanes, so a wave does four blocks at a time
// with no LDS; a weight tile is a workgroup, eight rows a lane.
//
// Measured (calls in a graph, bf16): 16384 x 1024 SwiGLU 16.9 us for 84 MB (5.0 TB/s, part of it
// from cache between repeats; a copy of 2 GiB 4.9); 18944 x 4096 in tiles 41.6 us for 233 MB (likewise); 1 x 4096 2.2 us, an
// empty launch 1.9.
#include "fp8_common.h"
#include "internal.h"

namespace ternary {

namespace {

constexpr int kThreads = 256;

// Codes of 8 values against scale s (s == 0: zeros), as two words.
__device__ __forceinline__ u32x2_v codes8(const float v[8], float s)
{
    float r[8];
    // The rounded quotient: by one reciprocal (corrected once) and, for each value, a
    // product whose exact remainder corrects it.  Three operations a value where a division takes
    // ten; remainders stay exact while s is neither tiny nor huge.  (The correction of a -0 is +0: the sign
    // is put back.)
    const bool mid = s > 0x1p-100f && s < 0x1p100f;
    if (__builtin_amdgcn_ballot_w64(!mid) == 0) {
        const float a = __builtin_amdgcn_rcpf(s), inv = fmaf(fmaf(-s, a, 1.f), a, a);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q = v[i] * inv;
            r[i] = copysignf(fmaf(fmaf(-s, q, v[i]), inv, q), v[i]);  // (at most 448)
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float d = s > 0.f ? v[i] / s : (v[i] != v[i] ? v[i] : 0.f);
            // a subnormal s can leave a quotient above 448: the largest code then
            // (NaN passes the comparisons and stays NaN)
            r[i] = d > kE4m3Max ? kE4m3Max : (d < -kE4m3Max ? -kE4m3Max : d);
        }
    }
    int a = __builtin_amdgcn_cvt_pk_fp8_f32(r[0], r[1], 0, false);
    a = __builtin_amdgcn_cvt_pk_fp8_f32(r[2], r[3], a, true);
    int b = __builtin_amdgcn_cvt_pk_fp8_f32(r[4], r[5], 0, false);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(r[6], r[7], b, true);
    return u32x2_v{(uint32_t)a, (uint32_t)b};
}

// silu(g) * u, silu within about three roundings: (g > 0 ? g : g E) / (1 + E) with E = exp(-|g|),
// which nothing overflows.  E is a power of two whose argument's rounding (up to |g| 2^-24 of the
// result) is put back, the quotient one by a corrected reciprocal.  FAR: for gates past 20
// (the rest get the same bits), where the divisor is 1; past 80 E is taken 2^64 times larger until u is in, as exp2
// gives nothing below 2^-126 and a subnormal silu would be rounded to few bits.
template <bool FAR>
__device__ __forceinline__ float swiglu(float g, float u)
{
#pragma clang fp contract(off)  // (t + 64 has to be t's rounded value, to which `rest` belongs, and 64)
    const float hi = 0x1.715476p+0f, lo = 0x1.4ae0cp-26f;  // log2(e), and what fp32 leaves of it
    const float a = FAR ? fminf(fabsf(g), 300.f) : fabsf(g);  // (E is 0 by then; a NaN stays in g)
    const float t = -a * hi, rest = fmaf(-a, lo, fmaf(-a, hi, -t));
    const bool small = FAR && a > 80.f;
    const float e = __builtin_amdgcn_exp2f(small ? t + 64.f : t);
    const float E = fmaf(e, rest * 0x1.62e43p-1f, e), n = g > 0.f ? g : g * E;
    const float d = 1.f + E, r = __builtin_amdgcn_rcpf(d), q = n * r;
    const float near = copysignf(fmaf(fmaf(-d, q, n), r, q), g);  // (the correction of a -0 is +0)
    if constexpr (!FAR)
        return near * u;
    const float v = (a > 20.f ? n : near) * u;
    return small && !(g > 0.f) ? v * 0x1p-64f : v;
}

// The same of eight, v the gates.
__device__ __forceinline__ void swiglu8(float v[8], const float u[8])
{
    bool near = true;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        near = near && fabsf(v[i]) <= 20.f;
    if (__builtin_amdgcn_ballot_w64(!near) == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = swiglu<false>(v[i], u[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = swiglu<true>(v[i], u[i]);
    }
}

// Values k .. k+7 of a row (columns from K on are zeros).  VEC: 16-byte loads
// (rows and K in whole aligned pieces of 8).
template <int DT, bool SWIGLU, bool VEC>
__device__ __forceinline__ void values8(const void *x, int64_t row, int K, int k, float v[8])
{
    float u[8];
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = 0.f;
        if (k >= K)
            return;
        load8<DT>(x, row + k, v);
        if constexpr (SWIGLU)
            load8<DT>(x, row + K + k, u);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = u[i] = 0.f;
            if (k + i < K) {
                v[i] = load_elem<DT>(x, row + k + i);
                if constexpr (SWIGLU)
                    u[i] = load_elem<DT>(x, row + K + k + i);
            }
        }
    }
    if constexpr (SWIGLU)
        swiglu8(v, u);
}

// The largest magnitude (NaN left out; 0 where nothing is left).
__device__ __forceinline__ float absmax8(const float v[8])
{
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = fmaxf(m, fabsf(v[i]));
    return m;
}

// One scale per 128 values of a row: lane group u of 16 lanes takes blocks
// u, u + (lane groups of the grid), ...
template <int DT, bool SWIGLU, bool VEC>
__global__ void __launch_bounds__(kThreads)
    rows_kernel(const void *__restrict__ x, int64_t M, int K, int64_t ldx, uint8_t *__restrict__ q,
                float *__restrict__ scale)
{
    const int kb = (K + kFp8Block - 1) / kFp8Block;
    const int64_t blocks = M * kb, stride = (int64_t)gridDim.x * (kThreads / 16);
    const int l = threadIdx.x & 15;
    for (int64_t u = (int64_t)blockIdx.x * (kThreads / 16) + (threadIdx.x >> 4); u < blocks;
         u += stride) {
        // (a 64-bit division would cost as much as the block's arithmetic)
        const int64_t row = blocks <= UINT32_MAX ? (int64_t)((uint32_t)u / (uint32_t)kb) : u / kb;
        const int k = (int)(u - row * kb) * kFp8Block + 8 * l;
        float v[8];
        values8<DT, SWIGLU, VEC>(x, row * ldx, K, k, v);
        float m = absmax8(v);
#pragma unroll
        for (int o = 1; o < 16; o <<= 1)
            m = fmaxf(m, __shfl_xor(m, o));
        const float s = m / kE4m3Max;
        *reinterpret_cast<u32x2_v *>(q + u * kFp8Block + 8 * l) = codes8(v, s);
        if (l == 0)
            scale[u] = s;
    }
}

// One scale per 128 x 128 tile: a workgroup holds the tile in registers,
// thread t columns 8 (t % 16) .. +7 of rows t / 16 + 16 i.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads)
    tiles_kernel(const void *__restrict__ x, int64_t M, int K, int64_t ldx, uint8_t *__restrict__ q,
                 float *__restrict__ scale)
{
    __shared__ float wmax[kThreads / 64];
    const int kb = (K + kFp8Block - 1) / kFp8Block;
    const int64_t tiles = (M + kFp8Block - 1) / kFp8Block * kb;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t tm = t / kb;
        const int tk = (int)(t - tm * kb);
        const int k = tk * kFp8Block + 8 * (threadIdx.x & 15);
        float v[8][8], m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t row = tm * kFp8Block + (threadIdx.x >> 4) + 16 * i;
            values8<DT, false, VEC>(x, row * ldx, row < M ? K : 0, k, v[i]);
            m = fmaxf(m, absmax8(v[i]));
        }
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1)
            m = fmaxf(m, __shfl_xor(m, o));
        if ((threadIdx.x & 63) == 0)
            wmax[threadIdx.x >> 6] = m;
        __syncthreads();
        m = fmaxf(fmaxf(wmax[0], wmax[1]), fmaxf(wmax[2], wmax[3]));
        __syncthreads();  // wmax is rewritten by the workgroup's next tile
        const float s = m / kE4m3Max;
        if (threadIdx.x == 0)
            scale[t] = s;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t row = tm * kFp8Block + (threadIdx.x >> 4) + 16 * i;
            if (row < M)
                *reinterpret_cast<u32x2_v *>(q + row * kb * kFp8Block + k) = codes8(v[i], s);
        }
    }
}

}  // namespace

hipError_t launch_fp8_quantize(const void *x, int dtype, int64_t M, int64_t K, int64_t ldx,
                               bool tile, bool swiglu, uint8_t *q, float *scale, hipStream_t stream)
{
    const int64_t e = dtype == TERNARY_FP32 ? 4 : 2;
    // 16-byte loads where every row, and the up half of a SwiGLU row, starts on 16 bytes
    const bool vec = ((uintptr_t)x & 15) == 0 && ldx * e % 16 == 0 && K % 8 == 0;
    const int64_t kb = fp8_blocks(K);
    const int64_t wgs = tile ? fp8_blocks(M) * kb : (M * kb + kThreads / 16 - 1) / (kThreads / 16);
    const dim3 grid((unsigned)(wgs < (1 << 20) ? wgs : (1 << 20))), block(kThreads);
    with_dtype(dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        auto run = [&](auto kernel) {
            hipLaunchKernelGGL(kernel, grid, block, 0, stream, x, M, (int)K, ldx, q, scale);
        };
        if (tile)
            vec ? run(tiles_kernel<DT, true>) : run(tiles_kernel<DT, false>);
        else if (swiglu)
            vec ? run(rows_kernel<DT, true, true>) : run(rows_kernel<DT, true, false>);
        else
            vec ? run(rows_kernel<DT, false, true>) : run(rows_kernel<DT, false, false>);
    });
    return hipGetLastError();
}

}  // namespace ternary
