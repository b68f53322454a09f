// The weighted sum of each token's expert rows:
//     out[t, n] = add[t, n] + sum_j weights[t, j] * y[slots[t, j], n]
// in fp32, j ascending, rounded once.  HBM-bound: every expert row is read
// once and every output written once.  A lane takes 8 columns of a token (one
// 16-byte load a row for 16-bit types).
//
// Measured (kernel trace, bf16): 2047 x 4096 of 8 rows a token 29.0 us for 151 MB (5.2
// TB/s, part of it from cache between repeats); 1 x 4096 4.2 us, an empty launch 1.9.
#include "fp8_common.h"
#include "internal.h"

namespace ternary {

namespace {

constexpr int kThreads = 256;

// VEC: rows in whole aligned pieces of 8 elements; else one element a lane.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads) combine_kernel(const CombineArgs a)
{
    constexpr int W = VEC ? 8 : 1;
    const int64_t per = a.N / W, units = (int64_t)a.T * per, stride = (int64_t)gridDim.x * kThreads;
    for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < units; u += stride) {
        const int64_t t = u / per, n = (u - t * per) * W;
        float acc[W];
#pragma unroll
        for (int i = 0; i < W; ++i)
            acc[i] = 0.f;
        if (a.add) {
            if constexpr (VEC)
                load8<DT>(a.add, t * a.N + n, acc);
            else
                acc[0] = load_elem<DT>(a.add, t * a.N + n);
        }
        for (int j = 0; j < a.k; ++j) {
            const int r = a.slots[t * a.k + j];
            if (r < 0 || r >= a.R)
                continue;
            const float w = a.weights[t * a.k + j];
            float v[W];
            if constexpr (VEC)
                load8<DT>(a.y, (int64_t)r * a.N + n, v);
            else
                v[0] = load_elem<DT>(a.y, (int64_t)r * a.N + n);
#pragma unroll
            for (int i = 0; i < W; ++i)
                acc[i] += w * v[i];
        }
        if constexpr (VEC) {
            store4<DT>(a.out, t * a.N + n, f32x4_t{acc[0], acc[1], acc[2], acc[3]});
            store4<DT>(a.out, t * a.N + n + 4, f32x4_t{acc[4], acc[5], acc[6], acc[7]});
        } else {
            store_elem<DT>(a.out, t * a.N + n, acc[0]);
        }
    }
}

}  // namespace

hipError_t launch_combine(const CombineArgs &a, int dtype, hipStream_t stream)
{
    const bool vec = a.N % 8 == 0 && (((uintptr_t)a.y | (uintptr_t)a.out | (uintptr_t)a.add) & 15) == 0;
    const int64_t units = (int64_t)a.T * (vec ? a.N / 8 : a.N), wgs = (units + kThreads - 1) / kThreads;
    const dim3 grid((unsigned)(wgs < (1 << 20) ? wgs : (1 << 20)));
    with_dtype(dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        if (vec)
            hipLaunchKernelGGL((combine_kernel<DT, true>), grid, dim3(kThreads), 0, stream, a);
        else
            hipLaunchKernelGGL((combine_kernel<DT, false>), grid, dim3(kThreads), 0, stream, a);
    });
    return hipGetLastError();
}

}  // namespace ternary
