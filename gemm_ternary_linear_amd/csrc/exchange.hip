// Rows sent to their places and back, with weights, and the gradients of that: with p =
// slots[t, j] the place of token t's j-th slot,
//     dispatch:           out[p] = w[t, j] x[t]
//     combine's gradient: dy[p] = w[t, j] g[t],  dw[t, j] = <y[p], g[t]>
//     dispatch's gradient: dx[t] = add[t] + sum_j w[t, j] g[p],  dw[t, j] = <x[t], g[p]>
// Products and sums in fp32, in an order that depends on the sizes alone, each output rounded once.  HBM-bound: every
// row is read once and every output written once, 16 bytes a lane.  Rows whose length or
// address is no multiple of 16 bytes go by the same pieces of eight elements, loaded at their own
// alignment (the memory unit takes any), and their last piece by elements.
//
// dispatch takes a piece of a token and stores it k times (x is read once; by places it would be read k times,
// from caches at best).  combine's gradient takes a wave a slot: no sums across waves, and
// as many waves as rows.  dispatch's gradient takes a workgroup a token, which holds its piece of x
// and of dx in registers while the k rows pass.
//
// Measured (calls in a graph, bf16, 8 slots a token; a copy's rate in brackets): dispatch 2047 x 4096 27.4 us (30.3), combine's gradient 55.4
// (57.3), dispatch's gradient 4096 x 2048 with weights and add 43.9 (37.2; one piece a thread 49).
#include "fp8_common.h"
#include "internal.h"
#include "places.h"
#include "rows.h"

namespace ternary {

namespace {

constexpr int kThreads = 256;
constexpr int64_t kMostWgs = 1 << 20;  // workgroups of a launch; they take what is left in turns

// The sum over a wave, in lane 63.
__device__ __forceinline__ float wave_add(float v)
{
    auto moved = [](float u, auto ctrl, auto rows) {
        return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, u), decltype(ctrl)::value,
                                                                     decltype(rows)::value, 0xf, false));
    };
    v += moved(v, std::integral_constant<int, 0x111>(), std::integral_constant<int, 0xf>());  // row_shr 1, 2, 4, 8
    v += moved(v, std::integral_constant<int, 0x112>(), std::integral_constant<int, 0xf>());
    v += moved(v, std::integral_constant<int, 0x114>(), std::integral_constant<int, 0xf>());
    v += moved(v, std::integral_constant<int, 0x118>(), std::integral_constant<int, 0xf>());
    v += moved(v, std::integral_constant<int, 0x142>(), std::integral_constant<int, 0xa>());  // row_bcast 15, 31
    v += moved(v, std::integral_constant<int, 0x143>(), std::integral_constant<int, 0xc>());
    return v;
}

template <int DT, bool WIDE, bool STREAM>
__global__ void __launch_bounds__(kThreads) dispatch_kernel(const ExchangeArgs a)
{
    const int64_t per = (a.N + 7) / 8, units = a.T * per, stride = (int64_t)gridDim.x * kThreads;
    for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < units; u += stride) {
        const int64_t t = u / per;
        const int n = (int)(u - t * per) * 8, left = a.N - n;
        const Raw<DT> x = load_piece<DT, WIDE>(a.x, t * a.N + n, left);
        float v[8];
        widen_piece(x, v);
        for (int j = blockIdx.y; j < a.k; j += gridDim.y) {
            const int p = a.slots[t * a.k + j];
            if (p < 0 || p >= a.R)
                continue;
            Raw<DT> y = x;
            if (a.weights) {
                const float w = a.weights[t * a.k + j];
                float s[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    s[i] = w * v[i];
                y = round_piece<DT>(s);
            }
            store_piece<DT, WIDE, STREAM>(a.out, (int64_t)p * a.N + n, left, y);
        }
    }
}

template <int DT, bool WIDE, bool STREAM>
__global__ void __launch_bounds__(kThreads) combine_back_kernel(const ExchangeArgs a)
{
    const int lane = threadIdx.x & 63;
    constexpr int W = kThreads / 64;
    const int64_t first = (int64_t)blockIdx.x * W + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (int64_t s = first; s < a.T * a.k; s += (int64_t)gridDim.x * W) {
        const int64_t t = s / a.k;
        const int p = a.slots[s];
        float sum = 0.f;
        if (p >= 0 && p < a.R) {
            const float w = a.weights[s];
            constexpr int B = DT == TERNARY_FP32 ? 2 : 4;  // pieces whose loads go out together
            for (int n0 = lane * 8; n0 < a.N; n0 += B * 512) {
                Raw<DT> g[B], y[B];
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    const int n = n0 + b * 512;
                    if (n < a.N) {
                        g[b] = load_piece<DT, WIDE>(a.grad, t * a.N + n, a.N - n);
                        y[b] = load_piece<DT, WIDE, STREAM>(a.x, (int64_t)p * a.N + n, a.N - n);
                    }
                }
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    const int n = n0 + b * 512;
                    if (n < a.N) {
                        float gv[8], yv[8];
                        widen_piece(g[b], gv);
                        widen_piece(y[b], yv);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            sum += gv[i] * yv[i];
                            gv[i] *= w;
                        }
                        store_piece<DT, WIDE, STREAM>(a.out, (int64_t)p * a.N + n, a.N - n, round_piece<DT>(gv));
                    }
                }
            }
        }
        sum = wave_add(sum);
        if (lane == 63)
            a.dweights[s] = sum;
    }
}

// WEIGHTED: rows times their weights, and the weights' gradient; else both left out.
template <int DT, bool WIDE, bool WEIGHTED>
__global__ void __launch_bounds__(kThreads) dispatch_back_kernel(const ExchangeArgs a)
{
    constexpr int C = 2, J = 4;  // pieces a thread holds at a time; rows whose loads go out together
    __shared__ float dots[kThreads / 64][TERNARY_MAX_TOP_K];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const int32_t *slots = a.slots + t * a.k;
        if (WEIGHTED && lane < a.k)
            dots[wave][lane] = 0.f;
        for (int base = 0; base < a.N; base += C * 8 * blockDim.x) {
            float acc[C][8], x[C][8];
            int n[C], left[C];
#pragma unroll
            for (int c = 0; c < C; ++c) {
                n[c] = base + (c * blockDim.x + threadIdx.x) * 8;
                left[c] = a.N - n[c];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    acc[c][i] = x[c][i] = 0.f;
                if (left[c] > 0) {
                    if (a.add)
                        widen_piece(load_piece<DT, WIDE>(a.add, t * a.N + n[c], left[c]), acc[c]);
                    if (WEIGHTED)
                        widen_piece(load_piece<DT, WIDE>(a.x, t * a.N + n[c], left[c]), x[c]);
                }
            }
            for (int j0 = 0; j0 < a.k; j0 += J) {
                Raw<DT> g[J][C] = {};
                float w[J];
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const int p = j0 + j < a.k ? slots[j0 + j] : -1;
                    const bool has = p >= 0 && p < a.R;
                    w[j] = WEIGHTED ? (has ? a.weights[t * a.k + j0 + j] : 0.f) : 1.f;
                    if (has)
#pragma unroll
                        for (int c = 0; c < C; ++c)
                            if (left[c] > 0)
                                g[j][c] = load_piece<DT, WIDE>(a.grad, (int64_t)p * a.N + n[c], left[c]);
                }
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    float dot = 0.f;
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        float v[8];
                        widen_piece(g[j][c], v);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            acc[c][i] += WEIGHTED ? w[j] * v[i] : v[i];
                            dot += WEIGHTED ? v[i] * x[c][i] : 0.f;
                        }
                    }
                    if (WEIGHTED && j0 + j < a.k) {
                        dot = wave_add(dot);
                        if (lane == 63)
                            dots[wave][j0 + j] += dot;
                    }
                }
            }
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (left[c] > 0)
                    store_piece<DT, WIDE>(a.out, t * a.N + n[c], left[c], round_piece<DT>(acc[c]));
        }
        if (WEIGHTED) {
            __syncthreads();
            if ((int)threadIdx.x < a.k) {
                const int p = slots[threadIdx.x];
                float sum = 0.f;
                for (int i = 0; i < waves; ++i)
                    sum += dots[i][threadIdx.x];
                a.dweights[t * a.k + threadIdx.x] = p >= 0 && p < a.R ? sum : 0.f;
            }
        }
        if (WEIGHTED)
            __syncthreads();  // (the sums are read before the next token's begin)
    }
}

bool wide_rows(const ExchangeArgs &a)
{
    return a.N % 8 == 0 && (((uintptr_t)a.x | (uintptr_t)a.grad | (uintptr_t)a.add | (uintptr_t)a.out) & 15) == 0;
}

// Runs f(dtype, wide rows, rows past the caches) as compile-time values.  16-bit rows of 64 MB or more go past the caches
// (us, past and not: dispatch 2047 x 4096 27.2 and 30.8, combine's gradient 56 and 61; of 34 MB 8.1 and 9.7, 15.5 and 13.3; fp32 dispatch of 65 MB
// 26.7 and 22.3).
template <class F>
void with_rows(const ExchangeArgs &a, int dtype, F f)
{
    const bool stream = dtype != TERNARY_FP32 && a.R * a.N >= (int64_t)32 << 20;
    with_dtype(dtype, [&](auto dt) {
        if (!wide_rows(a))
            f(dt, std::false_type(), std::false_type());
        else if (!stream)
            f(dt, std::true_type(), std::false_type());
        else
            f(dt, std::true_type(), std::true_type());
    });
}

}  // namespace

hipError_t launch_dispatch(const ExchangeArgs &a, int dtype, hipStream_t stream)
{
    const int64_t units = a.T * ((a.N + 7) / 8), wgs = (units + kThreads - 1) / kThreads;
    // few pieces: the stores of one are shared out over several threads (8 rows each: 4 x 4096 3.1 us, one thread 4.7; 33 x 4096 3.1 and 4.9)
    const int ways = wgs >= 512 ? 1 : (int)(512 / wgs < a.k ? 512 / wgs : a.k);
    const dim3 grid((unsigned)(wgs < kMostWgs ? wgs : kMostWgs), ways);
    with_rows(a, dtype, [&](auto dt, auto wide, auto past) {
        hipLaunchKernelGGL((dispatch_kernel<decltype(dt)::value, decltype(wide)::value, decltype(past)::value>), grid,
                           dim3(kThreads), 0, stream, a);
    });
    return hipGetLastError();
}

hipError_t launch_combine_back(const ExchangeArgs &a, int dtype, hipStream_t stream)
{
    const int64_t wgs = (a.T * a.k + kThreads / 64 - 1) / (kThreads / 64);
    const dim3 grid((unsigned)(wgs < kMostWgs ? wgs : kMostWgs));
    with_rows(a, dtype, [&](auto dt, auto wide, auto past) {
        hipLaunchKernelGGL((combine_back_kernel<decltype(dt)::value, decltype(wide)::value, decltype(past)::value>), grid,
                           dim3(kThreads), 0, stream, a);
    });
    return hipGetLastError();
}

hipError_t launch_dispatch_back(const ExchangeArgs &a, int dtype, hipStream_t stream)
{
    const dim3 grid((unsigned)(a.T < kMostWgs ? a.T : kMostWgs));
    const int threads = a.N <= 1024 ? 64 : a.N <= 2048 ? 128 : kThreads;  // two pieces a thread
    with_rows(a, dtype, [&](auto dt, auto wide, auto) {
        constexpr int DT = decltype(dt)::value;
        constexpr bool WIDE = decltype(wide)::value;
        if (a.weights)
            hipLaunchKernelGGL((dispatch_back_kernel<DT, WIDE, true>), grid, dim3(threads), 0, stream, a);
        else
            hipLaunchKernelGGL((dispatch_back_kernel<DT, WIDE, false>), grid, dim3(threads), 0, stream, a);
    });
    return hipGetLastError();
}

}  // namespace ternary
