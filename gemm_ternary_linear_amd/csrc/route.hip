// Routing tokens to experts on gfx950: scores, top-k, weights, and the token
// slots sorted by expert.
//
// A wave takes a token; lane l holds experts l, l + 64, ...  Scores, group
// worths and weights are 64-bit: among the thousands of choices of a batch some
// are between experts whose scores agree to 1e-7, which 32 bits would decide by
// their rounding; E exponentials a token in 64 bits cost little beside the
// latency of the choice itself.  top_k rounds of a wave-wide maximum (the larger score, then
// the lower index) pick the experts in order.
//
// Sorting needs no atomics whose order matters: a token takes an expert at
// most once, so the tokens of a chunk that take expert e are a bit mask, a
// slot's place among the chunk's is a population count of the lower bits, and
// the chunks' counts add up to the rest.  Up to kFusedTokens tokens one
// workgroup routes and sorts (one launch); more are routed by a workgroup per
// 16 tokens, whose masks go to the workspace, and placed by a second kernel, a
// workgroup per 64 tokens, each adding up the masks of all chunks itself
// (2 bytes per chunk and expert, from L2).  Beyond kFlatTokens that sum would
// grow with the square of the batch, so a kernel in between adds it up per
// 1024 tokens.
#include <cfloat>

#include "fp8_common.h"
#include "internal.h"

namespace ternary {

namespace {

constexpr int kWaves = 16, kThreads = kWaves * 64;
constexpr int kFusedTokens = 64;    // tokens one workgroup routes and sorts
constexpr int kChunk = 16;          // tokens of a mask
constexpr int kPlaceTokens = 64;    // tokens a workgroup places
constexpr int kSuper = 1024;        // tokens of a row of sums
constexpr int kFlatTokens = 8192;   // most tokens without the rows of sums
constexpr int kMaxE = TERNARY_MAX_EXPERTS, kMaxK = TERNARY_MAX_TOP_K;

__device__ __forceinline__ double shfl_xor_d(double v, int o) { return __shfl_xor(v, o); }

// The choices of one token (a wave): lane j < k gets its j-th expert and weight.
// `group_lds`: E doubles of this wave's (used where groups > 1).
template <int DT, int EP>
__device__ __forceinline__ void choose(const RouteArgs &a, int t, double *group_lds, int &my_id,
                                       float &my_w)
{
    const int lane = threadIdx.x & 63, E = a.E;
    double p[EP], c[EP];
    double mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < EP; ++i) {
        const int e = i * 64 + lane;
        float l = -INFINITY, b = 0.f;
        if (e < E) {
            l = load_elem<DT>(a.logits, (int64_t)t * E + e);
            if (a.bias)
                b = a.bias[e];
        }
        const bool open = l > -INFINITY && b > -INFINITY;  // NaN: false
        p[i] = open ? (double)fminf(l, FLT_MAX) : -INFINITY;
        c[i] = b;
        mx = fmax(mx, p[i]);
    }
    if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < EP; ++i) {
            const bool open = p[i] > -INFINITY;
            p[i] = open ? 1.0 / (1.0 + exp(-p[i])) : 0.0;
            c[i] = open ? p[i] + c[i] : -INFINITY;
        }
    } else {
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1)
            mx = fmax(mx, shfl_xor_d(mx, o));
        double z = 0.0;
        bool open[EP];
#pragma unroll
        for (int i = 0; i < EP; ++i) {
            open[i] = p[i] > -INFINITY;
            p[i] = open[i] ? exp(p[i] - mx) : 0.0;
            z += p[i];
        }
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1)
            z += shfl_xor_d(z, o);
#pragma unroll
        for (int i = 0; i < EP; ++i) {
            p[i] = open[i] ? p[i] / z : 0.0;
            c[i] = open[i] ? p[i] + c[i] : -INFINITY;
        }
    }

    if (a.groups > 1) {
        // lane g < groups: its group's two largest, then the group's rank among all
        const int per = E / a.groups;
#pragma unroll
        for (int i = 0; i < EP; ++i)
            if (i * 64 + lane < E)
                group_lds[i * 64 + lane] = c[i];
        __builtin_amdgcn_wave_barrier();
        double b1 = -INFINITY, b2 = -INFINITY;
        if (lane < a.groups)
            for (int i = 0; i < per; ++i) {
                const double v = group_lds[lane * per + i];
                b2 = fmax(b2, fmin(b1, v));
                b1 = fmax(b1, v);
            }
        const double worth = b2 > -INFINITY ? b1 + b2 : b1;
        int rank = 0;
        for (int g = 0; g < a.groups; ++g) {
            const double w = __shfl(worth, g);
            rank += w > worth || (w == worth && g < lane) ? 1 : 0;
        }
        const uint64_t kept = __builtin_amdgcn_ballot_w64(lane < a.groups && rank < a.top_groups);
#pragma unroll
        for (int i = 0; i < EP; ++i)
            if (!(kept >> ((i * 64 + lane) / per) & 1))
                c[i] = -INFINITY;
        __builtin_amdgcn_wave_barrier();
    }

    my_id = -1;
    double mine = 0.0, sum = 0.0;
    for (int j = 0; j < a.k; ++j) {
        double best = c[0];
        int id = lane;
#pragma unroll
        for (int i = 1; i < EP; ++i)
            if (c[i] > best)
                best = c[i], id = i * 64 + lane;
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) {
            const double ob = shfl_xor_d(best, o);
            const int oid = __shfl_xor(id, o);
            if (ob > best || (ob == best && oid < id))
                best = ob, id = oid;
        }
        if (best == -INFINITY)
            break;  // the same in every lane
        double w = 0.0;
#pragma unroll
        for (int i = 0; i < EP; ++i)
            if (i * 64 + lane == id)
                w = p[i], c[i] = -INFINITY;
        w = __shfl(w, id & 63);
        sum += w;
        if (lane == j)
            my_id = id, mine = w;
    }
    if (a.renormalize && sum > 0.0)
        mine /= sum;
    my_w = (float)(mine * (double)a.scale);
}

// Exclusive sums of n <= kMaxE counts in LDS (in place; the total to v[n]).
// Run by all threads of the workgroup.
__device__ __forceinline__ void scan_counts(int *v, int n)
{
    __syncthreads();
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x, per = (n + 63) / 64, lo = lane * per;
        int s = 0;
        for (int i = 0; i < per; ++i)
            s += lo + i < n ? v[lo + i] : 0;
        int incl = s;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int u = __shfl_up(incl, o);
            incl += lane >= o ? u : 0;
        }
        int run = incl - s;
        for (int i = 0; i < per; ++i)
            if (lo + i < n) {
                const int u = v[lo + i];
                v[lo + i] = run;
                run += u;
            }
        if (lane == 63)
            v[n] = incl;
    }
    __syncthreads();
}

// Few tokens: routes and sorts all of them in one workgroup.
template <int DT, int EP>
__global__ void __launch_bounds__(kThreads) route_few_kernel(const RouteArgs a)
{
    extern __shared__ __attribute__((aligned(16))) double group_lds[];
    __shared__ uint64_t mask[kMaxE];
    __shared__ int place[kMaxE + 1];
    __shared__ int16_t ids[kFusedTokens * kMaxK];
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, n = a.T * a.k;
    for (int e = tid; e < a.E; e += kThreads)
        mask[e] = 0;
    __syncthreads();
    for (int t = wave; t < a.T; t += kWaves) {
        int id;
        float w;
        choose<DT, EP>(a, t, group_lds + wave * a.E, id, w);
        if (lane < a.k) {
            a.ids[t * a.k + lane] = id;
            a.weights[t * a.k + lane] = w;
            ids[t * a.k + lane] = (int16_t)id;
            if (id >= 0)
                atomicOr((unsigned long long *)&mask[id], 1ull << t);
        }
    }
    __syncthreads();
    for (int e = tid; e < a.E; e += kThreads)
        place[e] = __popcll(mask[e]);
    scan_counts(place, a.E);
    for (int e = tid; e <= a.E; e += kThreads)
        a.offsets[e] = place[e];
    for (int s = tid; s < n; s += kThreads) {
        const int id = ids[s], t = s / a.k;
        int r = -1;
        if (id >= 0) {
            r = place[id] + __popcll(mask[id] & ((1ull << t) - 1));
            a.order[r] = s;
        }
        a.slots[s] = r;
        if (s >= place[a.E])
            a.order[s] = -1;
    }
}

// Many tokens: a wave each, and the masks of every 16 tokens, [T/16][E].
template <int DT, int EP>
__global__ void __launch_bounds__(kThreads) route_many_kernel(const RouteArgs a)
{
    extern __shared__ __attribute__((aligned(16))) double group_lds[];
    __shared__ uint32_t mask[kMaxE];
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int64_t t = (int64_t)blockIdx.x * kChunk + wave;
    for (int e = tid; e < a.E; e += kThreads)
        mask[e] = 0;
    __syncthreads();
    if (t < a.T) {
        int id;
        float w;
        choose<DT, EP>(a, (int)t, group_lds + wave * a.E, id, w);
        if (lane < a.k) {
            a.ids[t * a.k + lane] = id;
            a.weights[t * a.k + lane] = w;
            if (id >= 0)
                atomicOr(&mask[id], 1u << wave);
        }
    }
    __syncthreads();
    uint16_t *out = static_cast<uint16_t *>(a.workspace) + (int64_t)blockIdx.x * a.E;
    for (int e = tid; e < a.E; e += kThreads)
        out[e] = (uint16_t)mask[e];
}

__host__ __device__ inline int64_t chunks_of(int64_t T) { return (T + kChunk - 1) / kChunk; }
// The rows of sums follow the masks, from 16 bytes on.
__host__ __device__ inline int64_t mask_bytes(int64_t T, int64_t E)
{
    return (chunks_of(T) * E * 2 + 15) & ~(int64_t)15;
}

// Counts of every kSuper tokens, [T/1024][E].
__global__ void __launch_bounds__(256) route_sums_kernel(const RouteArgs a)
{
    const uint16_t *masks = static_cast<const uint16_t *>(a.workspace);
    int *sums = reinterpret_cast<int *>(static_cast<char *>(a.workspace) + mask_bytes(a.T, a.E));
    constexpr int PER = kSuper / kChunk;
    const int64_t chunks = chunks_of(a.T), first = (int64_t)blockIdx.x * PER;
    for (int e = threadIdx.x; e < a.E; e += 256) {
        int s = 0;
        for (int64_t c = first; c < first + PER && c < chunks; ++c)
            s += __popc(masks[c * a.E + e]);
        sums[(int64_t)blockIdx.x * a.E + e] = s;
    }
}

// Places the slots of 64 tokens.
__global__ void __launch_bounds__(kThreads) route_place_kernel(const RouteArgs a, bool flat)
{
    constexpr int PER = kPlaceTokens / kChunk;
    __shared__ int total[kMaxE + 1], before[kMaxE];
    __shared__ uint64_t mask[kMaxE];
    const uint16_t *masks = static_cast<const uint16_t *>(a.workspace);
    const int *sums =
        reinterpret_cast<const int *>(static_cast<const char *>(a.workspace) + mask_bytes(a.T, a.E));
    const int tid = threadIdx.x, E = a.E;
    const int64_t chunks = chunks_of(a.T), first = (int64_t)blockIdx.x * PER;
    for (int e = tid; e < E; e += kThreads)
        total[e] = before[e] = 0;
    __syncthreads();
    // threads: `parts` rows at a time, one expert each
    const int width = (E + 63) & ~63, parts = kThreads / width, e = tid % width, part = tid / width;
    if (part < parts && e < E) {
        int all = 0, low = 0;
        if (flat) {
            for (int64_t c = part; c < chunks; c += parts) {
                const int n = __popc(masks[c * E + e]);
                all += n;
                low += c < first ? n : 0;
            }
        } else {
            const int64_t supers = (a.T + kSuper - 1) / kSuper, own = first / (kSuper / kChunk);
            for (int64_t s = part; s < supers; s += parts) {
                const int n = sums[s * E + e];
                all += n;
                low += s < own ? n : 0;
            }
            for (int64_t c = own * (kSuper / kChunk) + part; c < first; c += parts)
                low += __popc(masks[c * E + e]);
        }
        atomicAdd(&total[e], all);
        atomicAdd(&before[e], low);
        if (part == 0) {
            uint64_t m = 0;
            for (int i = 0; i < PER; ++i)
                if (first + i < chunks)
                    m |= (uint64_t)masks[(first + i) * E + e] << (kChunk * i);
            mask[e] = m;
        }
    }
    scan_counts(total, E);
    if (blockIdx.x == 0)
        for (int i = tid; i <= E; i += kThreads)
            a.offsets[i] = total[i];
    const int64_t s0 = (int64_t)blockIdx.x * kPlaceTokens * a.k, n = (int64_t)a.T * a.k;
    for (int i = tid; i < kPlaceTokens * a.k && s0 + i < n; i += kThreads) {
        const int64_t s = s0 + i;
        const int id = a.ids[s], t = i / a.k;
        int r = -1;
        if (id >= 0) {
            r = total[id] + before[id] + __popcll(mask[id] & ((1ull << t) - 1));
            a.order[r] = (int)s;
        }
        a.slots[s] = r;
        if (s >= total[E])
            a.order[s] = -1;
    }
}

}  // namespace

int64_t route_workspace(int64_t T, int64_t E)
{
    if (T <= kFusedTokens)
        return 0;
    return mask_bytes(T, E) + (T <= kFlatTokens ? 0 : (T + kSuper - 1) / kSuper * E * 4);
}

hipError_t launch_route(const RouteArgs &a, int dtype, hipStream_t stream)
{
    const size_t lds = a.groups > 1 ? (size_t)kWaves * a.E * sizeof(double) : 0;
    const int ep = (a.E + 63) / 64;
    with_dtype(dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        auto run = [&](auto few, auto many) {
            if (a.T <= kFusedTokens)
                hipLaunchKernelGGL(few, dim3(1), dim3(kThreads), lds, stream, a);
            else
                hipLaunchKernelGGL(many, dim3((unsigned)chunks_of(a.T)), dim3(kThreads), lds, stream, a);
        };
        if (ep <= 1)
            run(route_few_kernel<DT, 1>, route_many_kernel<DT, 1>);
        else if (ep <= 2)
            run(route_few_kernel<DT, 2>, route_many_kernel<DT, 2>);
        else if (ep <= 4)
            run(route_few_kernel<DT, 4>, route_many_kernel<DT, 4>);
        else
            run(route_few_kernel<DT, 8>, route_many_kernel<DT, 8>);
    });
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.T <= kFusedTokens)
        return e;
    const bool flat = a.T <= kFlatTokens;
    if (!flat) {
        hipLaunchKernelGGL(route_sums_kernel, dim3((unsigned)((a.T + kSuper - 1) / kSuper)), dim3(256), 0,
                           stream, a);
        e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    hipLaunchKernelGGL(route_place_kernel, dim3((unsigned)((a.T + kPlaceTokens - 1) / kPlaceTokens)),
                       dim3(kThreads), 0, stream, a, flat);
    return hipGetLastError();
}

}  // namespace ternary
