// Routing tokens to experts on gfx950: scores, top-k, weights, and the token
// slots sorted by expert.
//
// A wave takes a token; a lane holds one to eight neighbouring experts.  Scores, group
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
// workgroup per 16 or 64 tokens, each adding up the masks of all chunks itself
// (2 bytes per chunk and expert, from L2, 16 bytes a load).  Beyond kFlatTokens that sum would
// grow with the square of the batch, so a kernel in between adds it up per
// 1024 tokens.
//
// Limits, us a call in a graph, experts x top_k behind the tokens.  One launch against two:
// 24 x 64 x 4 5.8 and 7.5, 24 x 256 x 8 12.9 and 12.5, 32 x 64 x 4 7.1 and 7.5, 32 x 256 x 8
// 17.0 and 12.7, 48 x 64 x 4 9.1 and 7.5, 64 x 64 x 4 11.1 and 7.5, 64 x 256 x 8 29.9 and 12.7;
// but called one after another from Python, where the second launch and its workspace weigh, 32 x
// 64 x 4 12.9 and (33 tokens) 16.8, 32 x 256 x 8 16.9 and 17.0.  So one launch up to 64 tokens
// of at most 64 experts, and up to 32 of more.  16 against 64 tokens placed a workgroup: 128 x 64 x 4 7.8 and 9.0,
// 4096 x 256 x 8 18.1 and 18.9, 8192 x 256 x 8 31.0 and 27.7, 100000 x 256 x 8 431 and 244.  Rows of
// sums against none: 8193 x 64 x 4 16.6 and 13.6, 8193 x 256 x 8 28.8 and 29.4, 12000 x 512 x 8
// 53.5 and 59.5, 32000 x 64 x 4 28.4 and 31.9, 100000 x 256 x 8 232 and 534.
//
// What 4096 x 256 x 8 by sigmoid with groups spends (kernel traces, parts left out in
// turn): 12.4 us to choose, of which 3.9 are seven of the eight rounds of maxima and 1.5 the
// 64-bit sigmoid; placing 64 tokens a workgroup took 8.4, of which 2.6 were adding up masks.
// Unrolling that sum further changed nothing.  The logits' bytes would take 1 us.
#include <cfloat>

#include "fp8_common.h"
#include "internal.h"

namespace ternary {

namespace {

constexpr int kWaves = 16, kThreads = kWaves * 64;
constexpr int kFusedTokens = 64;    // most tokens one workgroup routes and sorts
constexpr int kChunk = 16;          // tokens of a mask
constexpr int kWideTokens = 4096;   // most tokens placed 16 a workgroup; beyond, 64
constexpr int kSuper = 1024;        // tokens of a row of sums
constexpr int kFlatTokens = 8192;   // most tokens without the rows of sums
constexpr int kMaxE = TERNARY_MAX_EXPERTS, kMaxK = TERNARY_MAX_TOP_K;

// v of another lane by a data-parallel move (0 where there is none): CTRL
// 0x111, 0x112, 0x114, 0x118 one to eight lanes up a row of 16, 0x142 and 0x143 the last lane of a row
// and of two rows to those after it.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t moved(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double moved(double v)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint64_t m = (uint64_t)moved<CTRL, ROWS>((uint32_t)(b >> 32)) << 32 | moved<CTRL, ROWS>((uint32_t)b);
    return __builtin_bit_cast(double, m);
}

// f over a wave, in lane 63, where 0 changes nothing.
template <class T, class F>
__device__ __forceinline__ T wave_fold(T v, F f)
{
    v = f(v, moved<0x111, 0xf>(v));
    v = f(v, moved<0x112, 0xf>(v));
    v = f(v, moved<0x114, 0xf>(v));
    v = f(v, moved<0x118, 0xf>(v));
    v = f(v, moved<0x142, 0xa>(v));
    v = f(v, moved<0x143, 0xc>(v));
    return v;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
    v = wave_fold(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ double lane_value(double v, int lane)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(b >> 32), lane);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)b, lane);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_sum(double v)
{
    return lane_value(wave_fold(v, [](double a, double b) { return a + b; }), 63);
}
// Unsigned numbers in the order of the floating ones (never 0 for a number or -inf).
__device__ __forceinline__ uint32_t ordered(float v)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, v);
    return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t ordered(double v)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);  // (-0 is 0)
    return b >> 63 ? ~b : b | 0x8000000000000000ull;
}

// The choices of one token (a wave): lane j < k gets its j-th expert and weight.
// Lane l holds experts EP l .. EP l + EP - 1.  `group_lds`: E doubles of this wave's
// (used where groups > 1).
template <int DT, int EP>
__device__ __forceinline__ void choose(const RouteArgs &a, int t, double *group_lds, int &my_id,
                                       float &my_w)
{
    const int lane = threadIdx.x & 63, E = a.E, e0 = lane * EP;
    float l[EP], bias[EP];
#pragma unroll
    for (int i = 0; i < EP; ++i) {
        l[i] = -INFINITY, bias[i] = 0.f;
        if (e0 + i < E) {
            l[i] = load_elem<DT>(a.logits, (int64_t)t * E + e0 + i);
            if (a.bias)
                bias[i] = a.bias[e0 + i];
        }
    }
    bool open[EP];
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < EP; ++i) {
        open[i] = l[i] > -INFINITY && bias[i] > -INFINITY;  // NaN: false
        l[i] = open[i] ? fminf(l[i], FLT_MAX) : -INFINITY;
        mx = fmaxf(mx, l[i]);
    }
    double p[EP];  // probabilities (softmax: times z)
    double z = 1.0;
    if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < EP; ++i)
            p[i] = open[i] ? 1.0 / (1.0 + exp(-(double)l[i])) : 0.0;
    } else {
        const uint32_t m = wave_max(ordered(mx));
        mx = __builtin_bit_cast(float, m >> 31 ? m & 0x7fffffffu : ~m);
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < EP; ++i) {
            p[i] = open[i] ? exp((double)l[i] - (double)mx) : 0.0;
            sum += p[i];
        }
        z = wave_sum(sum);
#pragma unroll
        for (int i = 0; i < EP; ++i)
            p[i] = open[i] ? p[i] / z : 0.0;
    }
    double c[EP];
#pragma unroll
    for (int i = 0; i < EP; ++i)
        c[i] = open[i] ? p[i] + (double)bias[i] : -INFINITY;

    if (a.groups > 1) {
        // A group's worth, from its two largest.  Groups of whole lanes, a power of
        // two of them, meet by exchanges; others through LDS, a lane a group.
        const int per = E / a.groups, lanes = per / EP;
        double b1 = -INFINITY, b2 = -INFINITY;
        auto add = [&](double v) {
            b2 = fmax(b2, fmin(b1, v));
            b1 = fmax(b1, v);
        };
        const bool whole = per % EP == 0 && (lanes & (lanes - 1)) == 0;
        if (whole) {
#pragma unroll
            for (int i = 0; i < EP; ++i)
                add(c[i]);
            for (int o = 1; o < lanes; o <<= 1) {
                const double o1 = __shfl_xor(b1, o), o2 = __shfl_xor(b2, o);
                add(o1);
                b2 = fmax(b2, o2);  // o2 <= o1, which is in: it can only be second
            }
        } else {
#pragma unroll
            for (int i = 0; i < EP; ++i)
                if (e0 + i < E)
                    group_lds[e0 + i] = c[i];
            __builtin_amdgcn_wave_barrier();
            if (lane < a.groups)
                for (int i = 0; i < per; ++i)
                    add(group_lds[lane * per + i]);
        }
        const double worth = b2 > -INFINITY ? b1 + b2 : b1;
        const int mine = whole ? lane / lanes : lane;
        int rank = 0;
        for (int g = 0; g < a.groups; ++g) {
            const double w = lane_value(worth, whole ? g * lanes : g);
            rank += w > worth || (w == worth && g < mine) ? 1 : 0;
        }
        const uint64_t kept = __builtin_amdgcn_ballot_w64(mine < a.groups && rank < a.top_groups);
#pragma unroll
        for (int i = 0; i < EP; ++i) {
            const bool keep = whole ? rank < a.top_groups : (kept >> min((e0 + i) / per, 63) & 1) != 0;
            c[i] = keep ? c[i] : -INFINITY;
        }
    }

    // k rounds of the largest: by the high halves of the ordered scores, and only
    // where two lanes agree in those by the low halves and the index.
    uint64_t key[EP];
#pragma unroll
    for (int i = 0; i < EP; ++i)
        key[i] = c[i] > -INFINITY ? ordered(c[i]) : 0;
    my_id = -1;
    double mine = 0.0, sum = 0.0;
    for (int j = 0; j < a.k; ++j) {
        uint64_t best = key[0];
        int at = 0;
#pragma unroll
        for (int i = 1; i < EP; ++i)
            if (key[i] > best)
                best = key[i], at = i;
        const uint32_t hi = wave_max((uint32_t)(best >> 32));
        if (hi == 0)
            break;  // none left (the same in every lane)
        uint64_t with = __builtin_amdgcn_ballot_w64((uint32_t)(best >> 32) == hi);
        if (with & (with - 1)) {
            const uint32_t lo = (uint32_t)(best >> 32) == hi ? (uint32_t)best : 0;
            const uint32_t most = wave_max(lo);
            with = __builtin_amdgcn_ballot_w64((uint32_t)(best >> 32) == hi && (uint32_t)best == most);
        }
        const int from = __builtin_ctzll(with);  // the lowest lane holds the lowest index
        double w = 0.0;
#pragma unroll
        for (int i = 0; i < EP; ++i)
            if (at == i) {
                w = p[i];
                key[i] = lane == from ? 0 : key[i];
            }
        const int id = __builtin_amdgcn_readlane(e0 + at, from);
        w = lane_value(w, from);
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

// Most tokens of one launch.
inline int fused_tokens(int64_t E) { return E <= 64 ? kFusedTokens : kFusedTokens / 2; }

__host__ __device__ inline int64_t chunks_of(int64_t T) { return (T + kChunk - 1) / kChunk; }
// Masks lie in rows of whole 16 bytes; the rows of sums follow them.
__host__ __device__ inline int mask_row(int64_t E) { return (int)((E + 7) & ~(int64_t)7); }
__host__ __device__ inline int64_t mask_bytes(int64_t T, int64_t E) { return chunks_of(T) * mask_row(E) * 2; }

// Many tokens: a wave each, and the masks of every 16 tokens, [T/16][mask_row(E)].
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
    const int ld = mask_row(a.E);
    uint16_t *out = static_cast<uint16_t *>(a.workspace) + (int64_t)blockIdx.x * ld;
    for (int e = tid; e < ld; e += kThreads)
        out[e] = e < a.E ? (uint16_t)mask[e] : 0;
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
        // (no early end: the loads of 16 steps go out together)
#pragma unroll 16
        for (int i = 0; i < PER; ++i) {
            const int64_t c = first + i;
            const int n = __popc(masks[min(c, chunks - 1) * mask_row(a.E) + e]);
            s += c < chunks ? n : 0;
        }
        sums[(int64_t)blockIdx.x * a.E + e] = s;
    }
}

// Places the slots of TOKENS tokens.
template <int TOKENS>
__global__ void __launch_bounds__(kThreads) route_place_kernel(const RouteArgs a, bool flat)
{
    constexpr int PER = TOKENS / kChunk;
    __shared__ int total[kMaxE + 1], before[kMaxE];
    __shared__ uint64_t mask[kMaxE];
    const uint16_t *masks = static_cast<const uint16_t *>(a.workspace);
    const int *sums =
        reinterpret_cast<const int *>(static_cast<const char *>(a.workspace) + mask_bytes(a.T, a.E));
    const int tid = threadIdx.x, E = a.E;
    const int64_t chunks = chunks_of(a.T), first = (int64_t)blockIdx.x * PER;
    const int ld = mask_row(E);
    for (int e = tid; e < E; e += kThreads) {
        total[e] = before[e] = 0;
        uint64_t m = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (first + i < chunks)
                m |= (uint64_t)masks[(first + i) * ld + e] << (kChunk * i);
        mask[e] = m;
    }
    __syncthreads();
    // Masks are added up eight experts (16 bytes) a thread, as many rows at a time as
    // there are threads.
    const int width = ld / 8, rows = kThreads / width, row = tid / width, e8 = tid % width * 8;
    const int64_t own = first / (kSuper / kChunk);  // this workgroup's row of sums
    if (row < rows) {
        int all[8] = {}, low[8] = {};
        auto add = [&](int64_t c, bool to_all) {
            const u32x4_v m = *reinterpret_cast<const u32x4_v *>(masks + c * ld + e8);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int n = __popc(i & 1 ? m[i / 2] >> 16 : m[i / 2] & 0xffffu);
                all[i] += to_all ? n : 0;
                low[i] += c < first ? n : 0;
            }
        };
        if (flat) {
#pragma unroll 4
            for (int64_t c = row; c < chunks; c += rows)
                add(c, true);
        } else {
            for (int64_t c = own * (kSuper / kChunk) + row; c < first; c += rows)
                add(c, false);
            const int64_t supers = (a.T + kSuper - 1) / kSuper;
#pragma unroll 2
            for (int64_t s = row; s < supers; s += rows)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int n = e8 + i < E ? sums[s * E + e8 + i] : 0;
                    all[i] += n;
                    low[i] += s < own ? n : 0;
                }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (e8 + i < E) {
                if (all[i])
                    atomicAdd(&total[e8 + i], all[i]);
                if (low[i])
                    atomicAdd(&before[e8 + i], low[i]);
            }
    }
    scan_counts(total, E);
    if (blockIdx.x == 0)
        for (int i = tid; i <= E; i += kThreads)
            a.offsets[i] = total[i];
    const int64_t s0 = (int64_t)blockIdx.x * TOKENS * a.k, n = (int64_t)a.T * a.k;
    for (int i = tid; i < TOKENS * a.k && s0 + i < n; i += kThreads) {
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
    if (T <= fused_tokens(E))
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
            if (a.T <= fused_tokens(a.E))
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
    if (e != hipSuccess || a.T <= fused_tokens(a.E))
        return e;
    const bool flat = a.T <= kFlatTokens;
    if (!flat) {
        hipLaunchKernelGGL(route_sums_kernel, dim3((unsigned)((a.T + kSuper - 1) / kSuper)), dim3(256), 0,
                           stream, a);
        e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    auto place = [&](auto kernel, int tokens) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)((a.T + tokens - 1) / tokens)), dim3(kThreads), 0, stream, a,
                           flat);
    };
    if (a.T <= kWideTokens)
        place(route_place_kernel<16>, 16);
    else
        place(route_place_kernel<64>, 64);
    return hipGetLastError();
}

}  // namespace ternary
