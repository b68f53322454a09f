// Slots sorted by given indices: a stable counting sort of ids [T * k], an expert (or adapter) a key.
//
// A wave takes 64 slots at a time.  Which of them share a key is found without exchanges: a ballot
// per bit of the key, and the lanes that agree in all of them.  A slot's place among its wave's
// is what the wave has counted of its key before, in LDS, and a population count of the agreeing
// lower lanes; the waves' counts, and the workgroups', are added up in order.  No atomic's
// order shows in a result.
//
// Up to kOneSlots slots one workgroup does all (one launch).  More: a workgroup counts a chunk of
// slots into the workspace; sums over the chunks before each are made by the placing
// workgroups themselves where the chunks are few, else by a kernel in between.
//
// Measured (us in a graph): 64 x 1 of 32 keys 3.4, 8192 x 8 of 256 8.4, 32768 x 8 12.8, 100000 x 4 of 64 13.1; latency of one or two launches.  Limits: 4096
// slots in one launch and in two, 64 keys 5.8 and 6.0, 256 keys 7.5 and 7.0; sums by the placing workgroups and by a
// kernel, 64 chunks of 256 keys 8.5 and 10.1, 94 of 64 7.3 and 9.3, 128 of 256 9.4 and 11.0; chunks of 1024 and of 4096 slots, 65536 slots 8.5
// and 13.3, 262144 12.8 and 14.3, 400000 13.3 and 13.1.
#include "fp8_common.h"
#include "internal.h"
#include "places.h"

namespace ternary {

namespace {

constexpr int kWaves = 16, kThreads = kWaves * 64;
constexpr int kMaxE = TERNARY_MAX_EXPERTS;
constexpr int kSteps = 4;                        // slots a lane, at most
constexpr int kOneSlots = kThreads * kSteps;     // most slots of one workgroup alone
constexpr int64_t kSmallSlots = (int64_t)1 << 18;  // most slots in chunks of 1024; beyond, of 4096
constexpr int kFlatChunks = 128;                 // most chunks whose counts every workgroup adds up itself

inline int chunk_slots(int64_t n) { return n <= kSmallSlots ? kThreads : kThreads * kSteps; }
// Counts lie in rows of whole 16 bytes.
__host__ __device__ inline int count_row(int E) { return (E + 3) & ~3; }
inline int64_t chunks_of(int64_t n) { return (n + chunk_slots(n) - 1) / chunk_slots(n); }

// The lanes of the wave whose key is this lane's (keys below 2^bits; `has` false: none).
__device__ __forceinline__ uint64_t same_key(int key, bool has, int bits)
{
    uint64_t same = __builtin_amdgcn_ballot_w64(has);
    for (int b = 0; b < bits; ++b) {
        const uint64_t set = __builtin_amdgcn_ballot_w64((key >> b & 1) != 0);
        same &= (key >> b & 1) ? set : ~set;
    }
    return same;
}

// Exclusive sums of n <= kMaxE counts in LDS, in place, the total to v[n].  All threads call it.
__device__ __forceinline__ void scan_counts(int *v, int n)
{
    __syncthreads();
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x, per = (n + 63) / 64, lo = lane * per;
        int s = 0;
        for (int i = 0; i < per; ++i)
            s += lo + i < n ? v[lo + i] : 0;
        const int incl = wave_scan(s);
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

// Counts of every chunk of slots, [chunks][count_row(E)].
__global__ void __launch_bounds__(kThreads) sort_count_kernel(const SortArgs a, int chunk)
{
    __shared__ int count[kMaxE];
    for (int e = threadIdx.x; e < a.E; e += kThreads)
        count[e] = 0;
    __syncthreads();
    const int64_t s0 = (int64_t)blockIdx.x * chunk;
    for (int i = threadIdx.x; i < chunk && s0 + i < a.n; i += kThreads) {
        const int id = a.ids[s0 + i];
        if ((unsigned)id < (unsigned)a.E)
            atomicAdd(&count[id], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < count_row(a.E); e += kThreads)
        a.counts[(int64_t)blockIdx.x * count_row(a.E) + e] = e < a.E ? count[e] : 0;
}

// The counts become sums over the chunks before; the totals go to a row after the last.  A
// workgroup takes 16 keys, 64 threads each.
__global__ void __launch_bounds__(kThreads) sort_scan_kernel(const SortArgs a, int64_t chunks)
{
    __shared__ int part[64][17];
    const int e = blockIdx.x * 16 + (threadIdx.x & 15), row = threadIdx.x >> 4, col = threadIdx.x & 15;
    const int64_t per = (chunks + 63) / 64, lo = min(row * per, chunks), hi = min(lo + per, chunks);
    int s = 0;
    if (e < a.E)
        for (int64_t c = lo; c < hi; ++c)
            s += a.counts[c * count_row(a.E) + e];
    part[row][col] = s;
    __syncthreads();
    if (e < a.E) {
        int run = 0;
        for (int i = 0; i < row; ++i)
            run += part[i][col];
        for (int64_t c = lo; c < hi; ++c) {
            const int u = a.counts[c * count_row(a.E) + e];
            a.counts[c * count_row(a.E) + e] = run;
            run += u;
        }
        if (row == 63)
            a.counts[chunks * count_row(a.E) + e] = run;
    }
}

// Places the slots of a chunk, STEPS a lane.  How: ONE, this is the only chunk; FLAT, the counts of all
// chunks are added up here; SUMMED, they hold sums.
enum class How { ONE, FLAT, SUMMED };

template <int STEPS, How HOW>
__global__ void __launch_bounds__(kThreads) sort_place_kernel(const SortArgs a, int64_t chunks, int bits)
{
    __shared__ int count[kWaves][kMaxE];
    __shared__ int first[kMaxE + 1], before[kMaxE];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, E = a.E, ld = count_row(E);
    const int64_t s0 = (int64_t)blockIdx.x * (kThreads * STEPS) + wave * (64 * STEPS) + lane;
    int id[STEPS], rank[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int64_t s = s0 + i * 64;
        id[i] = s < a.n ? a.ids[s] : -1;
        if ((unsigned)id[i] >= (unsigned)E)
            id[i] = -1;
    }
    for (int i = tid; i < kWaves * E; i += kThreads)
        count[i / E][i % E] = 0;
    if constexpr (HOW != How::ONE)
        for (int e = tid; e < E; e += kThreads) {
            first[e] = HOW == How::SUMMED ? a.counts[chunks * ld + e] : 0;
            before[e] = HOW == How::SUMMED ? a.counts[(int64_t)blockIdx.x * ld + e] : 0;
        }
    __syncthreads();
    if constexpr (HOW == How::FLAT) {
        // four keys a thread, as many rows of counts at a time as there are threads
        const int width = ld / 4, rows = kThreads / width, row = tid / width, e4 = tid % width * 4;
        if (row < rows) {
            int all[4] = {}, low[4] = {};
#pragma unroll 4
            for (int c = row; c < (int)chunks; c += rows) {
                const int4 v = *reinterpret_cast<const int4 *>(a.counts + c * ld + e4);
                const int n[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    all[i] += n[i];
                    low[i] += c < (int)blockIdx.x ? n[i] : 0;
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (all[i]) {
                    atomicAdd(&first[e4 + i], all[i]);
                    if (low[i])
                        atomicAdd(&before[e4 + i], low[i]);
                }
        }
    }
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const uint64_t same = same_key(id[i], id[i] >= 0, bits);
        const uint64_t low = same & ((1ull << lane) - 1);
        int old = 0;
        // the lowest lane of a key counts for all of them
        if (id[i] >= 0 && low == 0)
            old = atomicAdd(&count[wave][id[i]], __popcll(same));
        const int lead = id[i] >= 0 ? __builtin_ctzll(same) : lane;
        rank[i] = __shfl(old, lead) + __popcll(low);
    }
    __syncthreads();
    for (int e = tid; e < E; e += kThreads) {
        int run = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const int u = count[w][e];
            count[w][e] = run;
            run += u;
        }
        if constexpr (HOW == How::ONE)
            first[e] = run, before[e] = 0;
    }
    scan_counts(first, E);
    if (blockIdx.x == 0)
        for (int e = tid; e <= E; e += kThreads)
            a.offsets[e] = first[e];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int64_t s = s0 + i * 64;
        if (s >= a.n)
            continue;
        int p = -1;
        if (id[i] >= 0) {
            p = first[id[i]] + before[id[i]] + count[wave][id[i]] + rank[i];
            a.order[p] = (int)s;
        }
        a.slots[s] = p;
        if (s >= first[E])
            a.order[s] = -1;
        if (a.ones)
            a.ones[s] = 1.f;
    }
}

}  // namespace

int64_t sort_slots_workspace(int64_t n, int64_t E)
{
    return n <= kOneSlots ? 0 : (chunks_of(n) + 1) * count_row((int)E) * 4;
}

hipError_t launch_sort_slots(const SortArgs &a, hipStream_t stream)
{
    const int bits = a.E > 1 ? 32 - __builtin_clz((unsigned)(a.E - 1)) : 0;
    if (a.n <= kOneSlots) {
        if (a.n <= kThreads)
            hipLaunchKernelGGL((sort_place_kernel<1, How::ONE>), dim3(1), dim3(kThreads), 0, stream, a, (int64_t)1, bits);
        else
            hipLaunchKernelGGL((sort_place_kernel<kSteps, How::ONE>), dim3(1), dim3(kThreads), 0, stream, a, (int64_t)1, bits);
        return hipGetLastError();
    }
    const int64_t chunks = chunks_of(a.n);
    const dim3 grid((unsigned)chunks);
    const int chunk = chunk_slots(a.n);
    hipLaunchKernelGGL(sort_count_kernel, grid, dim3(kThreads), 0, stream, a, chunk);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    if (chunk == kThreads && chunks <= kFlatChunks) {
        hipLaunchKernelGGL((sort_place_kernel<1, How::FLAT>), grid, dim3(kThreads), 0, stream, a, chunks, bits);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(sort_scan_kernel, dim3((unsigned)((a.E + 15) / 16)), dim3(kThreads), 0, stream, a, chunks);
    e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    if (chunk == kThreads)
        hipLaunchKernelGGL((sort_place_kernel<1, How::SUMMED>), grid, dim3(kThreads), 0, stream, a, chunks, bits);
    else
        hipLaunchKernelGGL((sort_place_kernel<kSteps, How::SUMMED>), grid, dim3(kThreads), 0, stream, a, chunks, bits);
    return hipGetLastError();
}

}  // namespace ternary
