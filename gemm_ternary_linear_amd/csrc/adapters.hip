// Low-rank adapters beside a shared projection, each token with its own, and their gradients.
// For a token t of adapter e (scale s, a [rank, K], b [N, rank]):
//     v = x a^T,  y = add + s v b^T
// and of a gradient g of y
//     dv = s g b,  db = s sum_t g^T v,  da = sum_t dv^T x,  dx = add + dv a.
//
// Tokens come sorted by adapter (offsets, order), so a tile of neighbouring places shares its
// weights.  Three kernels make up both directions:
//     down  a long row times the weights: v and dv.  Split along the row over workgroups where the tiles are few;
//           partial sums in fp32, added up in order by their readers.
//     up    v times the weights, added to a row: y and dx.
//     outer sums over an adapter's tokens: da and db.  Split into pieces of tokens; partial sums in fp32,
//           added up in order by a fourth kernel where an adapter has several.
// All products are on the matrix unit in 16 bits, their sums in fp32.  v and dv, which are fp32, enter it as
// two 16-bit numbers, cut and the nearest to what that left: 2^-16 off (bf16; fp16 2^-22), far below the
// outputs' own rounding, for twice the matrix cycles, of which there are plenty: the
// layer is bound by reading x and reading and writing y.  fp16 would lose what is small or large, so there
// v is first brought to below 2 by a power of two: a row's largest (up) or the piece's (outer).
//
// Operands that the matrix unit wants along the other axis than they lie in memory (b in down, a in up, both sides of
// outer) pass through LDS and are read transposed (ds_read_b64_tr_b16: of 16 lanes, lane l gives the
// address of four neighbours of row l / 4 at column 4 (l % 4), and receives column l of the four rows).
#include "fp8_common.h"
#include "internal.h"
#include "places.h"
#include "rows.h"

namespace ternary {

namespace {

constexpr int kWaves = 4, kThreads = kWaves * 64;
constexpr int kCols = 256;     // columns of an up workgroup at a time: 64 a wave
constexpr int kStep = 64;      // tokens of a step of outer
// An outer workgroup's threads, the fragments of 16 columns of a wave, and its columns (half of the waves each).
__host__ __device__ constexpr int outer_threads(int rf) { return rf > 4 ? 1024 : 512; }
__host__ __device__ constexpr int outer_frags(int rf) { return rf > 2 ? 2 : 4; }
__host__ __device__ constexpr int outer_cols(int rf) { return outer_threads(rf) / 128 * 16 * outer_frags(rf); }
inline int rank_frags(int64_t rank) { return rank <= 16 ? 1 : rank <= 32 ? 2 : rank <= 64 ? 4 : 8; }
constexpr int kMaxPiece = 1024;  // most tokens of a piece of outer

template <int DT>
__device__ __forceinline__ f32x4_t mfma(u32x4_v a, u32x4_v b, f32x4_t c)
{
    if constexpr (DT == TERNARY_FP16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

typedef short s16x4_v __attribute__((ext_vector_type(4)));

// Eight rows (from the lane group's first) of the column that the lane takes, transposed: `p` is the address of row
// l / 4, column 4 (l % 4) of the group's rows, `ld` elements between rows.
__device__ __forceinline__ u32x4_v read_transposed(const uint16_t *p, int ld)
{
#if defined(__HIP_DEVICE_COMPILE__)
    typedef __attribute__((address_space(3))) s16x4_v lds_s4;
    const s16x4_v lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)p);
    const s16x4_v hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)(p + 4 * ld));
    const u32x2_v l = __builtin_bit_cast(u32x2_v, lo), h = __builtin_bit_cast(u32x2_v, hi);
    return u32x4_v{l.x, l.y, h.x, h.y};
#else
    return u32x4_v{};
#endif
}

// Elements i .. i + 7 of a row of n that starts at p; 0 past its end.
template <bool WIDE>
__device__ __forceinline__ u32x4_v row_piece(const uint16_t *p, int i, int n)
{
    return load_piece<TERNARY_BF16, WIDE>(p, i, n - i).d[0];
}

// Two values as two 16-bit numbers each: cut, and the nearest to what that left.  (Of an infinity nothing is left, which the
// difference gives as NaN; the maximum makes that a finite number, which changes no sum with the infinity.)
template <int DT>
__device__ __forceinline__ void split(float a, float b, uint32_t &hi, uint32_t &lo)
{
    if constexpr (DT == TERNARY_FP16) {  // |a|, |b| < 2 or not finite
        hi = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(a, b));
        const float x = fmaxf(a - f16_bits_to_f32((uint16_t)hi), -1.f), y = fmaxf(b - f16_bits_to_f32((uint16_t)(hi >> 16)), -1.f);
        lo = (uint32_t)f32_to_f16_rne(x) | (uint32_t)f32_to_f16_rne(y) << 16;
    } else {
        const uint32_t u = __builtin_bit_cast(uint32_t, a), v = __builtin_bit_cast(uint32_t, b);
        const uint32_t m = u & 0xffff0000u, n = v & 0xffff0000u;
        hi = __builtin_amdgcn_perm(v, u, 0x07060302u);
        const float x = fmaxf(a - __builtin_bit_cast(float, m), -0x1p121f), y = fmaxf(b - __builtin_bit_cast(float, n), -0x1p121f);
        lo = (uint32_t)f32_to_bf16_rne(x) | (uint32_t)f32_to_bf16_rne(y) << 16;
    }
}

// fp32 rows [T, rank] held as `parts` (1, 2, 4 or 8) partial sums, `stride` elements apart.
struct Small {
    const float *p;
    int parts, rank;
    int64_t stride;
};
template <int PARTS>
__device__ __forceinline__ void load_parts(const Small &s, const float *p, int left, float v[8])
{
    // (all loads go out together, the sums are in order)
    if (s.rank % 4 == 0) {
        f32x4_t u[PARTS][2];
#pragma unroll
        for (int k = 0; k < PARTS; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                u[k][h] = 4 * h < left ? *reinterpret_cast<const f32x4_t *>(p + k * s.stride + 4 * h) : f32x4_t{};
#pragma unroll
        for (int k = 0; k < PARTS; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = k ? v[i] + u[k][i / 4][i % 4] : u[k][i / 4][i % 4];
    } else {
        float u[PARTS][8];
#pragma unroll
        for (int k = 0; k < PARTS; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                u[k][i] = i < left ? p[k * s.stride + i] : 0.f;
#pragma unroll
        for (int k = 0; k < PARTS; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = k ? v[i] + u[k][i] : u[k][i];
    }
}
__device__ __forceinline__ void load_small(const Small &s, int64_t t, int j0, float v[8])
{
    const float *p = s.p + t * s.rank + j0;
    if (s.parts == 1)
        load_parts<1>(s, p, s.rank - j0, v);
    else if (s.parts == 2)
        load_parts<2>(s, p, s.rank - j0, v);
    else if (s.parts == 4)
        load_parts<4>(s, p, s.rank - j0, v);
    else {
        float more[8];  // (in two batches, for fewer registers)
        load_parts<4>(s, p, s.rank - j0, v);
        load_parts<4>(s, p + 4 * s.stride, s.rank - j0, more);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] += more[i];
    }
}

// The largest finite |v[i]|, and the exponent that brings it to 1 .. 2 (0 where all are 0).
__device__ __forceinline__ float largest(const float v[8])
{
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = fmaxf(m, fabsf(v[i]));
    if (m == INFINITY) {
        m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            m = fmaxf(m, fabsf(v[i]) < INFINITY ? fabsf(v[i]) : 0.f);
    }
    return m;
}
__device__ __forceinline__ int exponent(float m) { return m > 0.f ? ilogbf(m) : 0; }

// Eight values, times 2^-ex, split, into a row of LDS: [hi: RP][lo: RP].
template <int DT, int RP>
__device__ __forceinline__ void put_split(uint16_t *row, int j0, const float v[8], int ex)
{
    u32x4_v h, l;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t hi, lo;
        if constexpr (DT == TERNARY_FP16)
            split<DT>(ldexpf(v[2 * i], -ex), ldexpf(v[2 * i + 1], -ex), hi, lo);
        else
            split<DT>(v[2 * i], v[2 * i + 1], hi, lo);
        h[i] = hi, l[i] = lo;
    }
    *reinterpret_cast<u32x4_v *>(row + j0) = h;
    *reinterpret_cast<u32x4_v *>(row + RP + j0) = l;
}

// The token at place p, or -1.
__device__ __forceinline__ int token_at(const int32_t *order, int p, int end, int T)
{
    const int t = p < end ? order[p] : -1;
    return t < T ? t : -1;
}

// ---------------------------------------------------------------- down

struct DownArgs {
    const uint16_t *x, *w;  // [T, L]; [E, rank, L], or (TR) [E, L, rank]
    const float *scale;
    const int32_t *offsets, *order;
    float *out;  // [splits][T, rank]
    int T, L, rank, E, splits;
};

// A workgroup takes 16 MF places and a share of the row; its waves take turns at 64 elements of it (whole
// cache lines), the next turn's loads under way meanwhile, and meet at the end.  Rows are loaded as they lie, eight
// neighbouring lanes a line, and pass through LDS into operands: loaded as operands, with neighbouring lanes
// in different rows, each lane would cost L1 an access.
//
// HBM-bound at small ranks; at larger ones the weights, read from L2 for every tile, weigh as much.  Measured (8191 tokens of 4096,
// in a graph; a copy's rate 13.5 us): rank 16 13.9, 32 15.0, 64 20.1 (in operands' layout 30.3), 128 41.
template <int DT, int RF, int MF, int WAVES, bool TR, bool WIDE>
__global__ void __launch_bounds__(WAVES * 64) down_kernel(const DownArgs a)
{
    constexpr int RP = RF * 16, PER = RP / 8, LD = TR ? RP + 8 : 64 + 8;
    constexpr int WG = TR ? 32 : RP < 32 ? RP : 32;  // rows of weights that pass through LDS at a time
    constexpr int STAGE = (WG * LD > 16 * MF * 72 ? WG * LD : 16 * MF * 72) * 2, SUMS = MF * 64 * 16;
    __shared__ __attribute__((aligned(16))) unsigned char lds[WAVES * (STAGE > SUMS ? STAGE : SUMS)];
    const int lane = threadIdx.x & 63, g = lane >> 4, col = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tile = blockIdx.x / a.splits, part = blockIdx.x - tile * a.splits;
    int e, r0, r1;
    if (!find_tile<16 * MF>(a.offsets, a.E, a.T, tile, e, r0, r1))
        return;
    int tok[2 * MF];
#pragma unroll
    for (int m = 0; m < 2 * MF; ++m)
        tok[m] = token_at(a.order, r0 + m * 8 + lane / 8, r1, a.T);
    f32x4_t acc[RF][MF] = {};
    const int steps = (a.L + 63) / 64;
    const int lo = (int)((int64_t)steps * part / a.splits), hi = (int)((int64_t)steps * (part + 1) / a.splits);
    const uint16_t *w = a.w + (int64_t)e * a.rank * a.L;
    uint16_t *stage = reinterpret_cast<uint16_t *>(lds) + wave * (STAGE / 2);
    u32x4_v nx[2 * MF], nw[2 * RF];
    auto fetch = [&](int i) {
        const int k0 = i * 64, k = k0 + lane % 8 * 8;
#pragma unroll
        for (int m = 0; m < 2 * MF; ++m)
            nx[m] = tok[m] >= 0 ? row_piece<WIDE>(a.x + (int64_t)tok[m] * a.L, k, a.L) : u32x4_v{};
#pragma unroll
        for (int q = 0; q < 2 * RF; ++q) {
            if constexpr (TR) {
                const int row = (lane + q * 64) / PER, j = (lane + q * 64) % PER * 8;
                nw[q] = k0 + row < a.L ? row_piece<WIDE>(w + (int64_t)(k0 + row) * a.rank, j, a.rank) : u32x4_v{};
            } else {
                const int j = q * 8 + lane / 8;
                nw[q] = j < a.rank ? row_piece<WIDE>(w + (int64_t)j * a.L, k, a.L) : u32x4_v{};
            }
        }
    };
    auto order = []() { asm volatile("" ::: "memory"); };  // (a wave's LDS accesses are in order)
    if (lo + wave < hi)
        fetch(lo + wave);
    for (int i = lo + wave; i < hi; i += WAVES) {
        u32x4_v xf[2][MF], wf[2][RF];
#pragma unroll
        for (int m = 0; m < 2 * MF; ++m)
            *reinterpret_cast<u32x4_v *>(stage + (m * 8 + lane / 8) * 72 + lane % 8 * 8) = nx[m];
        order();
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int m = 0; m < MF; ++m)
                xf[h][m] = *reinterpret_cast<const u32x4_v *>(stage + (m * 16 + col) * 72 + h * 32 + g * 8);
        order();
        // weights: 32 of the row (TR), or 32 of the rank, at a time
#pragma unroll
        for (int part = 0; part < (TR ? 2 : RP / WG); ++part) {
            constexpr int NQ = TR ? WG * PER / 64 : WG / 8;
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                const int p = TR ? (lane + q * 64) / PER * LD + (lane + q * 64) % PER * 8 : (q * 8 + lane / 8) * LD + lane % 8 * 8;
                *reinterpret_cast<u32x4_v *>(stage + p) = nw[part * NQ + q];
            }
            order();
            if constexpr (TR) {
#pragma unroll
                for (int f = 0; f < RF; ++f)
                    wf[part][f] = read_transposed(stage + (g * 8 + col / 4) * LD + f * 16 + col % 4 * 4, LD);
            } else {
#pragma unroll
                for (int f = 0; f < WG / 16; ++f)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        wf[h][part * (WG / 16) + f] = *reinterpret_cast<const u32x4_v *>(stage + (f * 16 + col) * LD + h * 32 + g * 8);
            }
            order();
        }
        if (i + WAVES < hi)
            fetch(i + WAVES);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int f = 0; f < RF; ++f)
#pragma unroll
                for (int m = 0; m < MF; ++m)
                    acc[f][m] = mfma<DT>(wf[h][f], xf[h][m], acc[f][m]);
    }
    // the waves' sums, 16 of the rank at a time
    f32x4_t *sums = reinterpret_cast<f32x4_t *>(lds);
    const float s = a.scale ? a.scale[e] : 1.f;
    float *out = a.out + (int64_t)part * a.T * a.rank;
#pragma unroll
    for (int f = 0; f < RF; ++f) {
        __syncthreads();
#pragma unroll
        for (int m = 0; m < MF; ++m)
            sums[(wave * MF + m) * 64 + lane] = acc[f][m];
        __syncthreads();
        for (int m = wave; m < MF; m += WAVES) {
            f32x4_t v = sums[m * 64 + lane];
#pragma unroll
            for (int u = 1; u < WAVES; ++u)
                v += sums[(u * MF + m) * 64 + lane];
            const int t = token_at(a.order, r0 + m * 16 + col, r1, a.T), j = f * 16 + g * 4;
            if (t >= 0) {
                if (a.rank % 4 == 0) {
                    if (j < a.rank)
                        *reinterpret_cast<f32x4_t *>(out + (int64_t)t * a.rank + j) = v * s;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (j + i < a.rank)
                            out[(int64_t)t * a.rank + j + i] = v[i] * s;
                }
            }
        }
    }
}

// ---------------------------------------------------------------- up

struct UpArgs {
    Small v;
    const uint16_t *w;  // [E, C, rank], or (TR) [E, rank, C]
    const float *scale;
    const int32_t *offsets, *order, *slots;
    const uint16_t *add;
    uint16_t *y;
    float *hidden;  // v's sums are written here, or NULL
    int T, C, rank, E;
    int chunks, per;  // runs of 256 columns; how many a workgroup takes
};

// A workgroup takes 16 MF places and runs of 256 columns, 64 a wave, whose weights stay in registers while the places
// pass.  Weights, what is added to and y go between memory and the wave as they lie, eight neighbouring lanes a line, and
// pass through LDS into operands and out of results, a wave by itself.
//
// HBM-bound.  Measured (8191 tokens, base and result, in a graph): 18944 columns 114 us at rank 16 (5.4 TB/s), 135 at rank 64, 179 at 128; 4096
// columns at rank 32 29.4 (4.6 TB/s).  In the operands' own layout, 64 L1 accesses an instruction, it took 164 at rank 64; without
// passing the caches 151.
template <int DT, int RF, int MF, bool TR, bool WIDE>
__global__ void __launch_bounds__(kThreads) up_kernel(const UpArgs a)
{
    constexpr int ROWS = MF * 16, RP = RF * 16, PER = RP / 8, LDV = 2 * RP + 8, LDO = 64 + 4;
    constexpr int QW = RP < 32 ? 1 : RP / 32, Q = 2 * RP / 32;  // operands of the weights, and of v
    // weights that pass through LDS at a time: rows of [rank, C] (TR), or columns
    constexpr int GR = TR ? (RP < 32 ? RP : 32) : (RP <= 32 ? 64 : 16), LDW = TR ? 64 + 8 : RP + 8;
    constexpr int STAGE = 16 * LDO * 4 > GR * LDW * 2 ? 16 * LDO * 4 : GR * LDW * 2;
    __shared__ __attribute__((aligned(16))) uint16_t sv[ROWS * LDV];
    __shared__ __attribute__((aligned(16))) unsigned char lds[kWaves * STAGE];
    __shared__ float factor[ROWS];
    __shared__ int toks[ROWS];
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, col = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int runs = (a.chunks + a.per - 1) / a.per;
    const int tile = blockIdx.x / runs, run = blockIdx.x - tile * runs;
    const int c0 = run * a.per, c1 = min(a.chunks, c0 + a.per);
    // tokens without an adapter, as many looked at by each tile as it has rows
    if (a.y != a.add && (int64_t)tile * ROWS < a.T)
        for (int row = tid / 32; row < ROWS; row += kThreads / 32) {
            const int64_t t = (int64_t)tile * ROWS + row;
            if (t >= a.T || (unsigned)a.slots[t] < (unsigned)a.T)
                continue;
            for (int n = c0 * kCols + tid % 32 * 8; n < min(c1 * kCols, a.C); n += kCols) {
                Raw<DT> v = {};
                if (a.add)
                    v = load_piece<DT, WIDE>(a.add, t * a.C + n, a.C - n);
                store_piece<DT, WIDE>(a.y, t * a.C + n, a.C - n, v);
            }
        }
    int e, r0, r1;
    if (!find_tile<ROWS>(a.offsets, a.E, a.T, tile, e, r0, r1))
        return;
    const float s = a.scale ? a.scale[e] : 1.f;
    // v, in 16-bit halves; RP / 8 threads a row
#pragma unroll
    for (int base = 0; base < ROWS * PER; base += kThreads) {
        const int i = base + tid, row = i / PER, j0 = i % PER * 8;
        if (ROWS * PER % kThreads != 0 && row >= ROWS)
            break;
        const int t = token_at(a.order, r0 + row, r1, a.T);
        float v[8] = {};
        if (t >= 0) {
            load_small(a.v, t, j0, v);
            if (a.hidden && run == 0)
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (j0 + k < a.rank)
                        a.hidden[(int64_t)t * a.rank + j0 + k] = v[k];
        }
        int ex = 0;
        if constexpr (DT == TERNARY_FP16) {
            float m = largest(v);
#pragma unroll
            for (int o = 1; o < PER; o <<= 1)
                m = fmaxf(m, __shfl_xor(m, o));
            ex = exponent(m);
        }
        put_split<DT, RP>(sv + row * LDV, j0, v, ex);
        if (j0 == 0)
            factor[row] = ldexpf(s, ex), toks[row] = t;
    }
    __syncthreads();
    const uint16_t *w = a.w + (int64_t)e * a.rank * a.C;
    uint16_t *sw = reinterpret_cast<uint16_t *>(lds + wave * STAGE);
    float *so = reinterpret_cast<float *>(lds + wave * STAGE);
    auto order = []() { asm volatile("" ::: "memory"); };  // (a wave's LDS accesses are in order)
    for (int c = c0; c < c1; ++c) {
        const int n0 = c * kCols + wave * 64, n = n0 + lane % 8 * 8;  // this wave's columns, this lane's
        constexpr int NW = TR ? RP / 8 : PER;
        u32x4_v raw[NW], wf[4][QW];
#pragma unroll
        for (int i = 0; i < NW; ++i)
            if constexpr (TR) {
                const int j = i * 8 + lane / 8;
                raw[i] = j < a.rank ? row_piece<WIDE>(w + (int64_t)j * a.C, n, a.C) : u32x4_v{};
            } else {
                const int r = (i * 64 + lane) / PER, j = (i * 64 + lane) % PER * 8;
                raw[i] = n0 + r < a.C ? row_piece<WIDE>(w + (int64_t)(n0 + r) * a.rank, j, a.rank) : u32x4_v{};
            }
        Raw<DT> base[MF][2];
#pragma unroll
        for (int m = 0; m < MF; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int t = toks[m * 16 + h * 8 + lane / 8];
                base[m][h] = Raw<DT>{};
                if (a.add && t >= 0)
                    base[m][h] = load_piece<DT, WIDE, (MF > 2)>(a.add, (int64_t)t * a.C + n, a.C - n);
            }
        // (rows of the matrix operand: f 16 + 0 .. 15)
#pragma unroll
        for (int p = 0; p < (TR ? RP : 64) / GR; ++p) {
            constexpr int NP = TR ? GR / 8 : GR * PER / 64;
            order();
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int at = TR ? (i * 8 + lane / 8) * LDW + lane % 8 * 8 : (i * 64 + lane) / PER * LDW + (i * 64 + lane) % PER * 8;
                *reinterpret_cast<u32x4_v *>(sw + at) = raw[p * NP + i];
            }
            order();
            // lane group g: j = 8 g on of 32; of a rank of 16 they are there twice (v's halves)
            if constexpr (TR) {
#pragma unroll
                for (int f = 0; f < 4; ++f)
                    wf[f][p] = read_transposed(sw + ((RP < 32 ? g & 1 : g) * 8 + col / 4) * LDW + f * 16 + col % 4 * 4, LDW);
            } else {
#pragma unroll
                for (int f = 0; f < GR / 16; ++f)
#pragma unroll
                    for (int q = 0; q < QW; ++q)
                        wf[p * (GR / 16) + f][q] =
                            *reinterpret_cast<const u32x4_v *>(sw + (f * 16 + col) * LDW + (RP < 32 ? (g & 1) * 8 : q * 32 + g * 8));
            }
        }
#pragma unroll
        for (int m = 0; m < MF; ++m) {
            if (r0 + m * 16 >= r1)
                break;
            f32x4_t acc[4] = {};
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const u32x4_v vf = *reinterpret_cast<const u32x4_v *>(sv + (m * 16 + col) * LDV + q * 32 + g * 8);
#pragma unroll
                for (int f = 0; f < 4; ++f)
                    acc[f] = mfma<DT>(wf[f][q % QW], vf, acc[f]);
            }
            const float by = factor[m * 16 + col];
            order();
#pragma unroll
            for (int f = 0; f < 4; ++f)
                *reinterpret_cast<f32x4_t *>(so + col * LDO + f * 16 + g * 4) = acc[f] * by;
            order();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int row = h * 8 + lane / 8, t = toks[m * 16 + row];
                const f32x4_t lo = *reinterpret_cast<const f32x4_t *>(so + row * LDO + lane % 8 * 8);
                const f32x4_t hi = *reinterpret_cast<const f32x4_t *>(so + row * LDO + lane % 8 * 8 + 4);
                float o[8];
                widen_piece(base[m][h], o);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    o[i] += i < 4 ? lo[i % 4] : hi[i % 4];
                if (t >= 0 && n < a.C)
                    store_piece<DT, WIDE, (MF > 2)>(a.y, (int64_t)t * a.C + n, a.C - n, round_piece<DT>(o));
            }
        }
    }
}

// ---------------------------------------------------------------- outer

struct OuterProblem {
    const uint16_t *d;  // [T, C]
    Small v;
    uint16_t *out;
    float *partial;     // [pieces of adapters with several][rank * C]
    const float *scale;
    int C, chunks;
};
struct OuterArgs {
    OuterProblem p[2];  // out [E, C, rank]; out [E, rank, C]
    const int32_t *offsets, *order;
    int T, rank, E;
    int piece, partials;  // tokens of a piece; pieces that `partial` has room for
};

// A workgroup takes a piece of an adapter's tokens and 256 columns (128 of ranks 33 to 64): 64 a wave (32 of ranks above
// 32), every second 32 tokens to each half of the waves, whose sums meet at the end.  Steps of 64 tokens pass through LDS as they lie, and both operands are
// read transposed; the next step's loads are under way meanwhile.
//
// Bound by the latency of a step's loads (1.6 waves a SIMD): 8191 tokens of 4096 + 4096 columns at rank 32 35 us for 134 MB (3.8 TB/s), rank 64
// 60; 512 tokens 8.
// BY_RANK: the output is [E, rank, C], else [E, C, rank].
template <int DT, int RF, bool WIDE, bool BY_RANK>
__device__ __forceinline__ void outer_piece(const OuterArgs &a, const OuterProblem &p, int idx, int c0, uint16_t *sd,
                                            uint16_t *sv, int *toks, float *most)
{
    constexpr int RP = RF * 16, LDV = 2 * RP + 8, CF = outer_frags(RF), THREADS = outer_threads(RF), HALF = THREADS / 128, COLS = outer_cols(RF), CP = COLS / 8, LDD = COLS + 16;
    constexpr int PER = RP / 8, NV = (kStep * PER + THREADS - 1) / THREADS, ND = kStep * CP / THREADS;
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, col = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), half = wave / HALF, cols = wave % HALF * (16 * CF);
    int e, r0, r1, pieces, number;
    if (!find_piece(a.offsets, a.E, a.T, a.piece, idx, e, r0, r1, pieces, number) || (pieces > 1 && number >= a.partials))
        return;
    const int len = (r1 - r0 + kStep - 1) / kStep * kStep;
    for (int i = tid; i < len; i += THREADS)
        toks[i] = token_at(a.order, r0 + i, r1, a.T);
    __syncthreads();
    int ex = -200;  // fp16: the exponent that v is brought down by, that of its largest so far
    u32x4_v nd[ND];
    float nv[NV][8];
    auto fetch = [&](int r) {
#pragma unroll
        for (int q = 0; q < ND; ++q) {
            const int row = (tid + q * THREADS) / CP, n = c0 + tid % CP * 8;
            const int t = toks[r - r0 + row];
            nd[q] = t >= 0 ? row_piece<WIDE>(p.d + (int64_t)t * p.C, n, p.C) : u32x4_v{};
        }
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const int i = tid + q * THREADS;
            const int t = i / PER < kStep ? toks[r - r0 + i / PER] : -1;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                nv[q][k] = 0.f;
            if (t >= 0)
                load_small(p.v, t, i % PER * 8, nv[q]);
        }
    };
    f32x4_t acc[CF][RF] = {};
    fetch(r0);
    for (int r = r0; r < r1; r += kStep) {
        if constexpr (DT == TERNARY_FP16) {
            float m = 0.f;
#pragma unroll
            for (int q = 0; q < NV; ++q)
                m = fmaxf(m, largest(nv[q]));
#pragma unroll
            for (int o = 1; o < 64; o <<= 1)
                m = fmaxf(m, __shfl_xor(m, o));
            if (lane == 0)
                most[wave] = m;
        }
        __syncthreads();
        if constexpr (DT == TERNARY_FP16) {
            float m = most[0];
#pragma unroll
            for (int w = 1; w < THREADS / 64; ++w)
                m = fmaxf(m, most[w]);
            const int now = m > 0.f ? max(ex, ilogbf(m)) : ex;
            if (now > ex) {
                const float down = ldexpf(1.f, ex - now);
#pragma unroll
                for (int c = 0; c < CF; ++c)
#pragma unroll
                    for (int f = 0; f < RF; ++f)
                        acc[c][f] *= down;
                ex = now;
            }
        }
#pragma unroll
        for (int q = 0; q < ND; ++q)
            *reinterpret_cast<u32x4_v *>(sd + (tid + q * THREADS) / CP * LDD + tid % CP * 8) = nd[q];
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const int i = tid + q * THREADS;
            if (i / PER < kStep)
                put_split<DT, RP>(sv + i / PER * LDV, i % PER * 8, nv[q], ex);
        }
        __syncthreads();
        if (r + kStep < r1)
            fetch(r + kStep);
        const int row = half * 32 + g * 8 + col / 4;
        u32x4_v df[CF];
#pragma unroll
        for (int c = 0; c < CF; ++c)
            df[c] = read_transposed(sd + row * LDD + cols + c * 16 + col % 4 * 4, LDD);
#pragma unroll
        for (int f = 0; f < RF; ++f)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const u32x4_v vf = read_transposed(sv + row * LDV + h * RP + f * 16 + col % 4 * 4, LDV);
#pragma unroll
                for (int c = 0; c < CF; ++c)
                    acc[c][f] = BY_RANK ? mfma<DT>(df[c], vf, acc[c][f]) : mfma<DT>(vf, df[c], acc[c][f]);
            }
    }
    const int64_t size = (int64_t)a.rank * p.C;
    const float by = ldexpf(p.scale ? p.scale[e] : 1.f, DT == TERNARY_FP16 ? ex : 0);
    f32x4_t *other = reinterpret_cast<f32x4_t *>(sd);  // the other half's sums, 16 of the rank at a time
#pragma unroll
    for (int f = 0; f < RF; ++f) {
        __syncthreads();
        if (half == 1)
#pragma unroll
            for (int c = 0; c < CF; ++c)
                other[(wave % HALF * CF + c) * 64 + lane] = acc[c][f];
        __syncthreads();
        if (half == 0)
#pragma unroll
            for (int c = 0; c < CF; ++c) {
                // four neighbours of the axis that lies contiguous in the output
                const int j = f * 16 + (BY_RANK ? col : g * 4), n = c0 + cols + c * 16 + (BY_RANK ? g * 4 : col);
                const int64_t i = BY_RANK ? (int64_t)j * p.C + n : (int64_t)n * a.rank + j;
                const int left = BY_RANK ? (j < a.rank ? p.C - n : 0) : (n < p.C ? a.rank - j : 0);
                const int line = BY_RANK ? p.C : a.rank;
                const f32x4_t v = (acc[c][f] + other[(wave * CF + c) * 64 + lane]) * by;
                if (left <= 0)
                    continue;
                if (pieces > 1) {
                    float *o = p.partial + number * size + i;
                    if (line % 4 == 0)
                        *reinterpret_cast<f32x4_t *>(o) = v;
                    else
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (k < left)
                                o[k] = v[k];
                } else {
                    uint16_t *o = p.out + e * size + i;
                    if (line % 4 == 0)
                        store4<DT>(o, 0, v);
                    else
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (k < left)
                                store_elem<DT>(o, k, v[k]);
                }
            }
    }
}

template <int DT, int RF, bool WIDE>
__global__ void __launch_bounds__(outer_threads(RF), 4) outer_kernel(const OuterArgs a)
{
    __shared__ __attribute__((aligned(16))) uint16_t sd[kStep * (outer_cols(RF) + 16)], sv[kStep * (RF * 32 + 8)];
    __shared__ int toks[kMaxPiece];
    __shared__ float most[outer_threads(RF) / 64];
    const int chunks = a.p[0].chunks + a.p[1].chunks, idx = blockIdx.x / chunks, at = blockIdx.x - idx * chunks;
    if (at < a.p[0].chunks)
        outer_piece<DT, RF, WIDE, false>(a, a.p[0], idx, at * outer_cols(RF), sd, sv, toks, most);
    else
        outer_piece<DT, RF, WIDE, true>(a, a.p[1], idx, (at - a.p[0].chunks) * outer_cols(RF), sd, sv, toks, most);
}

// Gradients of adapters with several pieces, and zeros for those without tokens: four neighbours a thread.
template <int DT>
__global__ void __launch_bounds__(kThreads) outer_sum_kernel(const OuterArgs a, int blocks0)
{
    const int which = (int)blockIdx.x >= blocks0, e = blockIdx.y;
    const OuterProblem &p = a.p[which];
    int pieces, first;
    expert_pieces(a.offsets, a.E, a.T, a.piece, e, pieces, first);
    if (pieces == 1)
        return;
    pieces = min(pieces, a.partials - first);
    const int64_t size = (int64_t)a.rank * p.C;
    const int64_t i = ((int64_t)(blockIdx.x - (which ? blocks0 : 0)) * kThreads + threadIdx.x) * 4;
    if (i >= size)
        return;
    float v[4] = {};
    uint16_t *o = p.out + e * size + i;
    if (size % 4 == 0) {
#pragma unroll 4
        for (int k = 0; k < pieces; ++k) {
            const f32x4_t u = *reinterpret_cast<const f32x4_t *>(p.partial + (first + k) * size + i);
#pragma unroll
            for (int q = 0; q < 4; ++q)
                v[q] += u[q];
        }
        store4<DT>(o, 0, f32x4_t{v[0], v[1], v[2], v[3]});
    } else {
        for (int k = 0; k < pieces; ++k)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                v[q] += i + q < size ? p.partial[(first + k) * size + i + q] : 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (i + q < size)
                store_elem<DT>(o, q, v[q]);
    }
}

// ---------------------------------------------------------------- few tokens

// Few tokens of small rank: down and up in one launch.  A workgroup of 16 waves takes 16 places: its waves share the rows of x,
// meet, and take 64 columns of y each.  Workgroups that share the places each compute v for themselves (from
// L2), which costs less than a second launch; b and what is added to are under way meanwhile.  Bound by a chain of loads (offsets,
// order, x and a, y): 1 token of 4096 x 4096, rank 16, 7.1 us in a graph, 64 tokens of 32 adapters 8.8.
struct FewArgs {
    AdapterArgs p;
    int chunks;  // runs of 1024 columns
};
constexpr int kFewWaves = 16, kFewCols = kFewWaves * 64;

template <int DT, int RF, bool WIDE>
__global__ void __launch_bounds__(kFewWaves * 64) few_kernel(const FewArgs f)
{
    constexpr int RP = RF * 16, PER = RP / 8, LD = 64 + 8, LDW = RP + 8, LDO = 64 + 4, LDV = 2 * RP + 8;
    constexpr int STAGE = (64 * LDW > 32 * LD ? 64 * LDW : 32 * LD) * 2 > 16 * LDO * 4 ? (64 * LDW > 32 * LD ? 64 * LDW : 32 * LD) * 2 : 16 * LDO * 4;
    static_assert(RF <= 2 && kFewWaves * STAGE >= kFewWaves * RF * 64 * 16);
    __shared__ __attribute__((aligned(16))) unsigned char lds[kFewWaves * STAGE];
    __shared__ __attribute__((aligned(16))) float sums[16 * (RP + 4)];
    __shared__ __attribute__((aligned(16))) uint16_t sv[16 * LDV];
    __shared__ float factor[16];
    const AdapterArgs &a = f.p;
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, col = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int tile = blockIdx.x / f.chunks, chunk = blockIdx.x - tile * f.chunks;
    // tokens without an adapter, 16 looked at by each tile, one a wave
    if (a.y != a.add && (int64_t)tile * 16 + wave < a.T) {
        const int64_t t = (int64_t)tile * 16 + wave;
        if ((unsigned)a.slots[t] >= (unsigned)a.T)
            for (int n = chunk * kFewCols + lane * 8; n < min((chunk + 1) * kFewCols, a.N); n += 512) {
                Raw<DT> v = {};
                if (a.add)
                    v = load_piece<DT, WIDE>(a.add, t * a.N + n, a.N - n);
                store_piece<DT, WIDE>(a.y, t * a.N + n, a.N - n, v);
            }
    }
    int e, r0, r1;
    if (!find_tile<16>(a.offsets, a.E, a.T, tile, e, r0, r1))
        return;
    int tok[2];  // of rows lane / 8 and 8 on
#pragma unroll
    for (int m = 0; m < 2; ++m)
        tok[m] = token_at(a.order, r0 + m * 8 + lane / 8, r1, a.T);
    const uint16_t *w = a.a + (int64_t)e * a.rank * a.K, *wb = a.b + (int64_t)e * a.rank * a.N;
    unsigned char *mine = lds + wave * STAGE;
    uint16_t *stage = reinterpret_cast<uint16_t *>(mine);
    float *so = reinterpret_cast<float *>(mine);
    auto order = []() { asm volatile("" ::: "memory"); };  // (a wave's LDS accesses are in order)
    const int n0 = chunk * kFewCols + wave * 64, n = n0 + lane % 8 * 8;  // this wave's columns, this lane's
    u32x4_v raw[PER];
    Raw<DT> base[2];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int r = (i * 64 + lane) / PER, j = (i * 64 + lane) % PER * 8;
        raw[i] = n0 + r < a.N ? row_piece<WIDE>(wb + (int64_t)(n0 + r) * a.rank, j, a.rank) : u32x4_v{};
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        base[h] = Raw<DT>{};
        if (a.add && tok[h] >= 0)
            base[h] = load_piece<DT, WIDE>(a.add, (int64_t)tok[h] * a.N + n, a.N - n);
    }
    constexpr int B = RF == 1 ? 4 : 2;  // steps whose loads go out together
    const int steps = (a.K + 63) / 64;
    f32x4_t acc[RF] = {};
    for (int i0 = wave; i0 < steps; i0 += B * kFewWaves) {
        u32x4_v nx[B][2], nw[B][2 * RF];
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const int i = i0 + b * kFewWaves, k = i * 64 + lane % 8 * 8;  // (past the last step: past the rows' end)
#pragma unroll
            for (int q = 0; q < 2 * RF; ++q) {
                const int j = q * 8 + lane / 8;
                nw[b][q] = j < a.rank ? row_piece<WIDE>(w + (int64_t)j * a.K, k, a.K) : u32x4_v{};
            }
#pragma unroll
            for (int m = 0; m < 2; ++m)
                nx[b][m] = tok[m] >= 0 ? row_piece<WIDE>(a.x + (int64_t)tok[m] * a.K, k, a.K) : u32x4_v{};
        }
#pragma unroll
        for (int b = 0; b < B; ++b) {
            if (i0 + b * kFewWaves >= steps)
                break;
            u32x4_v xf[2], wf[2][RF];
            order();
#pragma unroll
            for (int q = 0; q < 2 * RF; ++q)
                *reinterpret_cast<u32x4_v *>(stage + (q * 8 + lane / 8) * LD + lane % 8 * 8) = nw[b][q];
            order();
#pragma unroll
            for (int u = 0; u < RF; ++u)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    wf[h][u] = *reinterpret_cast<const u32x4_v *>(stage + (u * 16 + col) * LD + h * 32 + g * 8);
            order();
#pragma unroll
            for (int m = 0; m < 2; ++m)
                *reinterpret_cast<u32x4_v *>(stage + (m * 8 + lane / 8) * LD + lane % 8 * 8) = nx[b][m];
            order();
#pragma unroll
            for (int h = 0; h < 2; ++h)
                xf[h] = *reinterpret_cast<const u32x4_v *>(stage + col * LD + h * 32 + g * 8);
            order();
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int u = 0; u < RF; ++u)
                    acc[u] = mfma<DT>(wf[h][u], xf[h], acc[u]);
        }
    }
    // the waves' sums
    f32x4_t *parts = reinterpret_cast<f32x4_t *>(lds);
    __syncthreads();
#pragma unroll
    for (int u = 0; u < RF; ++u)
        parts[(wave * RF + u) * 64 + lane] = acc[u];
    __syncthreads();
    if (wave < RF) {
        f32x4_t v = parts[wave * 64 + lane];
#pragma unroll
        for (int u = 1; u < kFewWaves; ++u)
            v += parts[(u * RF + wave) * 64 + lane];
        *reinterpret_cast<f32x4_t *>(sums + col * (RP + 4) + wave * 16 + g * 4) = v;
    }
    __syncthreads();
    if (tid < 16 * PER) {
        const int row = tid / PER, j0 = tid % PER * 8, t = token_at(a.order, r0 + row, r1, a.T);
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] = sums[row * (RP + 4) + j0 + k];
        if (a.hidden && chunk == 0 && t >= 0)
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (j0 + k < a.rank)
                    a.hidden[(int64_t)t * a.rank + j0 + k] = v[k];
        int ex = 0;
        if constexpr (DT == TERNARY_FP16) {
            float m = largest(v);
#pragma unroll
            for (int o = 1; o < PER; o <<= 1)
                m = fmaxf(m, __shfl_xor(m, o));
            ex = exponent(m);
        }
        put_split<DT, RP>(sv + row * LDV, j0, v, ex);
        if (j0 == 0)
            factor[row] = ldexpf(a.scale ? a.scale[e] : 1.f, ex);
    }
    __syncthreads();
    u32x4_v wf[4];
    order();
#pragma unroll
    for (int i = 0; i < PER; ++i)
        *reinterpret_cast<u32x4_v *>(stage + (i * 64 + lane) / PER * LDW + (i * 64 + lane) % PER * 8) = raw[i];
    order();
#pragma unroll
    for (int u = 0; u < 4; ++u)
        wf[u] = *reinterpret_cast<const u32x4_v *>(stage + (u * 16 + col) * LDW + (RP < 32 ? (g & 1) * 8 : g * 8));
    f32x4_t out[4] = {};
#pragma unroll
    for (int q = 0; q < RF; ++q) {
        const u32x4_v vf = *reinterpret_cast<const u32x4_v *>(sv + col * LDV + q * 32 + g * 8);
#pragma unroll
        for (int u = 0; u < 4; ++u)
            out[u] = mfma<DT>(wf[u], vf, out[u]);
    }
    const float by = factor[col];
    order();
#pragma unroll
    for (int u = 0; u < 4; ++u)
        *reinterpret_cast<f32x4_t *>(so + col * LDO + u * 16 + g * 4) = out[u] * by;
    order();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int row = h * 8 + lane / 8;
        const f32x4_t lo = *reinterpret_cast<const f32x4_t *>(so + row * LDO + lane % 8 * 8);
        const f32x4_t hi = *reinterpret_cast<const f32x4_t *>(so + row * LDO + lane % 8 * 8 + 4);
        float o[8];
        widen_piece(base[h], o);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            o[i] += i < 4 ? lo[i % 4] : hi[i % 4];
        if (tok[h] >= 0 && n < a.N)
            store_piece<DT, WIDE>(a.y, (int64_t)tok[h] * a.N + n, a.N - n, round_piece<DT>(o));
    }
}

// ---------------------------------------------------------------- launches

inline int64_t up_to(int64_t n, int64_t m) { return (n + m - 1) / m; }
// Tiles of `rows` places that T places of E adapters may need.
inline int64_t tiles_of(int64_t T, int64_t E, int64_t rows) { return T / rows + (E < T ? E : T); }
inline bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }

// Fragments of 16 tokens of a down tile (us of all kernels for two and four: 8191 tokens of 4096 -> 18944 at rank 64 157 and 165, their gradients
// of 4096 x 4096 118 and 131; for two and one 157 and 161, 118 and 123; one where adapters have fewer tokens).  A workgroup has four waves;
// where tiles are few 16, so that there are few partial sums (1000 tokens at rank 16 13.3 us, with four 14.0; gradients of 2048 32.3 and 34.1; not
// of ranks above 32, which want the registers).
inline int down_rows(int64_t T, int64_t E) { return T <= 16 * E ? 1 : 2; }
inline int64_t down_tiles(int64_t T, int64_t E) { return up_to(T, 16 * down_rows(T, E)) + (E < T ? E : T) / 2; }
inline bool down_few(int64_t T, int64_t E, int64_t rank) { return rank <= 32 && down_tiles(T, E) < 192; }
// Workgroups that share a row: until there are enough waves, or a wave has a single step.
inline int down_splits(int64_t T, int64_t E, int64_t L, int64_t rank)
{
    const int64_t tiles = down_tiles(T, E), waves = down_few(T, E, rank) ? 16 : 4, steps = up_to(L, 64 * waves);
    int s = 1;
    while (s < 8 && s * 2 <= steps && s * tiles * waves < 1536)
        s *= 2;
    return s;
}
// Tokens of a piece: about 256 workgroups (of 8191 tokens, 4096 + 4096 columns; us of all gradients in a graph, for 192, 256 and 512: rank 32
// 96, 97 and 104; rank 16 86, 86 and 93; 4096 tokens of 16 adapters, rank 128, 104, 103 and 117 for 384).
inline int piece_tokens(int64_t T, int64_t K, int64_t N, int64_t rank)
{
    const int cols = outer_cols(rank_frags(rank));
    const int64_t chunks = up_to(K, cols) + up_to(N, cols), want = T * chunks / 256 / kStep * kStep;
    return (int)(want < 128 ? 128 : want > kMaxPiece ? kMaxPiece : want);
}
inline int64_t round256(int64_t n) { return (n + 255) & ~(int64_t)255; }
inline int64_t small_bytes(int64_t T, int64_t E, int64_t L, int64_t rank)
{
    return round256(T * rank * 4 * down_splits(T, E, L, rank));
}

// Runs f(dtype, fragments of 16 of the rank, wide rows) as compile-time values.
template <class F>
void with_rank(bool fp16, int rank, bool wide, F f)
{
    auto by_type = [&](auto dt) {
        auto by_width = [&](auto rf) {
            if (wide)
                f(dt, rf, std::true_type());
            else
                f(dt, rf, std::false_type());
        };
        if (rank <= 16)
            by_width(std::integral_constant<int, 1>());
        else if (rank <= 32)
            by_width(std::integral_constant<int, 2>());
        else if (rank <= 64)
            by_width(std::integral_constant<int, 4>());
        else
            by_width(std::integral_constant<int, 8>());
    };
    if (fp16)
        by_type(std::integral_constant<int, TERNARY_FP16>());
    else
        by_type(std::integral_constant<int, TERNARY_BF16>());
}

template <bool TR>
hipError_t launch_down(const DownArgs &d, bool fp16, hipStream_t stream)
{
    const int mf = down_rows(d.T, d.E);
    const bool few = down_few(d.T, d.E, d.rank);
    const bool wide = d.L % 8 == 0 && aligned16(d.x) && aligned16(d.w) && (!TR || d.rank % 8 == 0);
    const dim3 grid((unsigned)(tiles_of(d.T, d.E, 16 * mf) * d.splits));
    with_rank(fp16, d.rank, wide, [&](auto dt, auto rf, auto wd) {
        constexpr int DT = decltype(dt)::value, RF = decltype(rf)::value;
        constexpr bool WIDE = decltype(wd)::value;
        auto run = [&](auto kernel, int waves) {
            hipLaunchKernelGGL(kernel, grid, dim3(waves * 64), 0, stream, d);
        };
        if constexpr (RF <= 2) {
            if (few)
                return mf == 1 ? run(down_kernel<DT, RF, 1, 16, TR, WIDE>, 16) : run(down_kernel<DT, RF, 2, 16, TR, WIDE>, 16);
        }
        mf == 1 ? run(down_kernel<DT, RF, 1, 4, TR, WIDE>, 4) : run(down_kernel<DT, RF, 2, 4, TR, WIDE>, 4);
    });
    return hipGetLastError();
}

template <bool TR>
hipError_t launch_up(UpArgs u, bool fp16, hipStream_t stream)
{
    u.chunks = (int)up_to(u.C, kCols);
    // Large outputs: tiles of 64 places, past the caches (us, 64 and 32: 8191 tokens of 18944 columns at rank 64 165 and 197, 4096 of 8192
    // at rank 128 87 and 89, 5000 of 4096 33.0 and 33.4 at rank 16, 51.6 and 50.3 at 64; 3000 of 4096 23.4 and 21.3, 32.1 and 27.5; 300 11.6 and
    // 9.8).  Two runs of columns a workgroup where there are enough (18944 columns 135 us for up alone, one run 144).
    const int mf = (int64_t)u.T * u.C >= (int64_t)3 << 23 ? 4 : 2;
    const int64_t tiles = tiles_of(u.T, u.E, 16 * mf);
    const int64_t per = tiles * u.chunks / 2048;
    u.per = (int)(per < 1 ? 1 : per > 2 ? 2 : per);
    const bool wide = u.C % 8 == 0 && aligned16(u.w) && aligned16(u.add) && aligned16(u.y) && (TR || u.rank % 8 == 0);
    const dim3 grid((unsigned)(tiles * up_to(u.chunks, u.per)));
    with_rank(fp16, u.rank, wide, [&](auto dt, auto rf, auto wd) {
        constexpr int DT = decltype(dt)::value, RF = decltype(rf)::value;
        constexpr bool WIDE = decltype(wd)::value;
        if (mf == 2)
            hipLaunchKernelGGL((up_kernel<DT, RF, 2, TR, WIDE>), grid, dim3(kThreads), 0, stream, u);
        else
            hipLaunchKernelGGL((up_kernel<DT, RF, 4, TR, WIDE>), grid, dim3(kThreads), 0, stream, u);
    });
    return hipGetLastError();
}

// Whether one launch takes all.  Us in a graph, one launch and two (from Python, where a launch and a workspace cost the
// host 5: 10.1 and 15.1 wherever the kernels take less), 4096 -> N, 32 adapters.  Rank 16: 1 token -> 4096 7.3 and 7.8, 16 7.5 and
// 7.8, 64 9.1 and 8.5, 128 -> 1024 8.4 and 8.4, 128 -> 4096 10.1 and 8.9, 64 -> 18944 15.2 and 12.2.  Rank 32: 1 -> 4096 9.0 and 8.5,
// 4 9.2 and 8.6, 16 10.6 and 8.8, 64 11.8 and 10.5.
inline bool few_tokens(int64_t T, int64_t N, int64_t rank)
{
    return rank <= 16 ? T <= 128 && T * N <= 1 << 18 : rank <= 32 && T * N <= 1 << 14;
}

hipError_t launch_few(const AdapterArgs &a, hipStream_t stream)
{
    const FewArgs f = {a, (int)up_to(a.N, kFewCols)};
    const bool wide = a.K % 8 == 0 && a.N % 8 == 0 && a.rank % 8 == 0 && aligned16(a.x) && aligned16(a.a) && aligned16(a.b) &&
                      aligned16(a.add) && aligned16(a.y);
    const dim3 grid((unsigned)(tiles_of(a.T, a.E, 16) * f.chunks));
    with_rank(a.fp16, a.rank, wide, [&](auto dt, auto rf, auto wd) {
        if constexpr (decltype(rf)::value <= 2)
            hipLaunchKernelGGL((few_kernel<decltype(dt)::value, decltype(rf)::value, decltype(wd)::value>), grid,
                               dim3(kFewWaves * 64), 0, stream, f);
    });
    return hipGetLastError();
}

}  // namespace

int64_t adapters_workspace(int64_t T, int64_t K, int64_t N, int64_t rank, int64_t E)
{
    return few_tokens(T, N, rank) ? 0 : small_bytes(T, E, K, rank);
}

int64_t adapters_back_workspace(int64_t T, int64_t K, int64_t N, int64_t rank, int64_t E)
{
    const int64_t partials = 2 * T / piece_tokens(T, K, N, rank);
    return small_bytes(T, E, N, rank) + round256(partials * rank * N * 4) + round256(partials * rank * K * 4);
}

hipError_t launch_adapters(const AdapterArgs &a, hipStream_t stream)
{
    if (few_tokens(a.T, a.N, a.rank))
        return launch_few(a, stream);
    const int splits = down_splits(a.T, a.E, a.K, a.rank);
    float *v = static_cast<float *>(a.workspace);
    const DownArgs d = {a.x, a.a, nullptr, a.offsets, a.order, v, a.T, a.K, a.rank, a.E, splits};
    hipError_t e = launch_down<false>(d, a.fp16, stream);
    if (e != hipSuccess)
        return e;
    const UpArgs u = {{v, splits, a.rank, (int64_t)a.T * a.rank}, a.b, a.scale, a.offsets, a.order, a.slots, a.add, a.y,
                      a.hidden, a.T, a.N, a.rank, a.E, 0, 0};
    return launch_up<false>(u, a.fp16, stream);
}

hipError_t launch_adapters_back(const AdapterArgs &a, hipStream_t stream)
{
    const int piece = piece_tokens(a.T, a.K, a.N, a.rank), splits = down_splits(a.T, a.E, a.N, a.rank);
    const int partials = (int)(2 * (int64_t)a.T / piece), cols = outer_cols(rank_frags(a.rank));
    char *ws = static_cast<char *>(a.workspace);
    float *dv = reinterpret_cast<float *>(ws);
    ws += small_bytes(a.T, a.E, a.N, a.rank);
    float *part_b = reinterpret_cast<float *>(ws);
    ws += round256((int64_t)partials * a.rank * a.N * 4);
    float *part_a = reinterpret_cast<float *>(ws);
    const Small small = {dv, splits, a.rank, (int64_t)a.T * a.rank};
    hipError_t e = hipSuccess;
    const OuterArgs o = {{{a.grad, {a.hidden, 1, a.rank, 0}, a.db, part_b, a.scale, a.N, (int)up_to(a.N, cols)},
                          {a.x, small, a.da, part_a, nullptr, a.K, (int)up_to(a.K, cols)}},
                         a.offsets, a.order, a.T, a.rank, a.E, piece, partials};
    if (a.T) {
        const DownArgs d = {a.grad, a.b, a.scale, a.offsets, a.order, dv, a.T, a.N, a.rank, a.E, splits};
        e = launch_down<true>(d, a.fp16, stream);
        if (e != hipSuccess)
            return e;
        const bool wide = a.N % 8 == 0 && a.K % 8 == 0 && aligned16(a.grad) && aligned16(a.x);
        const dim3 grid((unsigned)(tiles_of(a.T, a.E, piece) * (o.p[0].chunks + o.p[1].chunks)));
        with_rank(a.fp16, a.rank, wide, [&](auto dt, auto rf, auto wd) {
            hipLaunchKernelGGL((outer_kernel<decltype(dt)::value, decltype(rf)::value, decltype(wd)::value>), grid,
                               dim3(outer_threads(decltype(rf)::value)), 0, stream, o);
        });
        e = hipGetLastError();
        if (e != hipSuccess)
            return e;
        const UpArgs u = {small, a.a, nullptr, a.offsets, a.order, a.slots, a.add, a.dx, nullptr, a.T, a.K, a.rank, a.E, 0, 0};
        e = launch_up<true>(u, a.fp16, stream);
        if (e != hipSuccess)
            return e;
    }
    const int blocks0 = (int)up_to((int64_t)a.rank * a.N, kThreads * 4), blocks1 = (int)up_to((int64_t)a.rank * a.K, kThreads * 4);
    const dim3 grid((unsigned)(blocks0 + blocks1), (unsigned)a.E);
    if (a.fp16)
        hipLaunchKernelGGL((outer_sum_kernel<TERNARY_FP16>), grid, dim3(kThreads), 0, stream, o, blocks0);
    else
        hipLaunchKernelGGL((outer_sum_kernel<TERNARY_BF16>), grid, dim3(kThreads), 0, stream, o, blocks0);
    return hipGetLastError();
}

}  // namespace ternary
