// Products of 8-bit activations on gfx950: with 8-bit weights (a scale per
// block of 128 x 128), and with the ternary weights of experts.
//
//     y[m, n] = sum_b xs[m, b] s(n, b) sum_{k in b} x[m, k] w[n, k]
//
// Sums are fp32 throughout.  The matrix unit's 8-bit forms do not keep them: of eight products
// that a lane holds side by side they align all to the largest and cut what falls 2^-14 below it, so
// that beside a factor of 448 one of 2^-6 counts for nothing (measured; up to 2^-11.4 of the sum
// of magnitudes, all of a sum whose large products cancel).  So both factors become fp16, which
// holds every e4m3 value and +-2, and v_mfma_f32_16x16x32_f16 adds their products, which are exact, in 24 bits.
// That unit has half the rate of the 8-bit one; what it costs is beside the kernels below.
//
// Four of those instructions multiply 16 channels (the A operand) by 16 rows of x (B) over one
// block of 128; their sums are then scaled and added to the running sums.
// A lane's four results are four channels of one row: the row's scale is one
// register and the four go out in one store.  Ternary codes become fp4 (+-2) in five vector operations a 16 codes, and
// fp16 by eight conversions; as the first give a word's odd codes, then its even ones, x's bytes are put in the
// same order (eight byte permutes per 16 rows x 128).  A lane holds 32 values of k of each operand, the
// same ones: of 8-bit weights k = 16 g .. and 64 + 16 g .. (16 each) in lane group g (lanes 16 g up).
#include "fp8_common.h"
#include "internal.h"
#include "places.h"

namespace ternary {

namespace {

// A lane's 32 values of a block, for four instructions.
struct Wide {
    f16x8_t q[4];
};
template <class A>
__device__ __forceinline__ f16x8_t join_halves(A a, A b, A c, A d)
{
    return __builtin_bit_cast(f16x8_t, u32x4_v{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b),
                                              __builtin_bit_cast(uint32_t, c), __builtin_bit_cast(uint32_t, d)});
}
// Eight e4m3 values (two registers), or eight fp4 values (one), as fp16.
__device__ __forceinline__ f16x8_t widen_fp8(int lo, int hi)
{
    return join_halves(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, false),
                       __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, true),
                       __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, false),
                       __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, true));
}
__device__ __forceinline__ f16x8_t widen_fp4(int v)
{
    return join_halves(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4((uint32_t)v, 1.f, 0),
                       __builtin_amdgcn_cvt_scalef32_pk_f16_fp4((uint32_t)v, 1.f, 1),
                       __builtin_amdgcn_cvt_scalef32_pk_f16_fp4((uint32_t)v, 1.f, 2),
                       __builtin_amdgcn_cvt_scalef32_pk_f16_fp4((uint32_t)v, 1.f, 3));
}
__device__ __forceinline__ Wide widen(u32x4_v a, u32x4_v b)
{
    return Wide{{widen_fp8((int)a.x, (int)a.y), widen_fp8((int)a.z, (int)a.w), widen_fp8((int)b.x, (int)b.y),
                 widen_fp8((int)b.z, (int)b.w)}};
}

// 32 of a block's k: 16 channels by 16 rows.
__device__ __forceinline__ f32x4_t mfma(f16x8_t w, f16x8_t x, f32x4_t d)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(w, x, d, 0, 0, 0);
}
// Chunks of 16 of a block of x that lane group g holds: the first, and how many on
// the second lies.  8-bit weights: as the same chunks of w; ternary ones: as the
// lane groups of w hold the codes 0, 64, 32 and 96 (and 31 more).
template <bool TERN>
__device__ __forceinline__ int first_chunk(int g)
{
    return TERN ? (g & 1) * 4 + (g & 2) : g;
}
constexpr int second_chunk(bool tern) { return tern ? 1 : 4; }

// Scale of a channel's fp4 products.
__device__ __forceinline__ float channel_scale(uint16_t s) { return 0.5f * f16_bits_to_f32(s); }

// 16 codes (one word) -> the fp4 words of its odd and of its even codes (the
// field (b1 b0) becomes (sign, magnitude) = (b1, b0 ^ b1) at a nibble's top).
__device__ __forceinline__ void codes_to_fp4(uint32_t w, int &odd, int &even)
{
    const uint32_t z = __builtin_amdgcn_bitop3_b32(w, w >> 1, 0x55555555u, 0x78);
    odd = (int)(z & 0xccccccccu);
    even = (int)((z << 2) & 0xccccccccu);
}

// 32 codes (two words) as fp16, per 16 odd then even.
__device__ __forceinline__ Wide widen_codes(uint32_t w0, uint32_t w1)
{
    int c[4];
    codes_to_fp4(w0, c[0], c[1]);
    codes_to_fp4(w1, c[2], c[3]);
    return Wide{{widen_fp4(c[0]), widen_fp4(c[1]), widen_fp4(c[2]), widen_fp4(c[3])}};
}

// 32 bytes of x in that order.
__device__ __forceinline__ Wide widen_odd_even(u32x4_v a, u32x4_v b)
{
    constexpr uint32_t odd = 0x07050301u, even = 0x06040200u;
    return widen(u32x4_v{__builtin_amdgcn_perm(a.y, a.x, odd), __builtin_amdgcn_perm(a.w, a.z, odd),
                         __builtin_amdgcn_perm(a.y, a.x, even), __builtin_amdgcn_perm(a.w, a.z, even)},
                 u32x4_v{__builtin_amdgcn_perm(b.y, b.x, odd), __builtin_amdgcn_perm(b.w, b.z, odd),
                         __builtin_amdgcn_perm(b.y, b.x, even), __builtin_amdgcn_perm(b.w, b.z, even)});
}
template <bool TERN>
__device__ __forceinline__ Wide x_operand(u32x4_v a, u32x4_v b)
{
    return TERN ? widen_odd_even(a, b) : widen(a, b);
}

// Four channels ch .. ch + 3 of a row of y (those past N are left out).
template <int DT>
__device__ __forceinline__ void put4(const Fp8Product &p, int row, int ch, f32x4_t s)
{
    const int64_t at = (int64_t)row * p.N + ch;
    if (p.N % 4 == 0) {
        if (ch < p.N)
            store4<DT>(p.y, at, s);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (ch + i < p.N)
                store_elem<DT>(p.y, at + i, s[i]);
    }
}

// The same for y's type as the argument gives it.
__device__ __forceinline__ void put4(const Fp8Product &p, int row, int ch, f32x4_t s)
{
    if (p.dtype == TERNARY_BF16)
        put4<TERNARY_BF16>(p, row, ch, s);
    else if (p.dtype == TERNARY_FP16)
        put4<TERNARY_FP16>(p, row, ch, s);
    else
        put4<TERNARY_FP32>(p, row, ch, s);
}

// Waits for this wave's loads from memory (those into LDS among them) and for its LDS
// reads, then for the workgroup's other waves.
__device__ __forceinline__ void meet()
{
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(7 << 4);  // vmcnt(0) lgkmcnt(0)
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

typedef __attribute__((address_space(3))) u32x4_v lds_u4;
typedef __attribute__((address_space(3))) void lds_void;

// One memory-to-LDS load: 16 bytes a lane from `src`, to lds + 16 * lane.
__device__ __forceinline__ void load_to_lds(const uint8_t *src, lds_u4 *lds)
{
#if defined(__HIP_DEVICE_COMPILE__)
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)src,
                                     (lds_void *)lds, 16, 0, 0);
#endif
}

// The same from a buffer resource.
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t rsrc, lds_u4 *lds, int voff, int soff)
{
#if defined(__HIP_DEVICE_COMPILE__)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void *)lds, 16, voff, soff,
                                             0, 0);
#endif
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void *base, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)bytes, 0x00020000);
}

// A row of a stage is 128 bytes, eight chunks of 16; chunk c of row r sits at
// c ^ swz(r), which spreads the rows that a fragment read touches over the banks.
__device__ __forceinline__ int swz(int r) { return r & 7; }

// ---------------------------------------------------------------- few rows
//
// Weights are read once, so the kernel is a stream of them: they go straight
// from memory to registers, a chunk of U blocks at a time with all its loads
// issued together, and the eight waves of a workgroup share K out (`ks` ways; the others
// take further channels) and meet once, in LDS.  A wave holds 16 FN channels x
// 16 MT rows.  x is read again (from L2) for every 16 FN channels; it passes
// through LDS, each wave's own part, because the operand's lane order (16 rows
// in neighbouring lanes) would cost a cache access per lane: at 45 rows of 18944 x 4096
// the accesses of L1, not HBM, bounded a kernel that loaded x like w (39 us).
//
// Measured (calls in a graph, bf16 outputs; behind each the time with the 8-bit matrix instruction): 1 row of 4096 x
// 4096 5.6 us (5.7); 45 rows of 18944 x 4096 20.7 (19.8; 3.8 TB/s); 64 experts of 2048 x 4096, 8 a
// token, 1 token 8.0 (6.9), 16 tokens 44 (37); of 4096 x 1024 with scales per 128, 33 tokens, 31 (25; 2.4 TB/s).

constexpr int kWaves = 8, kThreads = kWaves * 64;
// Blocks of a chunk: as many as leave room for two workgroups' x in a compute unit's LDS.
constexpr int thin_chunk(int mt) { return mt == 1 ? 4 : mt == 2 ? 2 : 1; }

typedef float f32x4_u __attribute__((ext_vector_type(4), aligned(4)));
typedef float f32x2_u __attribute__((ext_vector_type(2), aligned(4)));
// weights' scales are read by scalar loads: the same for a whole wave
typedef const __attribute__((address_space(4))) float constant_float;

// Values b0 .. b0 + U - 1 of a row of n; past its end 0.
template <int U>
__device__ __forceinline__ void load_scales(const float *row, int b0, int n, float v[U])
{
    static_assert(U == 1 || U == 2 || U == 4);
    if (n < U || b0 + U > n) {
#pragma unroll
        for (int i = 0; i < U; ++i)
            v[i] = row[min(b0 + i, n - 1)];
#pragma unroll
        for (int i = 0; i < U; ++i)
            v[i] = b0 + i < n ? v[i] : 0.f;
    } else if constexpr (U == 4) {
        const f32x4_u u = *reinterpret_cast<const f32x4_u *>(row + b0);
        v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
    } else if constexpr (U == 2) {
        const f32x2_u u = *reinterpret_cast<const f32x2_u *>(row + b0);
        v[0] = u.x, v[1] = u.y;
    } else {
        v[0] = row[b0];
    }
}

typedef uint16_t u16x4_u __attribute__((ext_vector_type(4), aligned(2)));

// Group scales (fp16) of blocks b0 .. b0 + U - 1 of a channel of n groups of `gb`
// blocks; past its end 0.
template <int U>
__device__ __forceinline__ void load_group_scales(const uint16_t *row, int b0, int gb, int n, uint16_t v[U])
{
    if (U == 4 && gb == 1 && b0 + U <= n) {
        const u16x4_u u = *reinterpret_cast<const u16x4_u *>(row + b0);
        v[0] = u.x, v[1] = u.y, v[2 % U] = u.z, v[3 % U] = u.w;
    } else {
#pragma unroll
        for (int i = 0; i < U; ++i)
            v[i] = row[min((b0 + i) / gb, n - 1)];
#pragma unroll
        for (int i = 0; i < U; ++i)
            v[i] = (b0 + i) / gb < n ? v[i] : (uint16_t)0;
    }
}

// TERN: ternary weights of experts (G: with group scales).
template <bool TERN, bool G, int MT, int FN>
__global__ void __launch_bounds__(kThreads, FN < 3 ? 4 : 2) thin_kernel(const Fp8Product p, int ks)
{
    constexpr int U = thin_chunk(MT);
    typedef float u_t __attribute__((ext_vector_type(U)));  // scales of a chunk
    // x's chunks, then (once they are done with) the waves' sums
    constexpr int XU4 = U * MT * 128, RU4 = FN * MT * 64;
    __shared__ __attribute__((aligned(16))) u32x4_v sx[kWaves * (XU4 > RU4 ? XU4 : RU4)];
    __shared__ __attribute__((aligned(16))) u_t ss[kWaves][MT][16];
    __shared__ __attribute__((aligned(16))) uint16_t sg[kWaves][G ? U : 1][G ? FN * 16 : 4];
    const int lane = threadIdx.x & 63, g = lane >> 4, col = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nb = p.nb, kpart = wave % ks, parts = kWaves / ks;
    // workgroups run over the channels first: those of one tile of rows are neighbours
    const int ntn = (p.N + 16 * FN * parts - 1) / (16 * FN * parts);
    const int slot = blockIdx.x / ntn, tm = TERN ? p.first + slot : slot;
    const int n0 = ((blockIdx.x - slot * ntn) * parts + wave / ks) * 16 * FN;
    int e = 0, r0 = tm * 16 * MT, r1 = min(p.M, r0 + 16 * MT);
    if constexpr (TERN)
        if (!find_tile<16 * MT>(p.offsets, p.E, p.M, tm, e, r0, r1))
            return;

    // This lane's weights: of channel col of each fragment, chunks like x's, or
    // a ternary slab's 16 bytes at 16 * lane.  (Channels past N repeat the last.)
    const u32x4_v *wp[FN];
#pragma unroll
    for (int i = 0; i < FN; ++i) {
        if constexpr (TERN) {
            const int blocks = (p.N + 15) / 16, blk = min(n0 / 16 + i, blocks - 1);
            wp[i] = reinterpret_cast<const u32x4_v *>(
                        p.w + ((int64_t)e * blocks + blk) * ((nb + 1) / 2) * kTileBytes) + lane;
        } else {
            wp[i] = reinterpret_cast<const u32x4_v *>(p.w + (int64_t)min(n0 + 16 * i + col, p.N - 1) * nb * kFp8Block) + g;
        }
    }
    constexpr int WL = TERN ? U / 2 : 2 * U;  // weight loads of a fragment and chunk
    u32x4_v w[FN][WL];
    auto load_w = [&](int b0) {  // (blocks past the last: the last again)
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int u = 0; u < WL; ++u) {
                if constexpr (TERN)
                    w[i][u] = wp[i][min(b0 / 2 + u, (nb - 1) / 2) * 64];
                else
                    w[i][u] = wp[i][min(b0 + u / 2, nb - 1) * 8 + 4 * (u & 1)];
            }
    };
    load_w(kpart * U);  // on their way while the rows of x are looked up

    // Rows of x.  Lane l loads chunk (l % 8) ^ (l / 8) of row l / 8 of eight rows
    // at a time (the swizzle of the stages below); rows past the last repeat it.
    auto x_row = [&](int r) -> int64_t {
        int64_t row = min(r0 + r, r1 - 1);
        if constexpr (TERN) {
            if (p.order)
                row = p.order[row] / p.top_k;
            row = row < 0 || row >= p.x_rows ? 0 : row;
        }
        return row;
    };
    const int rows = r1 - r0;
    const uint8_t *xp[2 * MT];
#pragma unroll
    for (int q = 0; q < 2 * MT; ++q)
        xp[q] = p.x + x_row(8 * q + (lane >> 3)) * nb * kFp8Block + 16 * ((lane & 7) ^ (lane >> 3));
    // Their scales: lanes 0 .. 15 load a fragment's, for all.
    const float *sp[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j)
        sp[j] = p.x_scale + x_row(16 * j + col) * nb;
    const int cg = first_chunk<TERN>(g);
    const int c0 = cg ^ (col & 7), c1 = (cg + second_chunk(TERN)) ^ (col & 7);
    lds_u4 *const lx = (lds_u4 *)sx + wave * (U * MT * 128);
    const int xa = (col >> 3) * 64 + (col & 7) * 8;
    constant_float *wsp[FN];  // w's scales of each fragment (16 channels are in one block)
#pragma unroll
    for (int i = 0; i < FN; ++i)
        wsp[i] = TERN ? nullptr : (constant_float *)(p.w_scale + (int64_t)(min(n0 + 16 * i, p.N - 1) / kFp8Block) * nb);

    f32x4_t acc[FN][MT];
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j)
            acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    // Blocks past the last load that again, and count with scales of 0 (all of them: 0 times an infinite one is NaN).
    for (int b0 = kpart * U; b0 < nb; b0 += ks * U) {
        float ws[FN][U];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int q = 0; q < 2 * MT; ++q)
                if (8 * q < rows)
                    load_to_lds(xp[q] + min(b0 + u, nb - 1) * kFp8Block, lx + (u * 2 * MT + q) * 64);
        if (lane < 16) {
            float v[MT][U];
#pragma unroll
            for (int j = 0; j < MT; ++j)
                load_scales<U>(sp[j], b0, nb, v[j]);
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                u_t t;
#pragma unroll
                for (int u = 0; u < U; ++u)
                    t[u] = v[j][u];
                ss[wave][j][lane] = t;
            }
        }
        if constexpr (!TERN)
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int u = 0; u < U; ++u)
                    ws[i][u] = b0 + u < nb ? wsp[i][min(b0 + u, nb - 1)] : 0.f;
        if constexpr (G)
            if (lane < 16 * FN) {  // a channel a lane
                uint16_t v[U];
                load_group_scales<U>(p.t_scale + ((int64_t)e * p.N + min(n0 + lane, p.N - 1)) * p.ngroups, b0,
                                     p.group / kFp8Block, p.ngroups, v);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    sg[wave][u][lane] = v[u];
            }
        // x is there once this wave's loads are done: no other wave reads it
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(7 << 4);
        __builtin_amdgcn_wave_barrier();
        u_t xs[MT];
#pragma unroll
        for (int j = 0; j < MT; ++j)
            xs[j] = ss[wave][j][col];
        uint32_t odd[TERN ? FN : 1][2];  // codes of a slab's second block
        f32x4_t gs[FN];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            auto w_operand = [&](int i) -> Wide {
                if constexpr (TERN) {
                    // A slab holds codes 64 q .. 64 q + 63 in lanes 16 q up; exchanging the
                    // halves of a wave (permlane32_swap) leaves a block's codes 0, 64, 32 and 96 (and
                    // 31 more) in its four lane groups.
                    if (u % 2)
                        return widen_codes(odd[i][0], odd[i][1]);
                    const u32x4_v r = w[i][u / 2];
                    const u32x2_v lo = __builtin_amdgcn_permlane32_swap(r.x, r.z, false, false);
                    const u32x2_v hi = __builtin_amdgcn_permlane32_swap(r.y, r.w, false, false);
                    odd[i][0] = lo.y, odd[i][1] = hi.y;
                    return widen_codes(lo.x, hi.x);
                } else {
                    return widen(w[i][2 * u], w[i][2 * u + 1]);
                }
            };
            auto x_at = [&](int j) -> Wide {
                return x_operand<TERN>(lx[(u * MT + j) * 128 + xa + c0], lx[(u * MT + j) * 128 + xa + c1]);
            };
#pragma unroll
            for (int i = 0; i < (G ? FN : 0); ++i) {
                const u32x2_v q = *reinterpret_cast<const u32x2_v *>(&sg[wave][G ? u : 0][16 * i + 4 * g]);
                gs[i] = f32x4_t{channel_scale((uint16_t)q.x), channel_scale((uint16_t)(q.x >> 16)),
                                channel_scale((uint16_t)q.y), channel_scale((uint16_t)(q.y >> 16))};
            }
            // Each fragment becomes fp16 once: the operand with fewer of them stays in registers.
            constexpr bool KEEP_X = MT <= FN;
            constexpr int KEPT = KEEP_X ? MT : FN, TURNS = KEEP_X ? FN : MT;
            Wide kept[KEPT];
#pragma unroll
            for (int k = 0; k < KEPT; ++k)
                kept[k] = KEEP_X ? x_at(k) : w_operand(k);
#pragma unroll
            for (int t = 0; t < TURNS; ++t) {
                const Wide turn = KEEP_X ? w_operand(t) : x_at(t);
                f32x4_t d[KEPT];
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int k = 0; k < KEPT; ++k)
                        d[k] = mfma(KEEP_X ? turn.q[q] : kept[k].q[q], KEEP_X ? kept[k].q[q] : turn.q[q],
                                    q ? d[k] : f32x4_t{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                for (int k = 0; k < KEPT; ++k) {
                    const int i = KEEP_X ? t : k, j = KEEP_X ? k : t;
                    const float f = TERN ? xs[j][u] : xs[j][u] * ws[i][u];
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        acc[i][j][c] += d[k][c] * (G ? f * gs[i][c] : f);
                }
            }
        }
        // (the next chunk's x goes where this one's has been read)
        __builtin_amdgcn_sched_barrier(0);
        if (b0 + ks * U < nb)
            load_w(b0 + ks * U);
    }
    __syncthreads();
    f32x4_t(*const red)[FN * MT][64] = reinterpret_cast<f32x4_t(*)[FN * MT][64]>(sx);
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j)
            red[wave][i * MT + j][lane] = acc[i][j];
    __syncthreads();
    // the waves' sums, in their order: fragment q of wave group q / (FN MT)
    for (int q = wave; q < parts * FN * MT; q += kWaves) {
        const int w0 = q / (FN * MT) * ks, fr = q % (FN * MT), i = fr / MT, j = fr % MT;
        f32x4_t s = red[w0][fr][lane];
        for (int w = 1; w < ks; ++w)
            s += red[w0 + w][fr][lane];
        const int row = r0 + 16 * j + col;
        const int ch = ((blockIdx.x - slot * ntn) * parts + q / (FN * MT)) * 16 * FN + 16 * i + 4 * g;
        if (row >= r1)
            continue;
        if constexpr (TERN && !G)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                s[k] *= channel_scale(p.t_scale[(int64_t)e * p.N + min(ch + k, p.N - 1)]);
        put4(p, row, ch, s);
    }
}

// Most threads of a launch, and `tiles` tiles of rows in launches of at most `most` each.
constexpr int64_t kMostThreads = (int64_t)1 << 31;
template <class F>
hipError_t launch_pieces(const Fp8Product &p, int64_t tiles, int64_t most, F launch)
{
    hipError_t e = hipSuccess;
    for (int64_t t = 0; t < tiles && e == hipSuccess; t += most) {
        Fp8Product part = p;
        part.first = (int)t;
        launch(part, tiles - t < most ? tiles - t : most);
        e = hipGetLastError();
    }
    return e;
}

// ks: ways to share K.  Each wave should have a chunk of its own, and the more
// channels a workgroup holds the fewer there are, so no more ways than chunks.
template <bool TERN, bool G, int MT, int FN>
hipError_t launch_thin(const Fp8Product &p, int64_t tiles, hipStream_t stream)
{
    constexpr int U = thin_chunk(MT);
    const int chunks = (p.nb + U - 1) / U;
    const int ks = chunks >= 8 ? 8 : chunks >= 4 ? 4 : chunks >= 2 ? 2 : 1;
    const int64_t ntn = (p.N + 16 * FN * (kWaves / ks) - 1) / (16 * FN * (kWaves / ks));
    // 8-bit weights: a tile of at most 48 rows, or up to 2^18 tiles of few channels: one launch
    return launch_pieces(p, tiles, TERN ? kMostThreads / kThreads / ntn : tiles, [&](const Fp8Product &part, int64_t n) {
        hipLaunchKernelGGL((thin_kernel<TERN, G, MT, FN>), dim3((unsigned)(n * ntn)), dim3(kThreads), 0, stream, part, ks);
    });
}

// Fragments of 16 channels a wave holds, 17 to 48 rows: F with the fewest rounds of F over the
// compute units, the larger of two (it reads x less often).  us, 45 rows (F = 1 to 5): 18944 x 4096
// 27.2, 26.3, 25.5, 29.6, 21.0; 16384 x 4096 23.0, 19.9, 24.8, 18.5, 20.0; 12288 x 4096 18.6, 18.9, 14.9,
// 17.0, 18.9; 8192 x 2048 8.3, 7.6, 8.7, 10.2, 11.0; 4096 x 4096 8.5, 10.6, 13.3, 15.2, 17.3.  Up to 16 rows a chunk
// is long, two workgroups share a compute unit and F = 1 is the best or near it (8 rows, F = 1 to 3: 18944 x 4096
// 19.5, 20.7, 20.0; 12288 x 4096 12.8, 12.4, 11.4; 8192 x 2048 5.8, 7.9, 9.9; 1024 x 8192 7.4, 12.6, 16.8).  64 rows: F = 1 where
// that is one round (4096 x 4096: 10.2, with 2 12.2), else 2 (18944 x 4096: 1 34.0, 2 29.3, 3 29.3; 128 rows of 4096 x
// 4096 16.7, 12.7, 15.9; 12288 x 4096 22.9, 21.2, 17.2, but 192 rows of 4096 x 1024 9.3, 8.5, 12.9).  Experts: F = 1 below 1024
// fragments (1 token, 8 of 16 of 1024 x 2048: 5.2, with 2 5.9; of 128 of 512 x 2048 5.5 and 6.4), else 2 (8 of 64 of 2048 x 4096
// 12.1 and 8.7; 16 tokens 66.8 and 44.4).
inline int thin_fragments(int64_t frags)
{
    const int64_t cus = device_cus();
    int best = 1;
    int64_t least = INT64_MAX;
    for (int f = 1; f <= 5; ++f) {
        const int64_t rounds = (frags + f * cus - 1) / (f * cus) * f;
        if (rounds <= least)
            least = rounds, best = f;
    }
    return best;
}

// Rows in tiles of 16 MT.
template <bool TERN, bool G, int MT>
hipError_t launch_thin(const Fp8Product &p, int64_t tiles, hipStream_t stream)
{
    const int64_t frags = (p.N + 15) / 16 * tiles;
    if constexpr (TERN) {
        return frags < 1024 ? launch_thin<TERN, G, MT, 1>(p, tiles, stream)
                            : launch_thin<TERN, G, MT, 2>(p, tiles, stream);
    } else if constexpr (MT == 1) {
        return launch_thin<TERN, G, MT, 1>(p, tiles, stream);
    } else if constexpr (MT == 4) {
        return frags <= device_cus() ? launch_thin<TERN, G, MT, 1>(p, tiles, stream)
                                     : launch_thin<TERN, G, MT, 2>(p, tiles, stream);
    } else {
        switch (thin_fragments(frags)) {
        case 1: return launch_thin<TERN, G, MT, 1>(p, tiles, stream);
        case 2: return launch_thin<TERN, G, MT, 2>(p, tiles, stream);
        case 3: return launch_thin<TERN, G, MT, 3>(p, tiles, stream);
        case 4: return launch_thin<TERN, G, MT, 4>(p, tiles, stream);
        default: return launch_thin<TERN, G, MT, 5>(p, tiles, stream);
        }
    }
}

// ---------------------------------------------------------------- many rows

// Measured (bf16 outputs; calls one after another): 2048 rows of 18944 x 4096 285 to 290 us (1.1
// PFLOP/s; 183 with the 8-bit matrix instruction and its sums), the matrix unit busy for 58 % of the compute units' cycles; 64
// experts of 2048 x 4096, 8 a token, 2047 tokens, 288 to 300 us (0.93 PFLOP/s; 205), busy for 51 %.  Parts
// left out in turn (experts in tiles of 64 places, 308): without the conversions to fp16 265 and 235, without the scaling 268 and 291,
// without either 250 and 230, at which the matrix unit's own rate is near (1.38 PFLOP/s in a bf16 library product).  Tiles of 256
// channels x 128 rows took 296, of 128 x 256 301.

// Tiles of TN channels x TM rows by WN x WM waves.
template <int TN_, int TM_, int WN_, int WM_>
struct Tile {
    static constexpr int TN = TN_, TM = TM_, WN = WN_, WM = WM_;
    static constexpr int THREADS = WN * WM * 64;
    static constexpr int FN = TN / WN / 16, FM = TM / WM / 16;  // fragments of a wave
    // Waves that a SIMD has registers for.  (With 512 registers a wave the compiler puts matrix results where
    // vector instructions have to fetch them from: 310 instead of 290 us at 2048 x 18944 x 4096.)
    static constexpr int WAVES = 2;
};

// Values b0 .. b0 + 3 of a row of n (past its end the last) that a whole workgroup reads.
__device__ __forceinline__ f32x4_t load_scales_uniform(const float *row, int b0, int n)
{
    constant_float *r = (constant_float *)row;
    return f32x4_t{r[min(b0, n - 1)], r[min(b0 + 1, n - 1)], r[min(b0 + 2, n - 1)], r[min(b0 + 3, n - 1)]};
}

// G: group-scaled ternary weights.
template <bool TERN, bool G, class C>
__global__ void __launch_bounds__(C::THREADS, C::WAVES) tile_kernel(const Fp8Product p)
{
    constexpr int TN = C::TN, TM = C::TM, FN = C::FN, FM = C::FM, THREADS = C::THREADS;
    constexpr int XI = TM * 8 / THREADS;                      // x loads of a thread and stage
    constexpr int WCH = TERN ? TN * 2 : TN * 8;               // 16-byte chunks of w in a stage
    constexpr int WI = (WCH + THREADS - 1) / THREADS;
    constexpr int QB = TERN ? 1 : (TN + 127) / 128;           // blocks of channels with scales of their own
    static_assert(TM * 8 % THREADS == 0 && (WCH % THREADS == 0 || WI == 1) && TM <= THREADS && TN <= THREADS);
    // One object per stage (x, then w): a load into one stage is then known not to
    // touch the others.
    constexpr int STAGE = TM * 8 + WCH;
    __shared__ __attribute__((aligned(16))) u32x4_v st0[STAGE], st1[STAGE];
    lds_u4 *const lx[2] = {(lds_u4 *)st0, (lds_u4 *)st1};
    lds_u4 *const lw[2] = {lx[0] + TM * 8, lx[1] + TM * 8};
    // Scales of eight steps: x's (times w's for 8-bit weights), a lane's FM rows
    // together, then a group's channels', a lane's FN fragments together.  They are read
    // and written right behind the waves' meeting: the compiler waits for every load into
    // LDS that is under way before it touches an object that none of them writes.
    typedef float fm_t __attribute__((ext_vector_type(FM)));
    constexpr int SF = QB * TM, SL = SF + (G ? TN : 0);
    __shared__ __attribute__((aligned(16))) float sf[8 * SL];

    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, col = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave % C::WN, wm = wave / C::WN;
    const int nb = p.nb;
    // Workgroup b runs on XCD b % 8 (each has an L2 of its own).  Dense: an XCD takes a
    // run of tiles, eight row tiles of a channel tile after the other, so that its 32 or
    // so workgroups at a time share 8 x tiles and a few w tiles, and w is read by one XCD
    // per eight row tiles.  Experts: it takes every eighth row tile (how many there are is only known
    // here), its channel tiles one after the other.
    const int ntn = (p.N + TN - 1) / TN;
    const int xcd = blockIdx.x & 7, slot = blockIdx.x >> 3;
    int tm, tn;
    if constexpr (TERN) {
        tm = p.first + slot / ntn * 8 + xcd;
        tn = slot % ntn;
    } else {
        const int ntm = (p.M + TM - 1) / TM;
        const int64_t tiles = (int64_t)ntm * ntn;
        const int64_t t = tiles * xcd / 8 + slot;
        if (t >= tiles * (xcd + 1) / 8)
            return;
        const int64_t band = (int64_t)8 * ntn;
        const int m0 = (int)(t / band) * 8, rows = min(8, ntm - m0), in = (int)(t % band);
        tm = m0 + in % rows;
        tn = in / rows;
    }
    const int n0 = tn * TN;
    int e = 0, r0 = tm * TM, r1 = min(p.M, r0 + TM);
    if constexpr (TERN)
        if (!find_tile<TM>(p.offsets, p.E, p.M, tm, e, r0, r1))
            return;

    auto x_row = [&](int r) -> int64_t {  // row of x of the tile's row r
        int64_t row = min(r0 + r, r1 - 1);
        if constexpr (TERN) {
            if (p.order)
                row = p.order[row] / p.top_k;
            row = row < 0 || row >= p.x_rows ? 0 : row;
        }
        return row;
    };
    // Sources (rows and channels past the last repeat it).  Gathered rows of x and the
    // experts' blocks have pointers of their own, a dense tile is one resource
    // with 32-bit offsets.
    constexpr int RS = THREADS / 8;        // rows between a thread's chunks of x
    const int rowbytes = nb * kFp8Block;   // at most 2^20
    static_assert(RS % 8 == 0, "the same chunk of each row");
    const uint8_t *xsrc[XI], *wsrc = nullptr;
    int xoff[XI], woff[WI];
    __amdgpu_buffer_rsrc_t xr, wr;
    if constexpr (TERN) {
#pragma unroll
        for (int i = 0; i < XI; ++i)
            xsrc[i] = p.x + x_row((tid >> 3) + i * RS) * rowbytes + 16 * ((tid & 7) ^ swz(tid >> 3));
        // 32 chunks of a block of 16 channels are a half slab, consecutive in memory
        static_assert(!TERN || WI == 1);
        const int blk = min(n0 / 16 + (tid >> 5), (p.N + 15) / 16 - 1);
        wsrc = p.w + ((int64_t)e * ((p.N + 15) / 16) + blk) * ((nb + 1) / 2) * kTileBytes + 16 * (tid & 31);
    } else {
        const int rows = r1 - r0, chans = min(TN, p.N - n0);
        xr = make_rsrc(p.x + (int64_t)r0 * rowbytes, (uint32_t)(rows * rowbytes));
#pragma unroll
        for (int i = 0; i < XI; ++i)
            xoff[i] = min((tid >> 3) + i * RS, rows - 1) * rowbytes + 16 * ((tid & 7) ^ swz(tid >> 3));
        wr = make_rsrc(p.w + (int64_t)n0 * rowbytes, (uint32_t)(chans * rowbytes));
#pragma unroll
        for (int i = 0; i < WI; ++i)
            woff[i] = min((tid >> 3) + i * RS, chans - 1) * rowbytes + 16 * ((tid & 7) ^ swz(tid >> 3));
    }
    const float *fsrc = p.x_scale + (tid < TM ? x_row(tid) : 0) * nb;
    const uint16_t *gsrc = G ? p.t_scale + ((int64_t)e * p.N + min(n0 + tid, p.N - 1)) * p.ngroups : nullptr;
    const int gsteps = G ? p.group / kFp8Block : 1;

    // One of the NP loads into a stage that a thread issues for step b.
    constexpr int NP = XI + WI;
    auto issue = [&](auto S, int b, int q) {
        constexpr int s = decltype(S)::value;
        if (q < XI) {
            lds_u4 *to = lx[s] + q * THREADS + wave * 64;
            if constexpr (TERN)
                load_to_lds(xsrc[q < XI ? q : 0] + b * kFp8Block, to);
            else
                load_to_lds(xr, to, xoff[q < XI ? q : 0], b * kFp8Block);
        } else {
            const int i = q - XI;
            lds_u4 *to = lw[s] + i * THREADS + wave * 64;
            if constexpr (!TERN)
                load_to_lds(wr, to, woff[q >= XI ? i : 0], b * kFp8Block);
            else if (WCH % THREADS == 0 || wave * 64 < WCH)
                load_to_lds(wsrc + (int64_t)b * (kTileBytes / 2), to);
        }
    };
    // The scales of four steps in registers (a row of x, and a channel, a thread).
    // (Group scales as loaded: a conversion here would wait for them, and with them
    // for all loads before.)
    struct Factors {
        f32x4_t x, w[QB];
        uint32_t g[4];
    };
    auto load_factors = [&](int b0) -> Factors {
        Factors r = {};
        if (wave < TM / 64 && b0 < nb) {
            float v[4];
            load_scales<4>(fsrc, b0, nb, v);
            r.x = f32x4_t{v[0], v[1], v[2], v[3]};
        }
        if constexpr (!TERN)
#pragma unroll
            for (int q = 0; q < QB; ++q)
                r.w[q] = load_scales_uniform(p.w_scale + (int64_t)min(n0 / 128 + q, (p.N - 1) / 128) * nb, b0, nb);
        if constexpr (G)
            if (wave < TN / 64) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    r.g[i] = gsrc[min((b0 + i) / gsteps, p.ngroups - 1)];
            }
        return r;
    };
    // row r = 16 (FM u + j) + c of the tile: entry j of (u, c)
    const int fpos = ((tid / (16 * FM)) * 16 + (tid & 15)) * FM + (tid >> 4) % FM;
    // channel 16 (FN u + i) + 4 g + k: entry 4 i + k of (u, g)
    const int gpos = ((tid / (16 * FN)) * 4 + (tid >> 2) % 4) * 4 * FN + (tid >> 4) % FN * 4 + tid % 4;
    auto store_factors = [&](const Factors &r, int b0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (wave < TM / 64)
#pragma unroll
                for (int q = 0; q < QB; ++q)
                    sf[((b0 + i) & 7) * SL + q * TM + fpos] = TERN ? r.x[i] : r.x[i] * r.w[q][i];
            if constexpr (G)
                if (wave < TN / 64)
                    sf[((b0 + i) & 7) * SL + SF + gpos] = channel_scale((uint16_t)r.g[i]);
        }
    };
    Factors next;

    f32x4_t acc[FN][FM];
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j)
            acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
    // Ternary: the codes of two fragments come by one load, 16 bytes of the first
    // fragment's in lanes 0 .. 31, of the second's in the others; exchanging the halves of
    // each (permlane32_swap) leaves a fragment with the codes 0, 64, 32 and 96 (and 31 more)
    // in its lane groups.
    static_assert(!TERN || FN % 2 == 0);
    const int xa = (wm * FM * 16 + col) * 8, cg = first_chunk<TERN>(g);
    const int c0 = cg ^ swz(col), c1 = (cg + second_chunk(TERN)) ^ swz(col);
    const int wa = TERN ? wn * FN * 32 + lane : (wn * FN * 16 + col) * 8;

    // Operands on their way from LDS: w's two fragments ahead (ternary: two
    // fragments by one load), all of x's, and the scales.
    u32x4_v rw[2][2], rx[FM][2];
    fm_t fn, f, fp;          // the next step's, this step's, the last one's
    // The matrix results of this fragment and of the one before, which are scaled behind this one's
    // matrix instructions: they are there by then.
    f32x4_t d[2][FM];
    typedef float g_t __attribute__((ext_vector_type(G ? 4 * FN : 4)));
    g_t gn, gs;  // its channels' scales: the next step's, this step's,
    f32x4_t gp;  // the last one's last fragment's
    auto read_w = [&](auto S, int i) {
        constexpr int s = decltype(S)::value;
        if constexpr (TERN) {
            if (i % 2 == 0)
                rw[0][0] = lw[s][wa + i * 32];
        } else {
            rw[i & 1][0] = lw[s][wa + i * 128 + c0];
            rw[i & 1][1] = lw[s][wa + i * 128 + c1];
        }
    };
    auto read_x = [&](auto S, int j) {
        constexpr int s = decltype(S)::value;
        rx[j][0] = lx[s][xa + j * 128 + c0];
        rx[j][1] = lx[s][xa + j * 128 + c1];
    };
    auto read_f = [&](int b) {
        fn = *reinterpret_cast<const fm_t *>(
            sf + (b & 7) * SL + (TERN ? 0 : (wn * FN * 16) / 128 * TM) + (wm * 16 + col) * FM);
        if constexpr (G)
            gn = *reinterpret_cast<const g_t *>(sf + (b & 7) * SL + SF + (wn * 4 + g) * 4 * FN);
    };
    u32x2_v odd_codes = {0, 0};  // of the second fragment of two
    auto w_operand = [&](int i) -> Wide {
        if constexpr (TERN) {
            u32x2_v w = odd_codes;
            if (i % 2 == 0) {
                const u32x4_v r = rw[0][0];
                const u32x2_v lo = __builtin_amdgcn_permlane32_swap(r.x, r.z, false, false);
                const u32x2_v hi = __builtin_amdgcn_permlane32_swap(r.y, r.w, false, false);
                w = u32x2_v{lo.x, hi.x};
                odd_codes = u32x2_v{lo.y, hi.y};
            }
            return widen_codes(w.x, w.y);
        } else {
            return widen(rw[i & 1][0], rw[i & 1][1]);
        }
    };
    // Value k of result j of fragment i of this step, or (i = -1) of the last one of the step before.
    auto scale_add = [&](int i, int j, int k) {
        const int c = i < 0 ? FN - 1 : i;
        const float by = i < 0 ? fp[j] : f[j];
        acc[c][j][k] += d[c & 1][j][k] * (G ? by * (i < 0 ? gp[k] : gs[G ? 4 * c + k : 0]) : by);
    };

    // Step b, from stage s.  A fragment is four matrix instructions a row fragment, by turns; each is
    // followed by the scaling of a value of the fragment before, so that neither waits for the other.
    // x's fragments become fp16 once a step, in front of their first instruction.  The
    // waves meet two fragments before the end, once the stage is read and the next one is there:
    // from then on this stage takes step b + 2, its loads spread over the instructions (issued
    // together they hold up the waves, whose turns in the load unit come one after another), and
    // the next step's first operands are read behind the last fragments' matrix instructions.
    auto step = [&](auto S, int b) {
        constexpr int s = decltype(S)::value;
        constexpr std::integral_constant<int, 1 - s> T;  // the next step's stage
        static_assert(FN % 2 == 0 && FN >= 4);
        Wide x[FM];
        fp = f;
        f = fn;
        if constexpr (G)
            gp = f32x4_t{gs[G ? 4 * FN - 4 : 0], gs[G ? 4 * FN - 3 : 0], gs[G ? 4 * FN - 2 : 0], gs[G ? 4 * FN - 1 : 0]};
        gs = gn;
#pragma unroll
        for (int i = 0; i < FN; ++i) {
            const Wide a = w_operand(i);
            if (i == FN - 2) {
                meet();
                read_f(b + 1);
                // scales ahead: loaded at the first step of four, put into LDS at the third
                if constexpr (s == 0) {
                    if (b & 2)
                        store_factors(next, b + 2);
                    else
                        next = load_factors(b + 4);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int j = 0; j < FM; ++j) {
                    if (i == 0 && q == 0)
                        x[j] = x_operand<TERN>(rx[j][0], rx[j][1]);
                    asm volatile("" : "+v"(x[j].q[q]));  // (nothing: keeps the instruction from moving up)
                    d[i & 1][j] = mfma(a.q[q], x[j].q[q], q ? d[i & 1][j] : zero);
                    if (i == FN - 1 && q == 3)
                        read_x(T, j);
                    scale_add(i - 1, j, q);
                    constexpr int SLOTS = 8 * FM;  // instructions of the last two fragments
                    const int slot = (i - (FN - 2)) * 4 * FM + q * FM + j;
#pragma unroll
                    for (int n = 0; n < NP; ++n)
                        if (i >= FN - 2 && slot == n * SLOTS / NP)
                            issue(S, min(b + 2, nb - 1), n);
                    asm volatile("" : "+v"(acc[i ? i - 1 : FN - 1][j]));  // (the same, down)
                    __builtin_amdgcn_sched_barrier(0);
                }
            if (i + 2 < FN)
                read_w(S, i + 2);
            else
                read_w(T, i + 2 - FN);
        }
    };

    // Every step loads a stage for two steps on; the last ones load the last step
    // again, into a stage that is not read (a branch there, or a second exit of the loop, had
    // the compiler copy the step).
    auto fill = [&](auto S) {
        constexpr int s = decltype(S)::value;
#pragma unroll
        for (int q = 0; q < NP; ++q)
            issue(S, min(s, nb - 1), q);
    };
    fill(std::integral_constant<int, 0>());
    next = load_factors(0);
    store_factors(next, 0);
    meet();
    fill(std::integral_constant<int, 1>());
    read_w(std::integral_constant<int, 0>(), 0);
    read_w(std::integral_constant<int, 0>(), 1);
    read_f(0);
#pragma unroll
    for (int j = 0; j < FM; ++j) {
        read_x(std::integral_constant<int, 0>(), j);
        f[j] = 0.f;
        d[1][j] = zero;  // (as a last fragment of a step before)
    }
    gs = 0.f;
    gp = zero;
    if constexpr (!G)
        gn = 0.f;
    int b = 0;
    for (; b + 2 <= nb; b += 2) {
        step(std::integral_constant<int, 0>(), b);
        step(std::integral_constant<int, 1>(), b + 1);
    }
    if (b < nb)
        step(std::integral_constant<int, 0>(), b);
#pragma unroll
    for (int j = 0; j < FM; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k)
            scale_add(FN - 1, j, k);
    meet();  // no load into LDS outlives the workgroup

#pragma unroll
    for (int i = 0; i < FN; ++i) {
        const int ch = n0 + (wn * FN + i) * 16 + 4 * g;
        f32x4_t cs = {1.f, 1.f, 1.f, 1.f};
        if constexpr (TERN && !G)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                cs[k] = channel_scale(p.t_scale[(int64_t)e * p.N + min(ch + k, p.N - 1)]);
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            const int row = r0 + (wm * FM + j) * 16 + col;
            if (row < r1)
                put4(p, row, ch, TERN && !G ? acc[i][j] * cs : acc[i][j]);
        }
    }
}

template <bool TERN, class C>
hipError_t launch_tiles(const Fp8Product &p, int64_t tiles, hipStream_t stream)
{
    const int ntn = (p.N + C::TN - 1) / C::TN;
    if constexpr (TERN) {
        // (whole eights of tiles a launch: tile t runs on XCD t % 8)
        return launch_pieces(p, tiles, kMostThreads / C::THREADS / ntn & ~(int64_t)7, [&](const Fp8Product &part, int64_t n) {
            const dim3 grid((unsigned)((n + 7) / 8 * 8 * ntn));
            if (p.group)
                hipLaunchKernelGGL((tile_kernel<true, true, C>), grid, dim3(C::THREADS), 0, stream, part);
            else
                hipLaunchKernelGGL((tile_kernel<true, false, C>), grid, dim3(C::THREADS), 0, stream, part);
        });
    } else {
        const int64_t wgs = (tiles * ntn + 7) / 8 * 8;
        if (wgs * C::THREADS > UINT32_MAX)
            return hipErrorInvalidValue;  // (an output of more than 2^37 elements)
        hipLaunchKernelGGL((tile_kernel<false, false, C>), dim3((unsigned)wgs), dim3(C::THREADS), 0, stream, p);
        return hipGetLastError();
    }
}

// Tiles of `rows` places that E experts of R places in all can need.
int64_t expert_tiles(const Fp8Product &p, int rows)
{
    return p.M / rows + (p.M < p.E ? p.M : p.E);
}

// Expected time of n tiles in rounds of `most`, as a multiple of a round's: between
// whole rounds and an even spread.
double rounds_of(int64_t n, int64_t most)
{
    return ((double)((n + most - 1) / most) + (n > most ? (double)n / most : 1.0)) / 2;
}

// Row tiles of `rows` that R places of E experts are expected to need: an expert's last is half full.
int64_t likely_tiles(const Fp8Product &p, int rows)
{
    const int64_t most = p.M < p.E ? p.M : p.E, n = p.M / rows + most / 2;
    return n > most ? n : most;
}

}  // namespace

// Which kernel: the least of what each is expected to take (us), fitted to times over M = 64 .. 4096 at
// 18944, 16384, 12288, 4096 and 256 x 4096, 1024 x 8192, 8192 x 2048 and 4096 x 1024; what it
// chose there was at most 7 % over the best.  Streamed, tiles of 64 rows and of 128, us: 64 rows of 4096 x 4096 10.2, 24.1 and 35.0; of
// 18944 x 4096 29.3, 25.5 and 35.9; 192 rows of 1024 x 8192 13.9, 43.8 and 64.3; 384 rows of 18944 x 4096 (tiles) 70.9
// and 59.4; 2048 rows 322 and 289; 4096 rows of 256 x 4096 26.8, 25.0 and 35.6.  Four stages of 64 rows instead of two were slower
// at every one of them (64 rows of 18944 x 4096 26.3, 192 rows 50.6 against 37.4).
hipError_t launch_fp8_linear(const Fp8Product &p, hipStream_t stream)
{
    if (p.M <= 16)
        return launch_thin<false, false, 1>(p, 1, stream);
    if (p.M <= 32)
        return launch_thin<false, false, 2>(p, 1, stream);
    if (p.M <= 48)
        return launch_thin<false, false, 3>(p, 1, stream);
    const int64_t cus = device_cus(), m64 = (p.M + 63) / 64, m128 = (p.M + 127) / 128;
    const int64_t n128 = ((int64_t)p.N + 127) / 128, frags = m64 * (((int64_t)p.N + 15) / 16);
    const double t_thin = 1.0 + (frags <= cus ? 0.24 * p.nb : (1.2 + 0.28 * p.nb) * rounds_of((frags + 1) / 2, cus));
    const double t_64 = 3.0 + p.nb * (m64 * n128 <= cus ? 0.66 : 1.06 * rounds_of(m64 * n128, 2 * cus));
    const double t_128 = 5.0 + p.nb * (m128 * n128 <= cus ? 0.93 : 1.75 * rounds_of(m128 * n128, 2 * cus));
    if (t_thin <= t_64 && t_thin <= t_128)
        return launch_thin<false, false, 4>(p, m64, stream);
    if (t_64 <= t_128)
        return launch_tiles<false, Tile<128, 64, 2, 2>>(p, m64, stream);
    return launch_tiles<false, Tile<128, 128, 2, 2>>(p, m128, stream);
}

// Likewise: streamed, K shared by eight waves, or tiles of 64 or 128 places; the latter from 112 places an
// expert on (with fewer an expert's only tile is seldom full).  Fitted at 64 experts of 2048 x 4096 and 4096 x 1024 (scales per
// 128), 16 of 1024 x 2048 and 128 of 512 x 2048 (per 128), 8 a token, 1 to 2047 tokens; at most 6 % over the best there.  us,
// streamed, 64 and 128: 2048 x 4096 at 16 tokens 44, 71 and 113, 100 68, 74 and 115, 128 78, 75 and 116, 1024 (tiles) 201 and 178, 2047
// 335 and 295; 4096 x 1024 at 128 46, 48 and 75, 192 58, 52 and 77, 2047 219 and 192; 16 of 1024 x 2048 at 64 12, 17 and 24.
hipError_t launch_linear_experts(const Fp8Product &p, hipStream_t stream)
{
    const int64_t cus = device_cus(), n128 = ((int64_t)p.N + 127) / 128;
    const int64_t t64 = likely_tiles(p, 64) * n128, t128 = likely_tiles(p, 128) * n128;
    const bool group = p.group != 0;
    const double t_thin = 3.0 + p.nb * (group ? 0.23 : 0.20) * likely_tiles(p, 16) * p.N / 32 / (2 * cus);
    const double t_64 = 3.0 + p.nb * (t64 <= cus ? 0.84 : (group ? 1.45 : 1.15) * rounds_of(t64, 2 * cus));
    const double t_128 = 5.0 + p.nb * (t128 <= cus ? 1.1 : (group ? 2.3 : 1.85) * rounds_of(t128, 2 * cus));
    const bool full = p.M >= 112 * (int64_t)p.E;
    if (t_thin <= t_64 && (t_thin <= t_128 || !full))
        return group ? launch_thin<true, true, 1>(p, expert_tiles(p, 16), stream)
                     : launch_thin<true, false, 1>(p, expert_tiles(p, 16), stream);
    if (t_64 <= t_128 || !full)
        return launch_tiles<true, Tile<128, 64, 2, 2>>(p, expert_tiles(p, 64), stream);
    return launch_tiles<true, Tile<128, 128, 2, 2>>(p, expert_tiles(p, 128), stream);
}

}  // namespace ternary
