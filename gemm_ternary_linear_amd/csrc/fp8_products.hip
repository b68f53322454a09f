// Products of 8-bit activations on gfx950: with 8-bit weights (a scale per
// block of 128 x 128), and with the ternary weights of experts.
//
//     y[m, n] = sum_b xs[m, b] s(n, b) sum_{k in b} x[m, k] w[n, k]
//
// One v_mfma_scale_f32_16x16x128_f8f6f4 multiplies 16 channels (the A operand)
// by 16 rows of x (B) over one block of 128; its fp32 sums are then scaled and
// added to the running sums, so no rounding but fp32's happens before the end.
// A lane's four results are four channels of one row: the row's scale is one
// register and the four go out in one store.  Ternary codes become fp4 (+-2,
// halved by the instruction's A scale) in five vector operations a 16 codes;
// as those give a word's odd codes, then its even ones, x's bytes are put in the
// same order (eight byte permutes per 16 rows x 128).  Lane group g (lanes 16 g
// up) holds k = 32 g .. 32 g + 31 of a block of an fp4 operand, and k = 16 g .. and
// 64 + 16 g .. (16 each) of an fp8 one.
#include "fp8_common.h"
#include "internal.h"

namespace ternary {

namespace {

constexpr int kFp8 = 0, kFp4 = 4;      // operand types of the matrix instruction
constexpr int kOne = 127, kHalf = 126;  // its E8M0 scales

// Places [r0, r1) of expert e that the idx-th tile of BM rows covers (tiles run
// expert by expert); false past the last.  Every lane of a wave calls it.
template <int BM>
__device__ __forceinline__ bool find_tile(const int32_t *offsets, int E, int R, int idx, int &e,
                                          int &r0, int &r1)
{
    const int lane = threadIdx.x & 63, per = (E + 63) / 64, lo = lane * per;
    int mine = 0;
    for (int i = 0; i < per; ++i)
        if (lo + i < E) {
            const int a = max(offsets[lo + i], 0), b = min(offsets[lo + i + 1], R);
            mine += b > a ? (b - a + BM - 1) / BM : 0;
        }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(incl, o);
        incl += lane >= o ? u : 0;
    }
    const uint64_t over = __builtin_amdgcn_ballot_w64(incl > idx);
    if (!over)
        return false;
    const int from = __builtin_ctzll(over);
    int left = idx - __shfl(incl - mine, from);
    for (int i = 0; i < per; ++i) {
        const int x = from * per + i;
        if (x >= E)
            break;
        const int a = max(offsets[x], 0), b = min(offsets[x + 1], R);
        const int tiles = b > a ? (b - a + BM - 1) / BM : 0;
        if (left >= 0 && left < tiles) {
            e = x;
            r0 = a + left * BM;
            r1 = min(b, r0 + BM);
            return true;
        }
        left -= tiles;
    }
    return false;
}

// 16 codes (one word) -> the fp4 words of its odd and of its even codes (the
// field (b1 b0) becomes (sign, magnitude) = (b1, b0 ^ b1) at a nibble's top).
__device__ __forceinline__ void codes_to_fp4(uint32_t w, int &odd, int &even)
{
    const uint32_t z = __builtin_amdgcn_bitop3_b32(w, w >> 1, 0x55555555u, 0x78);
    odd = (int)(z & 0xccccccccu);
    even = (int)((z << 2) & 0xccccccccu);
}

// 32 bytes of x in the order of the fp4 operand: per 16, odd then even.
__device__ __forceinline__ i32x8_v odd_even(u32x4_v a, u32x4_v b)
{
    i32x8_v r;
    r[0] = (int)__builtin_amdgcn_perm(a.y, a.x, 0x07050301u);
    r[1] = (int)__builtin_amdgcn_perm(a.w, a.z, 0x07050301u);
    r[2] = (int)__builtin_amdgcn_perm(a.y, a.x, 0x06040200u);
    r[3] = (int)__builtin_amdgcn_perm(a.w, a.z, 0x06040200u);
    r[4] = (int)__builtin_amdgcn_perm(b.y, b.x, 0x07050301u);
    r[5] = (int)__builtin_amdgcn_perm(b.w, b.z, 0x07050301u);
    r[6] = (int)__builtin_amdgcn_perm(b.y, b.x, 0x06040200u);
    r[7] = (int)__builtin_amdgcn_perm(b.w, b.z, 0x06040200u);
    return r;
}

__device__ __forceinline__ i32x8_v join(u32x4_v a, u32x4_v b)
{
    return i32x8_v{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}

constexpr int kWaves = 4, kThreads = kWaves * 64;

// A workgroup computes 16 channels x 16 MT rows; its waves share the K blocks
// out and meet in LDS.  Operands go straight from memory to registers.
template <bool TERN, int MT, int DT>
__global__ void __launch_bounds__(kThreads) stream_kernel(const Fp8Product p)
{
    __shared__ f32x4_t red[kWaves][MT][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, col = lane & 15;
    const int n0 = blockIdx.x * 16, nb = p.nb;
    int e = 0, r0 = blockIdx.y * 16 * MT, r1 = min(p.M, r0 + 16 * MT);
    if constexpr (TERN)
        if (!find_tile<16 * MT>(p.offsets, p.E, p.M, blockIdx.y, e, r0, r1))
            return;

    // this lane's row of x in each fragment (rows past the last repeat it; their
    // results are not stored)
    const uint8_t *xp[MT];
    const float *sp[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) {
        int64_t row = min(r0 + 16 * j + col, r1 - 1);
        if constexpr (TERN)
            if (p.order)
                row = p.order[row] / p.top_k;
        if constexpr (TERN)
            row = row < 0 || row >= p.x_rows ? 0 : row;
        xp[j] = p.x + row * nb * kFp8Block;
        sp[j] = p.x_scale + row * nb;
    }
    const int n = min(n0 + col, p.N - 1);  // this lane's channel of A
    const uint8_t *wp;
    if constexpr (TERN)
        wp = p.w + ((int64_t)e * ((p.N + 15) / 16) + blockIdx.x) * ((nb + 1) / 2) * kTileBytes;
    else
        wp = p.w + (int64_t)n * nb * kFp8Block;

    f32x4_t acc[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j)
        acc[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};

    for (int b = wave; b < nb; b += kWaves) {
        i32x8_v a;
        float ws[4] = {1.f, 1.f, 1.f, 1.f};
        if constexpr (TERN) {
            // lane group g: codes 32 g .. 32 g + 31 of the block
            const u32x2_v w = *reinterpret_cast<const u32x2_v *>(
                wp + (b >> 1) * kTileBytes + ((b & 1) * 2 + (g >> 1)) * 256 + col * 16 + (g & 1) * 8);
            int f[4];
            codes_to_fp4(w.x, f[0], f[1]);
            codes_to_fp4(w.y, f[2], f[3]);
            a = i32x8_v{f[0], f[1], f[2], f[3], 0, 0, 0, 0};
            if (p.group) {
                const int gi = (int)((int64_t)b * kFp8Block / p.group);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    ws[i] = f16_bits_to_f32(
                        p.t_scale[((int64_t)e * p.N + min(n0 + 4 * g + i, p.N - 1)) * p.ngroups + gi]);
            }
        } else {
            const u32x4_v *w = reinterpret_cast<const u32x4_v *>(wp + b * kFp8Block + 16 * g);
            a = join(w[0], w[4]);
            ws[0] = p.w_scale[(int64_t)(n0 / kFp8Block) * nb + b];
        }
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            const u32x4_v *xv = reinterpret_cast<const u32x4_v *>(xp[j] + b * kFp8Block + 16 * g);
            const float xs = sp[j][b];
            f32x4_t d;
            if constexpr (TERN)
                d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    a, odd_even(xv[0], xv[4]), zero, kFp4, kFp8, 0, kHalf, 0, kOne);
            else
                d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, join(xv[0], xv[4]), zero, kFp8,
                                                                     kFp8, 0, kOne, 0, kOne);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[j][i] += d[i] * (TERN ? xs * ws[i] : xs * ws[0]);
        }
    }
#pragma unroll
    for (int j = 0; j < MT; ++j)
        red[wave][j][lane] = acc[j];
    __syncthreads();
    // the waves' sums, in their order
    for (int j = wave; j < MT; j += kWaves) {
        f32x4_t s = red[0][j][lane];
        for (int w = 1; w < kWaves; ++w)
            s += red[w][j][lane];
        const int row = r0 + 16 * j + col, ch = n0 + 4 * g;
        if (row >= r1)
            continue;
        if constexpr (TERN)
            if (!p.group)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s[i] *= f16_bits_to_f32(p.t_scale[(int64_t)e * p.N + min(ch + i, p.N - 1)]);
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
}

template <bool TERN, int MT>
hipError_t launch_stream(const Fp8Product &p, int64_t tiles, hipStream_t stream)
{
    const unsigned nx = (unsigned)((p.N + 15) / 16);
    with_dtype(p.dtype, [&](auto dt) {
        hipLaunchKernelGGL((stream_kernel<TERN, MT, decltype(dt)::value>), dim3(nx, (unsigned)tiles),
                           dim3(kThreads), 0, stream, p);
    });
    return hipGetLastError();
}

// Tiles of `rows` places that E experts of R places in all can need.
int64_t expert_tiles(const Fp8Product &p, int rows)
{
    return p.M / rows + (p.M < p.E ? p.M : p.E);
}

}  // namespace

hipError_t launch_fp8_linear(const Fp8Product &p, hipStream_t stream)
{
    if (p.M <= 16)
        return launch_stream<false, 1>(p, 1, stream);
    return launch_stream<false, 4>(p, (p.M + 63) / 64, stream);
}

hipError_t launch_linear_experts(const Fp8Product &p, hipStream_t stream)
{
    if (p.M <= 16 * p.E)
        return launch_stream<true, 1>(p, expert_tiles(p, 16), stream);
    return launch_stream<true, 4>(p, expert_tiles(p, 64), stream);
}

}  // namespace ternary
