// Products of 8-bit activations on gfx950: with 8-bit weights (a scale per
// block of 128 x 128), and with the ternary weights of experts.
//
//     y[m, n] = sum_b xs[m, b] s(n, b) sum_{k in b} x[m, k] w[n, k]
//
// One v_mfma_scale_f32_16x16x128_f8f6f4 multiplies 16 channels (the A operand)
// by 16 rows of x (B) over one block of 128; its fp32 sums are then scaled and
// added to the running sums, so no rounding but fp32's happens before the end.
// A lane's four results are four channels of one row: the row's scale is one
// register and the four go out in one store.  Ternary codes become fp4 (+-2) in five vector operations a 16 codes;
// as those give a word's odd codes, then its even ones, x's bytes are put in the
// same order (eight byte permutes per 16 rows x 128).  Lane group g (lanes 16 g
// up) holds k = 32 g .. 32 g + 31 of a block of an fp4 operand, and k = 16 g .. and
// 64 + 16 g .. (16 each) of an fp8 one.
#include "fp8_common.h"
#include "internal.h"

namespace ternary {

namespace {

// One block of 128: 16 channels by 16 rows.  Without the instruction's own block
// scales (both arguments 0) it issues faster: in a loop with the scaling of its results,
// 4480 against 3883 TFLOP/s.  So an fp4 operand's +-2 stay, and half of each is left to
// the channel's scale.
template <bool TERN>
__device__ __forceinline__ f32x4_t mfma(i32x8_v w, i32x8_v x)
{
    const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, zero, TERN ? 4 : 0, 0, 0, 0, 0, 0);
}
// Scale of a channel's fp4 products.
__device__ __forceinline__ float channel_scale(uint16_t s) { return 0.5f * f16_bits_to_f32(s); }

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
                    ws[i] = channel_scale(
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
                d = mfma<true>(a, odd_even(xv[0], xv[4]));
            else
                d = mfma<false>(a, join(xv[0], xv[4]));
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
                    s[i] *= channel_scale(p.t_scale[(int64_t)e * p.N + min(ch + i, p.N - 1)]);
        put4<DT>(p, row, ch, s);
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

// ---------------------------------------------------------------- many rows

// Waits for everything this wave has loaded (LDS reads, and loads into LDS among
// them), then for the workgroup's other waves.
__device__ __forceinline__ void meet()
{
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(7 << 4);  // vmcnt(0) lgkmcnt(0)
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

typedef __attribute__((address_space(3))) u32x4_v lds_u4;
typedef __attribute__((address_space(3))) u32x2_v lds_u2;
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

template <int TN_, int TM_, int WN_, int WM_>
struct Tile {
    static constexpr int TN = TN_, TM = TM_, WN = WN_, WM = WM_;
    static constexpr int THREADS = WN * WM * 64;
    static constexpr int FN = TN / WN / 16, FM = TM / WM / 16;  // fragments of a wave
};

// weights' scales are read by scalar loads: the same for a whole workgroup
typedef const __attribute__((address_space(4))) float constant_float;
typedef float f32x4_u __attribute__((ext_vector_type(4), aligned(4)));

// Values b0 .. b0 + 3 of a row of n (unspecified past its end).
__device__ __forceinline__ f32x4_t load_scales(const float *row, int b0, int n)
{
    if (n < 4) {
        return f32x4_t{row[min(b0, n - 1)], row[min(b0 + 1, n - 1)], row[min(b0 + 2, n - 1)], row[n - 1]};
    }
    // the row's last four at its end, moved down
    const int at = min(b0, n - 4);
    f32x4_u u = *reinterpret_cast<const f32x4_u *>(row + at);
    if (at + 1 <= b0)
        u = u.yzww;
    if (at + 2 <= b0)
        u = u.yzww;
    if (at + 3 <= b0)
        u = u.yzww;
    return f32x4_t{u.x, u.y, u.z, u.w};
}
// The same for a row that a whole workgroup reads (scalar loads).
__device__ __forceinline__ f32x4_t load_scales_uniform(const float *row, int b0, int n)
{
    constant_float *r = (constant_float *)row;
    return f32x4_t{r[min(b0, n - 1)], r[min(b0 + 1, n - 1)], r[min(b0 + 2, n - 1)], r[min(b0 + 3, n - 1)]};
}

// G: group-scaled ternary weights.
template <bool TERN, bool G, int DT, class C>
__global__ void __launch_bounds__(C::THREADS, 2) tile_kernel(const Fp8Product p)
{
    constexpr int TN = C::TN, TM = C::TM, FN = C::FN, FM = C::FM, THREADS = C::THREADS;
    constexpr int XI = TM * 8 / THREADS;                      // x loads of a thread and stage
    constexpr int WCH = TERN ? TN * 2 : TN * 8;               // 16-byte chunks of w in a stage
    constexpr int WI = (WCH + THREADS - 1) / THREADS;
    constexpr int QB = TERN ? 1 : (TN + 127) / 128;           // blocks of channels with scales of their own
    static_assert(TM * 8 % THREADS == 0 && (WCH % THREADS == 0 || WI == 1) && TM <= THREADS && TN <= THREADS);
    // one object per stage: a load into one stage is then known not to touch the other
    __shared__ __attribute__((aligned(16))) u32x4_v sx0[TM * 8], sx1[TM * 8], sw0[WCH], sw1[WCH];
    // scales of eight steps: x's (times w's for 8-bit weights), a lane's FM
    // rows together, and a group's channels'.  Each is read by one load: a pair of loads that the
    // compiler merges loses the object it reads, and with it would wait for every stage in flight.
    typedef float fm_t __attribute__((ext_vector_type(FM)));
    __shared__ __attribute__((aligned(16))) fm_t sf[QB][8][TM / FM];
    __shared__ __attribute__((aligned(16))) f32x4_t sg[G ? 8 : 1][G ? TN / 4 : 1];

    lds_u4 *const lx[2] = {(lds_u4 *)sx0, (lds_u4 *)sx1}, *const lw[2] = {(lds_u4 *)sw0, (lds_u4 *)sw1};

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
        tm = slot / ntn * 8 + xcd;
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
    // dense: the last tile ends at M, so that every row of a tile exists (rows of
    // two tiles are computed by both, to the same bits)
    int e = 0, r0 = min(tm * TM, p.M - TM), r1 = r0 + TM;
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
    // Sources.  Gathered rows of x and the experts' blocks have pointers of
    // their own; a dense tile is one resource, each thread's rows a uniform
    // distance apart.
    constexpr int RS = THREADS / 8;        // rows between a thread's chunks of x
    const int rowbytes = nb * kFp8Block;   // at most 2^20
    static_assert(RS % 8 == 0, "the same chunk of each row");
    const uint8_t *xsrc[XI], *wsrc = nullptr;
    int woff[WI];
    const int off = (tid >> 3) * rowbytes + 16 * ((tid & 7) ^ swz(tid >> 3));
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
        xr = make_rsrc(p.x + (int64_t)r0 * rowbytes, (uint32_t)(TM * rowbytes));
        const int chans = min(TN, p.N - n0);  // (those past the last repeat it)
        wr = make_rsrc(p.w + (int64_t)n0 * rowbytes, (uint32_t)(chans * rowbytes));
#pragma unroll
        for (int i = 0; i < WI; ++i)
            woff[i] = min((tid >> 3) + i * RS, chans - 1) * rowbytes + 16 * ((tid & 7) ^ swz(tid >> 3));
    }
    const float *fsrc = p.x_scale + (tid < TM ? x_row(tid) : 0) * nb;
    const uint16_t *gsrc = G ? p.t_scale + ((int64_t)e * p.N + min(n0 + tid, p.N - 1)) * p.ngroups : nullptr;
    const int gsteps = G ? p.group / kFp8Block : 1;

    auto issue = [&](auto S, int b) {
        constexpr int s = decltype(S)::value;
#pragma unroll
        for (int i = 0; i < XI; ++i) {
            lds_u4 *to = lx[s] + i * THREADS + wave * 64;
            if constexpr (TERN)
                load_to_lds(xsrc[i] + b * kFp8Block, to);
            else
                load_to_lds(xr, to, off, i * RS * rowbytes + b * kFp8Block);
        }
#pragma unroll
        for (int i = 0; i < WI; ++i) {
            lds_u4 *to = lw[s] + i * THREADS + wave * 64;
            if constexpr (!TERN)
                load_to_lds(wr, to, woff[i], b * kFp8Block);
            else if (WCH % THREADS == 0 || wave * 64 < WCH)
                load_to_lds(wsrc + (int64_t)b * (kTileBytes / 2), to);
        }
    };
    f32x4_t fx = {0.f, 0.f, 0.f, 0.f}, fw[QB], gv = fx;
    auto load_factors = [&](int b0) {  // of steps b0 .. b0 + 3
        if (wave < TM / 64)
            fx = load_scales(fsrc, b0, nb);
        if constexpr (!TERN)
#pragma unroll
            for (int q = 0; q < QB; ++q)
                fw[q] = load_scales_uniform(p.w_scale + (int64_t)min(n0 / 128 + q, (p.N - 1) / 128) * nb, b0, nb);
        if constexpr (G)
            if (wave < TN / 64)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    gv[i] = channel_scale(gsrc[min(b0 + i, nb - 1) / gsteps]);
    };
    // row r = 16 (FM u + j) + c of the tile: entry j of (u, c)
    const int fpos = ((tid / (16 * FM)) * 16 + (tid & 15)) * FM + (tid >> 4) % FM;
    auto store_factors = [&](int b0) {
        if (wave < TM / 64)
#pragma unroll
            for (int q = 0; q < QB; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    reinterpret_cast<float *>(sf[q][(b0 + i) & 7])[fpos] = TERN ? fx[i] : fx[i] * fw[q][i];
        if constexpr (G)
            if (wave < TN / 64)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    reinterpret_cast<float *>(sg[(b0 + i) & 7])[tid] = gv[i];
    };

    f32x4_t acc[FN][FM];
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j)
            acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
    // Chunks of a row that lane group g holds: g and g + 4.  Ternary: the codes of
    // two fragments come by one load, 16 bytes of the first fragment's in lanes 0 .. 31, of the
    // second's in the others; exchanging the halves of each (permlane32_swap)
    // leaves a fragment with the codes 0, 64, 32 and 96 (and 31 more) in its lane
    // groups, so x's chunks are 0, 1, 4, 5 and those two further on.
    static_assert(!TERN || FN % 2 == 0);
    const int xa = (wm * FM * 16 + col) * 8, cg = TERN ? g + (g & 2) : g;
    const int c0 = cg ^ swz(col), c1 = (cg + (TERN ? 2 : 4)) ^ swz(col);
    const int wa = TERN ? wn * FN * 32 + lane : (wn * FN * 16 + col) * 8;

    // Operands on their way from LDS: w's two fragments ahead (ternary: two
    // fragments by one load), all of x's, and the scales.
    u32x4_v rw[2][2], rx[FM][2];
    fm_t fn, f, fp;          // the next step's, this step's, the last one's
    // matrix results not yet scaled, and two fragments' channels' scales.  A
    // result is scaled behind the second matrix instruction after its own: it is there by then.
    constexpr int LAG = 2;
    static_assert(FM >= LAG && FN * FM % 4 == 0);
    f32x4_t d[4], gs[2];
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
    auto read_f = [&](int b) { fn = sf[TERN ? 0 : (wn * FN * 16) / 128][b & 7][wm * 16 + col]; };
    u32x2_v odd_codes = {0, 0};  // of the second fragment of two
    auto w_operand = [&](int i) -> i32x8_v {
        if constexpr (TERN) {
            u32x2_v w = odd_codes;
            if (i % 2 == 0) {
                const u32x4_v r = rw[0][0];
                const u32x2_v lo = __builtin_amdgcn_permlane32_swap(r.x, r.z, false, false);
                const u32x2_v hi = __builtin_amdgcn_permlane32_swap(r.y, r.w, false, false);
                w = u32x2_v{lo.x, hi.x};
                odd_codes = u32x2_v{lo.y, hi.y};
            }
            int c[4];
            codes_to_fp4(w.x, c[0], c[1]);
            codes_to_fp4(w.y, c[2], c[3]);
            return i32x8_v{c[0], c[1], c[2], c[3], 0, 0, 0, 0};
        } else {
            return join(rw[i & 1][0], rw[i & 1][1]);
        }
    };
    auto scale_add = [&](int n, const fm_t &by) {  // result n of a step
        const int i = n / FM, j = n % FM;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            acc[i][j][k] += d[n & 3][k] * (G ? by[j] * gs[i & 1][k] : by[j]);
    };

    // Step b, from stage s.  Each matrix instruction is followed by the scaling of a
    // result of the fragment before, so that neither waits for the other.  The
    // waves meet two fragments before the end, once the stage is read and the next one is there:
    // from then on this stage takes step b + 2, and the next step's first
    // operands are read behind the last fragments' matrix instructions.
    auto step = [&](auto S, int b) {
        constexpr int s = decltype(S)::value;
        constexpr std::integral_constant<int, s ^ 1> T;
        static_assert(FN % 2 == 0 && FN >= 4);
        i32x8_v x[FM];
        fp = f;
        f = fn;
#pragma unroll
        for (int i = 0; i < FN; ++i) {
            const i32x8_v a = w_operand(i);
            f32x4_t gnew;
            if constexpr (G)
                gnew = sg[b & 7][(wn * FN + i) * 4 + g];
            if (i == FN - 2) {
                meet();
                issue(S, min(b + 2, nb - 1));
                if constexpr (s == 0) {
                    // scales ahead: loaded at the first step of four, put into LDS at the third
                    if (b & 2)
                        store_factors(b + 2);
                    else
                        load_factors(b + 4);
                }
                read_f(b + 1);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < FM; ++j) {
                const int n = i * FM + j;
                if (i == 0)
                    x[j] = TERN ? odd_even(rx[j][0], rx[j][1]) : join(rx[j][0], rx[j][1]);
                asm volatile("" : "+v"(x[j]));  // (nothing: keeps the instruction from moving up)
                d[n & 3] = mfma<TERN>(a, x[j]);
                if (i == FN - 1)
                    read_x(T, j);
                if (G && j == LAG)
                    gs[i & 1] = gnew;
                const int m = n >= LAG ? n - LAG : n - LAG + FN * FM;
                scale_add(m, n >= LAG ? f : fp);
                asm volatile("" : "+v"(acc[m / FM][m % FM]));  // (the same, down)
                __builtin_amdgcn_sched_barrier(0);
            }
            if (i + 2 < FN)
                read_w(S, i + 2);
            else
                read_w(T, i + 2 - FN);
        }
    };

    load_factors(0);
    store_factors(0);
    // Every step loads the stage of the step after the next; the last ones load the
    // last step again, into a stage that is not read (a branch there, or a second exit of the loop, had
    // the compiler copy the step).
    issue(std::integral_constant<int, 0>(), 0);
    issue(std::integral_constant<int, 1>(), min(1, nb - 1));
    meet();
    read_w(std::integral_constant<int, 0>(), 0);
    read_w(std::integral_constant<int, 0>(), 1);
    read_f(0);
#pragma unroll
    for (int j = 0; j < FM; ++j) {
        read_x(std::integral_constant<int, 0>(), j);
        f[j] = 0.f;
    }
    d[2] = d[3] = zero;
    gs[1] = zero;
    int b = 0;
    for (; b + 1 < nb; b += 2) {
        step(std::integral_constant<int, 0>(), b);
        step(std::integral_constant<int, 1>(), b + 1);
    }
    if (b < nb)
        step(std::integral_constant<int, 0>(), b);
#pragma unroll
    for (int n = FN * FM - LAG; n < FN * FM; ++n)
        scale_add(n, f);
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
                put4<DT>(p, row, ch, TERN && !G ? acc[i][j] * cs : acc[i][j]);
        }
    }
}

template <bool TERN, class C>
hipError_t launch_tiles(const Fp8Product &p, int64_t tiles, hipStream_t stream)
{
    const int ntn = (p.N + C::TN - 1) / C::TN;
    const int64_t wgs = TERN ? (tiles + 7) / 8 * 8 * ntn : (tiles * ntn + 7) / 8 * 8;
    if (wgs > INT32_MAX)
        return hipErrorInvalidValue;
    with_dtype(p.dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        if (TERN && p.group)
            hipLaunchKernelGGL((tile_kernel<TERN, TERN, DT, C>), dim3((unsigned)wgs), dim3(C::THREADS), 0, stream, p);
        else
            hipLaunchKernelGGL((tile_kernel<TERN, false, DT, C>), dim3((unsigned)wgs), dim3(C::THREADS), 0, stream, p);
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
    if (p.M < 256)
        return launch_stream<false, 4>(p, (p.M + 63) / 64, stream);
    return launch_tiles<false, Tile<256, 256, 2, 4>>(p, (p.M + 255) / 256, stream);
}

hipError_t launch_linear_experts(const Fp8Product &p, hipStream_t stream)
{
    if (p.M <= 16 * p.E)
        return launch_stream<true, 1>(p, expert_tiles(p, 16), stream);
    if (p.M <= 32 * p.E)
        return launch_stream<true, 4>(p, expert_tiles(p, 64), stream);
    return launch_tiles<true, Tile<256, 128, 4, 2>>(p, expert_tiles(p, 128), stream);
}

}  // namespace ternary
