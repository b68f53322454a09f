// Which places (rows sorted by expert) a workgroup has: device helpers of the kernels that
// walk tiles of them.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ternary {

// Inclusive sum over the lanes of a wave (row shifts, then each row's total to
// the rows after it).
__device__ __forceinline__ int wave_scan(int v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // row_shr 1, 2, 4, 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row_bcast 15, 31
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);
    return v;
}

// Places [r0, r1) of expert e that the idx-th tile of BM rows covers (tiles run
// expert by expert); false past the last.  Every lane of a wave calls it; lane l
// looks at experts EP l .. EP l + EP - 1.  Whatever the offsets hold, the places are within
// [0, R) and the expert within [0, E).
template <int BM, int EP>
__device__ __forceinline__ bool find_tile_of(const int32_t *offsets, int E, int R, int idx, int &e,
                                             int &r0, int &r1)
{
    const int lo = (threadIdx.x & 63) * EP;
    int o[EP + 1];
#pragma unroll
    for (int i = 0; i <= EP; ++i)
        o[i] = offsets[min(lo + i, E)];
    int mine = 0;
#pragma unroll
    for (int i = 0; i < EP; ++i) {
        const int a = max(o[i], 0), b = min(o[i + 1], R);
        mine += b > a ? (b - a + BM - 1) / BM : 0;
    }
    const int incl = wave_scan(mine);
    int left = idx - (incl - mine), fe = -1, f0 = 0, f1 = 0;
    const uint64_t here = __builtin_amdgcn_ballot_w64(left >= 0 && left < mine);
    if (!here)
        return false;
#pragma unroll
    for (int i = 0; i < EP; ++i) {
        const int a = max(o[i], 0), b = min(o[i + 1], R);
        const int tiles = b > a ? (b - a + BM - 1) / BM : 0;
        if (left >= 0 && left < tiles) {
            fe = lo + i;
            f0 = a + left * BM;
            f1 = min(b, f0 + BM);
        }
        left -= tiles;
    }
    const int from = __builtin_ctzll(here);
    e = __builtin_amdgcn_readlane(fe, from);
    r0 = __builtin_amdgcn_readlane(f0, from);
    r1 = __builtin_amdgcn_readlane(f1, from);
    return e >= 0;
}

template <int BM>
__device__ __forceinline__ bool find_tile(const int32_t *offsets, int E, int R, int idx, int &e,
                                          int &r0, int &r1)
{
    if (E <= 64)
        return find_tile_of<BM, 1>(offsets, E, R, idx, e, r0, r1);
    if (E <= 256)
        return find_tile_of<BM, 4>(offsets, E, R, idx, e, r0, r1);
    return find_tile_of<BM, 8>(offsets, E, R, idx, e, r0, r1);
}

// The idx-th piece of up to P places of one expert, as by find_tile, the expert's pieces alike but for multiples of
// 32; and its number of pieces, and where it has several the piece's number among the pieces of such experts.
template <int EP>
__device__ __forceinline__ bool find_piece_of(const int32_t *offsets, int E, int R, int P, int idx, int &e, int &r0,
                                              int &r1, int &pieces, int &number)
{
    const int lo = (threadIdx.x & 63) * EP;
    int o[EP + 1];
#pragma unroll
    for (int i = 0; i <= EP; ++i)
        o[i] = offsets[min(lo + i, E)];
    int n[EP], mine = 0, several = 0;
#pragma unroll
    for (int i = 0; i < EP; ++i) {
        const int a = max(o[i], 0), b = min(o[i + 1], R);
        n[i] = b > a ? (b - a + P - 1) / P : 0;
        mine += n[i];
        several += n[i] > 1 ? n[i] : 0;
    }
    int left = idx - (wave_scan(mine) - mine), before = wave_scan(several) - several;
    int fe = -1, f0 = 0, f1 = 0, fn = 0, fs = 0;
    const uint64_t here = __builtin_amdgcn_ballot_w64(left >= 0 && left < mine);
    if (!here)
        return false;
#pragma unroll
    for (int i = 0; i < EP; ++i) {
        if (left >= 0 && left < n[i]) {
            const int a = max(o[i], 0), b = min(o[i + 1], R), len = ((b - a + n[i] - 1) / n[i] + 31) & ~31;
            fe = lo + i;
            f0 = min(a + left * len, b);
            f1 = min(b, f0 + len);
            fn = n[i];
            fs = before + left;
        }
        left -= n[i];
        before += n[i] > 1 ? n[i] : 0;
    }
    const int from = __builtin_ctzll(here);
    e = __builtin_amdgcn_readlane(fe, from);
    r0 = __builtin_amdgcn_readlane(f0, from);
    r1 = __builtin_amdgcn_readlane(f1, from);
    pieces = __builtin_amdgcn_readlane(fn, from);
    number = __builtin_amdgcn_readlane(fs, from);
    return e >= 0;
}
__device__ __forceinline__ bool find_piece(const int32_t *offsets, int E, int R, int P, int idx, int &e, int &r0,
                                           int &r1, int &pieces, int &number)
{
    if (E <= 64)
        return find_piece_of<1>(offsets, E, R, P, idx, e, r0, r1, pieces, number);
    return find_piece_of<8>(offsets, E, R, P, idx, e, r0, r1, pieces, number);
}

// Expert e's number of such pieces, and the first one's number among those of experts with several.
template <int EP>
__device__ __forceinline__ void pieces_of_expert(const int32_t *offsets, int E, int R, int P, int e, int &pieces,
                                                 int &first)
{
    const int lo = (threadIdx.x & 63) * EP;
    int o[EP + 1];
#pragma unroll
    for (int i = 0; i <= EP; ++i)
        o[i] = offsets[min(lo + i, E)];
    int several = 0, mine = 0, before = 0;
#pragma unroll
    for (int i = 0; i < EP; ++i) {
        const int a = max(o[i], 0), b = min(o[i + 1], R), n = b > a ? (b - a + P - 1) / P : 0;
        if (lo + i == e)
            mine = n, before = several;
        several += n > 1 ? n : 0;
    }
    before += wave_scan(several) - several;
    const int from = e / EP;
    pieces = __builtin_amdgcn_readlane(mine, from);
    first = __builtin_amdgcn_readlane(before, from);
}
__device__ __forceinline__ void expert_pieces(const int32_t *offsets, int E, int R, int P, int e, int &pieces, int &first)
{
    if (E <= 64)
        pieces_of_expert<1>(offsets, E, R, P, e, pieces, first);
    else
        pieces_of_expert<8>(offsets, E, R, P, e, pieces, first);
}

}  // namespace ternary
