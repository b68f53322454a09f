// C ABI of the 8-bit layers and the experts (declared in include/ternary.h):
// host-side argument validation, then an asynchronous launch on the caller's
// stream.  Validation never dereferences a pointer and never calls HIP.
#include <stdint.h>

#include "../../include/ternary.h"
#include "check.h"
#include "internal.h"

using ternary::aligned;
using ternary::fp8_blocks;
using ternary::hip_status;
using ternary::kMaxDim;
using ternary::overlap;

namespace {

// Longest K of the products: K / 128 block scales of a row, and a row's bytes,
// stay far inside 32-bit offsets.
constexpr int64_t kMaxProductK = (int64_t)1 << 20;

// Bytes of an element, or 0 for an unknown type.
int64_t elem_bytes(int dtype)
{
    return dtype == TERNARY_BF16 || dtype == TERNARY_FP16 ? 2 : dtype == TERNARY_FP32 ? 4 : 0;
}

// Most places of the experts' products: a tile past the last stays inside 32 bits.
constexpr int64_t kMaxPlaces = (int64_t)1 << 30;

bool dim_ok(int64_t n, int64_t lo, int64_t hi = kMaxDim) { return n >= lo && n <= hi; }

}  // namespace

extern "C" {

int ternary_fp8_quantize(const void *x, int dtype, int64_t M, int64_t K, int64_t ldx, int block,
                         int act, uint8_t *q, float *scale, hipStream_t stream)
{
    const int64_t e = elem_bytes(dtype);
    if (!e)
        return TERNARY_ERR_DTYPE;
    const bool tile = block == TERNARY_BLOCK_TILE, swiglu = act == TERNARY_ACT_SWIGLU;
    if ((!tile && block != TERNARY_BLOCK_ROW) || (!swiglu && act != TERNARY_ACT_NONE) ||
        (tile && swiglu) || !dim_ok(M, 0) || !dim_ok(K, 1))
        return TERNARY_ERR_SHAPE;
    const int64_t row = swiglu ? 2 * K : K;
    if (ldx < row || ldx > ((int64_t)1 << 32))
        return TERNARY_ERR_SHAPE;
    if (M == 0)
        return TERNARY_OK;
    if (!x || !q || !scale)
        return TERNARY_ERR_NULL;
    if (!aligned(x, e) || !aligned(q, 16) || !aligned(scale, 4))
        return TERNARY_ERR_ALIGN;
    const int64_t kb = fp8_blocks(K), xbytes = ((M - 1) * ldx + row) * e,
                  qbytes = M * kb * ternary::kFp8Block, sbytes = 4 * kb * (tile ? fp8_blocks(M) : M);
    if (overlap(q, qbytes, x, xbytes) || overlap(scale, sbytes, x, xbytes) ||
        overlap(scale, sbytes, q, qbytes))
        return TERNARY_ERR_ALIAS;
    return hip_status(ternary::launch_fp8_quantize(x, dtype, M, K, ldx, tile, swiglu, q, scale, stream));
}

int ternary_fp8_linear(const uint8_t *x, const float *x_scale, const uint8_t *w,
                       const float *w_scale, int64_t M, int64_t N, int64_t K, void *y, int dtype,
                       hipStream_t stream)
{
    const int64_t e = elem_bytes(dtype);
    if (!e)
        return TERNARY_ERR_DTYPE;
    if (!dim_ok(M, 0) || !dim_ok(N, 0) || !dim_ok(K, 1, kMaxProductK) || K % ternary::kFp8Block)
        return TERNARY_ERR_SHAPE;
    if (M == 0 || N == 0)
        return TERNARY_OK;
    if (!x || !x_scale || !w || !w_scale || !y)
        return TERNARY_ERR_NULL;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(y, 16) || !aligned(x_scale, 4) ||
        !aligned(w_scale, 4))
        return TERNARY_ERR_ALIGN;
    const int64_t nb = K / ternary::kFp8Block, ybytes = e * M * N;
    if (overlap(y, ybytes, x, M * K) || overlap(y, ybytes, w, N * K) ||
        overlap(y, ybytes, x_scale, 4 * M * nb) || overlap(y, ybytes, w_scale, 4 * fp8_blocks(N) * nb))
        return TERNARY_ERR_ALIAS;
    ternary::Fp8Product p = {};
    p.x = x;
    p.x_scale = x_scale;
    p.w = w;
    p.w_scale = w_scale;
    p.y = y;
    p.dtype = dtype;
    p.M = (int)M;
    p.N = (int)N;
    p.nb = (int)nb;
    return hip_status(ternary::launch_fp8_linear(p, stream));
}

int64_t ternary_route_workspace(int64_t T, int64_t E)
{
    if (!dim_ok(T, 0) || !dim_ok(E, 1, TERNARY_MAX_EXPERTS))
        return TERNARY_ERR_SHAPE;
    return ternary::route_workspace(T, E);
}

int ternary_route(const void *logits, int dtype, int64_t T, int64_t E, const float *bias,
                  int score, int groups, int top_groups, int top_k, int renormalize, float scale,
                  int32_t *ids, float *weights, int32_t *offsets, int32_t *order, int32_t *slots,
                  void *workspace, hipStream_t stream)
{
    const int64_t e = elem_bytes(dtype);
    if (!e)
        return TERNARY_ERR_DTYPE;
    if (!dim_ok(T, 0) || !dim_ok(E, 1, TERNARY_MAX_EXPERTS) ||
        (score != TERNARY_SCORE_SOFTMAX && score != TERNARY_SCORE_SIGMOID) ||
        !dim_ok(groups, 1, TERNARY_MAX_EXPERT_GROUPS) || E % groups || !dim_ok(top_groups, 1, groups) ||
        !dim_ok(top_k, 1, TERNARY_MAX_TOP_K) || top_k > top_groups * (E / groups) ||
        T * top_k > INT32_MAX)
        return TERNARY_ERR_SHAPE;
    const int64_t wsbytes = ternary::route_workspace(T, E);
    if (!offsets || (T && (!logits || !ids || !weights || !order || !slots)) || (wsbytes && !workspace))
        return TERNARY_ERR_NULL;
    if (!aligned(logits, e) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4) ||
        !aligned(offsets, 4) || !aligned(order, 4) || !aligned(slots, 4) || (wsbytes && !aligned(workspace, 16)))
        return TERNARY_ERR_ALIGN;
    const int64_t lbytes = e * T * E, kbytes = 4 * T * top_k;
    const struct {
        const void *p;
        int64_t n;
    } out[6] = {{ids, kbytes}, {weights, kbytes}, {order, kbytes}, {slots, kbytes},
                {offsets, 4 * (E + 1)}, {workspace, wsbytes}};
    for (int i = 0; i < 6; ++i) {
        if (overlap(out[i].p, out[i].n, logits, lbytes) || (bias && overlap(out[i].p, out[i].n, bias, 4 * E)))
            return TERNARY_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i].p, out[i].n, out[j].p, out[j].n))
                return TERNARY_ERR_ALIAS;
    }
    const ternary::RouteArgs a = {logits, bias, ids, weights, offsets, order, slots, workspace,
                                  (int)T, (int)E, top_k, groups, top_groups, renormalize != 0,
                                  score == TERNARY_SCORE_SIGMOID, scale};
    return hip_status(ternary::launch_route(a, dtype, stream));
}

int ternary_linear_experts(const uint8_t *x, const float *x_scale, int64_t x_rows,
                           const uint8_t *tiled, const uint16_t *scale, int64_t E, int64_t N,
                           int64_t K, int64_t group_size, const int32_t *offsets,
                           const int32_t *order, int64_t R, int top_k, int rows, void *y,
                           int dtype, hipStream_t stream)
{
    const int64_t e = elem_bytes(dtype);
    if (!e)
        return TERNARY_ERR_DTYPE;
    if (group_size != -1 && group_size != 128 && group_size != 256)
        return TERNARY_ERR_GROUP;
    const bool tokens = rows == TERNARY_ROWS_TOKENS;
    if ((!tokens && rows != TERNARY_ROWS_SORTED) || !dim_ok(E, 1, TERNARY_MAX_EXPERTS) ||
        !dim_ok(N, 0) || !dim_ok(K, 1, kMaxProductK) || K % 4 ||
        (group_size > 0 && K % group_size) || !dim_ok(R, 0, kMaxPlaces) ||
        !dim_ok(x_rows, R ? 1 : 0, INT32_MAX) || (!tokens && x_rows < R) ||
        (tokens && !dim_ok(top_k, 1, TERNARY_MAX_TOP_K)))
        return TERNARY_ERR_SHAPE;
    if (R == 0 || N == 0)
        return TERNARY_OK;
    if (!x || !x_scale || !tiled || !scale || !offsets || (tokens && !order) || !y)
        return TERNARY_ERR_NULL;
    if (!aligned(x, 16) || !aligned(tiled, 16) || !aligned(y, 16) || !aligned(x_scale, 4) ||
        !aligned(scale, 2) || !aligned(offsets, 4) || (tokens && !aligned(order, 4)))
        return TERNARY_ERR_ALIGN;
    const int64_t nb = fp8_blocks(K), ng = group_size == -1 ? 1 : K / group_size, ybytes = e * R * N;
    if (overlap(y, ybytes, x, x_rows * nb * ternary::kFp8Block) ||
        overlap(y, ybytes, x_scale, 4 * x_rows * nb) ||
        overlap(y, ybytes, tiled, E * ternary::tiled_bytes(N, K)) ||
        overlap(y, ybytes, scale, 2 * E * N * ng) || overlap(y, ybytes, offsets, 4 * (E + 1)) ||
        (tokens && overlap(y, ybytes, order, 4 * R)))
        return TERNARY_ERR_ALIAS;
    ternary::Fp8Product p = {};
    p.x = x;
    p.x_scale = x_scale;
    p.w = tiled;
    p.t_scale = scale;
    p.y = y;
    p.dtype = dtype;
    p.M = (int)R;
    p.N = (int)N;
    p.nb = (int)nb;
    p.offsets = offsets;
    p.order = tokens ? order : nullptr;
    p.E = (int)E;
    p.group = group_size == -1 ? 0 : (int)group_size;
    p.ngroups = (int)ng;
    p.top_k = top_k;
    p.x_rows = (int)x_rows;
    return hip_status(ternary::launch_linear_experts(p, stream));
}

int ternary_combine(const void *y, int dtype, int64_t R, int64_t N, const int32_t *slots,
                    const float *weights, int64_t T, int top_k, const void *add, void *out,
                    hipStream_t stream)
{
    const int64_t e = elem_bytes(dtype);
    if (!e)
        return TERNARY_ERR_DTYPE;
    if (!dim_ok(T, 0) || !dim_ok(N, 0) || !dim_ok(R, 0, INT32_MAX) ||
        !dim_ok(top_k, 1, TERNARY_MAX_TOP_K))
        return TERNARY_ERR_SHAPE;
    if (T == 0 || N == 0)
        return TERNARY_OK;
    if ((R && !y) || !slots || !weights || !out)
        return TERNARY_ERR_NULL;
    if (!aligned(y, e) || !aligned(add, e) || !aligned(out, e) || !aligned(slots, 4) || !aligned(weights, 4))
        return TERNARY_ERR_ALIGN;
    const int64_t obytes = e * T * N;
    if (overlap(out, obytes, y, e * R * N) || overlap(out, obytes, slots, 4 * T * top_k) ||
        overlap(out, obytes, weights, 4 * T * top_k) ||
        (add && add != out && overlap(out, obytes, add, obytes)))
        return TERNARY_ERR_ALIAS;
    const ternary::CombineArgs a = {y, add, out, slots, weights, R, (int)T, top_k, (int)N};
    return hip_status(ternary::launch_combine(a, dtype, stream));
}

}  // extern "C"
