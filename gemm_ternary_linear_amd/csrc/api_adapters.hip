// C ABI of sorted slots, the exchange with experts and its gradients, and low-rank adapters (declared in
// include/ternary.h): host-side argument validation, then an asynchronous launch on the caller's
// stream.  Validation never dereferences a pointer and never calls HIP.
#include <initializer_list>

#include "../../include/ternary.h"
#include "check.h"
#include "internal.h"

using ternary::aligned;
using ternary::hip_status;
using ternary::kMaxDim;
using ternary::overlap;

namespace {

// Most elements of a matrix: offsets are 64-bit, grids stay inside the launch limits.
constexpr int64_t kMaxElems = (int64_t)1 << 38;

// Most columns of all adapters: a launch holds a workgroup for each of them and run of columns.
constexpr int64_t kMaxWidth = (int64_t)1 << 28;

int64_t elem_bytes(int dtype)
{
    return dtype == TERNARY_BF16 || dtype == TERNARY_FP16 ? 2 : dtype == TERNARY_FP32 ? 4 : 0;
}

bool dim_ok(int64_t n, int64_t lo, int64_t hi = kMaxDim) { return n >= lo && n <= hi; }

struct Range {
    const void *p;
    int64_t n;
};

// Whether an output overlaps an input or another output.  `same`: an input that may be exactly outs[0].
bool aliased(std::initializer_list<Range> outs, std::initializer_list<Range> ins, Range same = {nullptr, 0})
{
    const Range *first = outs.begin();
    if (same.p && same.p != first->p && overlap(first->p, first->n, same.p, same.n))
        return true;
    for (const Range *o = first; o != outs.end(); ++o) {
        if (!o->p)
            continue;
        if (o != first && same.p && overlap(o->p, o->n, same.p, same.n))
            return true;
        for (const Range &i : ins)
            if (i.p && overlap(o->p, o->n, i.p, i.n))
                return true;
        for (const Range *q = first; q != o; ++q)
            if (q->p && overlap(o->p, o->n, q->p, q->n))
                return true;
    }
    return false;
}

// What the exchange's functions have in common: TERNARY_OK, or an error.
int exchange_shape(int dtype, int64_t T, int64_t N, int64_t R, int top_k)
{
    if (!elem_bytes(dtype))
        return TERNARY_ERR_DTYPE;
    if (!dim_ok(T, 0) || !dim_ok(N, 0) || !dim_ok(top_k, 1, TERNARY_MAX_TOP_K) || !dim_ok(R, 0, INT32_MAX) ||
        T * top_k > INT32_MAX || T * N > kMaxElems || R * N > kMaxElems)
        return TERNARY_ERR_SHAPE;
    return TERNARY_OK;
}

int adapters_shape(int dtype, int64_t T, int64_t K, int64_t N, int64_t rank, int64_t E)
{
    if (dtype != TERNARY_BF16 && dtype != TERNARY_FP16)
        return TERNARY_ERR_DTYPE;
    if (!dim_ok(T, 0) || !dim_ok(K, 1) || !dim_ok(N, 1) || !dim_ok(rank, 1, TERNARY_MAX_RANK) ||
        !dim_ok(E, 1, TERNARY_MAX_EXPERTS) || T * K > kMaxElems || T * N > kMaxElems || E * (K + N) > kMaxWidth)
        return TERNARY_ERR_SHAPE;
    return TERNARY_OK;
}

}  // namespace

extern "C" {

int64_t ternary_sort_slots_workspace(int64_t T, int top_k, int64_t E)
{
    if (!dim_ok(T, 0) || !dim_ok(top_k, 1, TERNARY_MAX_TOP_K) || T * top_k > INT32_MAX ||
        !dim_ok(E, 1, TERNARY_MAX_EXPERTS))
        return TERNARY_ERR_SHAPE;
    return ternary::sort_slots_workspace(T * top_k, E);
}

int ternary_sort_slots(const int32_t *ids, int64_t T, int top_k, int64_t E, float *ones, int32_t *offsets,
                       int32_t *order, int32_t *slots, void *workspace, hipStream_t stream)
{
    const int64_t wsbytes = ternary_sort_slots_workspace(T, top_k, E);
    if (wsbytes < 0)
        return TERNARY_ERR_SHAPE;
    if (!offsets || (T && (!ids || !order || !slots)) || (wsbytes && !workspace))
        return TERNARY_ERR_NULL;
    if (!aligned(ids, 4) || !aligned(ones, 4) || !aligned(offsets, 4) || !aligned(order, 4) || !aligned(slots, 4) ||
        (wsbytes && !aligned(workspace, 16)))
        return TERNARY_ERR_ALIGN;
    const int64_t n = T * top_k, bytes = 4 * n;
    if (aliased({{offsets, 4 * (E + 1)}, {order, bytes}, {slots, bytes}, {ones, bytes}, {workspace, wsbytes}}, {{ids, bytes}}))
        return TERNARY_ERR_ALIAS;
    const ternary::SortArgs a = {ids, ones, offsets, order, slots, static_cast<int32_t *>(workspace), n, (int)E};
    return hip_status(ternary::launch_sort_slots(a, stream));
}

int ternary_dispatch(const void *x, int dtype, int64_t T, int64_t N, const int32_t *slots, const float *weights,
                     int top_k, int64_t R, void *out, hipStream_t stream)
{
    const int st = exchange_shape(dtype, T, N, R, top_k);
    if (st != TERNARY_OK)
        return st;
    if (T == 0 || N == 0 || R == 0)
        return TERNARY_OK;
    if (!x || !slots || !out)
        return TERNARY_ERR_NULL;
    const int64_t e = elem_bytes(dtype), kbytes = 4 * T * top_k;
    if (!aligned(x, e) || !aligned(out, e) || !aligned(slots, 4) || !aligned(weights, 4))
        return TERNARY_ERR_ALIGN;
    if (aliased({{out, e * R * N}}, {{x, e * T * N}, {slots, kbytes}, {weights, kbytes}}))
        return TERNARY_ERR_ALIAS;
    const ternary::ExchangeArgs a = {x, nullptr, nullptr, out, slots, weights, nullptr, T, R, (int)N, top_k};
    return hip_status(ternary::launch_dispatch(a, dtype, stream));
}

int ternary_dispatch_backward(const void *grad, int dtype, int64_t R, int64_t N, const int32_t *slots,
                              const float *weights, int64_t T, int top_k, const void *x, const void *add, void *dx,
                              float *dweights, hipStream_t stream)
{
    const int st = exchange_shape(dtype, T, N, R, top_k);
    if (st != TERNARY_OK)
        return st;
    if (T == 0)
        return TERNARY_OK;
    if ((R && N && !grad) || !slots || (N && !dx) || (N && (weights != nullptr) != (x != nullptr)) ||
        (weights != nullptr) != (dweights != nullptr))
        return TERNARY_ERR_NULL;
    const int64_t e = elem_bytes(dtype), kbytes = 4 * T * top_k, tbytes = e * T * N;
    if (!aligned(grad, e) || !aligned(x, e) || !aligned(add, e) || !aligned(dx, e) || !aligned(slots, 4) ||
        !aligned(weights, 4) || !aligned(dweights, 4))
        return TERNARY_ERR_ALIGN;
    if (aliased({{dx, tbytes}, {dweights, kbytes}},
                {{grad, e * R * N}, {x, tbytes}, {slots, kbytes}, {weights, kbytes}}, {add, tbytes}))
        return TERNARY_ERR_ALIAS;
    const ternary::ExchangeArgs a = {x, grad, add, dx, slots, weights, dweights, T, R, (int)N, top_k};
    return hip_status(ternary::launch_dispatch_back(a, dtype, stream));
}

int ternary_combine_backward(const void *grad, const void *y, int dtype, int64_t R, int64_t N, const int32_t *slots,
                             const float *weights, int64_t T, int top_k, void *dy, float *dweights, hipStream_t stream)
{
    const int st = exchange_shape(dtype, T, N, R, top_k);
    if (st != TERNARY_OK)
        return st;
    if (T == 0)
        return TERNARY_OK;
    if ((R && N && (!grad || !y || !dy)) || !slots || !weights || !dweights)
        return TERNARY_ERR_NULL;
    const int64_t e = elem_bytes(dtype), kbytes = 4 * T * top_k, rbytes = e * R * N;
    if (!aligned(grad, e) || !aligned(y, e) || !aligned(dy, e) || !aligned(slots, 4) || !aligned(weights, 4) ||
        !aligned(dweights, 4))
        return TERNARY_ERR_ALIGN;
    if (aliased({{dy, rbytes}, {dweights, kbytes}},
                {{grad, e * T * N}, {y, rbytes}, {slots, kbytes}, {weights, kbytes}}))
        return TERNARY_ERR_ALIAS;
    const ternary::ExchangeArgs a = {y, grad, nullptr, dy, slots, weights, dweights, T, R, (int)N, top_k};
    return hip_status(ternary::launch_combine_back(a, dtype, stream));
}

int64_t ternary_linear_adapters_workspace(int64_t T, int64_t K, int64_t N, int64_t rank, int64_t E)
{
    const int st = adapters_shape(TERNARY_BF16, T, K, N, rank, E);
    return st == TERNARY_OK ? ternary::adapters_workspace(T, K, N, rank, E) : st;
}

int64_t ternary_linear_adapters_backward_workspace(int64_t T, int64_t K, int64_t N, int64_t rank, int64_t E)
{
    const int st = adapters_shape(TERNARY_BF16, T, K, N, rank, E);
    return st == TERNARY_OK ? ternary::adapters_back_workspace(T, K, N, rank, E) : st;
}

int ternary_linear_adapters(const void *x, int dtype, int64_t T, int64_t K, int64_t N, int64_t rank, const void *a,
                            const void *b, int64_t E, const float *scale, const int32_t *offsets,
                            const int32_t *order, const int32_t *slots, const void *add, void *y, float *hidden,
                            void *workspace, hipStream_t stream)
{
    const int st = adapters_shape(dtype, T, K, N, rank, E);
    if (st != TERNARY_OK)
        return st;
    if (T == 0)
        return TERNARY_OK;
    const int64_t wsbytes = ternary::adapters_workspace(T, K, N, rank, E);
    if (!x || !a || !b || !offsets || !order || !slots || !y || (wsbytes && !workspace))
        return TERNARY_ERR_NULL;
    if (!aligned(x, 2) || !aligned(a, 2) || !aligned(b, 2) || !aligned(add, 2) || !aligned(y, 2) || !aligned(scale, 4) ||
        !aligned(offsets, 4) || !aligned(order, 4) || !aligned(slots, 4) || !aligned(hidden, 16) ||
        (wsbytes && !aligned(workspace, 16)))
        return TERNARY_ERR_ALIGN;
    if (aliased({{y, 2 * T * N}, {hidden, 4 * T * rank}, {workspace, wsbytes}},
                {{x, 2 * T * K}, {a, 2 * E * rank * K}, {b, 2 * E * N * rank}, {scale, 4 * E}, {offsets, 4 * (E + 1)},
                 {order, 4 * T}, {slots, 4 * T}},
                {add, 2 * T * N}))
        return TERNARY_ERR_ALIAS;
    ternary::AdapterArgs p = {};
    p.x = static_cast<const uint16_t *>(x);
    p.a = static_cast<const uint16_t *>(a);
    p.b = static_cast<const uint16_t *>(b);
    p.add = static_cast<const uint16_t *>(add);
    p.scale = scale;
    p.offsets = offsets;
    p.order = order;
    p.slots = slots;
    p.y = static_cast<uint16_t *>(y);
    p.hidden = hidden;
    p.workspace = workspace;
    p.T = (int)T;
    p.K = (int)K;
    p.N = (int)N;
    p.rank = (int)rank;
    p.E = (int)E;
    p.fp16 = dtype == TERNARY_FP16;
    return hip_status(ternary::launch_adapters(p, stream));
}

int ternary_linear_adapters_backward(const void *grad, const void *x, const float *hidden, int dtype, int64_t T,
                                     int64_t K, int64_t N, int64_t rank, const void *a, const void *b, int64_t E,
                                     const float *scale, const int32_t *offsets, const int32_t *order,
                                     const int32_t *slots, const void *add, void *dx, void *da, void *db,
                                     void *workspace, hipStream_t stream)
{
    const int st = adapters_shape(dtype, T, K, N, rank, E);
    if (st != TERNARY_OK)
        return st;
    const int64_t wsbytes = ternary::adapters_back_workspace(T, K, N, rank, E);
    if (!offsets || !da || !db || (T && (!grad || !x || !hidden || !a || !b || !order || !slots || !dx || !workspace)))
        return TERNARY_ERR_NULL;
    if (!aligned(grad, 2) || !aligned(x, 2) || !aligned(a, 2) || !aligned(b, 2) || !aligned(add, 2) || !aligned(dx, 2) ||
        !aligned(da, 16) || !aligned(db, 16) || !aligned(scale, 4) || !aligned(offsets, 4) || !aligned(order, 4) ||
        !aligned(slots, 4) || !aligned(hidden, 16) || !aligned(workspace, 16))
        return TERNARY_ERR_ALIGN;
    const int64_t abytes = 2 * E * rank * K, bbytes = 2 * E * N * rank;
    if (aliased({{dx, 2 * T * K}, {da, abytes}, {db, bbytes}, {workspace, wsbytes}},
                {{grad, 2 * T * N}, {x, 2 * T * K}, {hidden, 4 * T * rank}, {a, abytes}, {b, bbytes}, {scale, 4 * E},
                 {offsets, 4 * (E + 1)}, {order, 4 * T}, {slots, 4 * T}},
                {add, 2 * T * K}))
        return TERNARY_ERR_ALIAS;
    ternary::AdapterArgs p = {};
    p.x = static_cast<const uint16_t *>(x);
    p.a = static_cast<const uint16_t *>(a);
    p.b = static_cast<const uint16_t *>(b);
    p.grad = static_cast<const uint16_t *>(grad);
    p.add = static_cast<const uint16_t *>(add);
    p.scale = scale;
    p.offsets = offsets;
    p.order = order;
    p.slots = slots;
    p.dx = static_cast<uint16_t *>(dx);
    p.da = static_cast<uint16_t *>(da);
    p.db = static_cast<uint16_t *>(db);
    p.hidden = const_cast<float *>(hidden);
    p.workspace = workspace;
    p.T = (int)T;
    p.K = (int)K;
    p.N = (int)N;
    p.rank = (int)rank;
    p.E = (int)E;
    p.fp16 = dtype == TERNARY_FP16;
    return hip_status(ternary::launch_adapters_back(p, stream));
}

}  // extern "C"
