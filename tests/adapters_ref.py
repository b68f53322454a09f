"""Plain 64-bit definitions of sorted slots' exchange, its gradients and the low-rank adapters (numpy, CPU), and the
inputs their tests share.  No code of the library is used."""

import numpy as np
import torch

import fp8_ref as ref

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}  # half the smallest step
STEP = 2.0 ** -24   # a rounding to fp32, of the value
SUM = 2.0 ** -23    # an addition of the matrix unit, which may cut instead of rounding


def sort_slots(ids, E):
    """ref.sort_slots, where ids outside [0, E) count as none."""
    return ref.sort_slots(np.where((ids >= 0) & (ids < E), ids, -1).astype(np.int32), E)


def dispatch(x, w, slots):
    """float64 x [T, N], weights [T, k] -> rows [T * k, N]; rows without a slot NaN."""
    T, k = slots.shape
    out = np.full((T * k, x.shape[1]), np.nan)
    for t in range(T):
        for j in range(k):
            if slots[t, j] >= 0:
                out[slots[t, j]] = w[t, j] * x[t]
    return out


def combine(y, w, slots, add=0):
    has = slots >= 0
    return np.where(has[:, :, None], y[np.maximum(slots, 0)] * w[:, :, None], 0).sum(1) + add


def combine_backward(g, y, w, slots):
    """dy (NaN where no slot is), dweights."""
    has = slots >= 0
    dw = np.where(has, (np.where(has[:, :, None], y[np.maximum(slots, 0)], 0) * g[:, None, :]).sum(2), 0)
    return dispatch(g, w, slots), dw


def dispatch_backward(g, w, slots, x, add=0):
    """dx, dweights."""
    has = slots >= 0
    rows = np.where(has[:, :, None], g[np.maximum(slots, 0)], 0)
    return (rows * w[:, :, None]).sum(1) + add, (rows * x[:, None, :]).sum(2)


def adapters(x, a, b, s, of, add=0):
    """y [T, N], hidden [T, rank] (0 for tokens without an adapter); `of`: each token's adapter, or -1."""
    T, N, rank = x.shape[0], b.shape[1], a.shape[1]
    y, v = np.zeros((T, N)), np.zeros((T, rank))
    for e in range(a.shape[0]):
        at = of == e
        v[at] = x[at] @ a[e].T
        y[at] = s[e] * (v[at] @ b[e].T)
    return y + add, v


def adapters_backward(g, x, hidden, a, b, s, of, add=0):
    """dx, da, db, and dv."""
    dx, dv, da, db = np.zeros(x.shape), np.zeros(hidden.shape), np.zeros(a.shape), np.zeros(b.shape)
    for e in range(a.shape[0]):
        at = of == e
        dv[at] = s[e] * (g[at] @ b[e])
        dx[at] = dv[at] @ a[e]
        da[e] = dv[at].T @ x[at]
        db[e] = s[e] * (g[at].T @ hidden[at])
    return dx + add, da, db, dv


def wide(t):
    return t.double().cpu().numpy()


def routing(tl, ids, w, E):
    off, order, slots = sort_slots(ids, E)
    return tl.Routing(*(ref.dev(v) for v in (ids.astype(np.int32), w.astype(np.float32), off, order, slots)))


def guarded(shape, dtype, value=77.0, shift=0):
    """A tensor inside a buffer of `value`, `shift` elements off a 16-byte boundary, and the buffer."""
    n = int(np.prod(shape))
    buf = torch.full((n + 128,), value, dtype=dtype, device="cuda")
    return buf[64 + shift:64 + shift + n].view(shape), buf


def shifted(t, shift):
    """A copy of t whose first element lies `shift` elements off a 16-byte boundary."""
    if t is None or not shift:
        return t
    v, _ = guarded(t.shape, t.dtype, 0, shift)
    v.copy_(t)
    return v


def untouched(view, buf, value=77.0):
    """Whether the buffer around the view still holds its value."""
    lo = (view.data_ptr() - buf.data_ptr()) // buf.element_size()
    return bool((buf[:lo] == value).all()) and bool((buf[lo + view.numel():] == value).all())
