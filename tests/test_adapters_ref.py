"""The gradients' 64-bit formulas against differences of the forward definitions (CPU)."""

import numpy as np
import pytest

import adapters_ref as ar


def numeric(f, x, h=1e-5):
    """d f / d x by central differences, f a number."""
    g = np.zeros(x.shape)
    for i in np.ndindex(*x.shape):
        keep = x[i]
        x[i] = keep + h
        up = f()
        x[i] = keep - h
        g[i] = (up - f()) / (2 * h)
        x[i] = keep
    return g


def near(a, b):
    # f is at most quadratic in each argument: central differences are exact but for roundings, 1e-16 * |f| / h
    assert np.abs(a - b).max(initial=0) < 1e-7


@pytest.mark.parametrize("masked", [0, 2])
def test_exchange(masked):
    rng = np.random.default_rng(masked)
    T, k, E, N = 5, 3, 4, 6
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    ids[T - masked:] = -1
    ids[0, 1] = E + 3
    _, _, slots = ar.sort_slots(ids, E)
    x, w, y = rng.standard_normal((T, N)), rng.random((T, k)), rng.standard_normal((T * k, N))
    g, gr = rng.standard_normal((T, N)), rng.standard_normal((T * k, N))
    used = int((slots >= 0).sum())
    dy, dw = ar.combine_backward(g, y, w, slots)
    near(np.nan_to_num(dy), numeric(lambda: (ar.combine(y, w, slots) * g).sum(), y))
    near(dw, numeric(lambda: (ar.combine(y, w, slots) * g).sum(), w))
    assert np.isnan(dy[used:]).all()
    dx, dw = ar.dispatch_backward(gr, w, slots, x)
    near(dx, numeric(lambda: np.nansum(ar.dispatch(x, w, slots) * gr), x))
    near(dw, numeric(lambda: np.nansum(ar.dispatch(x, w, slots) * gr), w))


def test_adapters():
    rng = np.random.default_rng(3)
    T, K, N, rank, E = 7, 5, 4, 3, 3
    of = np.array([2, 0, -1, 2, 2, 0, -1])  # adapter 1 has no tokens
    x, a, b = rng.standard_normal((T, K)), rng.standard_normal((E, rank, K)), rng.standard_normal((E, N, rank))
    s, g = rng.random(E) + 0.5, rng.standard_normal((T, N))

    def f():
        return (ar.adapters(x, a, b, s, of)[0] * g).sum()

    dx, da, db, _ = ar.adapters_backward(g, x, ar.adapters(x, a, b, s, of)[1], a, b, s, of)
    for got, at in ((dx, x), (da, a), (db, b)):
        near(got, numeric(f, at))
    assert not da[1].any() and not db[1].any() and not dx[of < 0].any()
