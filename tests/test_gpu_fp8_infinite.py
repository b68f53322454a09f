"""Infinite block scales: the outputs that they reach are infinite with the block's sign, as by the definition, and not
NaN because of how many blocks a kernel takes at a time."""

import numpy as np
import pytest
import torch

import fp8_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tl():
    import gemm_ternary_linear_amd as tl
    return tl


@pytest.mark.parametrize("M", [1, 20, 40, 60, 300, 700])
@pytest.mark.parametrize("nb", [1, 3, 5])
def test_linear_infinite_scale(tl, M, nb):
    say(f"linear infinite scale M={M} nb={nb}")
    rng = np.random.default_rng(M + nb)
    N, K = 200, 128 * nb
    x, w = ref.codes_of(rng, M, K), ref.codes_of(rng, N, K)
    x[:, -1], w[:, -1] = ref.nearest_code(np.array(9.0)), ref.nearest_code(np.array(0.0))  # (sums may be any whole number)
    xs, ws = ref.scales_of(rng, M, nb), ref.scales_of(rng, 2, nb)
    ws[1, nb - 1] = np.inf
    xs[M // 2, 0] = np.inf
    y = np.zeros((M, N))
    with np.errstate(invalid="ignore"):
        for b in range(nb):
            s = ref.TABLE[x[:, 128 * b:128 * b + 128]] @ ref.TABLE[w[:, 128 * b:128 * b + 128]].T
            y += s * (xs[:, b, None].astype(np.float64) * np.repeat(ws[:, b], 128)[:N].astype(np.float64))
    assert np.isinf(y[:, 128:]).any()
    got = tl.fp8_linear(ref.fp8_dev(x), ref.dev(xs), ref.fp8_dev(w), ref.dev(ws), dtype=torch.float32).cpu().numpy()
    assert np.array_equal(got, y, equal_nan=True)


@pytest.mark.parametrize("T", [2, 300])
@pytest.mark.parametrize("K,g", [(128, 128), (384, 128), (640, 128), (768, 256)])
def test_experts_infinite_scale(tl, T, K, g):
    say(f"experts infinite scale T={T} K={K} g={g}")
    rng = np.random.default_rng(T + K)
    E, N, nb = 3, 70, K // 128
    ids = rng.integers(0, E, (T, 1)).astype(np.int32)
    off, order, slots = ref.sort_slots(ids, E)
    x, xs = ref.codes_of(rng, T, K), ref.scales_of(rng, T, nb)
    q = rng.integers(-1, 2, (E, N, K)).astype(np.int8)
    s = ref.scales_of(rng, E, N, K // g).astype(np.float16)
    s[:, 5, K // g - 1] = np.inf
    y = np.zeros((T, N))
    with np.errstate(invalid="ignore"):
        for r in range(T):
            t, e = order[r], ids[order[r], 0]
            for b in range(nb):
                cut = slice(128 * b, 128 * b + 128)
                y[r] += (q[e][:, cut] @ ref.TABLE[x[t, cut]]) * (xs[t, b].astype(np.float64) * s[e][:, 128 * b // g])
    codes = torch.stack([torch.from_numpy(ref.tile_codes(e)) for e in q]).cuda()
    r = tl.Routing(ref.dev(ids), ref.dev(np.zeros((T, 1), np.float32)), ref.dev(off), ref.dev(order), ref.dev(slots))
    assert np.isinf(y[:, 5]).any() and np.isfinite(np.delete(y, 5, 1)).all()
    got = tl.linear_experts(ref.fp8_dev(x), ref.dev(xs), codes, ref.dev(s), r, dtype=torch.float32).cpu().numpy()
    assert np.array_equal(got, y, equal_nan=True)
