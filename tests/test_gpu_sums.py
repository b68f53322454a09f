"""The products' inner sums: a factor that dwarfs the others beside it leaves their products whole.  A sum that
aligned its products to the largest and cut what falls 2^-14 below would lose them."""

import numpy as np
import pytest
import torch

import fp8_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def tl():
    import gemm_ternary_linear_amd as tl
    return tl


def code(v):
    return ref.nearest_code(np.asarray(v, np.float64))


def outliers(rng, x, big):
    """Puts +big and -big beside each other (within one aligned run of 8) into every row and block of 128 of the values
    x, at the places returned; every fourth row keeps only the first of its first block's two."""
    places = []
    for b in range(x.shape[1] // 128):
        p, q = 128 * b + 8 * rng.integers(16) + rng.choice(8, 2, replace=False)
        x[:, p], x[:, q] = big, -big
        if b == 0:
            x[3::4, q] = 0
        places += [p, q]
    return places


# every kernel of the products: few rows, then tiles of rows of each size
@pytest.mark.parametrize("M,N,K", [(1, 48, 512), (8, 80, 1024), (16, 4112, 128), (20, 100, 384), (33, 129, 256), (60, 200, 1664), (64, 18944, 128),
                                   (70, 16500, 256), (500, 1100, 384), (384, 6000, 256), (1030, 2050, 256), (2048, 2304, 128),
                                   # 17 to 48 rows: one to five fragments of channels a wave (on 256 compute units)
                                   (17, 8192, 256), (25, 12288, 384), (32, 16384, 128), (31, 18944, 256), (40, 8192, 128), (48, 12200, 256), (45, 16384, 384),
                                   (41, 18950, 256), (130, 8200, 384), (3000, 4100, 384), (381, 18943, 1152)])
def test_linear_outliers(tl, M, N, K):
    """Products of 2^16, cancelling, beside others of 225/64: every partial sum is a multiple of 2^-6 below 2^17, so
    sums of 24 bits are exact in any order, and every output bit is known."""
    say(f"linear outliers {M} {N} {K}")
    rng = np.random.default_rng(M + N + K)
    x, w = 1.875 * rng.choice([-1, 1], (M, K)), 1.875 * rng.choice([-1, 1], (N, K))
    w[:, outliers(rng, x, 256.0)] = 256.0
    xs, ws = np.full((M, K // 128), 2.0 ** -3, np.float32), np.full(((N + 127) // 128, K // 128), 2.0 ** -3, np.float32)
    y = x @ w.T / 64
    for name, dt in DT.items():
        got = tl.fp8_linear(ref.fp8_dev(code(x)), ref.dev(xs), ref.fp8_dev(code(w)), ref.dev(ws), dtype=dt)
        assert np.array_equal(got.double().cpu().numpy(), ref.rounded(y, dt)), name


@pytest.mark.parametrize("rows", ["tokens", "sorted"])
@pytest.mark.parametrize("T,E,k,N,K,g", [(1, 8, 2, 64, 512, -1), (2, 4, 2, 100, 384, 128), (9, 3, 1, 4112, 256, 256), (40, 16, 4, 33, 2048, -1),
                                         (200, 4, 2, 300, 640, -1), (300, 5, 2, 140, 512, 128), (700, 3, 2, 272, 768, 256),
                                         # tiles of 128 places
                                         (3000, 4, 2, 2100, 512, -1), (3001, 4, 2, 2100, 640, 128), (2000, 4, 3, 2050, 768, 256)])
def test_experts_outliers(tl, T, E, k, N, K, g, rows):
    """Factors of 448, cancelling, beside others of 7 x 2^-9: partial sums are multiples of 2^-9 below 2^10."""
    say(f"experts outliers {T} {E} {k} {N} {K} g={g} {rows}")
    rng = np.random.default_rng(T + E + N + K)
    ids = np.stack([rng.choice(E, k, replace=False) for _ in range(T)]).astype(np.int32)
    off, order, slots = ref.sort_slots(ids, E)
    x = 7 * 2.0 ** -9 * rng.choice([-1, 1], (T if rows == "tokens" else T * k, K))
    q = rng.integers(-1, 2, (E, N, K)).astype(np.int8)
    q[:, :, outliers(rng, x, 448.0)] = 1
    s = ref.scales_of(rng, *((E, N) if g == -1 else (E, N, K // g))).astype(np.float16)
    s[:] = s[..., :1] if g > 0 else s  # (one scale for all of a channel's groups: blocks' sums stay on one grid)
    xs = np.full((len(x), K // 128), 0.5, np.float32)
    y = np.zeros((T * k, N))
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        at = order[lo:hi] // k if rows == "tokens" else np.arange(lo, hi)
        y[lo:hi] = 0.5 * (x[at] @ q[e].T) * (s[e] if g == -1 else s[e][:, 0]).astype(np.float64)
    codes = torch.stack([torch.from_numpy(ref.tile_codes(e)) for e in q]).cuda()
    r = tl.Routing(ref.dev(ids), ref.dev(np.zeros((T, k), np.float32)), ref.dev(off), ref.dev(order), ref.dev(slots))
    for name, dt in DT.items():
        got = tl.linear_experts(ref.fp8_dev(code(x)), ref.dev(xs), codes, ref.dev(s), r, K=K, rows=rows, dtype=dt)
        assert np.array_equal(got.double().cpu().numpy(), ref.rounded(y, dt)), name
