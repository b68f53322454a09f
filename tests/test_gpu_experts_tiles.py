"""linear_experts where its tiles of 64 and of 128 places are chosen (many places times many channels): padded tokens, places
left as they were, NaN, indices that describe no routing."""

import numpy as np
import pytest
import torch

import fp8_ref as ref
import test_gpu_experts as few
from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tl():
    import gemm_ternary_linear_amd as tl
    return tl


# tiles of 64 places, of 64 with several rounds, of 128
SIZES = [(500, 4, 2, 1300, 384), (640, 8, 3, 1410, 256), (3001, 4, 2, 2100, 640)]


@pytest.mark.parametrize("rows", ["tokens", "sorted"])
@pytest.mark.parametrize("g", [-1, 128])
@pytest.mark.parametrize("T,E,k,N,K", SIZES)
def test_tiles_exact(tl, T, E, k, N, K, g, rows):
    few.test_experts_exact(tl, T, E, k, N, K, g, T // 9, 1, rows)


@pytest.mark.parametrize("T,E,k,N,K", [(500, 4, 2, 1300, 388), (2500, 4, 2, 2100, 132), (1500, 70, 3, 1301, 512)])
def test_tiles_odd(tl, T, E, k, N, K):
    few.test_experts_exact(tl, T, E, k, N, K, 256 if K % 256 == 0 else -1, 3, 3, "tokens")


@pytest.mark.parametrize("T,E,k,N,K", SIZES)
def test_tiles_rows_apart(tl, T, E, k, N, K):
    """A NaN in one token's x shows in that token's rows only; a NaN scale of an expert in that channel only."""
    say(f"experts' tiles NaN T={T}")
    rng = np.random.default_rng(T)
    ids = few.draw_ids(rng, T, E, k, 0, 0)
    xq, xs = ref.codes_of(rng, T, K), ref.scales_of(rng, T, K // 128)
    q = rng.integers(-1, 2, (E, N, K)).astype(np.int8)
    s = ref.scales_of(rng, E, N).astype(np.float16)
    y, _ = few.experts_ref(ref.wide(xq, xs), q, s, -1, ids, k, True)
    xq[T - 1, 200], xq[T // 2, 3] = 0x7f, 0xff
    s[2, 5] = np.nan
    off, order, _ = ref.sort_slots(ids, E)
    nan = np.zeros(y.shape, bool)
    nan[(order // k == T - 1) | (order // k == T // 2)] = True
    nan[off[2]:off[3], 5] = True
    codes = torch.stack([torch.from_numpy(ref.tile_codes(e)) for e in q]).cuda()
    got = tl.linear_experts(ref.fp8_dev(xq), ref.dev(xs), codes, ref.dev(s), few.routing(tl, ids, np.zeros(ids.shape, np.float32), E),
                            dtype=torch.float32).cpu().numpy()
    assert np.array_equal(np.isnan(got), nan) and np.array_equal(got[~nan], y[~nan])


@pytest.mark.parametrize("T,E,k,N,K", SIZES)
def test_tiles_foreign_indices(tl, T, E, k, N, K):
    """Offsets and order that describe no routing: nothing outside the arguments is written."""
    say(f"experts' tiles, foreign indices T={T}")
    rng = np.random.default_rng(T)
    xq, xs = ref.fp8_dev(ref.codes_of(rng, T, K)), ref.dev(ref.scales_of(rng, T, K // 128))
    codes = torch.stack([torch.from_numpy(ref.tile_codes(rng.integers(-1, 2, (N, K)).astype(np.int8))) for _ in range(E)]).cuda()
    s = ref.dev(ref.scales_of(rng, E, N).astype(np.float16))
    R = T * k
    r = few.routing(tl, few.draw_ids(rng, T, E, k, 0, 0), np.zeros((T, k), np.float32), E)
    order = torch.full((R,), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    order[::2] = -2 ** 31
    for off in ([0, R, -7, R + 100] + [2 ** 31 - 1] * (E - 3), [-2 ** 31, -5, -1] + [0] * (E - 2), list(range(E, -1, -1)), [R] * (E + 1)):
        bad = r._replace(offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), order=order)
        buf = torch.full((R * N + 64,), 77.0, device="cuda")
        tl.linear_experts(xq, xs, codes, s, bad, out=buf[32:32 + R * N].view(R, N))
        torch.cuda.synchronize()
        assert bool((buf[:32] == 77).all()) and bool((buf[32 + R * N:] == 77).all())
        if max(off) <= 0 or off[0] >= R:
            assert bool((buf == 77).all())
