"""linear_experts at the most places that it takes: their tiles are more than one launch may hold."""

import numpy as np
import pytest
import torch

import fp8_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [1, 40])  # streamed; in tiles of 128 places (80 GB of outputs)
def test_experts_most_places(N):
    import gemm_ternary_linear_amd as tl
    R, E, k, n, K = 1 << 30, 2, 32, 64, 8
    say(f"experts, {R} places of {N}")
    rng = np.random.default_rng(1)
    x, xs = ref.codes_of(rng, n, 128), ref.scales_of(rng, n, 1)
    x[:, K:] = 0
    q, s = rng.integers(-1, 2, (E, N, K)).astype(np.int8), ref.scales_of(rng, E, N).astype(np.float16)
    want = np.stack([ref.wide(x, xs)[:, :K] @ (q[e] * s[e].astype(np.float64)[:, None]).T for e in range(E)])
    codes = torch.stack([torch.from_numpy(ref.tile_codes(e)) for e in q]).cuda()
    order = torch.arange(n * k, dtype=torch.int32, device="cuda").repeat(R // (n * k))
    last = R - 5  # where the second expert's places begin
    offsets = torch.tensor([0, last, R], dtype=torch.int32, device="cuda")
    y = torch.full((R, N), 77.0, dtype=torch.float16, device="cuda")
    xd, xsd, sd = ref.fp8_dev(x), ref.dev(xs), ref.dev(s)
    st = tl.lib().ternary_linear_experts(xd.data_ptr(), xsd.data_ptr(), n, codes.data_ptr(), sd.data_ptr(), E, N, K, -1,
                                         offsets.data_ptr(), order.data_ptr(), R, k, 0, y.data_ptr(), tl.FP16,
                                         torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0
    rows = torch.from_numpy(want).cuda().half().repeat_interleave(k, 1)  # (whole numbers and quarters: exact)
    assert torch.equal(y[last:], rows[1][n * k - 5:])
    y[last:] = rows[0][n * k - 5:]
    for part in y.view(-1, n * k * N).split(1 << 14):
        assert bool((part == rows[0].reshape(-1)).all())
    del y, part
    torch.cuda.empty_cache()
