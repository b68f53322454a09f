"""fp8_quantize: the sign of a zero, whatever blocks its wave holds beside it."""

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


def codes(tl, x, **kw):
    return tl.fp8_quantize(torch.from_numpy(x).cuda(), **kw)[0].view(torch.uint8).cpu().numpy()


@pytest.mark.parametrize("block", ["row", "tile"])
@pytest.mark.parametrize("beside", ["values", "zeros", "infinity", "small"])
def test_negative_zero(tl, block, beside):
    """-0 beside other numbers is the code 0x80: -0 / s is -0.  Four blocks of a row share a wave."""
    say(f"-0 {block} {beside}")
    x = np.tile(np.linspace(-3, 5, 128, dtype=np.float32), (5, 4))
    x[:, ::5] = -0.0
    x[:, 1::5] = 0.0
    x[:, 2] = -1e-30  # (its quotient is below every code: -0 too)
    if beside == "zeros":
        x[:, 128:256] = 0
    elif beside == "infinity":
        x[1, 200] = np.inf
    elif beside == "small":
        x[:, 128:256] = 2.0 ** -120
    got = codes(tl, x, block=block)
    want, _ = ref.quantize(x, block == "tile")
    assert np.array_equal(np.where(got == 0xff, 0x7f, got), want)
    assert (got[0, :128:5] == 0x80).all() and (got[0, 1:128:5] == 0).all()


@pytest.mark.parametrize("vec", [True, False])
def test_negative_zero_swiglu(tl, vec):
    """silu of far negative gates underflows to -0, and silu(-0) is -0: the product's sign is the code's."""
    say(f"-0 swiglu {vec}")
    K = 256 if vec else 255
    g, u = np.full((3, K), 1.5, np.float32), np.ones((3, K), np.float32)
    g[:, 3:20] = -200
    g[:, 30:40] = -0.0
    g[:, 50:60] = 0.0
    u[:, 10:20] = -1
    u[:, 35:40] = -2
    u[:, 55:60] = -2
    g[2, 128:] = 0  # (a block with scale 0: its codes are 0 whatever the signs)
    got = codes(tl, np.concatenate([g, u], 1), act="swiglu")
    want = np.zeros(K, np.uint8)
    want[3:10] = want[30:35] = want[55:60] = 0x80
    low = [*range(3, 20), *range(30, 40), *range(50, 60)]
    assert (got[:, low] == want[low]).all(), got[:, low]
    assert (got[2, 128:] == 0).all() and (got[:2, 128:K] == 0x7e).all() and (got[:, :3] == 0x7e).all()
