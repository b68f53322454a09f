"""fp8_quantize's SwiGLU to fp32's own precision, down to where silu leaves fp32."""

import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tl():
    import gemm_ternary_linear_amd as tl
    return tl


@pytest.mark.parametrize("vec", [True, False])
def test_swiglu_precision(tl, vec):
    """A row of one value v is its scale times 448.  Roundings of v: exp2 within 2^-23, its corrected argument, the gate times
    it, 1 + it, the quotient, the product with up, v / 448: 8 x 2^-24 in all.  (448 s in 64 bits adds nothing; silu itself may be
    subnormal, the product is not.)"""
    say(f"swiglu precision {vec}")
    K = 128 if vec else 127
    gates = torch.cat([torch.linspace(-103, -60, 431), torch.linspace(-60, 60, 2407),
                       torch.tensor([-87.3, -87.34, -87.5, -88, -88.5, -88.72, -88.73, -89, -20.0001, -20, -19.9999, -1e-3, -1e-30, 1e-30, 1e-3,
                                     17.3, 17.4, 19.9999, 20, 20.0001, 88.8, 1e4, 3e38])]).float()
    up = torch.where(gates < -40, torch.tensor(1e30), torch.tensor(0.75))
    want = gates.double() / (1 + torch.exp(-gates.double())) * up.double()
    x = torch.cat([gates[:, None].expand(-1, K), up[:, None].expand(-1, K)], 1).contiguous()
    q, s = tl.fp8_quantize(x.cuda(), act="swiglu")
    got = s[:, 0].cpu().double() * 448 * torch.sign(want)
    off = (got - want).abs()
    bad = off > want.abs() * 8 * 2.0 ** -24
    assert not bad.any(), [(float(g), float(a), float(b)) for g, a, b in zip(gates[bad][:9], got[bad][:9], want[bad][:9])]
    codes = q.view(torch.uint8)[:, :K].cpu()
    assert (codes == torch.where(want < 0, 0xfe, 0x7e).to(torch.uint8)[:, None]).all()
