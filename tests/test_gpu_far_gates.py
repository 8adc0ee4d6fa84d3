"""Gates where the activation leaves fp32's normal numbers.  With z(g) as in tests/_block.py,
act(g) = g s(z) and s is taken as 0 where 1 + e^-z passes 2^126: there |g s| <= 87.4 * 2^-126 <
1.1e-36 for silu (less for gelu, whose |g| is about 10), and the slope s + g s (1 - s) z'(g) is at
most (1 + 10.2 * 23.9) 2^-126 < 3e-36 (gelu; silu 88.4 * 2^-126)."""

import numpy as np
import pytest
import torch

from tests._block import HALF, act_ref, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gates_at_the_end_of_fp32(act):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import token_routing_amd as mg
    far = torch.linspace(-80, -110, 256) if act == "silu" else torch.linspace(-5, -12, 256)
    I = far.numel()
    kept = torch.cat([far, torch.ones(I)]).bfloat16().view(1, 2 * I).cuda()
    dy = torch.ones(1, 8, dtype=torch.bfloat16, device="cuda")
    w = torch.full((1, 8, I), 0.125, dtype=torch.bfloat16, device="cuda")     # dH = 1
    m = torch.ones(1, dtype=torch.int32, device="cuda")
    f = (mg.GATED_SILU if act == "silu" else mg.GATED_GELU) | mg.GATED_HALVES
    da, h = mg.gated_bwd(dy, w, kept, m, None, 1, f)
    g = f64(far.bfloat16())
    a, d, ea, ed = act_ref(g, act)
    dg, du, hh = f64(da)[0, :I], f64(da)[0, I:], f64(h)[0]
    for got in (hh, du):
        assert (np.abs(got - a) <= (np.abs(a) + ea) * HALF + ea + 1.1e-36).all()
    assert (np.abs(dg - d) <= (np.abs(d) + ed) * HALF + ed + 3e-36).all()
    z = g if act == "silu" else 2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)
    assert (hh[z < -88] == 0).all() and (hh[z > -87] < 0).all()
