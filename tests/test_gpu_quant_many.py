"""quant_rows of more rows than one launch takes (weights of many experts): against the
definition in 64 bits, and the overlaps that no single launch sees."""

import pytest
import torch

pytestmark = pytest.mark.gpu

ROWS = (1 << 24) + 16


@pytest.fixture(scope="module")
def mg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import token_routing_amd as m
    m.load_library()
    return m


def want(x):
    v = x.double()
    m = v.abs().amax(-1, keepdim=True)
    # torch divides fp32 by a number as a product with its reciprocal; a quotient of 64 bits
    # rounded to 24 is the rounded real one (53 >= 2 * 24 + 2)
    return (torch.round(127 * v / torch.where(m > 0, m, 1.0)).to(torch.int8),
            (m[..., 0] / 127).float())


def test_many_rows(mg):
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(ROWS, 4, generator=g, device="cuda").bfloat16()[:, :3]    # rows 4 apart
    q, s = mg.quant_rows(x)
    codes, scales = want(x)
    assert torch.equal(q[:, :3], codes) and not q[:, 3:].any() and torch.equal(s, scales)


def test_many_weights(mg):
    g = torch.Generator(device="cuda").manual_seed(2)
    w = torch.randn(4, ROWS // 4, 5, generator=g, device="cuda")
    q = torch.full((4, ROWS // 4, 16), 9, dtype=torch.int8, device="cuda")
    got, s = mg.quant_rows(w, Q=q)
    codes, scales = want(w)
    assert got is q and torch.equal(q[..., :5], codes) and not q[..., 5:].any()
    assert torch.equal(s, scales)


def test_overlaps_of_different_launches(mg):
    """Q over rows of X that a later launch reads: refused as in one launch."""
    buf = torch.zeros(ROWS * 48, dtype=torch.uint8, device="cuda")
    x = buf[:ROWS * 32].view(torch.bfloat16).view(ROWS, 16)
    for at in ((ROWS - 8) * 32, 0):
        with pytest.raises(ValueError):
            mg.quant_rows(x, Q=buf[at:at + ROWS * 16].view(torch.int8).view(ROWS, 16))
    q = buf[ROWS * 32:].view(torch.int8).view(ROWS, 16)
    assert mg.quant_rows(x, Q=q)[0] is q
