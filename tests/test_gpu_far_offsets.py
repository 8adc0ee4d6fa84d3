"""Rows whose offset passes 2^31 elements: the gate, permute, unpermute and the
adapters on a few rows spread over 5 GB arrays, against the same rows packed
together (equal bit for bit: the same sums in the same order)."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import token_routing_amd as m
    m.load_library()
    return m


def test_gate_rows_far_apart(mg):
    T, E, ld = 1300, 64, 1 << 21                    # the last row starts at 2.7e9
    wide = torch.empty(T * ld, dtype=torch.bfloat16, device="cuda").view(T, ld)
    l = torch.randn(T, E, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    wide[:, 5:5 + E] = l
    ids, w, s = mg.moe_gate(wide[:, 5:5 + E], 4, renorm=True, want_scores=True)
    ids2, w2, s2 = mg.moe_gate(l, 4, renorm=True, want_scores=True)
    assert torch.equal(ids, ids2) and torch.equal(w, w2) and torch.equal(s, s2)
    assert torch.equal(mg.moe_gate_bwd(wide[:, 5:5 + E], ids, w, dscores=s, renorm=True),
                       mg.moe_gate_bwd(l, ids, w, dscores=s, renorm=True))


def test_permuted_rows_far_apart(mg):
    T, k, K, rows = 50, 3, 8191, 320000             # the last row starts at 2.6e9
    g = torch.Generator().manual_seed(2)
    at = torch.randperm(rows, generator=g)[:T * k]
    at[7] = rows - 1
    far, near = at.int().cuda(), torch.arange(T * k, dtype=torch.int32).cuda()
    X = torch.randn(T, K, generator=g).bfloat16().cuda()
    w = torch.rand(T * k, generator=g).cuda()
    big = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda")
    mg.permute(X, far, k, w, Xs=big)
    small, _ = mg.permute(X, near, k, w)
    assert torch.equal(big[at.cuda()], small)
    assert torch.equal(mg.unpermute(big, k, far, w, base=X), mg.unpermute(small, k, near, w, base=X))
    a, da = mg.permute_bwd(big, X, k, far, w)
    b, db = mg.permute_bwd(small, X, k, near, w)
    assert torch.equal(a, b) and torch.equal(da, db)
    other = torch.empty_like(big)
    a, da = mg.unpermute_bwd(X, big, k, far, w, dY=other)
    b, db = mg.unpermute_bwd(X, small, k, near, w)
    assert torch.equal(a[at.cuda()], b) and torch.equal(da, db)


def test_adapter_rows_far_apart(mg):
    n, L, R, K, N, ld = 90, 4, 16, 264, 328, 1 << 15
    T = 70000                                        # the last row starts at 2.3e9
    g = torch.Generator().manual_seed(3)
    rows = torch.sort(torch.randperm(T, generator=g)[:n]).values
    rows[-1] = T - 1
    ids = torch.full((T,), -1, dtype=torch.int32)
    ids[rows] = torch.randint(0, L, (n,), generator=g, dtype=torch.int32)
    r = mg.moe_route(ids.cuda().view(-1, 1), L, 16)
    r2 = mg.moe_route(ids[rows].cuda().view(-1, 1), L, 16)
    assert torch.equal(r["m_sizes"], r2["m_sizes"])
    A = (torch.randn(L, R, K, generator=g) / 16).bfloat16().cuda()
    B = torch.randn(L, N, R, generator=g).bfloat16().cuda()
    wide = torch.empty(T * ld, dtype=torch.bfloat16, device="cuda").view(T, ld)
    X, Y = wide[:, :K], wide[:, 1001:1001 + N]
    x = torch.randn(n, K, generator=g).bfloat16().cuda()
    y = torch.randn(n, N, generator=g).bfloat16().cuda()
    at = rows.cuda()
    wide[at, :K] = x
    wide[at, 1001:1001 + N] = y
    # a tile's size follows from rows per adapter, and splits from T: the same
    # sums only where both are the same, so the far rows are held to the bf16
    # result within one step
    _, H = mg.lora_fwd(X, A, B, r["m_sizes"], r["gather"], Y=Y, want_h=True)
    got = wide[at, 1001:1001 + N].double()
    y2, h2 = mg.lora_fwd(x, A, B, r2["m_sizes"], r2["gather"], base=y, want_h=True)
    assert torch.all((H[:n] - h2).abs() <= 2 * K * 2.0 ** -23 * h2.abs().max())
    assert torch.all((got - y2.double()).abs() <= 2.0 ** -7 * y2.double().abs() + 2.0 ** -10)
    dX = torch.empty(T * ld, dtype=torch.bfloat16, device="cuda").view(T, ld)[:, 77:77 + K]
    dX[at] = x
    _, dA, dB = mg.lora_bwd(X, Y, A, B, H, r["m_sizes"], r["gather"], dX=dX, fp32_grads=True)
    dy2 = wide[at, 1001:1001 + N].contiguous()
    dx2, dA2, dB2 = mg.lora_bwd(x, dy2, A, B, H[:n], r2["m_sizes"], r2["gather"], base=x,
                                fp32_grads=True)
    assert torch.all((dX[at].double() - dx2.double()).abs()
                     <= 2.0 ** -7 * dx2.double().abs() + 2.0 ** -10 * dx2.double().abs().max())
    for a, b in ((dA, dA2), (dB, dB2)):
        assert float((a - b).norm() / b.norm()) <= 2.0 ** -14
