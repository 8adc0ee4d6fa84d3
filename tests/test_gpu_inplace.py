"""Outputs that take the place of an input: the results of a call with buffers
of its own, bit for bit."""

import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def mg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import token_routing_amd as m
    m.load_library()
    return m


# T, k, K: one, two and four waves a row, up to eight picks and more
SORT = [(5, 1, 7), (40, 8, 515), (40, 9, 515), (33, 11, 2048), (20, 17, 129), (70, 64, 1003)]


def sorted_inputs(T, k, K, dtype):
    g = torch.Generator().manual_seed(T * k + K)
    dt = DT[dtype]
    scatter = torch.randperm(T * k, generator=g).int()
    scatter[::7] = -1                              # dropped slots
    return dict(X=torch.randn(T, K, generator=g).to(dt).cuda(), scatter=scatter.cuda(),
                rows=torch.randn(T * k, K, generator=g).to(dt).cuda(),
                w=torch.rand(T * k, generator=g).cuda())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,k,K", SORT)
def test_permute_gradient_over_its_input(mg, T, k, K, dtype):
    c = sorted_inputs(T, k, K, dtype)
    dX, dw = mg.permute_bwd(c["rows"], c["X"], k, c["scatter"], c["w"])
    X = c["X"].clone()
    got, dw2 = mg.permute_bwd(c["rows"], X, k, c["scatter"], c["w"], dX=X)
    assert got is X and torch.equal(X, dX) and torch.equal(dw2, dw)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,k,K", SORT)
def test_unpermute_gradient_over_its_input(mg, T, k, K, dtype):
    c = sorted_inputs(T, k, K, dtype)
    want = c["rows"].clone()                       # rows no slot maps to stay
    _, dw = mg.unpermute_bwd(c["X"], c["rows"], k, c["scatter"], c["w"], dY=want)
    Y = c["rows"].clone()
    _, dw2 = mg.unpermute_bwd(c["X"], Y, k, c["scatter"], c["w"], dY=Y)
    assert torch.equal(Y, want) and torch.equal(dw2, dw)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,k,K", SORT)
def test_unpermute_onto_its_base(mg, T, k, K, dtype):
    c = sorted_inputs(T, k, K, dtype)
    want = mg.unpermute(c["rows"], k, c["scatter"], c["w"], base=c["X"])
    X = c["X"].clone()
    mg.unpermute(c["rows"], k, c["scatter"], c["w"], base=X, out=X)
    assert torch.equal(X, want)


def test_adapter_gradients_beside_their_inputs(mg):
    """X, dY and dX as column slices of one matrix; dX over dY where no weight
    gradients are asked for; and the refusals."""
    T, L, R, K = 70, 3, 16, 72
    g = torch.Generator().manual_seed(1)

    def rnd(*s):
        return torch.randn(*s, generator=g).bfloat16().cuda()

    sizes = torch.tensor([30, 0, 40], dtype=torch.int32).cuda()
    X, dY, base, A, B = rnd(T, K), rnd(T, K), rnd(T, K), rnd(L, R, K), rnd(L, K, R)
    H = torch.randn(T, R, generator=g).cuda()
    want = mg.lora_bwd(X, dY, A, B, H, sizes, base=base)
    wide = torch.zeros(T, 3 * K + 5, dtype=torch.bfloat16, device="cuda")
    x, d, o = (wide[:, i * K + 2:(i + 1) * K + 2] for i in (0, 2, 1))
    x.copy_(X)
    d.copy_(dY)
    got = mg.lora_bwd(x, d, A, B, H, sizes, base=base, dX=o)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    over = dY.clone()
    mg.lora_bwd(None, over, A, B, None, sizes, base=base, dX=over, want_weights=False)
    assert torch.equal(over, want[0])
    for dX in (X, dY):
        with pytest.raises(Exception, match="moegg_lora_bwd"):
            mg.lora_bwd(X, dY, A, B, H, sizes, base=base, dX=dX)


# E, k, bias, groups, sigmoid, renorm
GATE = [(8, 2, False, 1, False, True), (60, 6, True, 1, False, False), (64, 8, True, 8, True, True),
        (128, 8, False, 1, True, False), (256, 8, True, 8, False, False),
        (511, 10, True, 1, True, False), (1024, 64, False, 8, False, True)]


@pytest.mark.parametrize("E,k,has_bias,groups,sigmoid,renorm", GATE)
def test_gate_scores_over_the_logits(mg, E, k, has_bias, groups, sigmoid, renorm):
    g = torch.Generator().manual_seed(E + k)
    T = 77
    l = torch.randn(T, E, generator=g) * 3
    l[torch.rand(T, E, generator=g) < 0.1] = -float("inf")
    l[5] = -float("inf")
    l = l.cuda()
    kw = dict(bias=torch.randn(E, generator=g).cuda() if has_bias else None, n_groups=groups,
              topk_groups=max(1, groups // 2), sigmoid=sigmoid, renorm=renorm)
    ids, w, s = mg.moe_gate(l, k, want_scores=True, **kw)
    over = l.clone()
    if has_bias or groups > 1:                     # the picks' logits are read behind the scores
        with pytest.raises(mg.MoeggError):
            mg.moe_gate(over, k, scores=over, **kw)
        assert torch.equal(over, l)
        return
    ids2, w2, s2 = mg.moe_gate(over, k, scores=over, **kw)
    assert s2 is over and torch.equal(over, s)
    assert torch.equal(ids2, ids) and torch.equal(w2, w)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("E,k,has_bias,groups,sigmoid,renorm", GATE)
def test_gate_gradient_over_an_input(mg, E, k, has_bias, groups, sigmoid, renorm, dtype):
    g = torch.Generator().manual_seed(2 * E + k)
    T = 77
    l = (torch.randn(T, E, generator=g) * 3).to(DT[dtype]).cuda()
    ids, w, s = mg.moe_gate(l, k, sigmoid=sigmoid, renorm=renorm, want_scores=True)
    gw, gs = torch.randn(T, k, generator=g).cuda(), torch.randn(T, E, generator=g).cuda()
    kw = dict(sigmoid=sigmoid, renorm=renorm)
    want = mg.moe_gate_bwd(l, ids, gw, dscores=gs, **kw)
    over = l.clone()
    mg.moe_gate_bwd(over, ids, gw, dscores=gs, dlogits=over, **kw)
    assert torch.equal(over, want)
    if dtype == "fp32":
        over = gs.clone()
        mg.moe_gate_bwd(l, ids, gw, dscores=over, dlogits=over, **kw)
        assert torch.equal(over, want)
