"""The gate (moegg_gate, moegg_gate_bwd) against a plain float64 evaluation.

Ids are compared for equality, ties included.  Bounds of the fp32 results: a
score is e^(l - m) / sum, where the argument's rounding (half a unit of
|l - m|) enters the exponent as it is, expf and the division are good to 2
units, and a sum over at most 16 values a lane and 6 steps over lanes to 24:
relative error <= (range + 32) * 2^-23 with range the row's largest |l - m|.
The log-sigmoid adds its own 4 units: <= (2 * range + 48) * 2^-23 with the
largest |log sigmoid|.  Gradients are products q (g - dot): the same relative
bound on q (|g| + sum q |g|), plus half a step of the output's type.
"""

import math

import numpy as np
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


def ref_gate(l, k, bias, groups, top_groups, scale, sigmoid, renorm):
    """ids, weights, scores of float64 logits l [T, E] (numpy), row by row."""
    T, E = l.shape
    l = np.where(np.isnan(l) | (l == np.inf), -np.inf, l)
    ids = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    scores = np.zeros((T, E))
    for t in range(T):
        row = l[t]
        live = row > -np.inf
        if sigmoid:
            logs = np.minimum(row, 0) - np.log1p(np.exp(-np.abs(row)))
        elif live.any():
            m = row[live].max()
            logs = row - m - np.log(np.exp(row[live] - m).sum())
        else:
            continue
        scores[t] = np.where(live, np.exp(logs), 0.0)
        key = row.copy() if bias is None and groups == 1 else scores[t] + (0 if bias is None else bias)
        ok = live & np.isfinite(key)
        if groups > 1:
            per = E // groups
            val = []
            for g in range(groups):
                kk = np.sort(key[g * per:(g + 1) * per][ok[g * per:(g + 1) * per]])[::-1][:2]
                val.append(kk.sum() if kk.size else -np.inf)
            best = sorted(range(groups), key=lambda g: (-val[g], g))[:top_groups]
            ok = ok & np.isin(np.arange(E) // per, best)
        order = sorted(np.nonzero(ok)[0], key=lambda e: (-key[e], e))[:k]
        ids[t, :len(order)] = order
        if order:
            x = logs[order]
            v = np.exp(x - x.max()) / np.exp(x - x.max()).sum() if renorm else np.exp(x)
            w[t, :len(order)] = scale * v
    return ids, w, scores


def rel_bound(l, sigmoid):
    fin = np.where(np.isfinite(l), l, np.nan)
    if sigmoid:
        with np.errstate(all="ignore"):
            r = np.nanmax(np.abs(np.minimum(fin, 0) - np.log1p(np.exp(-np.abs(fin)))), initial=1.0)
        return (2 * r + 48) * 2.0 ** -23
    with np.errstate(all="ignore"):
        r = np.nanmax(np.nanmax(fin, axis=1, initial=-1e9) - np.nanmin(fin, axis=1, initial=1e9),
                      initial=1.0)
    return (max(r, 1.0) + 32) * 2.0 ** -23


CASES = [
    # T, E, k, dtype, bias, groups, top_groups, sigmoid, renorm, scale
    (1, 8, 2, "bf16", False, 1, 1, False, True, 1.0),
    (5, 1, 1, "fp32", False, 1, 1, False, False, 1.0),
    (33, 8, 8, "fp16", False, 1, 1, False, False, 1.0),
    (37, 7, 3, "bf16", True, 1, 1, True, True, 2.5),
    (70, 60, 6, "bf16", False, 1, 1, False, True, 1.0),
    (17, 64, 64, "fp32", False, 1, 1, True, True, 1.0),
    (129, 128, 8, "bf16", False, 1, 1, False, True, 1.0),
    (65, 128, 37, "fp16", True, 1, 1, False, False, 0.5),
    (40, 160, 6, "fp32", True, 8, 3, False, False, 16.0),
    (66, 256, 8, "fp32", True, 8, 4, True, True, 2.5),
    (21, 256, 8, "bf16", False, 8, 4, True, True, 2.5),
    (9, 511, 10, "fp16", False, 1, 1, False, True, 1.0),
    (6, 1000, 64, "bf16", False, 1, 1, True, False, 1.0),
    (4, 1024, 5, "fp32", True, 64, 3, True, True, 1.0),
    (3, 12, 2, "fp32", False, 12, 2, False, True, 1.0),
]
IDS = ["-".join(str(x) for x in c) for c in CASES]


def make_logits(T, E, dtype, seed, masks=True):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn(T, E, generator=g) * 2
    if masks and T > 2 and E > 1:
        l[torch.rand(T, E, generator=g) < 0.15] = -math.inf
        l[1] = -math.inf                     # a token without any expert
        l[2] = -math.inf
        l[2, E // 2] = 0.5                   # one expert left
    return l.to(DT[dtype])


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_gate_forward(mg, case):
    T, E, k, dtype, has_bias, groups, top_groups, sigmoid, renorm, scale = case
    l = make_logits(T, E, dtype, 100 + T + E)
    g = torch.Generator().manual_seed(E)
    bias = torch.randn(E, generator=g) * 0.1 if has_bias else None
    ids, w, s = mg.moe_gate(l.cuda(), k, bias=None if bias is None else bias.cuda(),
                            n_groups=groups, topk_groups=top_groups, scale=scale, sigmoid=sigmoid,
                            renorm=renorm, want_scores=True)
    rids, rw, rs = ref_gate(l.double().numpy(), k, None if bias is None else bias.double().numpy(),
                            groups, top_groups, scale, sigmoid, renorm)
    assert np.array_equal(ids.cpu().numpy(), rids)
    rel = rel_bound(l.double().numpy(), sigmoid)
    assert np.all(np.abs(w.cpu().double().numpy() - rw) <= rel * np.abs(rw))
    assert np.all(np.abs(s.cpu().double().numpy() - rs) <= rel * rs)


def test_gate_ties_go_to_the_lowest_index(mg):
    l = torch.zeros(3, 130, dtype=torch.bfloat16)
    l[1] = -0.0
    l[1, ::2] = 0.0                          # -0 equals +0
    l[2, 64:] = 1.0
    ids, w, _ = mg.moe_gate(l.cuda(), 4, renorm=True)
    assert ids.cpu().tolist() == [[0, 1, 2, 3], [0, 1, 2, 3], [64, 65, 66, 67]]
    assert torch.equal(w.cpu(), torch.full((3, 4), 0.25))
    # equal keys and equal group values in 64 bits
    ids, _, _ = mg.moe_gate(l[:1, :128].cuda(), 4, n_groups=8, topk_groups=2, sigmoid=True)
    assert ids.cpu().tolist() == [[0, 1, 2, 3]]
    b = torch.zeros(130)
    b[7] = 2.0 ** -30                        # below a 32-bit rounding of the key
    ids, _, _ = mg.moe_gate(l[:1].cuda(), 3, bias=b.cuda(), sigmoid=True)
    assert ids.cpu().tolist() == [[7, 0, 1]]


def test_gate_extreme_and_odd_logits(mg):
    big = torch.finfo(torch.bfloat16).max
    l = torch.tensor([[big, -big, 0.0, 1.0], [-big] * 4, [-200.0, -300.0, -250.0, -math.inf],
                      [math.nan, 1.0, math.inf, 2.0]], dtype=torch.bfloat16)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids, w, s = mg.moe_gate(l[:3].cuda(), 3, renorm=True, want_scores=True, error_flags=err)
    assert int(err.item()) == 0
    assert ids.cpu().tolist() == [[0, 3, 2], [0, 1, 2], [0, 2, 1]]
    assert w.cpu()[0].tolist() == [1.0, 0.0, 0.0]
    assert torch.allclose(w.cpu()[1], torch.full((3,), 1 / 3), rtol=2.0 ** -22, atol=0)
    assert torch.isfinite(w).all() and torch.isfinite(s).all()
    # far sigmoids: their ratio stands although each underflows
    _, w, _ = mg.moe_gate(l[2:3].cuda(), 2, sigmoid=True, renorm=True)
    assert abs(w.sum().item() - 1) < 2 ** -22 and w[0, 0].item() > 0.999
    ids, w, s = mg.moe_gate(l[3:].cuda(), 3, want_scores=True, error_flags=err)
    assert int(err.item()) == mg.DERR_LOGIT
    assert ids.cpu().tolist() == [[3, 1, -1]] and w[0, 2].item() == 0
    assert s.cpu()[0, 0].item() == 0 and s.cpu()[0, 2].item() == 0
    err.zero_()
    b = torch.tensor([math.nan, 0.0, -math.inf, 0.0])
    ids, _, _ = mg.moe_gate(torch.ones(1, 4).cuda(), 4, bias=b.cuda(), error_flags=err)
    assert int(err.item()) == mg.DERR_LOGIT and ids.cpu().tolist() == [[1, 3, -1, -1]]


def test_gate_row_stride_stream_and_empty(mg):
    wide = torch.randn(50, 40, device="cuda")
    l = wide[:, 3:27]                        # rows of another matrix
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ids, w, _ = mg.moe_gate(l, 3, stream=side)
    d = mg.moe_gate_bwd(l, ids, w, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    ids2, w2, _ = mg.moe_gate(l.contiguous(), 3)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    assert torch.equal(d, mg.moe_gate_bwd(l.contiguous(), ids, w))
    e = torch.empty(0, 16, device="cuda")
    ids, w, s = mg.moe_gate(e, 2, want_scores=True)
    assert ids.shape == (0, 2) and w.shape == (0, 2) and s.shape == (0, 16)
    assert mg.moe_gate_bwd(e, ids, w).shape == (0, 16)


def ref_loss(l, ids, gw, gs, scale, sigmoid, renorm):
    """sum(weights * gw) + sum(scores * gs) of float64 logits; differentiable."""
    live = torch.isfinite(l)
    safe = torch.where(live, l, torch.zeros_like(l))
    if sigmoid:
        logs = torch.nn.functional.logsigmoid(safe)
    else:
        low = torch.where(live, safe, torch.full_like(l, -1e30))
        logs = torch.log_softmax(low, 1)
    ok = (ids >= 0) & torch.gather(live, 1, ids.clamp(min=0))
    x = torch.gather(logs, 1, ids.clamp(min=0))
    if renorm:
        w = torch.softmax(torch.where(ok, x, torch.full_like(x, -1e30)), 1)
    else:
        w = torch.exp(x)
    w = torch.where(ok, w, torch.zeros_like(w)) * scale
    loss = (w * gw).sum()
    if gs is not None:
        loss = loss + (torch.where(live, torch.exp(logs), torch.zeros_like(logs)) * gs).sum()
    return loss


@pytest.mark.parametrize("with_scores", [True, False], ids=["scores", "weights"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_gate_backward(mg, case, with_scores):
    T, E, k, dtype, _, _, _, sigmoid, renorm, scale = case
    l = make_logits(T, E, dtype, 200 + T + E)
    g = torch.Generator().manual_seed(7 * E)
    rids, _, _ = ref_gate(l.double().numpy(), k, None, 1, 1, scale, sigmoid, renorm)
    ids = torch.from_numpy(rids)
    gw = torch.randn(T, k, generator=g)
    gs = torch.randn(T, E, generator=g) if with_scores else None
    d = mg.moe_gate_bwd(l.cuda(), ids.cuda(), gw.cuda(), dscores=None if gs is None else gs.cuda(),
                        scale=scale, sigmoid=sigmoid, renorm=renorm).cpu().double()
    x = l.double().requires_grad_(True)
    args = (ids.long(), gw.double(), None if gs is None else gs.double(), scale, sigmoid, renorm)
    ref = torch.autograd.grad(ref_loss(x, *args), x)[0]
    ref = torch.where(torch.isfinite(x.detach()), ref, torch.zeros_like(ref))
    # the terms' magnitudes: every product that enters an element
    _, w, s = ref_gate(l.double().numpy(), k, None, 1, 1, 1.0, sigmoid, renorm)
    s, w = torch.from_numpy(s), torch.from_numpy(w)
    gabs = gw.double().abs() * abs(scale)
    mag = torch.zeros(T, E, dtype=torch.float64)
    one = w * (gabs + (w * gabs).sum(1, keepdim=True)) if renorm else w * gabs
    mag.scatter_add_(1, ids.clamp(min=0).long(), torch.where(ids >= 0, one, torch.zeros_like(one)))
    dsabs = torch.zeros(T, E, dtype=torch.float64) if gs is None else gs.double().abs()
    if not renorm:
        dsabs = dsabs.scatter_add(1, ids.clamp(min=0).long(),
                                  torch.where(ids >= 0, gabs, torch.zeros_like(gabs)))
    mag = mag + s * (dsabs + (0 if sigmoid else (s * dsabs).sum(1, keepdim=True)))
    # q, dot and the outer product each carry the relative bound once
    rel = 3 * rel_bound(l.double().numpy(), sigmoid)
    half = torch.finfo(DT[dtype]).eps / 2
    tiny = torch.finfo(DT[dtype]).smallest_normal * torch.finfo(DT[dtype]).eps
    # The reference's own arithmetic: with renorm autograd sends the weights'
    # gradient through the log-softmax of the whole row, where it cancels in
    # real numbers (an expert that was not picked has gradient 0) and leaves
    # the rounding of a float64 sum of E + k terms, each at most the row's
    # magnitudes together.
    own = (E + k + 8) * 2.0 ** -53 * (mag.sum(1, keepdim=True) + dsabs.sum(1, keepdim=True))
    bound = rel * mag * (1 + half) + half * ref.abs() + tiny + own
    assert torch.all((d - ref).abs() <= bound), float(((d - ref).abs() - bound).max())
    # the formula itself against differences of the loss along one direction
    v = torch.randn(T, E, generator=g, dtype=torch.float64)
    v = torch.where(torch.isfinite(x.detach()), v, torch.zeros_like(v))
    h = 1e-5
    diff = (ref_loss(x.detach() + h * v, *args) - ref_loss(x.detach() - h * v, *args)) / (2 * h)
    along = (ref * v).sum()
    assert abs(diff - along) <= 1e-6 * (1 + (ref * v).abs().sum()), (diff, along)


def test_gate_backward_odd_ids(mg):
    l = torch.randn(4, 16)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids = torch.tensor([[0, -1], [3, 3], [16, 2], [-1, -1]], dtype=torch.int32)
    gw = torch.ones(4, 2)
    d = mg.moe_gate_bwd(l.cuda(), ids.cuda(), gw.cuda(), sigmoid=True, error_flags=err).cpu()
    assert int(err.item()) == mg.DERR_EXPERT_ID
    s = torch.sigmoid(l.double())
    want = torch.zeros(4, 16, dtype=torch.float64)
    want[0, 0] = (s * (1 - s))[0, 0]
    want[1, 3] = 2 * (s * (1 - s))[1, 3]     # the same expert twice adds up
    want[2, 2] = (s * (1 - s))[2, 2]
    assert torch.allclose(d.double(), want, rtol=2.0 ** -20, atol=0)


def test_gate_feeds_route(mg):
    """Gate, then routing: padding tokens' slots are dropped."""
    l = make_logits(64, 16, "bf16", 5, masks=False)
    l[60:] = -math.inf
    ids, w, _ = mg.moe_gate(l.cuda(), 4, renorm=True)
    r = mg.moe_route(ids, 16)
    assert int(r["m_sizes"].sum().item()) == 240
    assert torch.all(r["scatter"].view(64, 4)[60:] == -1)
    assert torch.all(r["scatter"].view(64, 4)[:60] >= 0)
