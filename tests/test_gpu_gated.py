"""The gated feed-forward block (moegg_gated_fwd, moegg_gated_bwd) against 64-bit
evaluations: every form of what is kept, both activations, pairs and halves, odd
sizes, short and long groups, experts and slots without rows.  Bounds are those of
tests/_block.py; kept values are taken as they are by the backward, so that its only
sums are dH's."""

import numpy as np
import pytest
import torch

from tests._block import (HALF, U, act_ref, check, f64, gated_ref, grouped, join, pack_ref, routed,
                          sum_err, split, unpack_ref)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import token_routing_amd as m
    m.load_library()
    return m


def flags_of(mg, act, halves):
    return (mg.GATED_GELU if act == "gelu" else mg.GATED_SILU) | (mg.GATED_HALVES if halves else 0)


# T, k, E, K, I, act, halves
CASES = [
    (1, 1, 1, 1, 1, "silu", False),
    (1, 2, 8, 64, 32, "silu", True),
    (3, 2, 5, 130, 75, "gelu", True),
    (5, 1, 3, 133, 34, "silu", False),
    (64, 8, 128, 96, 40, "silu", False),
    (50, 2, 1024, 24, 16, "gelu", False),
    (300, 1, 2, 136, 264, "gelu", True),
    (300, 1, 2, 137, 261, "silu", False),
    (411, 2, 3, 200, 129, "silu", True),
    (640, 1, 1, 72, 128, "gelu", False),
    # few rows, reductions of several waves
    (6, 2, 6, 1032, 70, "silu", True),
    (4, 1, 2, 2056, 33, "gelu", False),
    (9, 1, 5, 1500, 21, "silu", False),
    # middle tiles with four stages
    (900, 2, 3, 72, 500, "silu", True),
    (1001, 3, 9, 603, 517, "gelu", False),
    (950, 2, 1, 640, 520, "silu", False),
    # middle and large tiles in both directions
    (500, 2, 3, 40, 2600, "silu", True),
    (1500, 1, 2, 24, 4001, "gelu", False),
    (1500, 1, 2, 48, 4000, "silu", True),
    (1500, 1, 2, 24, 8043, "silu", False),
    (1500, 1, 2, 40, 8040, "gelu", True),
]
IDS = ["-".join(map(str, c)) for c in CASES]


def inputs(mg, case, px=True, seed=0):
    T, k, E, K, I, act, halves = case
    r, order, experts, g = routed(mg, T, k, E, seed + sum(case[:5]))
    x = torch.randn(T if px else T * k, K, generator=g).bfloat16()
    w = (torch.randn(E, 2 * I, K, generator=g) * (2.0 / K ** 0.5)).bfloat16()
    return r, order, experts, g, x, w


@pytest.mark.parametrize("keep", [None, "bf16", "packed"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(mg, case, keep):
    T, k, E, K, I, act, halves = case
    px = keep != "bf16"                                  # expert-ordered rows in one of the forms
    r, order, experts, g, x, w = inputs(mg, case, px)
    S, n = T * k, order.size
    h = torch.full((S, I), 9.0, dtype=torch.bfloat16, device="cuda")
    Ip = (I + 31) // 32 * 32
    kept = None
    if keep == "bf16":
        kept = torch.full((S, 2 * I), 9.0, dtype=torch.bfloat16, device="cuda")
    elif keep == "packed":
        kept = (torch.full((S, 2 * Ip), 9, dtype=torch.int8, device="cuda"),
                torch.full((S, Ip // 16), 9, dtype=torch.uint8, device="cuda"))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got, out = mg.gated_fwd(x.cuda(), w.cuda(), r["m_sizes"], r["gather"] if px else None, k,
                            flags_of(mg, act, halves) | (mg.PERMUTE_X if px else 0), keep=keep,
                            H=h, kept=kept, error_flags=err)
    assert int(err) == 0 and got is h
    src = order // k if px else np.arange(n)
    a, mag = grouped(f64(x)[src], experts, f64(w), True)
    da = sum_err(mag, K)
    (gt, ut), (ge, ue) = split(a, halves), split(da, halves)
    ref, tol = gated_ref(gt, ut, ge, ue, act)
    check(got[:n], ref, tol, "H")
    assert (got[n:] == 9).all()
    if keep == "bf16":
        check(out[:n], a, da + (np.abs(a) + da) * HALF, "A")
        assert (out[n:] == 9).all()
    elif keep == "packed":
        q, s = (t.cpu().numpy() for t in out)
        assert (q[n:] == 9).all() and (s[n:] == 9).all()
        for part, v, e in ((0, gt, ge), (1, ut, ue)):
            pq, ps = q[:n, part * Ip:(part + 1) * Ip], s[:n, part * Ip // 32:(part + 1) * Ip // 32]
            step = np.exp2(ps.astype(float) - 127).repeat(32, 1)[:, :I]
            check(unpack_ref(pq, ps, I), v, step / 2 + e, "packed")
            assert (pq[:, I:] == 0).all()
            # the step of the exact values, or of values that far beside them
            lo = pack_ref(np.maximum(np.abs(v) - e, 0))[1]
            hi = pack_ref(np.abs(v) + e)[1]
            assert ((ps >= lo) & (ps <= hi)).all()


def test_packed_whole_numbers(mg):
    """Whole-number inputs, whose sums are exact: the codes are pack8's, bit for bit."""
    T, k, E, K, I = 300, 2, 3, 48, 70
    r, order, experts, g = routed(mg, T, k, E, 11)
    x = torch.randint(-4, 5, (T, K), generator=g).bfloat16()
    w = torch.randint(-4, 5, (E, 2 * I, K), generator=g).bfloat16()
    _, (q, s) = mg.gated_fwd(x.cuda(), w.cuda(), r["m_sizes"], r["gather"], k,
                             mg.PERMUTE_X | mg.GATED_SILU | mg.GATED_HALVES, keep="packed")
    a, _ = grouped(f64(x)[order // k], experts, f64(w), True)
    n = order.size
    for part, v in enumerate(split(a, True)):
        wq, ws = pack_ref(v)
        assert np.array_equal(q[:n].chunk(2, 1)[part].cpu().numpy(), wq)
        assert np.array_equal(s[:n].chunk(2, 1)[part].cpu().numpy(), ws)


def kept_values(g, S, I, halves, packed, spread=2.0):
    """Something kept (CPU tensors), and the gate and linear values it stands for."""
    gt, ut = (torch.randn(S, I, generator=g) * spread for _ in range(2))
    if packed:
        (gq, gs), (uq, us) = pack_ref(f64(gt)), pack_ref(f64(ut))
        kept = (torch.from_numpy(np.concatenate([gq, uq], 1)),
                torch.from_numpy(np.concatenate([gs, us], 1)))
        return kept, unpack_ref(gq, gs, I), unpack_ref(uq, us, I)
    gt, ut = gt.bfloat16(), ut.bfloat16()
    kept = torch.cat([gt, ut], 1) if halves else torch.stack([gt, ut], -1).flatten(1)
    return kept.contiguous(), f64(gt), f64(ut)


def to_cuda(kept):
    return kept.cuda() if isinstance(kept, torch.Tensor) else tuple(t.cuda() for t in kept)


def bwd_ref(gt, ut, dy, experts, w, act):
    """dg, du, H and their bounds for exact kept values."""
    dh, mag = grouped(dy, experts, w, False)
    eh = sum_err(mag, w.shape[1])
    a, d, ea, ed = act_ref(gt, act)
    dg, du, h = dh * ut * d, dh * a, a * ut
    eg = np.abs(ut) * (eh * (np.abs(d) + ed) + np.abs(dh) * ed)
    eu = eh * (np.abs(a) + ea) + np.abs(dh) * ea
    ehh = np.abs(ut) * ea
    return [(v, e + (np.abs(v) + e) * (HALF + 4 * U) + 1e-37)
            for v, e in ((dg, eg), (du, eu), (h, ehh))]


@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward(mg, case, packed):
    T, k, E, N, I, act, halves = case
    r, order, experts, g = routed(mg, T, k, E, 3 + sum(case[:5]))
    S, n = T * k, order.size
    py = packed != halves                                # dY in slot order in half of the cases
    kept, gt, ut = kept_values(g, S, I, halves, packed)
    dy = torch.randn(S, N, generator=g).bfloat16()
    w = (torch.randn(E, N, I, generator=g) / N ** 0.5).bfloat16()
    da = torch.full((S, 2 * I), 9.0, dtype=torch.bfloat16, device="cuda")
    h = torch.full((S, I), 9.0, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got, goth = mg.gated_bwd(dy.cuda(), w.cuda(), to_cuda(kept), r["m_sizes"], r["gather"], k,
                             flags_of(mg, act, halves) | (mg.PERMUTE_Y if py else 0), dA=da, H=h,
                             error_flags=err)
    assert int(err) == 0 and got is da and goth is h
    rows = f64(dy)[order if py else np.arange(n)]
    (dg, tg), (du, tu), (hh, th) = bwd_ref(gt[:n], ut[:n], rows, experts, f64(w), act)
    check(got[:n], join(dg, du, halves), join(tg, tu, halves), "dA")
    check(goth[:n], hh, th, "H")
    assert (got[n:] == 9).all() and (goth[n:] == 9).all()
    again, none = mg.gated_bwd(dy.cuda(), w.cuda(), to_cuda(kept), r["m_sizes"], r["gather"], k,
                               flags_of(mg, act, halves) | (mg.PERMUTE_Y if py else 0),
                               want_h=False)
    assert none is None and torch.equal(again[:n], got[:n])


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("T,I", [(300, 136), (300, 137), (20, 72), (20, 71)])
def test_backward_in_place(mg, T, I, halves):
    """dA may take A's place."""
    k, E, N = 1, 2, 64
    r, order, experts, g = routed(mg, T, k, E, T + I)
    kept, _, _ = kept_values(g, T, I, halves, False)
    dy = torch.randn(T, N, generator=g).bfloat16().cuda()
    w = torch.randn(E, N, I, generator=g).bfloat16().cuda()
    f = flags_of(mg, "gelu", halves)
    apart, h = mg.gated_bwd(dy, w, kept.cuda(), r["m_sizes"], None, k, f)
    a = kept.cuda()
    out, h2 = mg.gated_bwd(dy, w, a, r["m_sizes"], None, k, f, dA=a)
    n = order.size
    assert out is a and torch.equal(out[:n], apart[:n]) and torch.equal(h[:n], h2[:n])


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_differences(mg, act):
    """sum dA * D against (L(A + eD) - L(A - eD)) / 2e in 64 bits, L = sum dY * (act(g) u) W^T.

    The formula's own difference quotient is off by e^2 / 6 of its third derivative
    (|act'''| < 4, with values of a few units: below 1e-6 of the sum of magnitudes at
    e = 1e-4), the operator's dA by its bound at every element.
    """
    T, k, E, N, I = 70, 1, 2, 40, 48
    r, order, experts, g = routed(mg, T, k, E, 17, drop=False)
    kept, gt, ut = kept_values(g, T, I, False, False, spread=1.0)
    dy = torch.randn(T, N, generator=g).bfloat16()
    w = (torch.randn(E, N, I, generator=g) / N ** 0.5).bfloat16()
    da, _ = mg.gated_bwd(dy.cuda(), w.cuda(), kept.cuda(), r["m_sizes"], None, k,
                         flags_of(mg, act, False))
    rng = np.random.default_rng(0)
    dg, du = rng.standard_normal((2, T, I))

    def loss(t):
        a, _, _, _ = act_ref(gt + t * dg, act)
        y, _ = grouped(a * (ut + t * du), experts, f64(w).transpose(0, 2, 1), False)
        return (y * f64(dy)).sum()

    e = 1e-4
    want = (loss(e) - loss(-e)) / (2 * e)
    (rg, tg), (ru, tu), _ = bwd_ref(gt, ut, f64(dy), experts, f64(w), act)
    got = f64(da)
    g_, u_ = split(got, False)
    bound = (np.abs(dg) * tg + np.abs(du) * tu).sum()
    size = (np.abs(rg * dg) + np.abs(ru * du)).sum()
    assert abs((g_ * dg + u_ * du).sum() - want) <= bound + 1e-6 * size


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_far_gates(mg, act):
    """Gates far out, where the activation is 0 or g itself to the last bit."""
    I = 16
    gates = torch.tensor([-3e38, -1e30, -1e4, -200.0, 200.0, 1e4, 1e18, 0.0] * 2)
    kept = torch.cat([gates, torch.ones(I)]).bfloat16().view(1, 2 * I).cuda()
    dy = torch.ones(1, 8, dtype=torch.bfloat16, device="cuda")
    w = torch.full((1, 8, I), 0.25, dtype=torch.bfloat16, device="cuda")
    m = torch.ones(1, dtype=torch.int32, device="cuda")
    da, h = mg.gated_bwd(dy, w, kept, m, None, 1, flags_of(mg, act, True))
    g = f64(gates.bfloat16())
    big = g > 100
    dg, du = f64(da)[0, :I], f64(da)[0, I:]
    assert np.array_equal(dg, np.where(big, 2.0, np.where(g == 0, 1.0, 0.0)))
    assert np.array_equal(f64(h)[0], np.where(big, g, 0.0))
    assert np.array_equal(du, np.where(big, 2 * g, 0.0))


def test_values_that_are_not_numbers(mg):
    """A NaN row of X gives NaN in its own rows alone, kept ones among them."""
    T, K, I = 40, 64, 64
    g = torch.Generator().manual_seed(4)
    x = torch.randn(T, K, generator=g).bfloat16()
    x[5, 0] = float("nan")
    w = torch.randn(1, 2 * I, K, generator=g).bfloat16().cuda()
    m = torch.tensor([T], dtype=torch.int32, device="cuda")
    f = mg.GATED_SILU | mg.GATED_HALVES
    h, (q, s) = mg.gated_fwd(x.cuda(), w, m, None, 1, f, keep="packed")
    assert torch.isnan(h[5]).all() and torch.isfinite(h[:5]).all() and torch.isfinite(h[6:]).all()
    assert (s[5] == 255).all() and (s[:5] != 255).all() and (s[6:] != 255).all()
    dy = torch.randn(T, 32, generator=g).bfloat16().cuda()
    wd = torch.randn(1, 32, I, generator=g).bfloat16().cuda()
    da, h2 = mg.gated_bwd(dy, wd, (q, s), m, None, 1, f)
    for t in (da, h2):
        assert torch.isnan(t[5]).all()
        assert torch.isfinite(t[:5]).all() and torch.isfinite(t[6:]).all()


def test_operands_beside_16_bytes(mg):
    """Operands that begin 2 bytes off a 16-byte border give the same results."""
    T, k, E, K, I = 50, 2, 3, 64, 48
    r, order, experts, g = routed(mg, T, k, E, 23)
    n = order.size

    def off(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        out = flat[1:].view(t.shape)
        out.copy_(t)
        return out

    x = torch.randn(T, K, generator=g).bfloat16().cuda()
    w = torch.randn(E, 2 * I, K, generator=g).bfloat16().cuda()
    f = mg.GATED_SILU
    h, a = mg.gated_fwd(x, w, r["m_sizes"], r["gather"], k, f | mg.PERMUTE_X, keep="bf16")
    h2, a2 = mg.gated_fwd(off(x), off(w), r["m_sizes"], r["gather"], k, f | mg.PERMUTE_X,
                          keep="bf16", H=off(torch.zeros_like(h)), kept=off(torch.zeros_like(a)))
    assert torch.equal(h[:n], h2[:n]) and torch.equal(a[:n], a2[:n])
    dy = torch.randn(T * k, K, generator=g).bfloat16().cuda()
    wd = torch.randn(E, K, I, generator=g).bfloat16().cuda()
    d, hh = mg.gated_bwd(dy, wd, a, r["m_sizes"], r["gather"], k, f)
    d2, hh2 = mg.gated_bwd(off(dy), off(wd), off(a), r["m_sizes"], r["gather"], k, f)
    assert torch.equal(d[:n], d2[:n]) and torch.equal(hh[:n], hh2[:n])


def test_agrees_with_the_plain_forward(mg):
    """H and A of pairs are what grouped_gemm_fwd with and without GATED_SILU gives, to the
    bounds of both: the sums' order, one rounding each."""
    T, k, E, K, I = 600, 2, 3, 256, 128
    case = (T, k, E, K, I, "silu", False)
    r, order, experts, g, x, w = inputs(mg, case)
    n = order.size
    h, a = mg.gated_fwd(x.cuda(), w.cuda(), r["m_sizes"], r["gather"], k,
                        mg.PERMUTE_X | mg.GATED_SILU, keep="bf16")
    a2 = mg.grouped_gemm_fwd(x.cuda(), w.cuda(), r["m_sizes"], r["gather"], None, k, mg.PERMUTE_X)
    h2 = mg.grouped_gemm_fwd(x.cuda(), w.cuda(), r["m_sizes"], r["gather"], None, k,
                             mg.PERMUTE_X | mg.GATED_SILU)
    v, mag = grouped(f64(x)[order // k], experts, f64(w), True)
    e = sum_err(mag, K)
    (gt, ut), (ge, ue) = split(v, False), split(e, False)
    ref, tol = gated_ref(gt, ut, ge, ue, "silu")
    for t in (h, h2):
        check(t[:n], ref, tol)
    for t in (a, a2):
        check(t[:n], v, e + (np.abs(v) + e) * HALF)


def test_bad_gather(mg):
    T, k, E, K, I = 30, 2, 4, 32, 32
    case = (T, k, E, K, I, "silu", False)
    r, order, experts, g, x, w = inputs(mg, case)
    gather = r["gather"].clone()
    gather[4], gather[9] = -1, T * k
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    f = mg.GATED_SILU
    h, (q, s) = mg.gated_fwd(x.cuda(), w.cuda(), r["m_sizes"], r["gather"], k, f | mg.PERMUTE_X,
                             keep="packed")
    h2 = torch.full_like(h, 5.0)
    q2, s2 = torch.full_like(q, 5), torch.full_like(s, 5)
    mg.gated_fwd(x.cuda(), w.cuda(), r["m_sizes"], gather, k, f | mg.PERMUTE_X, keep="packed", H=h2,
                 kept=(q2, s2), error_flags=err)
    assert int(err) == mg.DERR_GATHER
    n = order.size
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[[4, 9]] = False
    for got, want in ((h2, h), (q2, q), (s2, s)):
        assert torch.equal(got[:n][keep], want[:n][keep]) and (got[[4, 9]] == 5).all()
    dy = torch.randn(T * k, 24, generator=g).bfloat16().cuda()
    wd = torch.randn(E, 24, I, generator=g).bfloat16().cuda()
    err.zero_()
    da = torch.full((T * k, 2 * I), 5.0, dtype=torch.bfloat16, device="cuda")
    mg.gated_bwd(dy, wd, (q, s), r["m_sizes"], gather, k, f | mg.PERMUTE_Y, dA=da, error_flags=err)
    assert int(err) == mg.DERR_GATHER and (da[[4, 9]] == 5).all()


def test_no_tokens(mg):
    e = torch.empty(0, 32, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(2, 16, 32, dtype=torch.bfloat16, device="cuda")
    m = torch.zeros(2, dtype=torch.int32, device="cuda")
    no = torch.empty(0, dtype=torch.int32, device="cuda")
    h, (q, s) = mg.gated_fwd(e, w, m, no, 1, mg.PERMUTE_X | mg.GATED_SILU, keep="packed")
    assert h.shape == (0, 8) and q.shape == (0, 64) and s.shape == (0, 2)
    da, h = mg.gated_bwd(torch.empty(0, 24, dtype=torch.bfloat16, device="cuda"),
                         torch.zeros(2, 24, 8, dtype=torch.bfloat16, device="cuda"), (q, s), m, no,
                         1, mg.GATED_SILU)
    assert da.shape == (0, 16) and h.shape == (0, 8)
