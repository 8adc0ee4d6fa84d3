"""Grouped products of 8-bit integers (moegg_grouped_gemm_i8) against exact sums in 64 bits.

The sum is exact; its conversion to fp32 and the two or three products with the
scales round by 2^-24 each, the result by 2^-8: |y| (2^-8 + 6 * 2^-24)."""

import numpy as np
import pytest
import torch

from tests._block import HALF, U, check, f64, gated_ref, grouped, routed, split

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import token_routing_amd as m
    m.load_library()
    return m


# T, k, E, K, N, form, act, halves
CASES = [
    (1, 1, 1, 16, 1, "plain", None, False),
    (1, 2, 8, 1024, 2048, "gated", "silu", False),
    (5, 2, 8, 112, 70, "gated", "gelu", True),
    (2, 1, 3, 32, 2, "gated", "silu", True),
    (64, 8, 128, 256, 192, "gated", "silu", False),
    (40, 3, 1024, 48, 40, "plain", None, False),
    (300, 1, 2, 208, 333, "plain", None, False),
    (257, 2, 3, 1008, 530, "scattered", None, False),
    (33, 2, 5, 64, 136, "scattered", None, False),
    (700, 1, 2, 336, 514, "gated", "silu", True),
    (700, 1, 2, 336, 516, "gated", "gelu", False),
    (520, 2, 4, 144, 1026, "gated", "gelu", True),
    (400, 2, 4, 80, 264, "sorted", None, False),
    (90, 2, 4, 80, 264, "sorted", "silu", False),
    # few rows: one to four of an expert at a time, reductions of parts and of several waves
    (1, 8, 128, 768, 256, "scattered", None, False),
    (1, 2, 4, 2064, 37, "plain", None, False),
    (6, 2, 6, 2064, 37, "plain", None, False),
    (3, 2, 4, 1040, 50, "gated", "silu", True),
    (7, 1, 5, 2096, 134, "gated", "gelu", False),
    (9, 2, 16, 2048, 130, "scattered", None, False),
    (4, 1, 1, 4112, 18, "sorted", "silu", False),
    (33, 1, 17, 1024, 65, "sorted", None, False),
    # middle tiles with four stages
    (900, 2, 3, 1152, 1001, "scattered", None, False),
    (900, 2, 3, 96, 1002, "gated", "silu", True),
    # sizes that take middle tiles (up to 128 rows a tile) and large ones
    (700, 2, 3, 64, 5000, "plain", None, False),
    (700, 2, 3, 64, 4998, "gated", "gelu", True),
    (1500, 1, 2, 48, 8008, "plain", None, False),
    (1500, 1, 2, 48, 8002, "gated", "silu", False),
    (1500, 1, 2, 48, 7704, "scattered", None, False),
]


@pytest.mark.parametrize("case", CASES, ids=["-".join(map(str, c)) for c in CASES])
def test_products(mg, case):
    T, k, E, K, N, form, act, halves = case
    r, order, experts, g = routed(mg, T, k, E, sum(case[:5]), drop=True)
    S = T * k
    in_order = form in ("scattered", "sorted")
    rows = S if in_order else T
    xq = torch.randint(-128, 128, (rows, K), generator=g, dtype=torch.int8)
    wq = torch.randint(-128, 128, (E, N, K), generator=g, dtype=torch.int8)
    xs = torch.rand(rows, generator=g) * 0.02 / 127 + 1e-4
    ws = torch.rand(E, N, generator=g) * 0.05 + 1e-3
    wt = torch.rand(S, generator=g) + 0.05
    flags = 0 if form == "sorted" else mg.PERMUTE_Y | mg.FUSE_MUL_POST if form == "scattered" \
        else mg.PERMUTE_X
    if act:
        flags |= mg.GATED_GELU if act == "gelu" else mg.GATED_SILU
        flags |= mg.GATED_HALVES if halves else 0
    cols = N // 2 if act else N
    out = torch.full((S, cols), 77.0, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    gather = None if form == "sorted" else r["gather"]
    got = mg.grouped_gemm_i8(xq.cuda(), xs.cuda(), wq.cuda(), ws.cuda(), r["m_sizes"], gather,
                             wt.cuda() if form == "scattered" else None, k, flags, Y=out,
                             error_flags=err)
    assert got is out and int(err) == 0
    n = order.size
    src = np.arange(n) if in_order else order // k
    y, _ = grouped(f64(xq)[src], experts, f64(wq), True)
    y = y * f64(xs)[src][:, None] * f64(ws)[experts]
    e = np.abs(y) * 6 * U
    if act:
        a, u = split(y, halves)
        ea, eu = split(e, halves)
        ref, tol = gated_ref(a, u, ea, eu, act)
        check(got[:n], ref, tol)
    elif form == "scattered":
        w = f64(wt)[order][:, None]
        check(got[torch.from_numpy(order).cuda()], y * w, np.abs(y * w) * (HALF + 6 * U))
        left = np.setdiff1d(np.arange(S), order)         # dropped slots
        assert (got[torch.from_numpy(left).cuda()] == 77).all()
        return
    else:
        check(got[:n], y, np.abs(y) * (HALF + 6 * U))
    assert (got[n:] == 77).all()                         # rows behind the last expert's


def test_largest_sums(mg):
    """-128 * -128 over the longest K stays in 32 bits."""
    K = 131056
    xq = torch.full((2, K), -128, dtype=torch.int8, device="cuda")
    wq = torch.full((1, 8, K), -128, dtype=torch.int8, device="cuda")
    one = torch.ones(8, device="cuda")
    m = torch.tensor([2], dtype=torch.int32, device="cuda")
    y = mg.grouped_gemm_i8(xq, one[:2], wq, one.view(1, 8), m, None, None, 1, 0)
    ref = 16384.0 * K
    assert (np.abs(f64(y) - ref) <= ref * (HALF + 2 * U)).all()


def test_from_values(mg):
    """Quantised from bf16 and multiplied: against the values that the codes stand for."""
    T, k, E, K, N = 129, 2, 4, 250, 96
    r, order, experts, g = routed(mg, T, k, E, 7)
    x = torch.randn(T, K, generator=g).bfloat16()
    w = torch.randn(E, N, K, generator=g).bfloat16()
    xq, xs = mg.quant_rows(x.cuda())
    wq, ws = mg.quant_rows(w.cuda())
    y = mg.grouped_gemm_i8(xq, xs, wq, ws, r["m_sizes"], r["gather"], None, k, mg.PERMUTE_X)
    xv = f64(xq) * f64(xs)[:, None]
    wv = f64(wq) * f64(ws)[:, :, None]
    ref, _ = grouped(xv[order // k], experts, wv, True)
    check(y[:order.size], ref, np.abs(ref) * (HALF + 6 * U) + 1e-12)
    # and near the product of the values themselves: half a code on each side
    true, _ = grouped(f64(x)[order // k], experts, f64(w), True)
    dx = f64(xs)[order // k][:, None] / 2
    dw = f64(ws)[experts] / 2
    ax = np.abs(f64(x)).sum(1)[order // k][:, None]
    aw = np.abs(f64(w)).sum(2)[experts]
    bound = ax * dw + aw * dx + K * dx * dw
    assert (np.abs(f64(y[:order.size]) - true) <= bound + np.abs(true) * 1.01 * HALF + bound * HALF).all()


def test_lost_rows_and_scales(mg):
    """A row whose values are not finite gives NaN outputs, and no other row does."""
    T, K, N = 40, 64, 72
    x = torch.randn(T, K, generator=torch.Generator().manual_seed(2))
    x[7, 3] = float("inf")
    xq, xs = mg.quant_rows(x.cuda())
    wq, ws = mg.quant_rows(torch.randn(1, N, K, generator=torch.Generator().manual_seed(3)).cuda())
    m = torch.tensor([T], dtype=torch.int32, device="cuda")
    y = mg.grouped_gemm_i8(xq, xs, wq, ws, m, None, None, 1, 0)
    nan = torch.isnan(y).all(1)
    assert nan[7] and int(nan.sum()) == 1 and torch.isfinite(y[~nan]).all()


def test_bad_device_data(mg):
    T, k, E, K, N = 30, 2, 4, 32, 64
    r, order, experts, g = routed(mg, T, k, E, 5, drop=False)
    xq = torch.randint(-5, 6, (T, K), generator=g, dtype=torch.int8).cuda()
    wq = torch.randint(-5, 6, (E, N, K), generator=g, dtype=torch.int8).cuda()
    xs, ws = torch.ones(T, device="cuda"), torch.ones(E, N, device="cuda")
    good = mg.grouped_gemm_i8(xq, xs, wq, ws, r["m_sizes"], r["gather"], None, k, mg.PERMUTE_X)
    gather = r["gather"].clone()
    gather[4], gather[9] = -1, T * k
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = torch.full_like(good, 5.0)
    mg.grouped_gemm_i8(xq, xs, wq, ws, r["m_sizes"], gather, None, k, mg.PERMUTE_X, Y=y,
                       error_flags=err)
    assert int(err) == mg.DERR_GATHER
    keep = torch.ones(T * k, dtype=torch.bool, device="cuda")
    keep[[4, 9]] = False
    assert torch.equal(y[keep], good[keep]) and (y[~keep] == 5).all()
    err.zero_()
    sizes = r["m_sizes"].clone()
    sizes[-1] += 3 * T * k
    mg.grouped_gemm_i8(xq, xs, wq, ws, sizes, r["gather"], None, k, mg.PERMUTE_X, Y=y,
                       error_flags=err)
    assert int(err) & mg.DERR_M_SIZES


def test_bad_gather_of_few_rows(mg):
    """As above where experts have one to three rows."""
    T, k, E, K, N = 4, 2, 4, 1040, 22
    r, order, experts, g = routed(mg, T, k, E, 6, drop=False)
    xq = torch.randint(-5, 6, (T, K), generator=g, dtype=torch.int8).cuda()
    wq = torch.randint(-5, 6, (E, N, K), generator=g, dtype=torch.int8).cuda()
    xs, ws = torch.ones(T, device="cuda"), torch.ones(E, N, device="cuda")
    for flags, cols in ((mg.PERMUTE_X, N), (mg.PERMUTE_X | mg.GATED_SILU, N // 2)):
        good = mg.grouped_gemm_i8(xq, xs, wq, ws, r["m_sizes"], r["gather"], None, k, flags)
        gather = r["gather"].clone()
        gather[1], gather[6] = -1, T * k
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        y = torch.full_like(good, 5.0)
        mg.grouped_gemm_i8(xq, xs, wq, ws, r["m_sizes"], gather, None, k, flags, Y=y,
                           error_flags=err)
        assert int(err) == mg.DERR_GATHER and y.shape[1] == cols
        keep = torch.ones(T * k, dtype=torch.bool, device="cuda")
        keep[[1, 6]] = False
        assert torch.equal(y[keep], good[keep]) and (y[~keep] == 5).all()
        err.zero_()
        sizes = r["m_sizes"].clone()
        sizes[0] = -3
        mg.grouped_gemm_i8(xq, xs, wq, ws, sizes, r["gather"], None, k, flags, Y=y,
                           error_flags=err)
        assert int(err) & mg.DERR_M_SIZES


def test_no_tokens(mg):
    e = torch.empty(0, 32, dtype=torch.int8, device="cuda")
    w = torch.zeros(2, 8, 32, dtype=torch.int8, device="cuda")
    y = mg.grouped_gemm_i8(e, torch.empty(0, device="cuda"), w, torch.ones(2, 8, device="cuda"),
                           torch.zeros(2, dtype=torch.int32, device="cuda"),
                           torch.empty(0, dtype=torch.int32, device="cuda"), None, 1, mg.PERMUTE_X)
    assert y.shape == (0, 8)
