"""dW from a packed X (moegg_grouped_gemm_dW_packed).  The values are expanded without
loss, so that it has to give what moegg_grouped_gemm_dW gives on them, and the 64-bit
product within the sums' bound."""

import numpy as np
import pytest
import torch

from tests._block import HALF, check, f64, pack_ref, routed, sum_err, unpack_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import token_routing_amd as m
    m.load_library()
    return m


# T, k, E, N, K, form, fp32
CASES = [
    (1, 1, 1, 1, 1, "x", False),
    (64, 8, 128, 64, 72, "x", False),                    # the short-reduction kernel
    (64, 2, 8, 70, 100, "x", True),                      # any shape
    (600, 2, 4, 264, 136, "x", False),
    (600, 2, 4, 264, 136, "y", True),
    (700, 1, 2, 128, 96, "none", False),
    (2100, 2, 3, 256, 64, "x", False),                   # split reductions
    (90, 3, 5, 33, 47, "y", False),
    (300, 2, 3, 2504, 40, "x", False),                   # expanded in expert order
    (300, 2, 3, 2496, 40, "x", True),                    # and in token order
    (1100, 8, 4, 24, 136, "x", False),
]


@pytest.mark.parametrize("case", CASES, ids=["-".join(map(str, c)) for c in CASES])
def test_dw(mg, case):
    T, k, E, N, K, form, fp32 = case
    r, order, experts, g = routed(mg, T, k, E, sum(case[:5]))
    S, n = T * k, order.size
    x = torch.randn(T if form == "x" else S, K, generator=g).bfloat16()
    dy = torch.randn(S, N, generator=g).bfloat16()
    xq, xs = mg.pack8(x.cuda())
    flags = {"x": mg.PERMUTE_X, "y": mg.PERMUTE_Y, "none": 0}[form]
    flags |= mg.DW_FP32_OUT if fp32 else 0
    gather = None if form == "none" else r["gather"]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = mg.grouped_gemm_dW_packed(xq, xs, dy.cuda(), r["m_sizes"], gather, k, flags, K=K,
                                    error_flags=err)
    assert int(err) == 0
    same = mg.grouped_gemm_dW(mg.unpack8(xq, xs, K), dy.cuda(), r["m_sizes"], gather, k, flags)
    if (N % 8, K % 8) == (0, 0):
        assert torch.equal(got, same)
    v = unpack_ref(*pack_ref(f64(x)), K)[order // k if form == "x" else np.arange(n)]
    rows = f64(dy)[order if form == "y" else np.arange(n)]
    ref, mag = np.zeros((E, N, K)), np.zeros((E, N, K))
    for e in np.unique(experts):
        at = experts == e
        ref[e] = rows[at].T @ v[at]
        mag[e] = np.abs(rows[at]).T @ np.abs(v[at])
    tol = sum_err(mag, S)
    for t in (got, same):
        check(t, ref, tol + (0 if fp32 else (np.abs(ref) + tol) * HALF))


def test_linear_in_x(mg):
    """sum dW * D = sum dY * (X D_e^T) for any D: the formula's own identity."""
    T, k, E, N, K = 130, 2, 3, 40, 64
    r, order, experts, g = routed(mg, T, k, E, 4)
    x = torch.randn(T, K, generator=g).bfloat16()
    dy = torch.randn(T * k, N, generator=g).bfloat16()
    xq, xs = mg.pack8(x.cuda())
    dw = mg.grouped_gemm_dW_packed(xq, xs, dy.cuda(), r["m_sizes"], r["gather"], k,
                                   mg.PERMUTE_X | mg.DW_FP32_OUT, K=K)
    d = np.random.default_rng(1).standard_normal((E, N, K))
    v = unpack_ref(*pack_ref(f64(x)), K)[order // k]
    rows = f64(dy)[:order.size]
    want = sum((rows[p] * (d[e] @ v[p])).sum() for p, e in enumerate(experts))
    size = sum((np.abs(rows[p]) * (np.abs(d[e]) @ np.abs(v[p]))).sum()
               for p, e in enumerate(experts))
    assert abs((f64(dw) * d).sum() - want) <= sum_err(size, T * k)


def test_bad_gather_and_empty(mg):
    T, k, E, N, K = 40, 2, 4, 32, 64
    r, order, experts, g = routed(mg, T, k, E, 6, drop=False)
    x = torch.randn(T, K, generator=g).bfloat16()
    dy = torch.randn(T * k, N, generator=g).bfloat16().cuda()
    xq, xs = mg.pack8(x.cuda())
    gather = r["gather"].clone()
    gather[5], gather[70] = T * k, -3
    dz = dy.clone()
    dz[[5, 70]] = 0
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = mg.grouped_gemm_dW_packed(xq, xs, dy, r["m_sizes"], gather, k, mg.PERMUTE_X, K=K,
                                    error_flags=err)
    assert int(err) == mg.DERR_GATHER
    want = mg.grouped_gemm_dW_packed(xq, xs, dz, r["m_sizes"], r["gather"], k, mg.PERMUTE_X, K=K)
    assert torch.equal(got, want)
    none = mg.grouped_gemm_dW_packed(xq[:0], xs[:0], dy[:0],
                                     torch.zeros(E, dtype=torch.int32, device="cuda"),
                                     r["gather"][:0], k, mg.PERMUTE_X, K=K)
    assert none.shape == (E, N, K) and (none == 0).all()
