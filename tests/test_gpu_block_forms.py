"""Forms of the feed-forward block beside those of its other tests: rows scattered without
weights, what is kept with the other permutation, the longest sums on the tiled kernels,
and outputs past 2^31 elements.  Bounds are those of tests/_block.py."""

import numpy as np
import pytest
import torch

from tests import _tiles as tiles
from tests._block import HALF, U, check, f64, gated_ref, grouped, routed, split, sum_err
from tests._block import pack_ref, unpack_ref
from tests.test_gpu_gated import CASES, IDS, bwd_ref, flags_of, inputs, join, kept_values, to_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import token_routing_amd as m
    m.load_library()
    return m


# T, k, E, K, N: vectors, small, four-stage, middle and large tiles
@pytest.mark.parametrize("T,k,E,K,N", [
    (1, 2, 4, 1040, 50), (9, 2, 16, 2048, 130), (257, 2, 3, 1008, 530), (33, 2, 5, 64, 137),
    (900, 2, 3, 1152, 1001), (700, 2, 3, 208, 5000), (1500, 1, 2, 272, 8008)])
def test_scattered_without_weights(mg, T, k, E, K, N):
    r, order, experts, g = routed(mg, T, k, E, T + N)
    S = T * k
    xq = torch.randint(-128, 128, (S, K), generator=g, dtype=torch.int8)
    wq = torch.randint(-128, 128, (E, N, K), generator=g, dtype=torch.int8)
    xs = torch.rand(S, generator=g) * 0.02 / 127 + 1e-4
    ws = torch.rand(E, N, generator=g) * 0.05 + 1e-3
    out = torch.full((S, N), 77.0, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    mg.grouped_gemm_i8(xq.cuda(), xs.cuda(), wq.cuda(), ws.cuda(), r["m_sizes"], r["gather"], None,
                       k, mg.PERMUTE_Y, Y=out, error_flags=err)
    assert int(err) == 0
    y, _ = grouped(f64(xq)[:order.size], experts, f64(wq), True)
    y = y * f64(xs)[:order.size, None] * f64(ws)[experts]
    check(out[torch.from_numpy(order).cuda()], y, np.abs(y) * (HALF + 6 * U))
    left = np.setdiff1d(np.arange(S), order)
    assert (out[torch.from_numpy(left).cuda()] == 77).all()


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows", [5, 130])
def test_longest_sums_of_tiles(mg, rows, gated):
    """-128 * -128 over the longest K in one accumulator of a matrix instruction."""
    K, N = 131056, 8
    xq = torch.full((rows, K), -128, dtype=torch.int8, device="cuda")
    wq = torch.full((1, N, K), -128, dtype=torch.int8, device="cuda")
    m = torch.tensor([rows], dtype=torch.int32, device="cuda")
    s = torch.full((rows,), 2.0 ** -14, device="cuda")
    one = torch.ones(1, N, device="cuda")
    y = mg.grouped_gemm_i8(xq, s, wq, one, m, None, None, 1, mg.GATED_SILU if gated else 0)
    v = np.full((rows, N), float(K))                     # 16384 K / 2^14
    if gated:
        e = v[:, ::2] * 6 * U
        check(y, *gated_ref(v[:, ::2], v[:, 1::2], e, e, "silu"))
    else:
        check(y, v, v * (HALF + 6 * U))


@pytest.mark.parametrize("keep", ["bf16", "packed"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward_kept_the_other_way(mg, case, keep):
    """bf16 kept with PERMUTE_X and packed without it."""
    T, k, E, K, I, act, halves = case
    px = keep == "bf16"
    r, order, experts, g, x, w = inputs(mg, case, px, seed=40)
    n, Ip = order.size, (I + 31) // 32 * 32
    h, kept = mg.gated_fwd(x.cuda(), w.cuda(), r["m_sizes"], r["gather"] if px else None, k,
                           flags_of(mg, act, halves) | (mg.PERMUTE_X if px else 0), keep=keep)
    a, mag = grouped(f64(x)[order // k if px else np.arange(n)], experts, f64(w), True)
    da = sum_err(mag, K)
    (gt, ut), (ge, ue) = split(a, halves), split(da, halves)
    check(h[:n], *gated_ref(gt, ut, ge, ue, act), "H")
    if keep == "bf16":
        check(kept[:n], a, da + (np.abs(a) + da) * HALF, "A")
        return
    q, s = (t[:n].cpu().numpy() for t in kept)
    for part, v, e in ((0, gt, ge), (1, ut, ue)):
        pq, ps = q[:, part * Ip:(part + 1) * Ip], s[:, part * Ip // 32:(part + 1) * Ip // 32]
        step = np.exp2(ps.astype(float) - 127).repeat(32, 1)[:, :I]
        check(unpack_ref(pq, ps, I), v, step / 2 + e, "packed")
        lo, hi = pack_ref(np.maximum(np.abs(v) - e, 0))[1], pack_ref(np.abs(v) + e)[1]
        assert ((ps >= lo) & (ps <= hi)).all()


@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward_the_other_way(mg, case, packed):
    """dY in slot order where the other test has it in expert order, and the reverse."""
    T, k, E, N, I, act, halves = case
    r, order, experts, g = routed(mg, T, k, E, 60 + sum(case[:5]))
    S, n, py = T * k, order.size, packed == halves
    kept, gt, ut = kept_values(g, S, I, halves, packed)
    dy = torch.randn(S, N, generator=g).bfloat16()
    w = (torch.randn(E, N, I, generator=g) / N ** 0.5).bfloat16()
    da, h = mg.gated_bwd(dy.cuda(), w.cuda(), to_cuda(kept), r["m_sizes"], r["gather"], k,
                         flags_of(mg, act, halves) | (mg.PERMUTE_Y if py else 0))
    (dg, tg), (du, tu), (hh, th) = bwd_ref(gt[:n], ut[:n], f64(dy)[order if py else np.arange(n)],
                                           experts, f64(w), act)
    check(da[:n], join(dg, du, halves), join(tg, tu, halves), "dA")
    check(h[:n], hh, th, "H")


def far_rows(S, row):
    """Rows at both ends and on either side of each 2^31st element of [S, row]."""
    at = list(range(3)) + list(range(S - 40, S))
    for i in range(1, S * row // 2 ** 31 + 1):
        b = i * 2 ** 31 // row
        at += range(max(b - 2, 0), min(b + 3, S))
    return torch.tensor(sorted(set(at)), device="cuda")


FAR = (131120, 16400)                                    # 2.15e9 elements of a plane


@pytest.mark.parametrize("form", ["plain", "scattered"])
def test_far_integers(mg, form):
    (S, N), K = FAR, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    xq = torch.randint(-128, 128, (S, K), generator=g, dtype=torch.int8, device="cuda")
    wq = torch.randint(-128, 128, (1, N, K), generator=g, dtype=torch.int8, device="cuda")
    xs = torch.rand(S, generator=g, device="cuda") + 0.1
    ws = torch.rand(1, N, generator=g, device="cuda") + 0.1
    m = torch.tensor([S], dtype=torch.int32, device="cuda")
    gather = torch.arange(S - 1, -1, -1, dtype=torch.int32, device="cuda")
    y = mg.grouped_gemm_i8(xq, xs, wq, ws, m, gather, None, 1,
                           mg.PERMUTE_Y if form == "scattered" else 0)
    at = far_rows(S, N)
    p = S - 1 - at if form == "scattered" else at
    ref = (xq[p].double() @ wq[0].double().t()) * xs[p].double()[:, None] * ws.double()
    tiles.check(y[at], ref, ref.abs() * (HALF + 6 * U))


def test_far_block(mg):
    """H past 2^31 elements, A and dA past 2^32, and the kept codes."""
    (S, I), K = FAR, 16
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(S, K, generator=g, device="cuda").bfloat16()
    w = torch.randn(1, 2 * I, K, generator=g, device="cuda").bfloat16()
    wd = torch.randn(1, K, I, generator=g, device="cuda").bfloat16()
    m = torch.tensor([S], dtype=torch.int32, device="cuda")
    f = mg.GATED_SILU | mg.GATED_HALVES
    at = far_rows(S, 2 * I)
    v, mag = x[at].double() @ w[0].double().t(), x[at].double().abs() @ w[0].double().abs().t()
    e = sum_err(mag, K)
    (gt, ut), (ge, ue) = tiles.split(v, True), tiles.split(e, True)
    dh, dmag = (x[at].double() @ wd[0].double(), x[at].double().abs() @ wd[0].double().abs())
    for keep in ("bf16", "packed"):
        h, kept = mg.gated_fwd(x, w, m, None, 1, f, keep=keep)
        tiles.check(h[at], *tiles.gated_ref(gt, ut, ge, ue, "silu"), "H")
        if keep == "bf16":
            tiles.check(kept[at], v, e + (v.abs() + e) * HALF, "A")
            kg, ku = tiles.split(kept[at].double(), True)
        else:
            parts = [[t[at].chunk(2, 1)[i] for t in kept] for i in range(2)]
            (kg, gs), (ku, us) = (tiles.unpack_ref(q, s, I) for q, s in parts)
            tiles.check(kg, gt, gs / 2 + ge, "gate codes")
            tiles.check(ku, ut, us / 2 + ue, "linear codes")
        da, h2 = mg.gated_bwd(x, wd, kept, m, None, 1, f, H=h)
        assert h2 is h
        (dg, tg), (du, tu), (hh, th) = tiles.bwd_ref(kg, ku, dh, sum_err(dmag, K), "silu")
        tiles.check(da[at], tiles.join(dg, du, True), tiles.join(tg, tu, True), "dA")
        tiles.check(h2[at], hh, th, "H again")
        del h, h2, da, kept


@pytest.mark.parametrize("T,K,N", [(3, 1040, 50), (90, 80, 136), (300, 64, 520), (1500, 48, 4000)])
def test_outputs_beside_16_bytes(mg, T, K, N):
    """Y, dA and H that begin 2 bytes off a 16-byte border, and nothing written beside them."""
    r, order, experts, g = routed(mg, T, 2, 3, T)
    S, n = 2 * T, order.size

    def off(rows, cols):
        flat = torch.full((rows * cols + 9,), 9.0, dtype=torch.bfloat16, device="cuda")
        return flat, flat[1:rows * cols + 1].view(rows, cols)

    xq, xs = mg.quant_rows(torch.randn(T, K, generator=g).cuda())
    wq, ws = mg.quant_rows(torch.randn(3, N, K, generator=g).cuda())
    for f, cols in ((0, N), (mg.GATED_SILU, N // 2)):
        flat, y = off(S, cols)
        args = (xq, xs, wq, ws, r["m_sizes"], r["gather"], None, 2, mg.PERMUTE_X | f)
        mg.grouped_gemm_i8(*args, Y=y)
        assert torch.equal(y[:n], mg.grouped_gemm_i8(*args)[:n]) and (y[n:] == 9).all()
        assert (flat[:1] == 9).all() and (flat[-8:] == 9).all()
    I = N // 2
    kept, _, _ = kept_values(g, S, I, False, True)
    dy = torch.randn(S, K, generator=g).bfloat16().cuda()
    wd = torch.randn(3, K, I, generator=g).bfloat16().cuda()
    args = (dy, wd, to_cuda(kept), r["m_sizes"], r["gather"], 2)
    for f in (mg.GATED_SILU, mg.GATED_GELU | mg.GATED_HALVES):
        (fa, da), (fh, h) = off(S, 2 * I), off(S, I)
        mg.gated_bwd(*args, f, dA=da, H=h)
        da2, h2 = mg.gated_bwd(*args, f)
        assert torch.equal(da[:n], da2[:n]) and torch.equal(h[:n], h2[:n])
        for flat, t in ((fa, da), (fh, h)):
            assert (t[n:] == 9).all() and (flat[:1] == 9).all() and (flat[-8:] == 9).all()
