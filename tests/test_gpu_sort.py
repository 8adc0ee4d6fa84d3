"""Token rows into expert order and back (moegg_permute, moegg_unpermute) and
their gradients against plain float64 evaluations.

Products of one weight and one value are exact in float64 and rounded once by
fp32 and once by the output's type, so permuted rows are compared bit for bit
with that arithmetic.  Sums of n terms in fp32 in any order are off by at most
n * 2^-24 * sum |terms| (fused products round no more often), plus half a step
of the output's type.
"""

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


# T, k, E, K, dtype, weighted, block_m
CASES = [
    (1, 1, 1, 1, "fp32", False, 0),
    (1, 8, 16, 2048, "bf16", True, 16),
    (7, 2, 4, 7, "bf16", True, 0),
    (50, 3, 9, 1003, "fp32", True, 16),
    (64, 8, 128, 2048, "bf16", False, 0),
    (33, 8, 100, 520, "fp16", True, 32),
    (20, 11, 12, 515, "bf16", True, 8),
    (129, 2, 8, 4099, "fp16", False, 128),
    (300, 4, 70, 264, "bf16", True, 128),
    (41, 17, 1024, 129, "fp32", True, 4),
    (37, 1, 3, 8192, "bf16", True, 0),
]
IDS = ["-".join(str(x) for x in c) for c in CASES]


def setup(mg, case, seed=0, drop=True):
    T, k, E, K, dtype, weighted, block_m = case
    g = torch.Generator().manual_seed(1000 + seed + T * K)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] if E >= k else
                       torch.randint(0, E, (k,), generator=g) for _ in range(T)]).to(torch.int32)
    if drop and T > 3:
        ids[1] = -1                          # a token without any expert
        ids[2, 0] = -1
    r = mg.moe_route(ids.cuda(), E, max(block_m, 1))
    w = (torch.rand(T * k, generator=g) + 0.1) if weighted else None
    pad = dict(offsets=r["offsets"], padded_offsets=r["padded_offsets"]) if block_m else {}
    rows = T * k + (E * (block_m - 1) if block_m else 0)
    # row of every slot, in plain python
    off, po = r["offsets"].tolist(), r["padded_offsets"].tolist()
    sc = r["scatter"].tolist()
    flat = ids.reshape(-1).tolist()
    want = [-1 if p < 0 else (p - off[e] + po[e] if block_m else p) for p, e in zip(sc, flat)]
    pads = []
    if block_m:
        m = r["m_sizes"].tolist()
        pads = [q for e in range(E) for q in range(po[e] + m[e], po[e + 1])]
    return g, r, w, pad, rows, np.array(want, dtype=np.int64), pads


def rnd(g, *shape, dtype):
    return torch.randn(*shape, generator=g).to(DT[dtype])


def cu(t):
    return None if t is None else t.cuda()


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_permute(mg, case):
    T, k, E, K, dtype, weighted, block_m = case
    g, r, w, pad, rows, want, pads = setup(mg, case)
    X = rnd(g, T, K, dtype=dtype)
    mark = 7.0
    Xs = torch.full((rows + 3, K), mark, dtype=DT[dtype], device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, row_map = mg.permute(X.cuda(), r["scatter"], k, cu(w), Xs=Xs, error_flags=err, **pad)
    assert out is Xs and int(err.item()) == 0
    assert row_map.cpu().tolist() == want.tolist()
    exp = torch.full((rows + 3, K), mark, dtype=DT[dtype])
    exp[pads] = 0
    v = X.float().repeat_interleave(k, 0)
    v = (v if w is None else v * w[:, None]).to(DT[dtype])
    keep = want >= 0
    exp[want[keep]] = v[torch.from_numpy(keep)]
    assert torch.equal(out.cpu(), exp)


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_permute_backward(mg, case):
    T, k, E, K, dtype, weighted, block_m = case
    g, r, w, pad, rows, want, pads = setup(mg, case, 1)
    X, D = rnd(g, T, K, dtype=dtype), rnd(g, rows, K, dtype=dtype)
    D[pads] = float("nan")                   # pad rows are not read
    row_map = torch.from_numpy(want).to(torch.int32)
    dX, dw = mg.permute_bwd(D.cuda(), X.cuda(), k, row_map.cuda(), cu(w))
    only, none = mg.permute_bwd(D.cuda(), None, k, row_map.cuda(), cu(w), want_dw=False)
    assert none is None and torch.equal(only, dX)
    check_collect(case, D, X, None, w, want, dX, dw)


def check_collect(case, rows_in, other, base, w, want, out, dw):
    T, k, E, K, dtype, _, _ = case
    half = torch.finfo(DT[dtype]).eps / 2
    idx = torch.from_numpy(np.maximum(want, 0))
    on = torch.from_numpy(want >= 0)[:, None]
    picked = torch.where(on, rows_in[idx].double(), torch.zeros((), dtype=torch.float64))
    terms = picked if w is None else picked * w.double()[:, None]
    terms = terms.view(T, k, K)
    ref, mag = terms.sum(1), terms.abs().sum(1)
    if base is not None:
        ref, mag = ref + base.double(), mag + base.double().abs()
    tiny = torch.finfo(DT[dtype]).smallest_normal * torch.finfo(DT[dtype]).eps
    bound = (k + 2) * 2.0 ** -24 * mag * (1 + half) + half * ref.abs() + tiny
    assert torch.all((out.cpu().double() - ref).abs() <= bound)
    if dw is not None:
        t = picked.view(T, k, K) * other.double()[:, None]
        err = (dw.cpu().double().view(T, k) - t.sum(2)).abs()
        assert torch.all(err <= (K + 1) * 2.0 ** -24 * t.abs().sum(2))


@pytest.mark.parametrize("with_base", [True, False], ids=["base", "nobase"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_unpermute(mg, case, with_base):
    T, k, E, K, dtype, weighted, block_m = case
    g, r, w, pad, rows, want, pads = setup(mg, case, 2)
    Y = rnd(g, rows, K, dtype=dtype)
    base = rnd(g, T, K, dtype=dtype) if with_base else None
    row_map = torch.from_numpy(want).to(torch.int32).cuda()
    out = mg.unpermute(Y.cuda(), k, row_map, cu(w), base=cu(base))
    check_collect(case, Y, None, base, w, want, out, None)
    if with_base:                            # onto the base in place
        buf = base.cuda()
        assert mg.unpermute(Y.cuda(), k, row_map, cu(w), base=buf, out=buf) is buf
        assert torch.equal(buf, out)
    if dtype == "bf16" and not with_base:    # the bf16 combine reads the same map
        c = mg.combine(Y.cuda(), k, row_map, cu(w), num_tokens=T)
        check_collect(case, Y, None, None, w, want, c, None)


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_unpermute_backward(mg, case):
    T, k, E, K, dtype, weighted, block_m = case
    g, r, w, pad, rows, want, pads = setup(mg, case, 3)
    dOut, Y = rnd(g, T, K, dtype=dtype), rnd(g, rows, K, dtype=dtype)
    row_map = torch.from_numpy(want).to(torch.int32)
    dY = torch.full((rows, K), 7.0, dtype=DT[dtype], device="cuda")
    out, dw = mg.unpermute_bwd(dOut.cuda(), Y.cuda(), k, row_map.cuda(), cu(w), dY=dY, **pad)
    exp = torch.full((rows, K), 7.0, dtype=DT[dtype])
    exp[pads] = 0
    v = dOut.float().repeat_interleave(k, 0)
    v = (v if w is None else v * w[:, None]).to(DT[dtype])
    keep = want >= 0
    exp[want[keep]] = v[torch.from_numpy(keep)]
    assert torch.equal(out.cpu(), exp)
    on = torch.from_numpy(keep)
    t = Y[torch.from_numpy(np.maximum(want, 0))].double() * dOut.double().repeat_interleave(k, 0)
    t = torch.where(on[:, None], t, torch.zeros_like(t))
    err = (dw.cpu().double() - t.sum(1)).abs()
    assert torch.all(err <= (K + 1) * 2.0 ** -24 * t.abs().sum(1))
    dY2 = torch.full((rows, K), 7.0, dtype=DT[dtype], device="cuda")
    out2, none = mg.unpermute_bwd(dOut.cuda(), None, k, row_map.cuda(), cu(w), dY=dY2,
                                  want_dw=False, **pad)
    assert none is None and torch.equal(out2, out)


def test_gradients_against_differences(mg):
    """<unpermute(permute(X, w)), G> along a direction in X and w, in fp32."""
    T, k, E, K = 24, 3, 6, 40
    g, r, w, pad, rows, want, _ = setup(mg, (T, k, E, K, "fp32", True, 8), 4, drop=False)
    X, G = torch.randn(T, K, generator=g), torch.randn(T, K, generator=g)
    u = torch.rand(T * k, generator=g)
    vX, vw, vu = (torch.randn(*s, generator=g) for s in ((T, K), (T * k,), (T * k,)))
    row_map = torch.from_numpy(want).to(torch.int32).cuda()

    def loss(X, w, u):
        xs, m = mg.permute(X.cuda(), r["scatter"], k, w.cuda(), block_m=8, **pad)
        assert torch.equal(m, row_map)
        y = mg.unpermute(xs, k, m, u.cuda())
        return (y.cpu().double() * G.double()).sum(), xs

    _, xs = loss(X, w, u)
    dY, du = mg.unpermute_bwd(G.cuda(), xs, k, row_map, u.cuda(), **pad)
    dX, dw = mg.permute_bwd(dY, X.cuda(), k, row_map, w.cuda())
    along = ((dX.cpu().double() * vX).sum() + (dw.cpu().double() * vw).sum()
             + (du.cpu().double() * vu).sum())
    h = 2.0 ** -7
    hi, _ = loss(X + h * vX, w + h * vw, u + h * vu)
    lo, _ = loss(X - h * vX, w - h * vw, u - h * vu)
    # the loss is a cubic form: the central difference is off by h^2 times its
    # third-order part <permute(vX, vw), vu G>, and by 8 roundings of 2^-24 of
    # the terms' magnitudes over h
    third, _ = loss(vX, vw, vu)
    mag = (X.abs().sum() + vX.abs().sum()) * 4 * k
    assert abs((hi - lo) / (2 * h) - along - h * h * third) <= 8 * 2.0 ** -24 * mag / h


def test_bad_rows_are_flagged_and_skipped(mg):
    T, k, E, K = 16, 2, 4, 72
    g, r, w, _, rows, want, _ = setup(mg, (T, k, E, K, "bf16", True, 0), 5, drop=False)
    X = rnd(g, T, K, dtype="bf16").cuda()
    sc = r["scatter"].clone()
    sc[5] = T * k + 9
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    Xs = torch.full((T * k, K), 7.0, dtype=torch.bfloat16, device="cuda")
    m = torch.empty_like(sc)
    mg.permute(X, sc, k, w.cuda(), Xs=Xs, row_map=m, error_flags=err)
    assert int(err.item()) == mg.DERR_GATHER and m[5].item() == -1
    assert torch.equal(torch.cat([m[:5], m[6:]]), torch.cat([sc[:5], sc[6:]]))
    assert mg.permute(X, sc, k, w.cuda(), Xs=Xs)[1] is sc
    assert torch.all(Xs[want[5]] == 7.0)
    for call in (lambda e: mg.permute_bwd(Xs, X, k, sc, w.cuda(), error_flags=e),
                 lambda e: mg.unpermute_bwd(X, Xs, k, sc, w.cuda(), error_flags=e)):
        err.zero_()
        _, dw = call(err)
        assert int(err.item()) == mg.DERR_GATHER and dw[5].item() == 0
    err.zero_()
    mg.unpermute(Xs, k, sc, w.cuda(), error_flags=err)
    assert int(err.item()) == mg.DERR_GATHER
    # a padded Xs with fewer rows than the layout needs
    po = torch.tensor([0, 16, 32, 48, 64], dtype=torch.int32, device="cuda")
    err.zero_()
    short = torch.full((40, K), 7.0, dtype=torch.bfloat16, device="cuda")
    _, m = mg.permute(X, r["scatter"], k, None, offsets=r["offsets"], padded_offsets=po, Xs=short,
                      error_flags=err)
    assert int(err.item()) == mg.DERR_GATHER
    assert int(m.max().item()) < 40


def test_empty_and_one_stream(mg):
    for T, k in ((0, 2), (0, 1)):
        X = torch.empty(T, 64, dtype=torch.float16, device="cuda")
        sc = torch.empty(0, dtype=torch.int32, device="cuda")
        Xs, m = mg.permute(X, sc, k)
        assert Xs.shape == (0, 64) and m.shape == (0,)
        assert mg.unpermute(Xs, k, m).shape == (0, 64)
        dX, dw = mg.permute_bwd(Xs, X, k, m)
        assert dX.shape == (0, 64) and dw.shape == (0,)
    # no tokens, but a padded layout: every row is a pad row
    z = torch.zeros(3, dtype=torch.int32, device="cuda")
    po = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    Xs = torch.full((10, 64), 7.0, dtype=torch.float16, device="cuda")
    mg.permute(torch.empty(0, 64, dtype=torch.float16, device="cuda"), z[:0], 2, offsets=z,
               padded_offsets=po, Xs=Xs)
    assert torch.all(Xs[:8] == 0) and torch.all(Xs[8:] == 7.0)
    case = (40, 4, 8, 136, "bf16", True, 16)
    g, r, w, pad, rows, want, _ = setup(mg, case, 6)
    X = rnd(g, 40, 136, dtype="bf16").cuda()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    Xs, m = mg.permute(X, r["scatter"], 4, block_m=16, stream=side, **pad)
    y = mg.unpermute(Xs, 4, m, w.cuda(), stream=side)
    side.synchronize()
    Xs2, m2 = mg.permute(X, r["scatter"], 4, block_m=16, **pad)
    assert torch.equal(m, m2) and torch.equal(y, mg.unpermute(Xs2, 4, m2, w.cuda()))


def test_unaligned_rows(mg):
    """Rows that start at any element, not at 16 bytes."""
    case = (30, 2, 4, 264, "bf16", True, 0)
    g, r, w, _, rows, want, _ = setup(mg, case, 7)
    X = rnd(g, 30, 264, dtype="bf16")
    flat = torch.zeros(30 * 264 + 3, dtype=torch.bfloat16, device="cuda")
    flat[3:] = X.cuda().view(-1)
    odd = flat[3:].view(30, 264)
    a, _ = mg.permute(X.cuda(), r["scatter"], 2, w.cuda(), Xs=torch.zeros(60, 264, dtype=X.dtype,
                                                                         device="cuda"))
    b, m = mg.permute(odd, r["scatter"], 2, w.cuda(), Xs=torch.zeros(60, 264, dtype=X.dtype,
                                                                     device="cuda"))
    assert torch.equal(a, b)
    base = flat[3:].view(30, 264)
    assert torch.equal(mg.unpermute(a, 2, m, w.cuda(), base=base),
                       mg.unpermute(a, 2, m, w.cuda(), base=X.cuda()))
