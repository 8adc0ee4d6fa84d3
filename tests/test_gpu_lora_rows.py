"""Rows without an adapter (ids that routing dropped): a new Y or dX holds their
base row, bit for bit; a given one keeps what it held.  The other rows equal
those of a call that adds in place to a copy of base."""

import pytest
import torch

from test_gpu_lora import DT, mg  # noqa: F401  (mg is the fixture)

pytestmark = pytest.mark.gpu


def poisoned(shape, dtype):
    """Leaves a freed block of NaN for the next allocation of this size."""
    t = torch.full(shape, float("nan"), dtype=dtype, device="cuda")
    torch.cuda.synchronize()
    del t


# T, L, R, K, N, dtype, what is dropped
CASES = [
    (60, 4, 16, 136, 264, "bf16", "fifth"),        # tiles of 16 rows, odd columns
    (300, 2, 16, 128, 192, "fp16", "fifth"),       # tiles of 64 rows, whole columns
    (300, 2, 24, 200, 131, "bf16", "fifth"),
    (1000, 3, 64, 64, 2560, "bf16", "half"),       # several column groups
    (257, 5, 128, 72, 640, "fp16", "half"),
    (130, 2, 256, 64, 320, "bf16", "fifth"),
    (50, 3, 8, 64, 64, "bf16", "all"),
    (1, 1, 4, 8, 8, "bf16", "all"),
    (64, 3, 8, 64, 64, "bf16", "last"),            # one row without an adapter
]


def make(mg, case):
    T, L, R, K, N, dtype, what = case
    g = torch.Generator().manual_seed(T + N)
    dt = DT[dtype]
    ids = torch.randint(0, L, (T,), generator=g, dtype=torch.int32)
    off = dict(fifth=torch.arange(T) % 5 == 0, half=torch.rand(T, generator=g) < 0.5,
               all=torch.ones(T, dtype=torch.bool), last=torch.arange(T) == T - 1)[what]
    ids[off] = -1
    r = mg.moe_route(ids.cuda().view(T, 1), L, 16)

    def rnd(*s):
        return torch.randn(*s, generator=g).to(dt).cuda()

    return dict(X=rnd(T, K), A=rnd(L, R, K), B=rnd(L, N, R), m=r["m_sizes"], gather=r["gather"],
                base=rnd(T, N), dY=rnd(T, N), dbase=rnd(T, K), off=off.cuda())


@pytest.mark.parametrize("sorted_rows", [False, True], ids=["gather", "sorted"])
@pytest.mark.parametrize("case", CASES, ids=["-".join(str(x) for x in c) for c in CASES])
def test_new_outputs_hold_base(mg, case, sorted_rows):
    c = make(mg, case)
    T, gather, off = c["X"].shape[0], c["gather"], c["off"]
    if sorted_rows:                                # rows behind the adapters' are the dropped ones
        gather = None
        off = torch.arange(T, device="cuda") >= int(c["m"].sum())
    assert off.any()
    want = c["base"].clone()
    mg.lora_fwd(c["X"], c["A"], c["B"], c["m"], gather, Y=want)
    assert torch.equal(want[off], c["base"][off])  # a given Y keeps them
    poisoned(want.shape, want.dtype)
    Y, H = mg.lora_fwd(c["X"], c["A"], c["B"], c["m"], gather, base=c["base"], want_h=True)
    assert torch.equal(Y, want)
    dwant = c["dbase"].clone()
    mg.lora_bwd(None, c["dY"], c["A"], c["B"], None, c["m"], gather, dX=dwant, want_weights=False)
    assert torch.equal(dwant[off], c["dbase"][off])
    poisoned(dwant.shape, dwant.dtype)
    dX, dA, dB = mg.lora_bwd(c["X"], c["dY"], c["A"], c["B"], H, c["m"], gather, base=c["dbase"])
    assert torch.equal(dX, dwant)
    assert torch.isfinite(dA).all() and torch.isfinite(dB).all()


def test_a_given_output_keeps_its_rows(mg):
    """A Y and dX apart from base, given by the caller: rows without an adapter are left alone."""
    c = make(mg, CASES[1])
    off = c["off"]
    Y = torch.full_like(c["base"], 7.0)
    mg.lora_fwd(c["X"], c["A"], c["B"], c["m"], c["gather"], base=c["base"], Y=Y)
    new, _ = mg.lora_fwd(c["X"], c["A"], c["B"], c["m"], c["gather"], base=c["base"])
    assert torch.all(Y[off] == 7) and torch.equal(Y[~off], new[~off])
    dX = torch.full_like(c["dbase"], 7.0)
    kw = dict(base=c["dbase"], want_weights=False)
    mg.lora_bwd(None, c["dY"], c["A"], c["B"], None, c["m"], c["gather"], dX=dX, **kw)
    new, _, _ = mg.lora_bwd(None, c["dY"], c["A"], c["B"], None, c["m"], c["gather"], **kw)
    assert torch.all(dX[off] == 7) and torch.equal(dX[~off], new[~off])


def test_strided_base_and_bad_entries(mg):
    """base with a row stride; rows whose gather entry was spoiled count as rows without an adapter."""
    c = make(mg, CASES[2])
    N = c["base"].shape[1]
    wide = torch.full((c["base"].shape[0], N + 13), 3.0, dtype=c["base"].dtype, device="cuda")
    base = wide[:, 5:5 + N]
    base.copy_(c["base"])
    gather = c["gather"].clone()
    lost = int(gather[4])
    gather[4] = -7
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = c["base"].clone()
    mg.lora_fwd(c["X"], c["A"], c["B"], c["m"], gather, Y=want, error_flags=err)
    assert int(err.item()) == mg.DERR_GATHER and torch.equal(want[lost], c["base"][lost])
    poisoned(want.shape, want.dtype)
    Y, _ = mg.lora_fwd(c["X"], c["A"], c["B"], c["m"], gather, base=base)
    assert torch.equal(Y, want)


def test_few_rows_without_an_adapter_among_many(mg):
    """300001 rows of one adapter but for three: one or two workgroups look for
    them, in more than one piece each."""
    T, K = 300001, 8
    ids = torch.zeros(T, 1, dtype=torch.int32)
    lost = [17, 150000, T - 1]
    ids[lost] = -1
    r = mg.moe_route(ids.cuda(), 1, 16)
    g = torch.Generator().manual_seed(1)
    X = torch.randn(T, K, generator=g).bfloat16().cuda()
    A = torch.randn(1, 4, K, generator=g).bfloat16().cuda()
    B = torch.randn(1, 16, 4, generator=g).bfloat16().cuda()
    base = torch.randn(T, 16, generator=g).bfloat16().cuda()
    want = base.clone()
    mg.lora_fwd(X, A, B, r["m_sizes"], r["gather"], Y=want)
    poisoned(want.shape, want.dtype)
    Y, _ = mg.lora_fwd(X, A, B, r["m_sizes"], r["gather"], base=base)
    assert torch.equal(Y[lost], base[lost]) and torch.equal(Y, want)


def test_captured_with_changing_routing(mg):
    """One graph, replayed while the rows without an adapter change."""
    c = make(mg, CASES[1])
    T = c["X"].shape[0]
    args = (c["X"], c["A"], c["B"], c["m"], c["gather"])
    mg.lora_fwd(*args, base=c["base"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Y, _ = mg.lora_fwd(*args, base=c["base"])
    for drop in (0, 7, 150, T):
        ids = torch.arange(T, dtype=torch.int32) % 2
        ids[:drop] = -1
        r = mg.moe_route(ids.cuda().view(T, 1), 2, 16)
        c["m"].copy_(r["m_sizes"])
        c["gather"].copy_(r["gather"])
        Y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        want = c["base"].clone()
        mg.lora_fwd(*args, Y=want)
        assert torch.equal(Y, want), drop


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), 0.0])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T", [40, 300])
def test_rank_zero_takes_nothing_from_its_adapter(mg, T, dtype, scale):
    """An adapter of rank 0 leaves base as it is and has zero gradients, also
    where its place holds NaN weights and a scale that is not a number."""
    dt = DT[dtype]
    g = torch.Generator().manual_seed(T)
    L, R, K, N = 3, 16, 64, 192

    def rnd(*s):
        return torch.randn(*s, generator=g).to(dt).cuda()

    X, dY, base, dbase, A, B = rnd(T, K), rnd(T, N), rnd(T, N), rnd(T, K), rnd(L, R, K), rnd(L, N, R)
    A[1], B[1] = float("nan"), float("nan")
    ids = (torch.arange(T, dtype=torch.int32) % L).cuda()
    r = mg.moe_route(ids.view(T, 1), L, 16)
    ranks = torch.tensor([16, 0, 7], dtype=torch.int32).cuda()
    good = torch.tensor([1.5, 1.0, 0.5]).cuda()
    bad = torch.tensor([1.5, scale, 0.5]).cuda()
    out = {}
    for name, scales in (("good", good), ("bad", bad)):
        Y, H = mg.lora_fwd(X, A, B, r["m_sizes"], r["gather"], ranks=ranks, scales=scales,
                           base=base, want_h=True)
        out[name] = (Y, H, *mg.lora_bwd(X, dY, A, B, H, r["m_sizes"], r["gather"], ranks=ranks,
                                        scales=scales, base=dbase))
    none = ids == 1
    Y, _, dX, dA, dB = out["bad"]
    assert torch.equal(Y[none], base[none]) and torch.equal(dX[none], dbase[none])
    assert not dA[1].any() and not dB[1].any()
    for a, b in zip(out["good"], out["bad"]):
        assert torch.equal(a, b)
