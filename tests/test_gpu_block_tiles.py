"""The feed-forward block where workgroups take several tiles and each tile several
reduction stages, for every tile shape, kept form and direction: the ring of stages is
refilled, the next tile's copies start before this tile's epilogue, and the tables of two
tiles alternate.  Every output element is compared with 64-bit values (bounds of
tests/_block.py), and a second call has to give the same bits.  Which kernel each case
takes is asserted in tests/test_block_shapes.py."""

import pytest
import torch

from tests import _tiles as r
from tests._block import HALF, U
from tests._tiles import check, gated_ref, grouped, join, split, sum_err, unpack_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import token_routing_amd as m
    m.load_library()
    return m


def flags_of(mg, c):
    if c["act"] is None:
        return 0
    return (mg.GATED_GELU if c["act"] == "gelu" else mg.GATED_SILU) | (
        mg.GATED_HALVES if c["halves"] else 0)


def routing(c, g):
    """m_sizes and a gather of every slot, in no order."""
    sizes = torch.tensor(c["sizes"], dtype=torch.int32, device="cuda")
    return sizes, torch.randperm(r.rows_of(c), generator=g, device="cuda").to(torch.int32)


def normal(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).bfloat16()


def filled(shape, dtype=torch.bfloat16):
    return torch.full(shape, 9, dtype=dtype, device="cuda")


def same_again(outs, again):
    for a, b in zip(outs, again):
        assert torch.equal(a, b)


def select(op):
    cases = [c for c in r.CASES if c["op"] == op]
    return pytest.mark.parametrize("c", cases, ids=[r.name(c) for c in cases])


@select("fwd")
def test_forward(mg, c):
    g = torch.Generator(device="cuda").manual_seed(c["depth"] + c["cols"])
    S, k, n, K, I = r.rows_of(c), c["topk"], sum(c["sizes"]), c["depth"], c["cols"]
    m, gather = routing(c, g)
    x = normal(g, S // k if c["px"] else S, K)
    w = normal(g, len(c["sizes"]), 2 * I, K, std=2 / K ** 0.5)
    Ip = (I + 31) // 32 * 32

    def call():
        kept = None
        if c["keep"] == "bf16":
            kept = filled((S, 2 * I))
        elif c["keep"] == "packed":
            kept = filled((S, 2 * Ip), torch.int8), filled((S, Ip // 16), torch.uint8)
        h = filled((S, I))
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        mg.gated_fwd(x, w, m, gather if c["px"] else None, k,
                     flags_of(mg, c) | (mg.PERMUTE_X if c["px"] else 0), keep=c["keep"], H=h,
                     kept=kept, error_flags=err)
        assert int(err) == 0
        return [h] + (list(kept) if isinstance(kept, tuple) else [] if kept is None else [kept])

    outs = call()
    src = gather[:n].long() // k if c["px"] else torch.arange(n, device="cuda")
    a, mag = grouped(c, x[src], w, True)
    da = sum_err(mag, K)
    (gt, ut), (ge, ue) = split(a, c["halves"]), split(da, c["halves"])
    check(outs[0][:n], *gated_ref(gt, ut, ge, ue, c["act"]), "H")
    if c["keep"] == "bf16":
        check(outs[1][:n], a, da + (a.abs() + da) * HALF, "A")
    elif c["keep"] == "packed":
        q, s = outs[1:]
        for part, v, e in ((0, gt, ge), (1, ut, ue)):
            pq, ps = q[:n, part * Ip:(part + 1) * Ip], s[:n, part * Ip // 32:(part + 1) * Ip // 32]
            back, step = unpack_ref(pq, ps, I)
            check(back, v, step / 2 + e, "packed")
            assert (pq[:, I:] == 0).all()
            # no wider step than the largest value of its block asks for, its bound included
            top = torch.nn.functional.pad(v.abs() + e, (0, Ip - I)).view(n, -1, 32).amax(2)
            widest = torch.exp2(ps.double() - 127) * 63.5
            assert (top >= widest).all()
    for t in outs:
        assert (t[n:] == 9).all()
    same_again(outs, call())


@select("i8")
def test_integers(mg, c):
    g = torch.Generator(device="cuda").manual_seed(c["depth"] + c["cols"])
    S, k, n, K = r.rows_of(c), c["topk"], sum(c["sizes"]), c["depth"]
    N, E = r.out_cols(c), len(c["sizes"])
    m, gather = routing(c, g)
    scattered = c["form"] == "scattered"
    rows = S if scattered else S // k
    xq = torch.randint(-128, 128, (rows, K), generator=g, dtype=torch.int8, device="cuda")
    wq = torch.randint(-128, 128, (E, N, K), generator=g, dtype=torch.int8, device="cuda")
    xs = torch.rand(rows, generator=g, device="cuda") * 0.02 / 127 + 1e-4
    ws = torch.rand(E, N, generator=g, device="cuda") * 0.05 + 1e-3
    wt = torch.rand(S, generator=g, device="cuda") + 0.05 if scattered else None
    flags = flags_of(mg, c) | (mg.PERMUTE_Y | mg.FUSE_MUL_POST if scattered else mg.PERMUTE_X)

    def call():
        y = filled((S, c["cols"]))
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        mg.grouped_gemm_i8(xq, xs, wq, ws, m, gather, wt, k, flags, Y=y, error_flags=err)
        assert int(err) == 0
        return y

    got = call()
    slots = gather[:n].long()
    src = torch.arange(n, device="cuda") if scattered else slots // k
    y, _ = grouped(c, xq[src], wq, True)
    owner = torch.repeat_interleave(torch.arange(E, device="cuda"), m.long())
    y = y * xs.double()[src][:, None] * ws.double()[owner]
    if scattered:
        y = y * wt.double()[slots][:, None]
        check(got[slots], y, y.abs() * (HALF + 6 * U))
        assert (got[gather[n:].long()] == 9).all()
    else:
        if c["act"]:
            (gt, ut), (ge, ue) = split(y, c["halves"]), split(y.abs() * 6 * U, c["halves"])
            check(got[:n], *gated_ref(gt, ut, ge, ue, c["act"]))
        else:
            check(got[:n], y, y.abs() * (HALF + 6 * U))
        assert (got[n:] == 9).all()
    same_again([got], [call()])


@select("bwd")
def test_backward(mg, c):
    g = torch.Generator(device="cuda").manual_seed(c["depth"] + c["cols"])
    S, k, n, N, I = r.rows_of(c), c["topk"], sum(c["sizes"]), c["depth"], c["cols"]
    m, gather = routing(c, g)
    dy = normal(g, S, N)
    w = normal(g, len(c["sizes"]), N, I, std=1 / N ** 0.5)
    gt, ut = normal(g, S, I, std=2.0), normal(g, S, I, std=2.0)
    Ip = (I + 31) // 32 * 32
    if c["kept"] == "packed":
        parts = [mg.pack8(t) for t in (gt, ut)]
        kept = tuple(torch.cat([a, b], 1) for a, b in zip(*parts))
        gt, ut = (unpack_ref(q, s, I)[0] for q, s in parts)
        assert kept[0].shape == (S, 2 * Ip)
    else:
        kept = join(gt, ut, c["halves"]).contiguous()
        gt, ut = gt.double(), ut.double()

    def call():
        a = kept.clone() if c["kept"] == "place" else kept
        da = a if c["kept"] == "place" else filled((S, 2 * I))
        h = filled((S, I))
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        mg.gated_bwd(dy, w, a, m, gather, k, flags_of(mg, c) | (mg.PERMUTE_Y if c["py"] else 0),
                     dA=da, H=h, error_flags=err)
        assert int(err) == 0
        return [da, h]

    outs = call()
    dh, mag = grouped(c, dy[gather[:n].long()] if c["py"] else dy[:n], w, False)
    (dg, tg), (du, tu), (h, th) = r.bwd_ref(gt[:n], ut[:n], dh, sum_err(mag, N), c["act"])
    check(outs[0][:n], join(dg, du, c["halves"]), join(tg, tu, c["halves"]), "dA")
    check(outs[1][:n], h, th, "H")
    left = kept[n:] if c["kept"] == "place" else 9
    assert (outs[0][n:] == left).all() and (outs[1][n:] == 9).all()
    same_again(outs, call())
