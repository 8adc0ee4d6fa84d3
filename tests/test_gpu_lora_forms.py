"""Every form of the adapters' kernels that the sizes select, against the float64
evaluation of test_gpu_lora: ranks of 65 to 256, whole and odd sizes, few and
many rows an adapter, launches whose workgroups take several runs of columns,
reductions cut over workgroups at odd lengths, and outputs past the last-level
cache.  Then gradients against differences of the library's own forwards.

Bounds are those of test_gpu_lora, element by element.  For long reductions
they are wide, so the relative Frobenius error is held as well: a stored value
is off by at most half a step, h or dh by the part that its two 16-bit halves
leave out, and an fp32 sum of n terms by n * 2^-23 of its largest partial sum;
partial sums of terms of random sign stay below twice the result in the
Frobenius norm.
"""

import pytest
import torch

from test_gpu_lora import DT, U, Case, close, mg  # noqa: F401  (mg is the fixture)

pytestmark = pytest.mark.gpu


def close_norm(got, ref, rel):
    err = float((got.detach().cpu().double() - ref).norm() / ref.norm())
    assert err <= rel, err


# T, L, R, K, N, dtype, ragged
BOTH = [
    # ranks of 65 to 128: odd and whole, few and many rows an adapter
    (40, 3, 72, 264, 328, "bf16", True),
    (200, 3, 100, 515, 264, "fp16", True),
    (60, 4, 96, 512, 768, "bf16", True),
    (60, 4, 128, 512, 768, "fp16", False),
    (130, 2, 128, 1024, 640, "fp16", False),
    (160, 2, 96, 640, 1024, "bf16", True),
    (4100, 3, 128, 128, 192, "bf16", True),
    # ranks of 129 to 256
    (45, 9, 130, 200, 264, "bf16", True),
    (50, 4, 256, 512, 512, "bf16", True),
    (50, 3, 200, 448, 576, "fp16", False),
    (150, 2, 256, 576, 448, "fp16", True),
    (150, 2, 160, 576, 640, "bf16", True),
    # whole sizes up to rank 64, two blocks of rows a tile
    (200, 2, 16, 512, 576, "fp16", True),
    (200, 2, 32, 576, 512, "fp16", False),
    (200, 2, 64, 512, 768, "fp16", True),
    (200, 2, 64, 768, 512, "bf16", True),
    # a reduction of odd length cut over several workgroups
    (20, 3, 24, 2051, 2051, "bf16", True),
    (20, 3, 7, 2051, 1999, "fp16", False),
    (70, 2, 100, 2051, 2051, "bf16", False),
]


def name(c):
    return "-".join(str(x) for x in c)


def check_forward(mg, c):
    y, e, h, he = c.forward(c.base)
    Y, H = mg.lora_fwd(c.X.cuda(), c.A.cuda(), c.B.cuda(), c.m_sizes, c.gather,
                       base=c.base.cuda(), want_h=True, **c.args())
    close(Y, y, e)
    close(H, h, he)
    rel = c.half + c.part + 2 * (c.K + c.R) * U
    close_norm(Y, y, rel)
    close_norm(H, h, 2 * c.K * U)
    buf = c.base.cuda()                        # in place, H not asked for
    mg.lora_fwd(c.X.cuda(), c.A.cuda(), c.B.cuda(), c.m_sizes, c.gather, Y=buf, **c.args())
    assert torch.equal(buf, Y)


def check_backward(mg, c, fp32):
    H = c.forward(c.base)[2].float()
    (dx, ex), (dA, eA), (dB, eB) = c.backward(H)
    args = (c.X.cuda(), c.dY.cuda(), c.A.cuda(), c.B.cuda(), H.cuda(), c.m_sizes, c.gather)
    gx, gA, gB = mg.lora_bwd(*args, base=c.dbase.cuda(), fp32_grads=fp32, **c.args())
    half = 0.0 if fp32 else c.half
    close(gx, dx, ex)
    close(gA, dA, eA + half * (dA.abs() + eA) + (0 if fp32 else c.floor))
    close(gB, dB, eB + half * (dB.abs() + eB) + (0 if fp32 else c.floor))
    close_norm(gx, dx, c.half + c.part + 2 * (c.N + c.R) * U)
    close_norm(gA, dA, half + c.part + 2 * (c.N + c.T) * U)
    close_norm(gB, dB, half + c.part + 2 * c.T * U)


@pytest.mark.parametrize("case", BOTH, ids=[name(c) for c in BOTH])
def test_forms_forward(mg, case):
    check_forward(mg, Case(mg, *case, seed=sum(case[:5])))


@pytest.mark.parametrize("fp32", [False, True], ids=["same", "fp32"])
@pytest.mark.parametrize("case", BOTH, ids=[name(c) for c in BOTH])
def test_forms_backward(mg, case, fp32):
    check_backward(mg, Case(mg, *case, seed=10 + sum(case[:5])), fp32)


# T, L, R, the short and the long side, dtype, ragged: workgroups of the product
# into the long side take two runs of 256 columns or more, the last one whole,
# partial or odd.
WIDE = [
    (2048, 2, 16, 64, 6400, "bf16", True),
    (2048, 2, 16, 72, 6403, "fp16", False),
    (1024, 64, 16, 64, 4160, "fp16", True),
    (2048, 2, 32, 64, 6400, "fp16", True),
    (2048, 2, 24, 64, 6408, "bf16", False),
    (2048, 2, 64, 64, 6400, "bf16", True),
    (2048, 2, 64, 136, 6400, "fp16", False),
    (2048, 2, 60, 65, 6411, "bf16", True),
    (1024, 64, 64, 64, 4096, "bf16", False),
    (1024, 2, 128, 64, 8192, "bf16", True),
    (1024, 2, 96, 64, 8256, "fp16", False),
    (1024, 2, 100, 72, 8195, "bf16", True),
    (1024, 64, 128, 64, 4096, "bf16", True),
    (512, 2, 256, 64, 8192, "bf16", False),
    (512, 2, 136, 72, 8200, "fp16", True),
    (1024, 64, 256, 64, 4096, "fp16", True),
]


@pytest.mark.parametrize("case", WIDE, ids=[name(c) for c in WIDE])
def test_several_runs_forward(mg, case):
    check_forward(mg, Case(mg, *case, seed=3 + sum(case[:5])))


@pytest.mark.parametrize("case", WIDE, ids=[name(c) for c in WIDE])
def test_several_runs_backward(mg, case):
    T, L, R, short, wide, dtype, ragged = case
    check_backward(mg, Case(mg, T, L, R, wide, short, dtype, ragged, seed=4 + sum(case[:5])), True)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("R", [16, 64])
def test_outputs_past_the_last_level_cache(mg, R, dtype):
    """4099 rows of 16640 columns, 273 MB of base and output, both directions; sampled rows."""
    T, L, C, K = 4099, 3, 16640, 64
    g = torch.Generator().manual_seed(R)
    dt = DT[dtype]
    ids = torch.randint(0, L, (T,), generator=g, dtype=torch.int32)
    r = mg.moe_route(ids.cuda().view(T, 1), L, 16)
    small = torch.randn(T, K, generator=g).to(dt)
    down = (torch.randn(L, R, K, generator=g) * K ** -0.5).to(dt)      # A, or B transposed
    up = torch.randn(L, C, R, generator=g).to(dt)
    base = torch.randn(T, C, generator=g).to(dt)
    half, part = torch.finfo(dt).eps / 2, 2.0 ** -17 if dtype == "bf16" else 2.0 ** -22
    Y, H = mg.lora_fwd(small.cuda(), down.cuda(), up.cuda(), r["m_sizes"], r["gather"],
                       base=base.cuda(), want_h=True)
    # the same numbers as a dX: dY = small, B = down^T, A = up^T
    dX, _, _ = mg.lora_bwd(None, small.cuda(), up.transpose(1, 2).contiguous().cuda(),
                           down.transpose(1, 2).contiguous().cuda(), None, r["m_sizes"],
                           r["gather"], base=base.cuda(), want_weights=False)
    for i in list(range(0, T, 97)) + [T - 1]:
        a = int(ids[i])
        x, A, B = small[i].double(), down[a].double(), up[a].double()
        h = A @ x
        y = base[i].double() + B @ h
        low = K * U * (A.abs() @ x.abs()) + h.abs() * (part + (R + 3) * U)
        if dtype == "fp16":
            low = low + h.abs().max() * 2.0 ** -39
        e = 1.001 * (B.abs() @ low)
        e = e + half * (y.abs() + e) + U * base[i].double().abs() + 2.0 ** -24
        for out in (Y, dX):
            assert torch.all((out[i].cpu().double() - y).abs() <= e), i


@pytest.mark.parametrize("R", [5, 16, 96])
@pytest.mark.parametrize("which", ["X", "A", "B"])
def test_gradients_against_differences_of_the_forward(mg, which, R):
    """The forward is linear in each of X, A and B, so the difference of two
    forwards along a direction v is exactly 2 dY(v) but for the stored values'
    rounding, half a step each.  With G that difference itself, <G, dY(v)> has
    no cancellation and is held against <gradient, v>.  X, A, B and v hold
    small integers (over powers of two): their sums are exact in bf16."""
    T, L, K, N = 50, 3, 72, 40
    g = torch.Generator().manual_seed(R)
    ids = torch.randint(0, L, (T,), generator=g, dtype=torch.int32)
    r = mg.moe_route(ids.cuda().view(T, 1), L, 16)

    def ints(*shape, top, scale):
        return (torch.randint(-top, top + 1, shape, generator=g) * scale).bfloat16()

    p = dict(X=ints(T, K, top=4, scale=0.25), A=ints(L, R, K, top=4, scale=0.125),
             B=ints(L, N, R, top=4, scale=0.25))
    v = ints(*p[which].shape, top=4, scale={"X": 0.25, "A": 0.125, "B": 0.25}[which])
    scales = torch.tensor([0.5, 1.0, 2.0]).cuda()
    zero = torch.zeros(T, N, dtype=torch.bfloat16).cuda()

    def forward(sign, want_h=False):
        q = dict(p)
        q[which] = p[which] + sign * v
        assert torch.equal(q[which].double(), p[which].double() + sign * v.double())
        return mg.lora_fwd(q["X"].cuda(), q["A"].cuda(), q["B"].cuda(), r["m_sizes"], r["gather"],
                           scales=scales, base=zero, want_h=want_h)

    hi, lo = forward(1)[0].cpu().double(), forward(-1)[0].cpu().double()
    H = forward(0, True)[1]
    G = ((hi - lo) / 2).bfloat16()
    dX, dA, dB = mg.lora_bwd(p["X"].cuda(), G.cuda(), p["A"].cuda(), p["B"].cuda(), H, r["m_sizes"],
                             r["gather"], scales=scales,
                             base=torch.zeros(T, K, dtype=torch.bfloat16).cuda(), fp32_grads=True)
    grad = dict(X=dX, A=dA, B=dB)[which].cpu().double()
    Gd = G.double()
    diff = ((hi - lo) / 2 * Gd).sum()
    along = (grad * v.double()).sum()
    # rounding of the two forwards; of dX (bf16) or of the parts of dh and H (2^-17,
    # sums of up to T + N + R terms in fp32)
    bound = 2.0 ** -8 * ((hi.abs() + lo.abs()) / 2 * Gd.abs()).sum()
    one = 2.0 ** -8 if which == "X" else 0.0
    mag = torch.zeros(())
    for i in range(T):
        a = int(ids[i])
        x, A, B = (t.double().abs() for t in (p["X"][i], p["A"][a], p["B"][a]))
        w = v.double().abs()
        h = (A @ w[i]) if which == "X" else (w[a] @ x) if which == "A" else (A @ x)
        b = w[a] if which == "B" else B
        mag = mag + scales[a].item() * (Gd[i].abs() @ (b @ h))
    bound = bound + one * (grad * v.double()).abs().sum() + (2.0 ** -17 + (T + N + R + K) * U) * mag
    assert diff > 20 * bound                   # the comparison says something
    assert abs(diff - along) <= bound, (float(diff), float(along), float(bound))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("R", [9, 16, 40])
def test_fp32_gradients_hold_fp32_values(mg, R, dtype):
    """One row an adapter, so that dB is scale * dY * H and dA is dh * X, one
    product an element: dY has a single column that is not zero, so dh is
    fp32(scale * dY * B) with a full mantissa, and H is any fp32 value.  bf16
    parts hold all 24 bits and fp16 parts leave 2^-22 at most; adding up to
    three parts' products and the scale round once each (2^-23)."""
    T, K, N = 37, 72, 40
    g = torch.Generator().manual_seed(R)
    dt = DT[dtype]
    X = (torch.randn(T, K, generator=g) + 3).to(dt)
    dY = torch.zeros(T, N, dtype=dt)
    dY[torch.arange(T), torch.randint(0, N, (T,), generator=g)] = 1.5
    A, B = torch.randn(T, R, K, generator=g).to(dt), torch.randn(T, N, R, generator=g).to(dt)
    H = torch.rand(T, R, generator=g) + 0.5
    s = torch.rand(T, generator=g) + 0.5
    sizes = torch.ones(T, dtype=torch.int32).cuda()
    _, dA, dB = mg.lora_bwd(X.cuda(), dY.cuda(), A.cuda(), B.cuda(), H.cuda(), sizes, None,
                            scales=s.cuda(), want_dx=False, fp32_grads=True)
    part = 0.0 if dtype == "bf16" else 2.0 ** -22
    dB_ref = s.double()[:, None, None] * dY.double()[:, :, None] * H.double()[:, None, :]
    dh = s.double()[:, None] * torch.einsum("tn,tnr->tr", dY.double(), B.double())
    dA_ref = dh[:, :, None] * X.double()[:, None, :]
    for got, ref in ((dA, dA_ref), (dB, dB_ref)):
        rel = (got.cpu().double() - ref).abs() / ref.abs().clamp(min=1e-30)
        assert float(rel[ref != 0].max()) <= part + 5 * U
        assert torch.all(got.cpu()[ref == 0] == 0)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows", [1, 40], ids=["one-row", "many-rows"])
@pytest.mark.parametrize("R", [9, 16, 24, 64, 128, 256])
def test_outputs_where_base_and_adapter_cancel(mg, R, rows, dtype):
    """base is minus the adapter's product, rounded, so the output is what that
    rounding left: it shows every bit that h or dh loses on its way into the
    product.  Each output column takes one rank (the others' weights are zero),
    so there is one product an element.  bf16 parts hold all 24 bits of h and
    fp16 parts leave 2^-22 at most; adding up to three parts, the scale and base
    round five times (2^-23 each, of the product), dh once more."""
    L, K, N = 7, 72, 136
    T = L * rows
    g = torch.Generator().manual_seed(R + rows)
    dt = DT[dtype]
    half, part = torch.finfo(dt).eps / 2, 0.0 if dtype == "bf16" else 2.0 ** -22
    tiny = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps
    one = torch.arange(L).repeat_interleave(rows)
    sizes = torch.full((L,), rows, dtype=torch.int32).cuda()
    s = torch.rand(L, generator=g) + 0.5
    X = torch.randn(T, K, generator=g).to(dt)
    A = torch.randn(L, R, K, generator=g).to(dt)
    B = torch.zeros(L, N, R)
    pick = torch.randint(0, R, (L, N), generator=g)
    B.scatter_(2, pick[:, :, None], torch.rand(L, N, 1, generator=g) + 0.5)
    B = B.to(dt)

    def check(got, base, prod, bound):
        ref = base.double() + prod
        err = (got.cpu().double() - ref).abs()
        assert torch.all(err <= half * ref.abs() * (1 + half) + bound + tiny), float(err.max())

    zero = torch.zeros(T, N, dtype=dt).cuda()
    H = mg.lora_fwd(X.cuda(), A.cuda(), B.cuda(), sizes, scales=s.cuda(), base=zero,
                    want_h=True)[1]
    prod = s.double()[one][:, None] * torch.stack(
        [B[a].double() @ H[t].cpu().double() for t, a in enumerate(one.tolist())])
    base = (-prod).to(dt)
    Y, _ = mg.lora_fwd(X.cuda(), A.cuda(), B.cuda(), sizes, scales=s.cuda(), base=base.cuda())
    check(Y, base, prod, (part + 5 * U) * prod.abs())

    # dX: dY has one column that is not zero, so dh is one product; A one rank a column
    dY = torch.zeros(T, N, dtype=dt)
    dY[torch.arange(T), torch.randint(0, N, (T,), generator=g)] = 1.5
    B2 = torch.randn(L, N, R, generator=g).to(dt)
    A2 = torch.zeros(L, R, K)
    pick = torch.randint(0, R, (L, K), generator=g)
    A2.scatter_(1, pick[:, None, :], torch.rand(L, 1, K, generator=g) + 0.5)
    A2 = A2.to(dt)
    dh = torch.stack([s.double()[a] * (dY[t].double() @ B2[a].double())
                      for t, a in enumerate(one.tolist())])
    prod = torch.stack([dh[t] @ A2[a].double() for t, a in enumerate(one.tolist())])
    base = (-prod).to(dt)
    dX, _, _ = mg.lora_bwd(None, dY.cuda(), A2.cuda(), B2.cuda(), None, sizes, scales=s.cuda(),
                           base=base.cuda(), want_weights=False)
    check(dX, base, prod, (part + 6 * U) * prod.abs())
