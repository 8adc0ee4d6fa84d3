"""Low-rank adapters (moegg_lora_fwd, moegg_lora_bwd) against a plain float64
evaluation, adapter by adapter.

Bounds: an fp32 sum of n terms is off by at most n * 2^-23 * sum |terms| (one
unit a term, as the matrix instructions need not round to nearest).  h or dh
enters the next product as two 16-bit parts.  In bf16 (8 bits of significand)
the high part of a value in [2^e, 2^(e+1)) leaves at most 2^(e-8), and the low
part of such a rest, at least 2^(e-9) in size, is off by at most 2^-8 * 2^(e-9)
= 2^(e-17): 2^-17 of the value.  In fp16 (11 bits) it is 2^-23, taken as 2^-22
(fp16 parts are scaled to the row's or column's largest
magnitude, of which at most 2^-39 more is lost).  A value stored in a 16-bit
type is off by half a step.
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = 2.0 ** -23


@pytest.fixture(scope="module")
def mg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import token_routing_amd as m
    m.load_library()
    return m


class Case:
    def __init__(self, mg, T, L, R, K, N, dtype, ragged, seed, drop=False, gather=True):
        g = torch.Generator().manual_seed(seed)
        dt = DT[dtype]
        self.T, self.L, self.R, self.K, self.N, self.dt = T, L, R, K, N, dt
        ids = torch.randint(0, L, (T,), generator=g, dtype=torch.int32)
        if L > 3:
            ids[ids == 1] = 2                  # an adapter without rows
        if drop and T > 4:
            ids[::5] = -1                      # rows of no adapter
        self.ids = ids
        r = mg.moe_route(ids.cuda().view(T, 1), L, 16)
        self.m_sizes, self.gather = r["m_sizes"], r["gather"]
        self.order = [int(i) for i in self.gather.cpu()]
        if not gather:                         # rows in adapter order already
            self.gather, self.order = None, list(range(T))
        self.sizes = self.m_sizes.cpu().tolist()
        self.rank = [R] * L
        if ragged:
            cyc = [R, max(1, R // 2), 0, max(1, R - 1)]
            self.rank = [cyc[a % 4] for a in range(L)]
        self.ranks = torch.tensor(self.rank, dtype=torch.int32).cuda() if ragged else None
        self.scale = torch.rand(L, generator=g) + 0.5
        self.scales = self.scale.cuda()
        self.X = torch.randn(T, K, generator=g).to(dt)
        self.A = (torch.randn(L, R, K, generator=g) * K ** -0.5).to(dt)
        self.B = torch.randn(L, N, R, generator=g).to(dt)
        self.dY = (torch.randn(T, N, generator=g) * 0.1).to(dt)
        self.base = torch.randn(T, N, generator=g).to(dt)
        self.dbase = (torch.randn(T, K, generator=g) * 0.1).to(dt)
        if ragged:                             # past the rank nothing is read into results
            for a in range(L):
                self.A[a, self.rank[a]:] = float("nan")
                self.B[a, :, self.rank[a]:] = float("nan")
        self.half = torch.finfo(dt).eps / 2
        self.part = 2.0 ** -17 if dtype == "bf16" else 2.0 ** -22
        self.floor = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps

    def segments(self):
        o = 0
        for a, m in enumerate(self.sizes):
            yield a, self.rank[a], float(self.scale[a]), self.order[o:o + m], slice(o, o + m)
            o += m

    def args(self):
        return dict(ranks=self.ranks, scales=self.scales)

    def forward(self, base):
        """y, its bound, h and its bound."""
        y, e = base.double(), torch.zeros(self.T, self.N, dtype=torch.float64)
        h = torch.zeros(self.T, self.R, dtype=torch.float64)
        he = torch.zeros_like(h)
        for a, r, s, rows, seg in self.segments():
            x, A, B = self.X[rows].double(), self.A[a, :r].double(), self.B[a, :, :r].double()
            hh = x @ A.T
            hb = self.K * U * (x.abs() @ A.abs().T)
            h[seg, :r], he[seg, :r] = hh, hb
            y[rows] += s * (hh @ B.T)
            low = hh.abs() * (self.part + (self.R + 3) * U)
            if self.dt == torch.float16 and r:
                low = low + hh.abs().amax(1, keepdim=True) * 2.0 ** -39
            e[rows] += 1.001 * s * ((hb + low) @ B.abs().T)
        e += self.half * (y.abs() + e) + self.floor + U * base.double().abs()
        return y, e, h, he

    def backward(self, H):
        dx, ex = self.dbase.double(), torch.zeros(self.T, self.K, dtype=torch.float64)
        dA = torch.zeros(self.L, self.R, self.K, dtype=torch.float64)
        dB = torch.zeros(self.L, self.N, self.R, dtype=torch.float64)
        eA, eB = torch.zeros_like(dA), torch.zeros_like(dB)
        H = H.double()
        for a, r, s, rows, seg in self.segments():
            if not rows or not r:
                continue
            x, dy = self.X[rows].double(), self.dY[rows].double()
            A, B, h = self.A[a, :r].double(), self.B[a, :, :r].double(), H[seg, :r]
            dh = s * (dy @ B)
            hb = (self.N + 1) * U * s * (dy.abs() @ B.abs())
            dx[rows] += dh @ A
            low = dh.abs() * (self.part + (self.R + 3) * U)
            if self.dt == torch.float16:
                low = low + dh.abs().amax() * 2.0 ** -39
            ex[rows] += 1.001 * ((hb + low) @ A.abs())
            n = len(rows) + 20
            dA[a, :r] = dh.T @ x
            low = dh.abs() * (self.part + n * U)
            hlow = h.abs() * (self.part + n * U)
            if self.dt == torch.float16:
                low = low + dh.abs().amax() * 2.0 ** -39
                hlow = hlow + h.abs().amax() * 2.0 ** -39
            eA[a, :r] = 1.001 * ((hb + low).T @ x.abs())
            dB[a, :, :r] = s * (dy.T @ h)
            eB[a, :, :r] = 1.001 * s * (dy.abs().T @ hlow)
        ex += self.half * (dx.abs() + ex) + self.floor + U * self.dbase.double().abs()
        return (dx, ex), (dA, eA), (dB, eB)


def close(got, ref, err):
    d = (got.detach().cpu().double() - ref).abs()
    assert torch.all(d <= err), float((d - err).max())


# T, L, R, K, N, dtype, ragged
CASES = [
    (1, 1, 1, 8, 8, "bf16", False),
    (3, 2, 2, 9, 67, "fp16", False),
    (1, 1, 16, 2048, 2048, "bf16", False),
    (1, 3, 8, 100, 70, "fp16", True),
    (7, 5, 4, 515, 264, "bf16", True),
    (33, 1, 24, 1024, 136, "fp16", False),
    (64, 32, 16, 1536, 1024, "bf16", False),
    (64, 70, 16, 264, 520, "bf16", True),
    (100, 6, 17, 129, 1003, "bf16", True),
    (130, 3, 33, 640, 333, "fp16", True),
    (200, 8, 64, 512, 768, "bf16", True),
    (77, 2, 130, 200, 264, "bf16", False),
    (90, 2, 256, 136, 72, "fp16", True),
    (1500, 2, 16, 136, 264, "bf16", True),     # several chunks of the gradients
    (1100, 1, 40, 72, 130, "fp16", False),
    (40, 300, 5, 64, 64, "bf16", False),       # more adapters than rows
    (2100, 1000, 8, 40, 72, "bf16", False),
]
IDS = ["-".join(str(x) for x in c) for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(mg, case):
    c = Case(mg, *case, seed=sum(case[:5]))
    y, e, h, he = c.forward(c.base)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    Y, H = mg.lora_fwd(c.X.cuda(), c.A.cuda(), c.B.cuda(), c.m_sizes, c.gather,
                       base=c.base.cuda(), want_h=True, error_flags=err, **c.args())
    assert int(err.item()) == 0
    close(Y, y, e)
    close(H, h, he)
    buf = c.base.cuda()                        # in place, H not asked for
    out, none = mg.lora_fwd(c.X.cuda(), c.A.cuda(), c.B.cuda(), c.m_sizes, c.gather, Y=buf,
                            **c.args())
    assert out is buf and none is None and torch.equal(buf, Y)


@pytest.mark.parametrize("fp32", [False, True], ids=["same", "fp32"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward(mg, case, fp32):
    c = Case(mg, *case, seed=10 + sum(case[:5]))
    H = c.forward(c.base)[2].float()
    (dx, ex), (dA, eA), (dB, eB) = c.backward(H)
    args = (c.X.cuda(), c.dY.cuda(), c.A.cuda(), c.B.cuda(), H.cuda(), c.m_sizes, c.gather)
    gx, gA, gB = mg.lora_bwd(*args, base=c.dbase.cuda(), fp32_grads=fp32, **c.args())
    close(gx, dx, ex)
    half = 0.0 if fp32 else c.half
    assert gA.dtype == gB.dtype == (torch.float32 if fp32 else c.dt)
    close(gA, dA, eA + half * (dA.abs() + eA) + (0 if fp32 else c.floor))
    close(gB, dB, eB + half * (dB.abs() + eB) + (0 if fp32 else c.floor))
    buf = c.dbase.cuda()
    only, na, nb = mg.lora_bwd(None, args[1], args[2], args[3], None, c.m_sizes, c.gather, dX=buf,
                               want_weights=False, **c.args())
    assert na is None and nb is None and only is buf and torch.equal(buf, gx)
    nx, wA, wB = mg.lora_bwd(*args, want_dx=False, fp32_grads=fp32, **c.args())
    assert nx is None and torch.equal(wA, gA) and torch.equal(wB, gB)


@pytest.mark.parametrize("case", [CASES[3], CASES[8], CASES[12]], ids=[IDS[3], IDS[8], IDS[12]])
def test_rows_in_adapter_order_and_strides(mg, case):
    """No gather_idx, and X, base and Y as column slices of wider matrices at odd offsets."""
    c = Case(mg, *case, seed=99, gather=False)
    y, e, _, _ = c.forward(c.base)
    X = torch.zeros(c.T, c.K + 5, dtype=c.dt, device="cuda")[:, 3:3 + c.K]
    base = torch.zeros(c.T, c.N + 9, dtype=c.dt, device="cuda")[:, 1:1 + c.N]
    wide = torch.full((c.T, c.N + 7), 7.0, dtype=c.dt, device="cuda")
    Y = wide[:, 5:5 + c.N]
    X.copy_(c.X)
    base.copy_(c.base)
    mg.lora_fwd(X, c.A.cuda(), c.B.cuda(), c.m_sizes, None, base=base, Y=Y, **c.args())
    close(Y, y, e)
    assert torch.all(wide[:, :5] == 7) and torch.all(wide[:, 5 + c.N:] == 7)
    H = c.forward(c.base)[2].float().cuda()
    dY = torch.zeros(c.T, c.N + 3, dtype=c.dt, device="cuda")[:, 2:2 + c.N]
    dY.copy_(c.dY)
    dx = torch.full((c.T, c.K + 6), 7.0, dtype=c.dt, device="cuda")
    inner = dx[:, 1:1 + c.K]
    inner.copy_(c.dbase)
    (rx, ex), (rA, eA), (rB, eB) = c.backward(H.cpu())
    _, gA, gB = mg.lora_bwd(X, dY, c.A.cuda(), c.B.cuda(), H, c.m_sizes, None, dX=inner,
                            fp32_grads=True, **c.args())
    close(inner, rx, ex)
    close(gA, rA, eA)
    close(gB, rB, eB)
    assert torch.all(dx[:, :1] == 7) and torch.all(dx[:, 1 + c.K:] == 7)


def test_rows_without_an_adapter_keep_their_output(mg):
    c = Case(mg, 60, 4, 16, 136, 264, "bf16", False, 5, drop=True)
    y, e, _, _ = c.forward(c.base)
    buf = c.base.cuda()
    mg.lora_fwd(c.X.cuda(), c.A.cuda(), c.B.cuda(), c.m_sizes, c.gather, Y=buf, scales=c.scales)
    close(buf, y, e)
    off = c.ids < 0
    assert off.any() and torch.equal(buf.cpu()[off], c.base[off])


def test_large_and_odd_values(mg):
    """h past fp16's range stays finite; a row's infinity stays in its row; rank 0 is base."""
    T, L, R, K, N = 20, 3, 8, 64, 40
    g = torch.Generator().manual_seed(3)
    X = torch.full((T, K), 200.0).half()
    A = (torch.rand(L, R, K, generator=g) * 50 + 50).half()        # h about 1e6
    B = (torch.randn(L, N, R, generator=g) * 1e-4).half()
    sizes = torch.tensor([7, 6, 7], dtype=torch.int32)
    ranks = torch.tensor([8, 0, 5], dtype=torch.int32)
    base = torch.randn(T, N, generator=g).half()
    Y, H = mg.lora_fwd(X.cuda(), A.cuda(), B.cuda(), sizes.cuda(), None, ranks=ranks.cuda(),
                       base=base.cuda(), want_h=True)
    assert H.max().item() > 70000 and torch.isfinite(Y).all()
    o = 0
    for a, (m, r) in enumerate(zip(sizes.tolist(), ranks.tolist())):
        seg = slice(o, o + m)
        h = X[seg].double() @ A[a, :r].double().T
        ref = base[seg].double() + h @ B[a, :, :r].double().T
        mag = h.abs() @ B[a, :, :r].double().abs().T
        bound = 2.0 ** -11 * ref.abs() + (2.0 ** -21 + (K + R + 4) * U) * mag + 2.0 ** -23 + 1e-6
        assert torch.all((Y[seg].cpu().double() - ref).abs() <= bound)
        o += m
    assert torch.equal(Y[7:13].cpu(), base[7:13])
    X2 = X.clone()
    X2[2, 5] = float("inf")
    X2[15, 1] = float("nan")
    Y2, _ = mg.lora_fwd(X2.cuda(), A.cuda(), B.cuda(), sizes.cuda(), None, ranks=ranks.cuda(),
                        base=base.cuda())
    keep = [i for i in range(T) if i not in (2, 15)]
    assert torch.equal(Y2[keep], Y[keep])
    assert not torch.isfinite(Y2[2]).any() and torch.isnan(Y2[15]).all()


def test_bad_metadata_is_flagged(mg):
    c = Case(mg, 50, 4, 16, 72, 72, "bf16", False, 8)
    args = (c.X.cuda(), c.A.cuda(), c.B.cuda())
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for gather, sizes, ranks, bit in (
            (c.gather.clone().index_fill_(0, torch.tensor([3], device="cuda"), 50), c.m_sizes,
             None, mg.DERR_GATHER),
            (c.gather.clone().index_fill_(0, torch.tensor([3], device="cuda"), -2), c.m_sizes,
             None, mg.DERR_GATHER),
            (c.gather, torch.tensor([30, 30, 2, 1], dtype=torch.int32).cuda(), None,
             mg.DERR_M_SIZES),
            (c.gather, torch.tensor([3, -9, 2, 1], dtype=torch.int32).cuda(), None,
             mg.DERR_M_SIZES),
            (c.gather, torch.tensor([2 ** 31 - 1] * 4, dtype=torch.int32).cuda(), None,
             mg.DERR_M_SIZES),
            (c.gather, c.m_sizes, torch.tensor([16, 17, 2, -1], dtype=torch.int32).cuda(),
             mg.DERR_RANK)):
        err.zero_()
        _, H = mg.lora_fwd(*args, sizes, gather, ranks=ranks, base=c.base.cuda(), want_h=True,
                           error_flags=err)
        assert int(err.item()) == bit
        err.zero_()
        mg.lora_bwd(args[0], c.dY.cuda(), args[1], args[2], torch.zeros_like(H), sizes, gather,
                    ranks=ranks, base=c.dbase.cuda(), error_flags=err)
        assert int(err.item()) == bit


def test_no_rows(mg):
    A = torch.zeros(3, 8, 40, dtype=torch.bfloat16, device="cuda")
    B = torch.zeros(3, 24, 8, dtype=torch.bfloat16, device="cuda")
    X = torch.empty(0, 40, dtype=torch.bfloat16, device="cuda")
    dY = torch.empty(0, 24, dtype=torch.bfloat16, device="cuda")
    sizes = torch.zeros(3, dtype=torch.int32, device="cuda")
    Y, H = mg.lora_fwd(X, A, B, sizes, base=dY, want_h=True)
    assert Y.shape == (0, 24) and H.shape == (0, 8)
    dA = torch.full_like(A, 7.0)
    dB = torch.full_like(B, 7.0)
    dX, _, _ = mg.lora_bwd(X, dY, A, B, H, sizes, base=X, dA=dA, dB=dB)
    assert dX.shape == (0, 40) and not dA.any() and not dB.any()


def test_gradients_against_differences(mg):
    """<Y, G> along one direction in X, A and B, from forwards of the library itself."""
    T, L, R, K, N = 48, 3, 6, 72, 40
    c = Case(mg, T, L, R, K, N, "bf16", False, 21)
    G = c.dY
    zero_y, zero_x = torch.zeros(T, N), torch.zeros(T, K)
    g = torch.Generator().manual_seed(4)
    vX = torch.randn(T, K, generator=g).to(c.dt)
    vA = (torch.randn(L, R, K, generator=g) * K ** -0.5).to(c.dt)
    vB = torch.randn(L, N, R, generator=g).to(c.dt)

    def loss(X, A, B):
        Y = torch.zeros(T, N, dtype=torch.float64)
        mag = 0.0
        for a, r, s, rows, _ in c.segments():
            h = X[rows] @ A[a].T
            Y[rows] = s * (h @ B[a].T)
            mag += (s * ((X[rows].abs() @ A[a].abs().T) @ B[a].abs().T) * G[rows].double().abs()).sum()
        return (Y * G.double()).sum(), mag

    H = mg.lora_fwd(c.X.cuda(), c.A.cuda(), c.B.cuda(), c.m_sizes, c.gather, scales=c.scales,
                    base=zero_y.to(c.dt).cuda(), want_h=True)[1]
    dX, dA, dB = mg.lora_bwd(c.X.cuda(), G.cuda(), c.A.cuda(), c.B.cuda(), H, c.m_sizes, c.gather,
                             scales=c.scales, base=zero_x.to(c.dt).cuda(), fp32_grads=True)
    along = ((dX.cpu().double() * vX.double()).sum() + (dA.cpu().double() * vA.double()).sum()
             + (dB.cpu().double() * vB.double()).sum())
    h = 2.0 ** -8
    X, A, B = c.X.double(), c.A.double(), c.B.double()
    hi, _ = loss(X + h * vX.double(), A + h * vA.double(), B + h * vB.double())
    lo, _ = loss(X - h * vX.double(), A - h * vA.double(), B - h * vB.double())
    third, _ = loss(vX.double(), vA.double(), vB.double())   # cubic: the difference's only error
    # dX is rounded to bf16 (half a step, 2^-9... of each element); dA, dB carry 2^-17
    bound = 2.0 ** -8 * (dX.cpu().double() * vX.double()).abs().sum() + 2.0 ** -14 * (
        (dA.cpu().double() * vA.double()).abs().sum() + (dB.cpu().double() * vB.double()).abs().sum())
    bound = bound + 2.0 ** -14 * (loss(X, A, vB.double())[1] + loss(vX.double(), A, B)[1]
                                  + loss(X, vA.double(), B)[1])
    assert abs((hi - lo) / (2 * h) - h * h * third - along) <= bound


def test_repeatable_and_on_a_side_stream(mg):
    c = Case(mg, 700, 5, 32, 264, 520, "bf16", True, 31)
    a = (c.X.cuda(), c.A.cuda(), c.B.cuda(), c.m_sizes, c.gather)
    base, dbase, dY = c.base.cuda(), c.dbase.cuda(), c.dY.cuda()
    Y, H = mg.lora_fwd(*a, base=base, want_h=True, **c.args())
    ref = mg.lora_bwd(a[0], dY, a[1], a[2], H, c.m_sizes, c.gather, base=dbase, **c.args())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(2):
        Y2, H2 = mg.lora_fwd(*a, base=base, want_h=True, stream=side, **c.args())
        got = mg.lora_bwd(a[0], dY, a[1], a[2], H2, c.m_sizes, c.gather, base=dbase, stream=side,
                          **c.args())
        side.synchronize()
        assert torch.equal(Y, Y2)
        for p, q in zip(ref, got):
            assert torch.equal(p, q)
