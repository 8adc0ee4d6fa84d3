"""Rows in 8-bit integers (moegg_quant_rows) and packed blocks (moegg_pack8,
moegg_unpack8) against their definitions in 64 bits: codes, scales and bytes have to
be equal, so has every value read back in bf16 and fp32."""

import numpy as np
import pytest
import torch

from tests._block import f64, pack_ref, unpack_ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def mg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import token_routing_amd as m
    m.load_library()
    return m


def values(rows, cols, dtype, seed, extra=0):
    """Values of very different rows, zeros and ties among them; `extra` columns beside."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols + extra, generator=g) * torch.exp2(
        torch.randint(-12, 12, (rows, 1), generator=g).float())
    x[torch.rand(rows, cols + extra, generator=g) < 0.05] = 0.0
    if rows > 2:
        x[2] = 0.0
    if rows > 3:
        x[3] = torch.randint(-127, 128, (cols + extra,), generator=g).float() + 0.5
    if rows > 4:
        x[4] = -127.5                                    # the border of a step's choice
    return x.to(DT[dtype])


SIZES = [(1, 1), (1, 31), (3, 32), (5, 33), (64, 2048), (7, 2049), (9, 70), (33, 8192), (6, 8200),
         (2, 20011), (300, 16), (1001, 203)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,cols", SIZES)
def test_quant_rows(mg, rows, cols, dtype):
    x = values(rows, cols, dtype, rows * cols, extra=5)
    d = x.cuda()[:, :cols]                               # rows cols + 5 apart
    q, s = mg.quant_rows(d)
    v = f64(x[:, :cols])
    m = np.abs(v).max(1)
    want = np.rint(np.where(m[:, None] > 0, 127 * v / np.where(m > 0, m, 1)[:, None], 0))
    assert q.shape == (rows, (cols + 15) // 16 * 16)
    assert np.array_equal(q[:, :cols].cpu().numpy(), want)
    assert (q[:, cols:] == 0).all()
    assert np.array_equal(s.cpu().numpy(), np.float32(m) / np.float32(127))


def test_quant_rows_ties_in_64_bits(mg):
    """fp32 quotients whose product with 127 / m rounds to a tie that they are not."""
    g = torch.Generator().manual_seed(3)
    m = (torch.rand(4096, 1, generator=g) + 1).float()
    k = torch.randint(0, 127, (4096, 15), generator=g).double() + 0.5
    x = torch.cat([m, (k * m.double() / 127).float()], 1)
    x[:, 8:] = torch.nextafter(x[:, 8:], torch.zeros(()))
    q, _ = mg.quant_rows(x.cuda())
    v = f64(x)
    assert np.array_equal(q.cpu().numpy(), np.rint(127 * v / np.abs(v).max(1)[:, None]))


def test_quant_rows_largest(mg):
    """Rows whose 127 / m is below fp32's normal numbers, or just above."""
    g = torch.Generator().manual_seed(9)
    m = torch.exp2(torch.rand(600, 1, generator=g, dtype=torch.float64) * 3 + 124.999).float()
    x = torch.cat([m, (torch.rand(600, 63, generator=g) * 2 - 1) * m], 1)
    k = torch.randint(0, 127, (600, 32), generator=g).double() + 0.5
    x[:, 32:] = (k * m.double() / 127).float()
    assert torch.isfinite(x).all()
    q, s = mg.quant_rows(x.cuda())
    v = f64(x)
    assert np.array_equal(q.cpu().numpy(), np.rint(127 * v / np.abs(v).max(1)[:, None]))
    assert np.array_equal(s.cpu().numpy(), np.abs(x.numpy()).max(1) / np.float32(127))


def test_quant_rows_far_values(mg):
    x = torch.zeros(8, 40)
    x[0, 3], x[0, 4] = 3.4028234e38, -1.7e38
    x[1, 0], x[1, 1] = 1e-45, -1e-45                     # subnormal: 127 / m overflows
    x[2, 5], x[2, 6] = 3e-37, 1e-38
    x[3, 7] = float("inf")
    x[4, 8] = float("nan")
    x[5, 9], x[5, 10] = float("-inf"), 1.0
    x[6, 39], x[6, 0] = -2.0, 1e-30
    q, s = mg.quant_rows(x.cuda())
    v = f64(x)[[0, 1, 2, 6]]
    want = np.rint(127 * v / np.abs(v).max(1)[:, None])
    assert np.array_equal(q.cpu().numpy()[[0, 1, 2, 6], :40], want)
    bad = [3, 4, 5]
    assert torch.isnan(s[bad]).all() and (q[bad] == 0).all()
    assert s[7] == 0 and (q[7] == 0).all()


def test_quant_weights(mg):
    w = torch.randn(3, 5, 40, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    q, s = mg.quant_rows(w)
    q2, s2 = mg.quant_rows(w.view(15, 40))
    assert q.shape == (3, 5, 48) and s.shape == (3, 5)
    assert torch.equal(q.view(15, 48), q2) and torch.equal(s.view(15), s2)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,cols", SIZES)
def test_pack_and_back(mg, rows, cols, dtype):
    x = values(rows, cols, dtype, rows + cols, extra=3)
    q, s = mg.pack8(x.cuda()[:, :cols])
    want_q, want_s = pack_ref(f64(x[:, :cols]))
    assert np.array_equal(q.cpu().numpy(), want_q)
    assert np.array_equal(s.cpu().numpy(), want_s)
    v = unpack_ref(want_q, s.cpu().numpy(), cols)
    for out in (torch.bfloat16, torch.float32):
        assert np.array_equal(f64(mg.unpack8(q, s, cols, out)), v)
    half = mg.unpack8(q, s, cols, torch.float16)
    assert np.array_equal(f64(half), f64(torch.from_numpy(v).clamp(-65504, 65504).half()))
    # half a step from what was packed
    step = np.exp2(s.cpu().numpy().astype(float) - 127).repeat(32, 1)[:, :cols]
    assert (np.abs(v - f64(x[:, :cols])) <= step / 2).all()


def test_unpack_into_wider_rows(mg):
    x = values(9, 70, "bf16", 5)
    q, s = mg.pack8(x.cuda())
    out = torch.full((9, 80), 7.0, dtype=torch.bfloat16, device="cuda")
    mg.unpack8(q, s, 70, X=out[:, 3:73])
    assert torch.equal(out[:, 3:73], mg.unpack8(q, s, 70))
    assert (out[:, :3] == 7).all() and (out[:, 73:] == 7).all()


def test_pack_far_values(mg):
    x = torch.zeros(7, 64)
    x[0, 1] = float("inf")                               # its block alone is lost
    x[0, 40] = 1.5
    x[1, 33] = float("nan")
    x[2, 0], x[2, 1] = 3.4028234e38, 1e30
    x[3, 0], x[3, 1] = 1e-45, -2.0 ** -126               # the smallest step is 2^-126
    x[4, 0], x[4, 1] = 2.0 ** -120, 2.0 ** -127
    x[5, 0], x[5, 1] = 65504.0, -3.0
    q, s = mg.pack8(x.cuda())
    want_q, want_s = pack_ref(f64(x))
    assert np.array_equal(q.cpu().numpy(), want_q)
    v = f64(mg.unpack8(q, s, 64, torch.float32))
    assert np.isnan(v[0, :32]).all() and v[0, 40] == 1.5
    assert np.isnan(v[1, 32:]).all() and (v[1, :32] == 0).all()
    ref = unpack_ref(want_q, s.cpu().numpy(), 64)
    assert np.array_equal(v, ref, equal_nan=True)
    assert v[2, 0] == 127 * 2.0 ** 121
    assert float(mg.unpack8(q, s, 64, torch.float16)[5, 0]) == 65504.0


def test_far_rows(mg):
    """Rows past 2^31 elements."""
    rows, cols = (1 << 31) // 4096 + 40, 4096
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    tail = values(40, cols, "bf16", 9)
    x[-40:] = tail.cuda()
    q, s = mg.pack8(x)
    want, _ = pack_ref(f64(tail))
    assert np.array_equal(q[-40:].cpu().numpy(), want)
    back = mg.unpack8(q, s, cols)
    assert np.array_equal(f64(back[-40:]), unpack_ref(want, s[-40:].cpu().numpy(), cols))
    q2, s2 = mg.quant_rows(x)
    q3, s3 = mg.quant_rows(tail.cuda())
    assert torch.equal(q2[-40:], q3) and torch.equal(s2[-40:], s3)
