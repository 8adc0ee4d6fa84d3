"""Calls of the feed-forward block in which workgroups take tile after tile, each of
several reduction stages: the cases, which kernel each takes, and 64-bit references
and bounds (those of tests/_block.py) on the GPU.

A case's `sizes` are the experts' rows, `rows` those of its tensors (at least their
sum), `depth` the reduction, `cols` the outputs' columns (of one part where gated).
"""

import ctypes
import os
import subprocess

import torch

from tests._block import BLOCK, HALF, U
from tests._util import gamma

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SMALL, MIDDLE, DEEP, LARGE, VECTORS = range(5)
TILE = {SMALL: 32, MIDDLE: 128, DEEP: 128, LARGE: 256}
STAGE = 128                                              # bytes of a row in one stage


def many(n, lo, hi, step):
    """n experts of lo .. hi rows, one of them without rows."""
    return [0 if i == 7 else lo + i * step % (hi - lo + 1) for i in range(n)]


def fwd(shape, sizes, depth, cols, keep, act="silu", halves=False, px=True, topk=1):
    return dict(op="fwd", shape=shape, sizes=sizes, depth=depth, cols=cols, keep=keep, act=act,
                halves=halves, px=px, topk=topk)


def i8(shape, sizes, depth, cols, form, act=None, halves=False, topk=1):
    return dict(op="i8", shape=shape, sizes=sizes, depth=depth, cols=cols, form=form, act=act,
                halves=halves, topk=topk)


def bwd(shape, sizes, depth, cols, kept, act="silu", halves=False, py=False, topk=1):
    return dict(op="bwd", shape=shape, sizes=sizes, depth=depth, cols=cols, kept=kept, act=act,
                halves=halves, py=py, topk=topk)


CASES = [
    # large tiles: two stages in the ring; 3, 4, 5 and 6 of them, whole and ragged
    fwd(LARGE, [2300], 200, 9000, "bf16", halves=True),
    fwd(LARGE, [700, 0, 1603], 136, 9000, "packed", act="gelu", topk=3),
    fwd(LARGE, [2300], 264, 8997, None, act="gelu", halves=True),
    fwd(LARGE, [1100, 1203], 192, 9003, "packed"),
    fwd(LARGE, [1100, 1203], 328, 9005, "bf16", px=False),
    i8(LARGE, [2300], 400, 9000, "gated", "silu", True),
    i8(LARGE, [700, 0, 1603], 272, 18001, "scattered", topk=3),
    i8(LARGE, [2300], 528, 18000, "plain"),
    i8(LARGE, [1100, 1203], 640, 9001, "gated", "gelu"),
    bwd(LARGE, [2300], 200, 18000, "bf16", halves=True, py=True),
    bwd(LARGE, [700, 0, 1603], 136, 18000, "packed", act="gelu", topk=3),
    bwd(LARGE, [2300], 264, 17997, "place", act="gelu"),
    bwd(LARGE, [1100, 1203], 328, 18001, "packed", halves=True, py=True),
    # middle tiles: two workgroups a compute unit
    fwd(MIDDLE, many(60, 100, 150, 7), 136, 1224, "bf16", act="gelu", topk=2),
    fwd(MIDDLE, many(60, 100, 150, 7), 200, 1221, "packed", halves=True),
    fwd(MIDDLE, many(60, 100, 150, 7), 328, 1224, None),
    i8(MIDDLE, many(60, 100, 150, 7), 400, 1222, "gated", "gelu", True),
    i8(MIDDLE, many(60, 100, 150, 7), 272, 2440, "scattered", topk=2),
    bwd(MIDDLE, many(60, 100, 150, 7), 136, 2440, "packed", py=True),
    bwd(MIDDLE, many(60, 100, 150, 7), 200, 2440, "packed", act="gelu", halves=True),
    # four stages in the ring: the backward's other forms of these calls, and calls with
    # more tiles than the rule expects of them
    bwd(DEEP, many(60, 100, 150, 7), 328, 2440, "bf16", act="gelu", halves=True),
    bwd(DEEP, many(60, 100, 150, 7), 392, 2437, "place"),
    bwd(DEEP, many(60, 100, 150, 7), 328, 2437, "packed", act="gelu", topk=2),
    fwd(DEEP, [129, 129, 129], 456, 4096, "packed"),
    fwd(DEEP, [129, 129, 129], 584, 4093, "bf16", act="gelu", halves=True),
    i8(DEEP, [129, 129, 129], 912, 4096, "gated", "silu"),
    i8(DEEP, [129, 129, 129], 784, 8188, "plain"),
    bwd(DEEP, [129, 129, 129], 456, 8192, "packed", py=True),
    bwd(DEEP, [129, 129, 129], 584, 8189, "place", act="gelu", halves=True),
    fwd(SMALL, [33, 33, 33], 392, 6144, "bf16"),
    fwd(SMALL, [33, 33, 33], 584, 6141, "packed", act="gelu", halves=True),
    i8(SMALL, [33, 33, 33], 784, 6144, "gated", "silu", True),
    i8(SMALL, [33, 33, 33], 912, 6141, "scattered"),
    bwd(SMALL, [33, 33, 33], 392, 7296, "packed", act="gelu", halves=True),
    bwd(SMALL, [33, 33, 33], 584, 7293, "bf16", py=True),
    # the vectors of a few rows
    i8(VECTORS, [1, 0, 1, 1, 0, 0, 0, 1], 2304, 12001, "plain", topk=2),
    i8(VECTORS, [16] + [0] * 8, 2064, 7000, "gated", "silu"),
    fwd(VECTORS, [3, 0, 1, 2, 5, 0, 0, 1], 1032, 5000, None, act="gelu", topk=2),
]


def name(c):
    form = c.get("form") or c.get("keep") or c.get("kept") or "none"
    shape = ["small", "middle", "deep", "large", "vectors"][c["shape"]]
    return f"{c['op']}-{shape}-{c['depth']}-{c['cols']}-{form}"


def rows_of(c):
    """Rows of the tensors: some behind the last expert's."""
    n, k = sum(c["sizes"]) + 2, c["topk"]
    return (n + k - 1) // k * k


def gated(c):
    return c["op"] == "fwd" or c.get("form") == "gated"


def out_cols(c):
    """Columns of the product's tiles: rows of W."""
    return c["cols"] * 2 if gated(c) else c["cols"]


def stages(c):
    """Reduction stages of a tile."""
    return -(-c["depth"] * (1 if c["op"] == "i8" else 2) // STAGE)


def tiles(c):
    bm = TILE[c["shape"]]
    bn = bm if bm > 32 else 256 if gated(c) else 128
    return sum(-(-m // bm) for m in c["sizes"]) * -(-out_cols(c) // bn)


def vector_groups(c):
    """Work items of the vector kernel: 4 rows by 16 columns (8 where gated)."""
    cols = 8 if gated(c) else 16
    return sum(-(-m // 4) for m in c["sizes"]) * -(-c["cols"] // cols)


def load_rules(folder):
    """The library's own rules (csrc/block_shape.h), compiled for the host."""
    src, lib = os.path.join(folder, "rules.cpp"), os.path.join(folder, "rules.so")
    with open(src, "w") as f:
        f.write('#include "block_shape.h"\n'
                'extern "C" int shape(int64_t S, int E, int cols, int small, double most, int cus)\n'
                '{ return moegg::tile_shape(S, E, cols, small, most, cus); }\n'
                'extern "C" int bwd_shape(int64_t S, int E, int cols, int two, int cus)\n'
                '{ return moegg::bwd_shape(S, E, cols, 128, 0.9, two, cus); }\n'
                'extern "C" int vec(int64_t S, int E, int cols, int gated, int64_t row, int cus)\n'
                '{ return moegg::vec_pays(S, E, cols, gated, row, cus); }\n')
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I",
                           os.path.join(ROOT, "token_routing_amd", "csrc"), src, "-o", lib])
    rules = ctypes.CDLL(lib)
    i64, i32 = ctypes.c_int64, ctypes.c_int
    rules.shape.argtypes = [i64, i32, i32, i32, ctypes.c_double, i32]
    rules.bwd_shape.argtypes = [i64, i32, i32, i32, i32]
    rules.vec.argtypes = [i64, i32, i32, i32, i64, i32]
    return rules


def shape_taken(rules, c, cus):
    S, E, cols = rows_of(c), len(c["sizes"]), out_cols(c)
    serving = c["op"] == "i8" or (c["op"] == "fwd" and c["keep"] is None)
    row = -(-c["depth"] // 8) * 16 if c["op"] != "i8" else c["depth"]
    if serving and rules.vec(S, E, cols, gated(c), row, cus):
        return VECTORS
    if c["op"] == "bwd":
        return rules.bwd_shape(S, E, cols, c["kept"] == "packed" and cols % 8 == 0, cus)
    return rules.shape(S, E, cols, 256 if gated(c) else 128, 0.75, cus)


# ---------------------------------------------------------------- references on the GPU

def grouped(c, x, w, transposed):
    """x[p] times its expert's w and the same of magnitudes, in 64 bits."""
    n = sum(c["sizes"])
    cols = w.shape[1] if transposed else w.shape[2]
    out = torch.zeros(n, cols, dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(out)
    p = 0
    for e, m in enumerate(c["sizes"]):
        if m:
            we = w[e].double()
            we = we.t().contiguous() if transposed else we
            xe = x[p:p + m].double()
            out[p:p + m] = xe @ we
            mag[p:p + m] = xe.abs() @ we.abs()
        p += m
    return out, mag


def sum_err(mag, n):
    return 2 * gamma(n + 1) * mag


def act_ref(g, act):
    """act(g), act'(g) and the bounds of their errors in fp32 (tests/_block.py)."""
    if act == "silu":
        z, dz = g, torch.ones_like(g)
    else:
        k = 2 * (2 / torch.pi) ** 0.5
        z, dz = k * (g + 0.044715 * g ** 3), k * (1 + 3 * 0.044715 * g ** 2)
    s = torch.sigmoid(z)
    a, t = g * s, s * (1 - s)
    d = s + g * t * dz
    e = (16 * z.abs() + 16) * U
    ad = (g * dz).abs() * (2 * e * s + U + 6 * U * t) + s * (e + 2 * U)
    return a, d, a.abs() * (e + 2 * U), ad


def gated_ref(g, u, eg, eu, act):
    a, _, ea, _ = act_ref(g, act)
    ea = ea + 1.2 * eg                                   # |act'| < 1.13
    h = a * u
    err = u.abs() * ea + a.abs() * eu + ea * eu
    return h, err + (h.abs() + err) * (HALF + 2 * U) + 1e-37


def bwd_ref(g, u, dh, eh, act):
    """dg, du and H with their bounds, for exact kept values."""
    a, d, ea, ed = act_ref(g, act)
    dg, du, h = dh * u * d, dh * a, a * u
    eg = u.abs() * (eh * (d.abs() + ed) + dh.abs() * ed)
    eu = eh * (a.abs() + ea) + dh.abs() * ea
    return [(v, e + (v.abs() + e) * (HALF + 4 * U) + 1e-37)
            for v, e in ((dg, eg), (du, eu), (h, u.abs() * ea))]


def split(a, halves):
    n = a.shape[1] // 2
    return (a[:, :n], a[:, n:]) if halves else (a[:, 0::2], a[:, 1::2])


def join(f, s, halves):
    return torch.cat([f, s], 1) if halves else torch.stack([f, s], -1).flatten(1)


def unpack_ref(q, s, cols):
    step = torch.exp2(s.double() - 127).repeat_interleave(BLOCK, 1)
    return (q.double() * step)[:, :cols], step[:, :cols]


def check(got, ref, tol, what=""):
    got = got.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.isfinite(got).all(), what
    over = (got - ref).abs() - tol
    at = int(over.argmax())
    assert float(over.flatten()[at]) <= 0, (what, divmod(at, got.shape[1]), float(got.flatten()[at]),
                                            float(ref.flatten()[at]), float(tol.flatten()[at]))
