"""Plain 64-bit evaluations of the feed-forward block's operators, and their error bounds.

Bounds count roundings: u = 2^-24 for fp32, half a step 2^-8 for bf16.  A sum of
n products in fp32, in any order, is off by at most 2 gamma(n) sum |terms| (a factor
2 over the recursive bound, as the other products' tests have it).

The sigmoid s(z) = 1 / (1 + e^-z) is computed with z off by 4 u |z| (its products),
the exponent's argument by another 2 u |z|, and v_exp_f32, the sum and v_rcp_f32 by
about 2 u each; d log s / d z <= 1, so s is off by (8 |z| + 8) u relative to itself.
SIG doubles that.  act(g) = g s adds one rounding.
"""

import numpy as np
import torch

from tests._util import gamma

U = 2.0 ** -24
HALF = 2.0 ** -8
BLOCK = 32


def routed(mg, T, k, E, seed, drop=True, block=128):
    """Ids (some slots dropped), the GPU's routing and per-slot expert order in numpy."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    if E > 3:
        ids[ids == 2] = 1                                # an expert without rows
    if drop and T > 4:
        ids[1] = -1                                      # a token without experts
        ids[3, 0] = -1
    r = mg.moe_route(ids.cuda(), E, block)
    flat = ids.reshape(-1).numpy()
    live = np.nonzero(flat >= 0)[0]
    order = live[np.argsort(flat[live], kind="stable")]  # slot at each sorted position
    return r, order, flat[order], g


def sigma(g, act):
    """z(g), s(z) and z'(g) in 64 bits."""
    if act == "silu":
        z, dz = g, np.ones_like(g)
    else:
        c = 2 * np.sqrt(2 / np.pi)
        z, dz = c * (g + 0.044715 * g ** 3), c * (1 + 3 * 0.044715 * g ** 2)
    return z, 1 / (1 + np.exp(-z)), dz


def sig_err(z):
    return (16 * np.abs(z) + 16) * U


def act_ref(g, act):
    """act(g), act'(g) and bounds of their errors in fp32 for an exact g."""
    z, s, dz = sigma(g, act)
    a = g * s
    t = s * (1 - s)
    d = s + g * t * dz
    # s (1 - s): s off by e s, 1 - s by e s + u; the product g t z' by 4 roundings more
    e = sig_err(z)
    ad = np.abs(g * dz) * (2 * e * s + U + 6 * U * t) + s * (e + 2 * U)
    return a, d, np.abs(a) * (e + 2 * U), ad


def split(a, halves):
    n = a.shape[1] // 2
    return (a[:, :n], a[:, n:]) if halves else (a[:, 0::2], a[:, 1::2])


def join(f, s, halves):
    return np.concatenate([f, s], 1) if halves else np.stack([f, s], -1).reshape(f.shape[0], -1)


def grouped(rows, experts, W, transposed):
    """(rows[p] times W[experts[p]], the same of absolute values) in 64 bits."""
    out = np.zeros((rows.shape[0], W.shape[1] if transposed else W.shape[2]))
    mag = np.zeros_like(out)
    for e in np.unique(experts):
        at = experts == e
        w = W[e].T if transposed else W[e]
        out[at] = rows[at] @ w
        mag[at] = np.abs(rows[at]) @ np.abs(w)
    return out, mag


def sum_err(mag, n):
    return 2 * gamma(n + 1) * mag


def gated_ref(g, u, eg, eu, act):
    """H = act(g) u and the bound of a bf16 H whose g and u are off by eg and eu."""
    a, d, ea, _ = act_ref(g, act)
    ea = ea + 1.2 * eg                                   # |act'| < 1.13
    h = a * u
    err = np.abs(u) * ea + np.abs(a) * eu + ea * eu
    return h, err + (np.abs(h) + err) * (HALF + 2 * U) + 1e-37


def pack_ref(x):
    """Codes and bytes of moegg_pack8 in 64 bits."""
    rows, cols = x.shape
    n = (cols + BLOCK - 1) // BLOCK
    b = np.zeros((rows, n * BLOCK))
    b[:, :cols] = x
    b = b.reshape(rows, n, BLOCK)
    finite = np.isfinite(b).all(2)
    b = np.where(finite[:, :, None], b, 0.0)
    top = np.abs(b).max(2)
    e = np.full(top.shape, -126, dtype=np.int64)
    nz = top > 0
    e[nz] = np.floor(np.log2(top[nz])).astype(np.int64) - 7
    for _ in range(3):
        e = np.where(np.rint(top * np.exp2(-e.astype(float))) > 127, e + 1, e)
    e = np.clip(e, -126, 121)
    q = np.clip(np.rint(b * np.exp2(-e.astype(float))[:, :, None]), -127, 127)
    s = np.where(finite, e + 127, 255)
    return q.reshape(rows, -1).astype(np.int8), s.astype(np.uint8)


def unpack_ref(q, s, cols):
    v = q.astype(np.float64).reshape(q.shape[0], -1, BLOCK)
    v = v * np.where(s == 255, np.nan, np.exp2(s.astype(np.float64) - 127))[:, :, None]
    return v.reshape(q.shape[0], -1)[:, :cols]


def f64(t):
    return t.detach().double().cpu().numpy()


def check(got, ref, tol, what=""):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.isfinite(got).all(), what
    over = np.abs(got - ref) - tol
    at = np.unravel_index(np.argmax(over), over.shape) if over.size else None
    assert over.size == 0 or over[at] <= 0, (what, at, got[at], ref[at], tol[at])
