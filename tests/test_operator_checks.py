"""Refusals of the gate, permute, unpermute and adapter entry points: every call here
fails on the host, before anything is enqueued."""

import ctypes
import math
import os

import pytest

EINVAL, ESHAPE = 1, 2
BF16, FP16, FP32 = 0, 1, 2
P = ctypes.c_void_p(1 << 20)             # never dereferenced
P2 = ctypes.c_void_p(1 << 21)
ODD = ctypes.c_void_p((1 << 20) + 1)
TWO = ctypes.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def lib():
    import token_routing_amd as mg
    if not os.path.exists(mg.LIB_PATH):
        from token_routing_amd import build
        build.build()
    return mg.load_library()


def gate(lib, logits=P, dtype=BF16, ld=64, bias=None, T=10, E=64, k=4, groups=1, top=1, scale=1.0,
         flags=0, ids=P, w=P, scores=None):
    return lib.moegg_gate(logits, dtype, ld, bias, T, E, k, groups, top, scale, flags, ids, w,
                          scores, None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), ESHAPE), (dict(E=0), ESHAPE), (dict(E=1025, ld=1025), ESHAPE),
    (dict(k=0), ESHAPE), (dict(k=65, E=128, ld=128), ESHAPE), (dict(E=3, k=4), ESHAPE),
    (dict(ld=63), ESHAPE), (dict(ld=1 << 50), ESHAPE), (dict(T=1 << 30), ESHAPE),
    (dict(T=1 << 26, k=1), ESHAPE),
    (dict(groups=0), ESHAPE), (dict(groups=5), ESHAPE), (dict(groups=65, E=130, ld=130), ESHAPE),
    (dict(groups=8, top=9), ESHAPE), (dict(groups=8, top=0), ESHAPE),
    (dict(groups=32, top=1), ESHAPE),          # two experts a group, four picks
    (dict(dtype=3), EINVAL), (dict(dtype=-1), EINVAL), (dict(flags=4), EINVAL),
    (dict(scale=math.nan), EINVAL), (dict(scale=math.inf), EINVAL),
    (dict(logits=None), EINVAL), (dict(logits=ODD), EINVAL), (dict(logits=TWO, dtype=FP32), EINVAL),
    (dict(ids=None), EINVAL), (dict(w=None), EINVAL), (dict(w=TWO), EINVAL),
    (dict(scores=TWO), EINVAL), (dict(bias=TWO), EINVAL),
])
def test_gate_refusals(lib, kw, want):
    assert gate(lib, **kw) == want


def test_gate_no_tokens(lib):
    assert gate(lib, T=0, logits=None, ids=None, w=None) == 0


def gate_bwd(lib, logits=P, dtype=BF16, ld=64, ids=P, dw=P, ds=None, T=10, E=64, k=4, scale=1.0,
             flags=0, out=P):
    return lib.moegg_gate_bwd(logits, dtype, ld, ids, dw, ds, T, E, k, scale, flags, out, None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), ESHAPE), (dict(k=65, E=128, ld=128), ESHAPE), (dict(ld=1), ESHAPE),
    (dict(dtype=7), EINVAL), (dict(flags=8), EINVAL), (dict(scale=-math.inf), EINVAL),
    (dict(ids=None), EINVAL), (dict(dw=None), EINVAL), (dict(out=None), EINVAL),
    (dict(out=ODD), EINVAL), (dict(ds=TWO), EINVAL), (dict(logits=None), EINVAL),
])
def test_gate_bwd_refusals(lib, kw, want):
    assert gate_bwd(lib, **kw) == want


def permute(lib, X=P, dtype=BF16, sc=P, w=None, off=None, pad=None, T=10, k=2, E=8, K=64, rows=20,
            Xs=P, row_map=P):
    return lib.moegg_permute(X, dtype, sc, w, off, pad, T, k, E, K, rows, Xs, row_map, None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), ESHAPE), (dict(k=0), ESHAPE), (dict(K=0), ESHAPE), (dict(rows=-1), ESHAPE),
    (dict(rows=1 << 31), ESHAPE), (dict(K=1 << 30, rows=1 << 20), ESHAPE),
    (dict(T=1 << 30, k=4), ESHAPE), (dict(dtype=3), EINVAL),
    (dict(off=P), EINVAL), (dict(pad=P), EINVAL),               # one of the two
    (dict(off=P, pad=P, row_map=None), EINVAL),
    (dict(off=P, pad=P, E=0), ESHAPE), (dict(off=P, pad=P, E=1025), ESHAPE),
    (dict(off=TWO, pad=P), EINVAL), (dict(T=0, off=P, pad=P, Xs=None), EINVAL),
    (dict(X=None), EINVAL), (dict(X=ODD), EINVAL), (dict(X=TWO, dtype=FP32), EINVAL),
    (dict(sc=None), EINVAL), (dict(Xs=None), EINVAL), (dict(w=TWO), EINVAL),
    (dict(row_map=TWO), EINVAL),
    (dict(off=P, pad=P, sc=P, row_map=P), EINVAL),              # the map over its own input
    (dict(T=1 << 24, k=1, K=1), ESHAPE),                        # more workgroups than a launch
])
def test_permute_refusals(lib, kw, want):
    assert permute(lib, **kw) == want


def test_backward_and_unpermute_refusals(lib):
    f = lib.moegg_permute_bwd
    assert f(P, BF16, P, P, None, -1, 2, 64, 20, P, P, None, None) == ESHAPE
    assert f(P, 9, P, P, None, 10, 2, 64, 20, P, P, None, None) == EINVAL
    assert f(P, BF16, None, P, None, 10, 2, 64, 20, P, P, None, None) == EINVAL   # dw reads X
    assert f(None, BF16, P, P, None, 10, 2, 64, 20, P, P, None, None) == EINVAL
    assert f(P, BF16, P, P, None, 10, 2, 64, 20, None, P, None, None) == EINVAL
    assert f(P, FP32, P, P, None, 10, 2, 64, 20, TWO, P, None, None) == EINVAL
    assert f(None, BF16, None, None, None, 0, 2, 64, 0, None, None, None, None) == 0
    f = lib.moegg_unpermute
    assert f(P, BF16, P, None, None, 10, 0, 64, 20, P, None, None) == ESHAPE
    assert f(P, BF16, P, None, ODD, 10, 2, 64, 20, P, None, None) == EINVAL
    assert f(P, BF16, None, None, None, 10, 2, 64, 20, P, None, None) == EINVAL
    assert f(None, BF16, None, None, None, 0, 2, 64, 0, None, None, None) == 0
    f = lib.moegg_unpermute_bwd
    assert f(P, BF16, P, P, None, P, None, 10, 2, 8, 64, 20, P, P, None, None) == EINVAL
    assert f(P, BF16, None, P, None, None, None, 10, 2, 8, 64, 20, P, P, None, None) == EINVAL
    assert f(P, BF16, P, P, None, P, P, 10, 2, 2000, 64, 20, P, P, None, None) == ESHAPE
    assert f(P, BF16, P, P, None, None, None, 10, 2, 8, 64, 20, None, P, None, None) == EINVAL


def test_python_argument_checks():
    import torch
    import token_routing_amd as mg
    cpu = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        mg.moe_gate(cpu, 2)
    with pytest.raises(ValueError):
        mg.permute(cpu, torch.zeros(8, dtype=torch.int32), 2)
    with pytest.raises(ValueError):
        mg._dtype_code(torch.zeros(2, dtype=torch.float64), "x")
    with pytest.raises(ValueError):
        mg.lora_fwd(cpu, torch.zeros(1, 2, 8), torch.zeros(1, 3, 2),
                    torch.zeros(1, dtype=torch.int32), base=torch.zeros(4, 3))
    # checks of layout, on tensors that need no GPU (index -1 is the CPU)
    assert mg._rows_arg(torch.zeros(4, 9)[:, 2:5], "x", torch.float32, (4, 3), -1)[1] == 9
    assert mg._rows_arg(torch.zeros(4, 9)[2:3, 2:5], "x", torch.float32, (1, 3), -1)[1] >= 3
    for t in (torch.zeros(3, 4).t(), torch.zeros(1, 3).expand(4, 3), torch.zeros(4, 6)[:, ::2]):
        with pytest.raises(ValueError):
            mg._rows_arg(t, "x", torch.float32, (4, 3), -1)
    with pytest.raises(ValueError):
        mg._slots_arg(torch.zeros(4, 4).t(), "w", torch.float32, 16, -1)
    with pytest.raises(ValueError):
        mg._arg(torch.zeros(4, 4), "w", torch.float32, (4, 5), -1)


def lora(lib, X=P, ldx=64, A=P, B=P, m=P, gather=P, ranks=None, scales=None, dtype=BF16, T=10, L=4,
         R=16, K=64, N=96, base=P, ldb=96, Y=P, ldy=96, H=None, ws=P, size=1 << 20):
    return lib.moegg_lora_fwd(X, ldx, A, B, m, gather, ranks, scales, dtype, T, L, R, K, N, base,
                              ldb, Y, ldy, H, ws, size, None, None)


EUNSUP, EWS = 3, 4


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), ESHAPE), (dict(T=1 << 31), ESHAPE), (dict(L=0), ESHAPE), (dict(L=1025), ESHAPE),
    (dict(R=0), ESHAPE), (dict(R=257), ESHAPE), (dict(K=7), ESHAPE), (dict(N=7), ESHAPE),
    (dict(ldx=63), ESHAPE), (dict(ldy=95), ESHAPE), (dict(ldb=95, Y=ODD), ESHAPE),
    (dict(ldx=1 << 40), ESHAPE), (dict(T=1, ldx=1 << 31), ESHAPE),
    (dict(T=1 << 28), ESHAPE), (dict(L=1024, R=256, K=1 << 30, ldx=1 << 30), ESHAPE),
    (dict(T=(1 << 31) - 1, N=1 << 20, ldy=1 << 20, ldb=1 << 20), ESHAPE),
    (dict(dtype=FP32), EUNSUP), (dict(dtype=5), EINVAL),
    (dict(X=None), EINVAL), (dict(A=None), EINVAL), (dict(B=None), EINVAL), (dict(m=None), EINVAL),
    (dict(Y=None), EINVAL), (dict(X=ODD), EINVAL), (dict(A=ODD), EINVAL), (dict(B=ODD), EINVAL),
    (dict(Y=ODD), EINVAL), (dict(base=ODD), EINVAL), (dict(m=TWO), EINVAL),
    (dict(gather=TWO), EINVAL), (dict(ranks=TWO), EINVAL), (dict(scales=TWO), EINVAL),
    (dict(H=TWO), EINVAL), (dict(ldb=100), EINVAL),             # base is Y, other strides
    (dict(ws=None), EWS), (dict(size=10), EWS), (dict(ws=TWO), EWS),
])
def test_lora_refusals(lib, kw, want):
    assert lora(lib, **kw) == want


def test_lora_no_rows(lib):
    assert lora(lib, T=0, X=None, Y=None, base=None, ws=None, size=0) == 0


def lora_bwd(lib, X=P, ldx=64, dY=P, lddy=96, A=P, B=P, H=P, m=P, gather=P, ranks=None, scales=None,
             dtype=BF16, T=10, L=4, R=16, K=64, N=96, base=P2, ldb=64, dX=P2, lddx=64, dA=P, dB=P,
             flags=0, ws=P, size=1 << 20):
    return lib.moegg_lora_bwd(X, ldx, dY, lddy, A, B, H, m, gather, ranks, scales, dtype, T, L, R,
                              K, N, base, ldb, dX, lddx, dA, dB, flags, ws, size, None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), ESHAPE), (dict(L=0), ESHAPE), (dict(R=300), ESHAPE), (dict(lddy=95), ESHAPE),
    (dict(ldx=63), ESHAPE), (dict(lddx=63), ESHAPE), (dict(ldb=63, dX=TWO), ESHAPE),
    (dict(dtype=FP32), EUNSUP), (dict(dtype=-1), EINVAL), (dict(flags=2), EINVAL),
    (dict(dA=None), EINVAL), (dict(dB=None), EINVAL), (dict(X=None), EINVAL), (dict(H=None), EINVAL),
    (dict(dY=None), EINVAL), (dict(A=None), EINVAL), (dict(B=None), EINVAL), (dict(m=None), EINVAL),
    (dict(dX=ODD, base=None), EINVAL), (dict(base=ODD), EINVAL), (dict(dA=ODD), EINVAL),
    (dict(dB=TWO, flags=1), EINVAL), (dict(H=TWO), EINVAL), (dict(ldb=80), EINVAL),
    (dict(ws=None), EWS), (dict(size=100), EWS), (dict(X=P, dX=P, base=TWO), EINVAL),
])
def test_lora_bwd_refusals(lib, kw, want):
    assert lora_bwd(lib, **kw) == want


def test_lora_workspace_sizes(lib):
    f, b = lib.moegg_lora_workspace_bytes, lib.moegg_lora_bwd_workspace_bytes

    def area(n):                             # n fp32 and a piece of 8 behind them
        return (n * 4 + 32 + 255) // 256 * 256

    # 64 rows over 32 adapters: 36 tiles of 16 rows, 8 workgroups a tile
    assert f(64, 32, 16, 4096, 4096) == area(8 * 64 * 16)
    # 72 tiles of 32 rows: four workgroups a tile; 264 of them: one each
    assert f(2048, 8, 64, 4096, 4096) == area(4 * 2048 * 64)
    assert f(8192, 8, 64, 4096, 4096) == area(8192 * 64)
    assert f(0, 4, 16, 64, 64) == 0 and b(0, 4, 16, 64, 64) == 0
    assert f(-1, 4, 16, 64, 64) == 0 and b(10, 4, 300, 64, 64) == 0 and f(10, 4, 16, 7, 64) == 0
    # dh alone up to one chunk of rows, then at most 2 T / chunk partial sums
    assert b(128, 1, 16, 64, 96) == area(128 * 16)
    chunk = 4096 * 64 // 384 // 32 * 32 + 32
    assert b(4096, 4, 32, 4096, 4096) == (area(2 * 4096 * 32) + 4096 * 32 * 4
                                          + 2 * 4096 // chunk * 32 * 8192 * 4)
    # a size just below what is needed
    need = f(64, 32, 16, 4096, 4096)
    assert lora(lib, T=64, L=32, K=4096, N=4096, ldx=4096, ldy=4096, ldb=4096,
                size=need - 1) == EWS
