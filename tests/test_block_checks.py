"""Refusals of the feed-forward block's entry points: every call here fails on the host,
before anything is enqueued."""

import ctypes
import os

import pytest
import torch

EINVAL, ESHAPE, EUNSUPPORTED, EWORKSPACE = 1, 2, 3, 4
BF16, FP16, FP32 = 0, 1, 2
PX, PY, MUL, SILU, GELU, HALVES = 1, 2, 4, 32, 64, 128


def at(n, off=0):
    """Address of a far apart, never dereferenced operand."""
    return ctypes.c_void_p((n << 40) + off)


@pytest.fixture(scope="module")
def lib():
    import token_routing_amd as mg
    if not os.path.exists(mg.LIB_PATH):
        from token_routing_amd import build
        build.build()
    return mg.load_library()


def quant(lib, X=at(1), dtype=BF16, ld=64, rows=10, K=64, Q=at(2), s=at(3)):
    return lib.moegg_quant_rows(X, dtype, ld, rows, K, Q, s, None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), ESHAPE), (dict(rows=1 << 24), ESHAPE), (dict(K=0), ESHAPE),
    (dict(ld=63), ESHAPE), (dict(ld=1 << 50), ESHAPE), (dict(dtype=3), EINVAL),
    (dict(dtype=-1), EINVAL), (dict(X=None), EINVAL), (dict(X=at(1, 1)), EINVAL),
    (dict(X=at(1, 2), dtype=FP32), EINVAL), (dict(Q=None), EINVAL), (dict(Q=at(2, 8)), EINVAL),
    (dict(s=None), EINVAL), (dict(s=at(3, 2)), EINVAL), (dict(Q=at(1)), EINVAL),
    (dict(s=at(2, 16)), EINVAL), (dict(s=at(1, 4)), EINVAL), (dict(K=2**31 - 1, ld=2**31), ESHAPE),
])
def test_quant_refusals(lib, kw, want):
    assert quant(lib, **kw) == want


def pack(lib, X=at(1), dtype=BF16, ld=64, rows=10, cols=64, Q=at(2), s=at(3)):
    return lib.moegg_pack8(X, dtype, ld, rows, cols, Q, s, None)


def unpack(lib, X=at(1), dtype=BF16, ld=64, rows=10, cols=64, Q=at(2), s=at(3)):
    return lib.moegg_unpack8(Q, s, rows, cols, X, dtype, ld, None)


@pytest.mark.parametrize("call", [pack, unpack])
@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), ESHAPE), (dict(rows=1 << 31), ESHAPE), (dict(cols=0), ESHAPE),
    (dict(ld=63), ESHAPE), (dict(ld=1 << 50), ESHAPE), (dict(dtype=3), EINVAL),
    (dict(X=None), EINVAL), (dict(X=at(1, 1)), EINVAL), (dict(Q=None), EINVAL),
    (dict(Q=at(2, 8)), EINVAL), (dict(s=None), EINVAL), (dict(Q=at(1)), EINVAL),
    (dict(s=at(1, 100)), EINVAL), (dict(cols=2**31 - 1, ld=2**31, rows=1), ESHAPE),
])
def test_pack_refusals(lib, call, kw, want):
    assert call(lib, **kw) == want


def test_nothing_to_do(lib):
    assert quant(lib, rows=0, X=None, Q=None, s=None) == 0
    assert pack(lib, rows=0, X=None, Q=None, s=None) == 0
    assert unpack(lib, rows=0, X=None, Q=None, s=None) == 0
    assert i8(lib, T=0, X=None, W=None, m=None, Y=None, ga=None) == 0
    assert fwd(lib, T=0, X=None, W=None, m=None, H=None, ga=None) == 0
    assert bwd(lib, T=0, dY=None, W=None, m=None, dA=None, ga=None, A=None) == 0


def i8(lib, X=at(1), xs=at(2), W=at(3), ws=at(4), m=at(5), ga=at(6), w=None, T=10, k=2, E=4, N=64,
       K=32, flags=PX, Y=at(7)):
    return lib.moegg_grouped_gemm_i8(X, xs, W, ws, m, ga, w, T, k, E, N, K, flags, Y, None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), ESHAPE), (dict(k=0), ESHAPE), (dict(E=0), ESHAPE), (dict(E=1025), ESHAPE),
    (dict(N=0), ESHAPE), (dict(K=0), ESHAPE), (dict(K=24), ESHAPE), (dict(K=131072), ESHAPE),
    (dict(T=1 << 30, k=4), ESHAPE), (dict(T=1 << 27, K=16), ESHAPE), (dict(N=1 << 27, K=16), ESHAPE),
    (dict(flags=8), EINVAL), (dict(flags=16), EINVAL), (dict(flags=PX | PY), EINVAL),
    (dict(flags=MUL), EINVAL), (dict(flags=PX | MUL), EINVAL), (dict(flags=PY | MUL), EINVAL),
    (dict(flags=PX | SILU | GELU), EINVAL), (dict(flags=PX | HALVES), EINVAL),
    (dict(flags=PY | SILU), EINVAL), (dict(flags=PY | MUL | GELU, w=at(8)), EINVAL),
    (dict(flags=PX | SILU, N=63), ESHAPE), (dict(ga=None), EINVAL), (dict(X=None), EINVAL),
    (dict(xs=None), EINVAL), (dict(xs=at(2, 2)), EINVAL), (dict(W=None), EINVAL),
    (dict(ws=None), EINVAL), (dict(m=None), EINVAL), (dict(Y=None), EINVAL),
    (dict(X=at(1, 8)), ESHAPE), (dict(W=at(3, 8)), ESHAPE), (dict(Y=at(7, 1)), ESHAPE),
    (dict(Y=at(1)), EINVAL), (dict(Y=at(3, 64)), EINVAL), (dict(Y=at(4)), EINVAL),
])
def test_i8_refusals(lib, kw, want):
    assert i8(lib, **kw) == want


def fwd(lib, X=at(1), W=at(2), m=at(3), ga=at(4), T=10, k=2, E=4, I=32, K=64, flags=PX | SILU,
        H=at(5), A=None, Aq=None, As=None, ws=None, n=0):
    return lib.moegg_gated_fwd(X, W, m, ga, T, k, E, I, K, flags, H, A, Aq, As, ws, n, None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), ESHAPE), (dict(k=0), ESHAPE), (dict(E=1025), ESHAPE), (dict(I=0), ESHAPE),
    (dict(I=1 << 30), ESHAPE), (dict(I=-5), ESHAPE), (dict(K=0), ESHAPE),
    (dict(T=1 << 30, k=4), ESHAPE), (dict(T=1 << 25), ESHAPE), (dict(I=1 << 24), ESHAPE),
    (dict(flags=PX), EINVAL), (dict(flags=PX | HALVES), EINVAL), (dict(flags=PX | SILU | GELU), EINVAL),
    (dict(flags=PY | SILU), EINVAL), (dict(flags=PX | SILU | MUL), EINVAL),
    (dict(flags=PX | SILU | 8), EINVAL), (dict(ga=None), EINVAL), (dict(X=None), EINVAL),
    (dict(W=None), EINVAL), (dict(m=None), EINVAL), (dict(H=None), EINVAL),
    (dict(X=at(1, 1)), EINVAL), (dict(H=at(5, 1)), EINVAL), (dict(A=at(6, 1)), EINVAL),
    (dict(Aq=at(6)), EINVAL), (dict(As=at(6)), EINVAL), (dict(A=at(8), Aq=at(6), As=at(7)), EINVAL),
    (dict(Aq=at(6, 8), As=at(7)), EINVAL),
    (dict(K=63), EWORKSPACE), (dict(K=63, ws=at(8), n=100), EWORKSPACE),
    (dict(X=at(1, 2)), EWORKSPACE), (dict(W=at(2, 4)), EWORKSPACE),
    (dict(K=63, ws=at(8, 8), n=1 << 30), EINVAL),
    (dict(H=at(1)), EINVAL), (dict(A=at(5)), EINVAL), (dict(A=at(2)), EINVAL),
    (dict(Aq=at(6), As=at(6, 10)), EINVAL), (dict(K=63, ws=at(5), n=1 << 30), EINVAL),
])
def test_gated_fwd_refusals(lib, kw, want):
    assert fwd(lib, **kw) == want


def bwd(lib, dY=at(1), W=at(2), m=at(3), ga=at(4), A=at(5), Aq=None, As=None, T=10, k=2, E=4, N=64,
        I=32, flags=SILU, dA=at(6), H=at(7), ws=None, n=0):
    return lib.moegg_gated_bwd(dY, W, m, ga, A, Aq, As, T, k, E, N, I, flags, dA, H, ws, n, None,
                               None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), ESHAPE), (dict(E=0), ESHAPE), (dict(N=0), ESHAPE), (dict(I=0), ESHAPE),
    (dict(T=1 << 24), ESHAPE), (dict(N=1 << 25, I=64), ESHAPE),
    (dict(flags=0), EINVAL), (dict(flags=SILU | GELU), EINVAL), (dict(flags=PX | SILU), EINVAL),
    (dict(flags=SILU | MUL), EINVAL), (dict(flags=PY | SILU, ga=None), EINVAL),
    (dict(A=None), EINVAL), (dict(Aq=at(8)), EINVAL), (dict(Aq=at(8), As=at(9)), EINVAL),
    (dict(A=None, Aq=at(8)), EINVAL), (dict(A=None, Aq=at(8, 2), As=at(9)), EINVAL),
    (dict(dY=None), EINVAL), (dict(W=None), EINVAL), (dict(m=None), EINVAL), (dict(dA=None), EINVAL),
    (dict(dY=at(1, 1)), EINVAL), (dict(dA=at(6, 1)), EINVAL), (dict(H=at(7, 1)), EINVAL),
    (dict(N=63), EWORKSPACE), (dict(I=31), EWORKSPACE), (dict(dY=at(1, 2)), EWORKSPACE),
    (dict(N=63, ws=at(10), n=64), EWORKSPACE), (dict(N=63, ws=at(10, 4), n=1 << 30), EINVAL),
    (dict(dA=at(1)), EINVAL), (dict(dA=at(2)), EINVAL), (dict(dA=at(5, 2)), EINVAL),
    (dict(H=at(5)), EINVAL), (dict(H=at(6)), EINVAL), (dict(H=at(1, 2)), EINVAL),
    (dict(A=None, Aq=at(8), As=at(9), dA=at(8)), EINVAL),
    (dict(N=63, ws=at(6), n=1 << 30), EINVAL),
])
def test_gated_bwd_refusals(lib, kw, want):
    assert bwd(lib, **kw) == want


def dw(lib, X=at(1), xs=at(2), dY=at(3), m=at(4), ga=at(5), T=10, k=2, E=4, N=64, K=32, flags=PX,
       out=at(6), ws=at(7), n=1 << 30):
    return lib.moegg_grouped_gemm_dW_packed(X, xs, dY, m, ga, T, k, E, N, K, flags, out, ws, n, None,
                                            None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), ESHAPE), (dict(E=0), ESHAPE), (dict(K=0), ESHAPE), (dict(T=1 << 26), ESHAPE),
    (dict(flags=MUL), EUNSUPPORTED), (dict(flags=16), EINVAL), (dict(flags=PX | PY), EINVAL),
    (dict(ga=None), EINVAL), (dict(out=None), EINVAL), (dict(m=None), EINVAL),
    (dict(out=at(6, 1)), EINVAL), (dict(out=at(6, 2), flags=PX | 8), EINVAL),
    (dict(X=None), EINVAL), (dict(xs=None), EINVAL), (dict(dY=None), EINVAL),
    (dict(X=at(1, 8)), EINVAL), (dict(dY=at(3, 1)), EINVAL), (dict(ws=at(7, 8)), EINVAL),
    (dict(ws=None, n=0), EWORKSPACE), (dict(n=100), EWORKSPACE),
    (dict(out=at(1)), EINVAL), (dict(out=at(3)), EINVAL), (dict(ws=at(3)), EINVAL),
    (dict(ws=at(6)), EINVAL),
])
def test_dw_packed_refusals(lib, kw, want):
    assert dw(lib, **kw) == want


def test_workspace_sizes(lib):
    f = lib.moegg_gated_fwd_workspace_bytes
    assert f(-1, 2, 4, 32, 64, PX) == 0 and f(10, 2, 4, 0, 64, PX) == 0
    assert f(10, 2, 4, 1 << 30, 64, PX) == 0
    assert f(10, 2, 4, 3, 63, PX) == 10 * 128 + 4 * 6 * 128
    assert f(10, 2, 4, 3, 63, 0) == 20 * 128 + 4 * 6 * 128
    b = lib.moegg_gated_bwd_workspace_bytes
    assert b(10, 2, 0, 32, 64) == 0
    assert b(10, 2, 4, 63, 7) == 20 * 128 + 4 * 63 * 16
    d = lib.moegg_grouped_gemm_dW_packed_workspace_bytes
    assert d(10, 2, 4, 0, 64, 0) == 0
    assert d(10, 2, 4, 64, 32, PX) == 10 * 32 * 2            # token order
    assert d(10, 2, 4, 64, 32, 0) == d(10, 2, 4, 64, 32, PY) == 20 * 32 * 2
    assert d(10, 2, 4, 4096, 32, PX) == 20 * 32 * 2          # expert order
    assert d(10, 2, 4, 63, 31, PX) == 20 * 31 * 2


def test_binding_refuses():
    """Types, shapes and devices, before the library is asked."""
    import token_routing_amd as mg
    cpu = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mg.quant_rows(cpu)
    with pytest.raises(ValueError):
        mg.quant_rows(cpu.to(torch.int32))
    with pytest.raises(ValueError):
        mg.pack8(cpu)
    with pytest.raises(ValueError):
        mg.unpack8(torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4, 1, dtype=torch.uint8), 8)
    with pytest.raises(ValueError):
        mg.gated_fwd(cpu, torch.zeros(1, 3, 8, dtype=torch.bfloat16), None, None, 1, 32)
    with pytest.raises(ValueError):
        mg.gated_fwd(cpu, torch.zeros(1, 4, 8, dtype=torch.bfloat16), None, None, 1, 32, keep="int8")


@pytest.mark.parametrize("call,kw,want", [
    (quant, dict(K=(1 << 30) + 1, ld=1 << 31), ESHAPE),
    (pack, dict(cols=(1 << 30) + 1, ld=1 << 31), ESHAPE),
    (unpack, dict(cols=(1 << 30) + 1, ld=1 << 31), ESHAPE),
    (i8, dict(Y=at(5)), EINVAL), (i8, dict(Y=at(6)), EINVAL),
    (i8, dict(Y=at(8), flags=PY | MUL, w=at(8)), EINVAL),
    (fwd, dict(H=at(3)), EINVAL), (fwd, dict(A=at(4)), EINVAL),
    (fwd, dict(Aq=at(4, 16), As=at(7)), EINVAL),
    (bwd, dict(dA=at(3)), EINVAL), (bwd, dict(H=at(4), flags=PY | SILU), EINVAL),
    (bwd, dict(N=63, ws=at(4), n=1 << 30, flags=PY | SILU), EINVAL),
    (dw, dict(out=at(4)), EINVAL), (dw, dict(ws=at(5)), EINVAL),
])
def test_far_columns_and_index_overlaps(lib, call, kw, want):
    assert call(lib, **kw) == want


def test_workspace_of_negative_sizes(lib):
    assert lib.moegg_gated_fwd_workspace_bytes(10, 2, 4, -2**31, 64, PX) == 0
    assert lib.moegg_gated_bwd_workspace_bytes(10, 2, 4, 64, -2**31) == 0
