"""Refusals of the gate, permute and unpermute entry points: every call here
fails on the host, before anything is enqueued."""

import ctypes
import math
import os

import pytest

EINVAL, ESHAPE = 1, 2
BF16, FP16, FP32 = 0, 1, 2
P = ctypes.c_void_p(1 << 20)             # never dereferenced
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
        mg._flat(torch.zeros(4, 4).t())
