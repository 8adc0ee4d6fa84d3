"""Refusals of outputs that overlap an input which is read after they are
written.  Every call here fails on the host, before anything is enqueued."""

import ctypes
import os

import pytest

EINVAL = 1
BF16 = 0


@pytest.fixture(scope="module")
def lib():
    import token_routing_amd as mg
    if not os.path.exists(mg.LIB_PATH):
        from token_routing_amd import build
        build.build()
    return mg.load_library()


T, L, R, K, N = 10, 4, 16, 64, 64
AT = 1 << 20                                       # never dereferenced
FAR = ctypes.c_void_p(1 << 24)


def bwd(lib, X, ldx, dY, lddy, dX, lddx):
    # no workspace: a call that passes the other checks is refused for that
    # (EWORKSPACE) and enqueues nothing either
    p = ctypes.c_void_p
    return lib.moegg_lora_bwd(p(X), ldx, p(dY), lddy, FAR, FAR, FAR, FAR, FAR, None, None, BF16, T,
                              L, R, K, N, p(dX), lddx, p(dX), lddx, FAR, FAR, 0, None, 0, None, None)


@pytest.mark.parametrize("dX,lddx", [
    (AT, K),                                       # the same matrix
    (AT + 2 * 8, K),                               # begins inside it
    (AT - 2 * K * (T - 1), K),                     # ends in its first row
    (AT + 2 * K * (T - 1), K),                     # begins in its last
    (AT + 6, 100),                                 # another stride across it
])
@pytest.mark.parametrize("over", ["X", "dY"])
def test_adapter_gradient_over_its_input(lib, over, dX, lddx):
    other = AT + (1 << 20)
    args = (AT, K, other, N) if over == "X" else (other, K, AT, N)
    assert bwd(lib, *args, dX, lddx) == EINVAL


@pytest.mark.parametrize("dX,lddx,ld", [
    (AT + 2 * K * T, K, K),                        # right behind
    (AT - 2 * K * T, K, K),                        # right in front
    (AT + 2 * K, 200, 200),                        # column slices of one matrix
    (AT - 2 * K, 200, 200),
    (AT + 2 * 200 * 3 + 2 * K, 200, 200),          # some rows further down, beside
])
@pytest.mark.parametrize("over", ["X", "dY"])
def test_adapter_gradient_beside_its_input(lib, over, dX, lddx, ld):
    other = AT + (1 << 20)
    args = (AT, ld, other, N) if over == "X" else (other, K, AT, ld)
    assert bwd(lib, *args, dX, lddx) == 4          # EWORKSPACE: past the overlap check


FP32 = 2


def gate(lib, logits, dtype, ld, scores, T=10, E=64, bias=None, groups=1):
    p = ctypes.c_void_p
    return lib.moegg_gate(p(logits), dtype, ld, bias, T, E, 2, groups, 1, 1.0, 0, FAR, FAR,
                          p(scores), None, None)


@pytest.mark.parametrize("dtype,ld,scores,bias,groups", [
    (FP32, 64, AT, FAR, 1),                        # in place, but the logits are read again
    (FP32, 64, AT, None, 8),
    (FP32, 80, AT, None, 1),                       # other rows
    (FP32, 64, AT + 4, None, 1),
    (FP32, 64, AT - 4, None, 1),
    (FP32, 64, AT + 4 * 639, None, 1),             # the last logit
    (BF16, 64, AT, None, 1),                       # another type
    (BF16, 64, AT + 2 * 636, None, 1),
])
def test_gate_scores_across_the_logits(lib, dtype, ld, scores, bias, groups):
    assert gate(lib, AT, dtype, ld, scores, bias=bias, groups=groups) == EINVAL


@pytest.mark.parametrize("dtype,ld,out", [
    (FP32, 80, AT), (FP32, 64, AT + 4), (BF16, 64, AT - 2), (BF16, 65, AT),
])
def test_gate_gradient_across_the_logits(lib, dtype, ld, out):
    p = ctypes.c_void_p
    assert lib.moegg_gate_bwd(p(AT), dtype, ld, FAR, FAR, None, 10, 64, 2, 1.0, 0, p(out), None,
                              None) == EINVAL


# 10 tokens of 64 bf16 columns (1280 bytes), two picks each (2560 bytes)
SORTED = AT + (1 << 20)


def sort_call(lib, name, tok, other, rows):
    p, none = ctypes.c_void_p, None
    if name == "permute":
        return lib.moegg_permute(p(tok), BF16, FAR, none, none, none, 10, 2, 0, 64, 20, p(rows),
                                 none, none, none)
    if name == "permute_bwd":
        return lib.moegg_permute_bwd(p(rows), BF16, p(other), FAR, none, 10, 2, 64, 20, p(tok), FAR,
                                     none, none)
    if name == "unpermute":
        return lib.moegg_unpermute(p(rows), BF16, FAR, none, p(other), 10, 2, 64, 20, p(tok), none,
                                   none)
    return lib.moegg_unpermute_bwd(p(tok), BF16, p(other), FAR, none, none, none, 10, 2, 0, 64, 20,
                                   p(rows), FAR, none, none)


@pytest.mark.parametrize("shift", [0, 2, -2, 1278, -2558])
@pytest.mark.parametrize("name", ["permute", "permute_bwd", "unpermute", "unpermute_bwd"])
def test_token_rows_across_sorted_rows(lib, name, shift):
    """tok at AT, the 20 sorted rows from `shift` bytes behind it."""
    assert sort_call(lib, name, AT, SORTED + (1 << 18), AT + shift) == EINVAL


@pytest.mark.parametrize("name,shift", [("permute_bwd", 128), ("permute_bwd", -2),
                                        ("unpermute", 2), ("unpermute", -1278),
                                        ("unpermute_bwd", 128), ("unpermute_bwd", -2558)])
def test_output_beside_its_place(lib, name, shift):
    """The input that the output may replace, but not row for row."""
    out = SORTED if name == "unpermute_bwd" else AT
    tok, rows = (AT, SORTED)
    assert sort_call(lib, name, tok, out + shift, rows) == EINVAL


def test_no_tokens_overlap_nothing(lib):
    """An empty X that begins inside Xs (an empty slice of one buffer)."""
    p, none = ctypes.c_void_p, None
    assert lib.moegg_permute(p(AT + 128), BF16, FAR, none, none, none, 0, 2, 0, 64, 20, p(AT), none,
                             none, none) == 0
