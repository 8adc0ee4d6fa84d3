"""Buffers that a gated call would not write, or does not have, are refused by the binding."""

import pytest
import torch

import token_routing_amd as mg

X = torch.zeros(4, 8, dtype=torch.bfloat16)
W = torch.zeros(1, 64, 8, dtype=torch.bfloat16)
A = torch.zeros(4, 64, dtype=torch.bfloat16)
PAIR = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 2, dtype=torch.uint8)


@pytest.mark.parametrize("keep,kept", [(None, A), (None, PAIR), ("packed", A), ("bf16", PAIR)])
def test_buffers_of_another_form(keep, kept):
    with pytest.raises(ValueError, match="kept does not fit"):
        mg.gated_fwd(X, W, None, None, 1, mg.GATED_SILU, keep=keep, kept=kept)


def test_nothing_kept():
    with pytest.raises(ValueError, match="kept must be"):
        mg.gated_bwd(X, torch.zeros(1, 8, 32, dtype=torch.bfloat16), None, None, None, 1,
                     mg.GATED_SILU)
