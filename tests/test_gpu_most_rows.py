"""The most rows that an expert can have: num_tokens * topk = 2^31 - 8 slots, all to one expert,
so that a row count rounded up to whole tiles passes 32 bits."""

import pytest
import torch

pytestmark = pytest.mark.gpu

T, K_TOP = 107374182, 20                                 # 2147483640 slots


@pytest.fixture(scope="module")
def mg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import token_routing_amd as m
    m.load_library()
    return m


@pytest.mark.parametrize("gated", [False, True])
def test_one_expert_of_all_slots(mg, gated):
    """Every row of the output.  Scales are powers of two and the sums whole numbers below 2^24,
    so that the plain result is the rounded sum; gated, each row is its token's own product."""
    S, K = T * K_TOP, 16
    g = torch.Generator(device="cuda").manual_seed(0)
    xq = torch.randint(-128, 128, (T, K), generator=g, dtype=torch.int8, device="cuda")
    wq = torch.randint(-128, 128, (1, 2 if gated else 1, K), generator=g, dtype=torch.int8,
                       device="cuda")
    xs = torch.full((T,), 2.0 ** -6, device="cuda")
    ws = torch.full(wq.shape[:2], 2.0 ** -6, device="cuda")
    gather = torch.arange(S, dtype=torch.int32, device="cuda")
    m = torch.tensor([S], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = torch.full((S, 1), 9.0, dtype=torch.bfloat16, device="cuda")
    mg.grouped_gemm_i8(xq, xs, wq, ws, m, gather, None, K_TOP,
                       mg.PERMUTE_X | (mg.GATED_SILU if gated else 0), Y=y, error_flags=err)
    assert int(err) == 0
    del gather
    # the same tokens once each, in pieces
    parts = []
    for a in range(0, T, 1 << 22):
        x = xq[a:a + (1 << 22)]
        if gated:
            n = x.shape[0]
            parts.append(mg.grouped_gemm_i8(x, xs[:n], wq, ws,
                                            torch.tensor([n], dtype=torch.int32, device="cuda"), None,
                                            None, 1, mg.GATED_SILU))
        else:
            v = (x.int() * wq[0, 0].int()).sum(1, keepdim=True)
            parts.append((v.float() * 2.0 ** -12).bfloat16())
    want = torch.cat(parts)
    assert torch.equal(y.view(T, K_TOP), want.expand(T, K_TOP))


@pytest.mark.parametrize("K,N", [(8, 8), (3, 1)], ids=["tiles", "any shape"])
@pytest.mark.parametrize("first", [0, 30])
def test_forward_of_all_slots(mg, K, N, first):
    """The bf16 forward: small whole numbers, whose sums of at most 128 bf16 holds."""
    S = T * K_TOP
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randint(-4, 5, (T, K), generator=g, dtype=torch.int8, device="cuda").bfloat16()
    w = torch.randint(-4, 5, (2, N, K), generator=g, device="cuda").bfloat16()
    gather = torch.arange(S, dtype=torch.int32, device="cuda")
    m = torch.tensor([first, S - first], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = torch.full((S, N), 9.0, dtype=torch.bfloat16, device="cuda")
    mg.grouped_gemm_fwd(x, w, m, gather, None, K_TOP, mg.PERMUTE_X, Y=y, error_flags=err)
    assert int(err) == 0
    del gather
    y = y.view(T, K_TOP, N)
    for a in range(0, T, 1 << 24):
        v = x[a:a + (1 << 24)].float()
        want = (v @ w[1].float().t()).bfloat16()[:, None, :].expand(-1, K_TOP, -1)
        if a == 0 and first:
            want = want.contiguous()
            want.view(-1, N)[:first] = (v[:2] @ w[0].float().t()).bfloat16().repeat_interleave(
                K_TOP, 0)[:first]
        assert torch.equal(y[a:a + (1 << 24)], want)
