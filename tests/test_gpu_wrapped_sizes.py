"""m_sizes whose sum passes 32 bits: clipped to the S rows there are, as any sum past S, and
reported; results are those of the clipped sizes, bit for bit, for every kernel that reads
sizes."""

import pytest
import torch

pytestmark = pytest.mark.gpu

BIG = 2 ** 31 - 1
# sums of 2^32 - 1, 2^32 + 2 (which wraps to 2), and far past both
SIZES = [[3, BIG, BIG, 1], [0, BIG, BIG, 4], [BIG] * 4, [5, 2 ** 30, 2 ** 30, BIG]]


@pytest.fixture(scope="module")
def mg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import token_routing_amd as m
    m.load_library()
    return m


def clipped(sizes, S):
    out, left = [], S
    for m in sizes:
        out.append(min(m, left))
        left -= out[-1]
    return out


# T, K, N: tiles, tiles of long reductions, odd sizes, few rows
@pytest.mark.parametrize("T,K,N", [(300, 128, 256), (40, 64, 72), (150, 33, 47), (3, 1040, 64)])
@pytest.mark.parametrize("sizes", SIZES, ids=["two", "wraps_to_two", "four", "halves"])
def test_wrapped_sizes(mg, T, K, N, sizes):
    k, E, S = 2, 4, 2 * T
    g = torch.Generator(device="cuda").manual_seed(T)
    nb, px = torch.bfloat16, mg.PERMUTE_X
    x = torch.randn(T, K, generator=g, device="cuda").to(nb)
    w = torch.randn(E, N, K, generator=g, device="cuda").to(nb)
    w2 = torch.randn(E, 2 * N, K, generator=g, device="cuda").to(nb)
    dy = torch.randn(S, N, generator=g, device="cuda").to(nb)
    a = torch.randn(S, 2 * K, generator=g, device="cuda").to(nb)
    gather = torch.randperm(S, generator=g, device="cuda").to(torch.int32)
    wt = torch.rand(S, generator=g, device="cuda")
    xq, xs = mg.quant_rows(x)
    wq, ws = mg.quant_rows(w)
    sq, ss = mg.quant_rows(torch.randn(S, K, generator=g, device="cuda"))
    pq, ps = mg.pack8(x)

    def packed(m, err):
        h, kept = mg.gated_fwd(x, w2, m, gather, k, px | mg.GATED_SILU, keep="packed",
                               error_flags=err)
        return (h, *kept)

    calls = {
        "fwd": lambda m, e: mg.grouped_gemm_fwd(x, w, m, gather, None, k, px, error_flags=e),
        "dX": lambda m, e: mg.grouped_gemm_dX(dy, w, m, gather, k, px, error_flags=e),
        "dW": lambda m, e: mg.grouped_gemm_dW(x, dy, m, gather, k, px, error_flags=e),
        "dW unsplit": lambda m, e: mg.grouped_gemm_dW(x, dy, m, gather, k, px, split=False,
                                                      error_flags=e),
        "dW packed": lambda m, e: mg.grouped_gemm_dW_packed(pq, ps, dy, m, gather, k, px, K=K,
                                                            error_flags=e),
        "i8": lambda m, e: mg.grouped_gemm_i8(xq, xs, wq, ws, m, gather, None, k, px,
                                              error_flags=e),
        "i8 scattered": lambda m, e: mg.grouped_gemm_i8(sq, ss, wq, ws, m, gather, wt, k,
                                                        mg.PERMUTE_Y | mg.FUSE_MUL_POST,
                                                        error_flags=e),
        "gated packed": packed,
        "gated": lambda m, e: mg.gated_fwd(x, w2, m, gather, k, px | mg.GATED_GELU,
                                           error_flags=e)[0],
        "gated bwd": lambda m, e: mg.gated_bwd(dy, w, a, m, gather, k,
                                               mg.GATED_SILU | mg.PERMUTE_Y, error_flags=e),
    }
    good = torch.tensor(clipped(sizes, S), dtype=torch.int32, device="cuda")
    bad = torch.tensor(sizes, dtype=torch.int32, device="cuda")
    for name, call in calls.items():
        flags = torch.zeros(2, dtype=torch.int32, device="cuda")
        want, got = call(good, flags[:1]), call(bad, flags[1:])
        assert flags.tolist() == [0, mg.DERR_M_SIZES], name
        for t, u in zip(*(v if isinstance(v, tuple) else (v,) for v in (got, want))):
            assert torch.equal(t, u), name
