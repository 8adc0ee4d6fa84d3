"""The gate, routing, permute, grouped GEMMs, per-expert adapters and unpermute
run together as one layer, forward and backward, against float64 autograd; the
same step captured in a graph; and two calls at once.

Layer: ids, w = gate(logits); y[s] = W_e x + s_e B_e A_e x for slot s of expert
e; out[t] = base[t] + sum_j w[s] y[s].  Tolerance of the whole: every stage
stores bf16, off by at most half a step, 2^-8 of the value, and a product of
random operands keeps the relative Frobenius error of its inputs; a result
behind n stored stages is held to (n + 1) * 2^-8, the fp32 sums being far
below that.
"""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import token_routing_amd as m
    m.load_library()
    return m


T, E, k, K, N, R, BM = 150, 6, 2, 128, 192, 16, 16


def make(seed):
    g = torch.Generator().manual_seed(seed)

    def rnd(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g) * std).to(dtype)

    d = dict(logits=rnd(T, E, dtype=torch.float32), X=rnd(T, K), W=rnd(E, N, K, std=K ** -0.5),
             A=rnd(E, R, K, std=K ** -0.5), B=rnd(E, N, R, std=R ** -0.5), base=rnd(T, N),
             G=rnd(T, N, std=0.1))
    d["logits"][T - 3:] = -float("inf")            # padding tokens
    d["scales"] = torch.rand(E, generator=g) + 0.5
    return {n: t.cuda() for n, t in d.items()}


def step(mg, d, padded, stream=None):
    """Forward and backward of the layer; returns everything that it computes."""
    kw = dict(stream=stream)
    ids, w, _ = mg.moe_gate(d["logits"], k, renorm=True, **kw)
    r = mg.moe_route(ids, E, BM, **kw)
    pad = dict(offsets=r["offsets"], padded_offsets=r["padded_offsets"]) if padded else {}
    xs, row_map = mg.permute(d["X"], r["scatter"], k, Xs=d.get("Xs"), block_m=BM if padded else None,
                             **pad, **kw)
    rows = xs.shape[0]
    m = r["padded_offsets"].diff() if padded else r["m_sizes"]
    # dropped slots' rows at the end belong to no expert: keep them defined
    y = mg.grouped_gemm_fwd(xs, d["W"], m, None, None, 1, 0, Y=d.get("Y"), **kw)
    y, h = mg.lora_fwd(xs, d["A"], d["B"], m, None, scales=d["scales"], Y=y, want_h=True, **kw)
    out = mg.unpermute(y, k, row_map, w, base=d["base"], **kw)
    dy, dw = mg.unpermute_bwd(d["G"], y, k, row_map, w, dY=d.get("dY"), **pad, **kw)
    dxs = mg.grouped_gemm_dX(dy, d["W"], m, None, 1, 0, dX=d.get("dXs"), **kw)
    dW = mg.grouped_gemm_dW(xs, dy, m, None, 1, 0, **kw)
    dxs, dA, dB = mg.lora_bwd(xs, dy, d["A"], d["B"], h, m, None, scales=d["scales"], dX=dxs, **kw)
    dX, _ = mg.permute_bwd(dxs, None, k, row_map, want_dw=False, **kw)
    dl = mg.moe_gate_bwd(d["logits"], ids, dw.view(T, k), renorm=True, **kw)
    assert rows == xs.shape[0]
    return dict(ids=ids, w=w, out=out, dX=dX, dW=dW, dA=dA, dB=dB, dl=dl)


def reference(d, ids):
    f = {n: t.cpu().double() for n, t in d.items()}
    leaves = {n: f[n].requires_grad_(True) for n in ("logits", "X", "W", "A", "B")}
    live = torch.isfinite(leaves["logits"].detach())
    ids = ids.cpu().long()
    ok = ids >= 0
    l = torch.where(live, leaves["logits"], torch.zeros_like(leaves["logits"]))
    x = torch.gather(l, 1, ids.clamp(min=0))
    w = torch.where(ok, torch.softmax(x, 1), torch.zeros_like(x))
    out = f["base"].clone()
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        y = leaves["X"][t] @ (leaves["W"][e].T + f["scales"][e] * leaves["A"][e].T @ leaves["B"][e].T)
        out = out.index_add(0, t, w[t, j][:, None] * y)
    (out * f["G"]).sum().backward()
    return dict(w=w.detach(), out=out.detach(), dX=leaves["X"].grad, dW=leaves["W"].grad,
                dA=leaves["A"].grad, dB=leaves["B"].grad, dl=leaves["logits"].grad)


# stages of bf16 stored before a result: y (twice: product, adapter), out; dy,
# dxs (twice), dX; the weights' gradients behind dy and their own rounding; dl
# behind y (twice)
STAGES = dict(w=0, out=3, dX=4, dW=2, dA=2, dB=2, dl=2)


@pytest.mark.parametrize("padded", [False, True], ids=["sorted", "padded"])
def test_layer_forward_and_backward(mg, padded):
    d = make(1)
    got = step(mg, d, padded)
    ref = reference(d, got["ids"])
    assert torch.all(got["ids"][T - 3:] == -1) and torch.all(got["ids"][:T - 3] >= 0)
    assert torch.equal(got["out"][T - 3:], d["base"][T - 3:])
    for n, stages in STAGES.items():
        a, b = got[n].cpu().double(), ref[n]
        b = torch.where(torch.isfinite(b), b, torch.zeros_like(b))
        err = float((a - b).norm() / b.norm())
        assert err <= (stages + 1) * 2.0 ** -8, (n, err)


@pytest.mark.parametrize("padded", [False, True], ids=["sorted", "padded"])
def test_layer_in_a_graph(mg, padded):
    """Captured once, replayed with new inputs between eager work, every replay
    equal to the eager step bit for bit."""
    d = make(2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(mg, d, padded)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(mg, d, padded)
    for seed in (3, 4, 5):
        new = make(seed)
        for n in d:
            d[n].copy_(new[n])
        graph.replay()
        torch.cuda.synchronize()
        kept = {n: t.clone() for n, t in captured.items()}
        eager = step(mg, {n: t.clone() for n, t in d.items()}, padded)
        torch.cuda.synchronize()
        for n in eager:
            assert torch.equal(kept[n], eager[n]), (seed, n)


def test_two_steps_at_once(mg):
    """Two streams run steps of their own at the same time."""
    a, b = make(6), make(7)
    ra, rb = step(mg, a, True), step(mg, b, True)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(3):
        got.append((step(mg, a, False, stream=s1), step(mg, b, False, stream=s2)))
    torch.cuda.synchronize()
    for ga, gb in got:
        for n in ("ids", "w", "out", "dX", "dl"):
            assert torch.equal(ga[n], ra[n]) and torch.equal(gb[n], rb[n]), n


def test_adapters_of_requests_share_one_routing(mg):
    """The rows of a batch grouped once, used for two projections of different width."""
    g = torch.Generator().manual_seed(8)
    rows, L = 70, 9
    ids = torch.randint(0, L, (rows,), generator=g, dtype=torch.int32)
    r = mg.moe_route(ids.cuda().view(-1, 1), L, 16)
    X = torch.randn(rows, 256, generator=g).bfloat16().cuda()
    wide = torch.randn(rows, 3 * 128, generator=g).bfloat16().cuda()      # q, k, v side by side
    before = wide.clone()
    for part in (0, 2):
        A = (torch.randn(L, 8, 256, generator=g) / 16).bfloat16().cuda()
        B = torch.randn(L, 128, 8, generator=g).bfloat16().cuda()
        view = wide[:, part * 128:(part + 1) * 128]
        mg.lora_fwd(X, A, B, r["m_sizes"], r["gather"], Y=view)
        ref = before[:, part * 128:(part + 1) * 128].double().cpu()
        for i, a in enumerate(ids.tolist()):
            ref[i] += B[a].double().cpu() @ (A[a].double().cpu() @ X[i].double().cpu())
        err = float((view.cpu().double() - ref).norm() / ref.norm())
        assert err <= 2.0 ** -8
    assert torch.equal(wide[:, 128:256], before[:, 128:256])
