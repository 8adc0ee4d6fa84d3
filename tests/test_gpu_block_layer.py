"""The block's operators as they are used together: a training step (routing, gated
forward that keeps 8 bits, packed input, down projection, combine, and all gradients)
and the serving layer in 8-bit integers; captured in a graph with replays, on another
stream, and as two graphs of their own workspaces."""

import numpy as np
import pytest
import torch

from tests._block import f64, grouped, routed, split

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import token_routing_amd as m
    m.load_library()
    return m


class Layer:
    def __init__(self, mg, T=96, k=2, E=4, K=128, I=72, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.mg, self.T, self.k, self.E, self.K, self.I = mg, T, k, E, K, I
        self.ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32).cuda()
        self.ids[3, 1] = -1
        self.x = torch.randn(T, K, generator=g).bfloat16().cuda()
        self.w1 = (torch.randn(E, 2 * I, K, generator=g) / K ** 0.5).bfloat16().cuda()
        self.w2 = (torch.randn(E, K, I, generator=g) / I ** 0.5).bfloat16().cuda()
        self.wt = (torch.rand(T * k, generator=g) + 0.1).cuda()
        self.dout = torch.randn(T, K, generator=g).bfloat16().cuda()
        self.i1 = mg.quant_rows(self.w1)
        self.i2 = mg.quant_rows(self.w2)

    def train(self):
        mg, k, f = self.mg, self.k, self.mg.GATED_SILU
        r = mg.moe_route(self.ids, self.E)
        m, ga = r["m_sizes"], r["gather"]
        xq = mg.pack8(self.x)
        h, kept = mg.gated_fwd(self.x, self.w1, m, ga, k, f | mg.PERMUTE_X, keep="packed")
        y = mg.grouped_gemm_fwd(h, self.w2, m, ga, None, k, 0)
        out = mg.combine(y, k, r["scatter"], self.wt)
        dy, dwt = mg.combine_bwd(self.dout, y, k, r["scatter"], self.wt)
        da, h2 = mg.gated_bwd(dy, self.w2, kept, m, ga, k, f)
        dw2 = mg.grouped_gemm_dW(h2, dy, m, ga, k, 0)
        dw1 = mg.grouped_gemm_dW_packed(*xq, da, m, ga, k, mg.PERMUTE_X, K=self.K)
        dxs = mg.grouped_gemm_dX(da, self.w1, m, ga, k, 0)
        dx = mg.combine(dxs, k, r["scatter"])
        return [out, dwt, dw1, dw2, dx]

    def serve(self):
        mg, k = self.mg, self.k
        r = mg.moe_route(self.ids, self.E)
        q, s = mg.quant_rows(self.x)
        h = mg.grouped_gemm_i8(q, s, *self.i1, r["m_sizes"], r["gather"], None, k,
                               mg.PERMUTE_X | mg.GATED_SILU)
        q, s = mg.quant_rows(h)
        y = mg.grouped_gemm_i8(q, s, *self.i2, r["m_sizes"], r["gather"], self.wt, k,
                               mg.PERMUTE_Y | mg.FUSE_MUL_POST)
        live = (self.ids.reshape(-1) >= 0)
        return [torch.where(live[:, None], y, torch.zeros_like(y))]

    def reference(self):
        """The training step in 64 bits, by autograd, with nothing rounded or kept in 8 bits."""
        x = self.x.double().cpu().requires_grad_()
        w1 = self.w1.double().cpu().requires_grad_()
        w2 = self.w2.double().cpu().requires_grad_()
        wt = self.wt.double().cpu().requires_grad_()
        out = torch.zeros(self.T, self.K, dtype=torch.float64)
        ids = self.ids.cpu()
        for t in range(self.T):
            for j in range(self.k):
                e = int(ids[t, j])
                if e < 0:
                    continue
                a = w1[e] @ x[t]
                g, u = a[0::2], a[1::2]
                y = w2[e] @ (g * torch.sigmoid(g) * u)
                out = out.index_add(0, torch.tensor([t]), (wt[t * self.k + j] * y)[None])
        loss = (out * self.dout.double().cpu()).sum()
        return [out.detach()] + list(torch.autograd.grad(loss, (wt, w1, w2, x)))


def test_training_step(mg):
    """Outputs near the unrounded step.  Relative to the whole tensor: each of up to five
    roundings to bf16 on the way costs at most 2^-8, and reading g and u back from 8 bits
    at most half a step, 1 / 128 of their block's largest: 5 * 2^-8 + 2^-7 for the forward
    and the gradients behind one such product, half as much again behind a second."""
    layer = Layer(mg)
    for got, ref in zip(layer.train(), layer.reference()):
        ref = ref.numpy()
        off = np.linalg.norm(f64(got) - ref) / np.linalg.norm(ref)
        assert off <= 1.5 * (5 * 2.0 ** -8 + 2.0 ** -7), off


def test_serving_layer(mg):
    """Near the layer in 64 bits: four roundings to codes (half of 1 / 127 of a row's
    largest value, which is below 5 times its root mean square here: 5 / 254 each) and
    three to bf16."""
    layer = Layer(mg, T=80)
    out = f64(layer.serve()[0])
    r, order, experts = None, [], []
    ids = layer.ids.cpu().reshape(-1).numpy()
    slots = np.nonzero(ids >= 0)[0]
    a, _ = grouped(f64(layer.x)[slots // layer.k], ids[slots], f64(layer.w1), True)
    g, u = split(a, False)
    y, _ = grouped(g / (1 + np.exp(-g)) * u, ids[slots], f64(layer.w2), True)
    y *= f64(layer.wt)[slots][:, None]
    assert (out[ids < 0] == 0).all()
    off = np.linalg.norm(out[slots] - y) / np.linalg.norm(y)
    assert off <= 4 * 5 / 254 + 3 * 2.0 ** -8, off


@pytest.mark.parametrize("form", ["train", "serve"])
def test_graph(mg, form):
    """Captured once, replayed with eager work between: every replay is the eager result."""
    layer = Layer(mg, seed=2)
    run = getattr(layer, form)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run()
    for k in range(4):
        layer.x.copy_(torch.randn(layer.T, layer.K,
                                  generator=torch.Generator().manual_seed(k)).bfloat16())
        want = run()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
        run()


def test_two_graphs(mg):
    """Two captured steps replayed one after the other keep their own results."""
    layers = [Layer(mg, seed=5), Layer(mg, T=60, seed=6)]
    wants, graphs, outs = [x.train() for x in layers], [], []
    for layer in layers:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(layer.train())
        graphs.append(graph)
    for k in (0, 1, 1, 0, 1):
        graphs[k].replay()
    torch.cuda.synchronize()
    for out, want in zip(outs, wants):
        for a, b in zip(out, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("form", ["train", "serve"])
def test_two_streams(mg, form):
    """Two layers at once, each on a stream of its own."""
    layers = [Layer(mg, seed=7), Layer(mg, T=200, seed=8)]
    want = [getattr(x, form)() for x in layers]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for layer, s in zip(layers, streams):
        with torch.cuda.stream(s):
            got.append(getattr(layer, form)())
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_given_buffers(mg):
    """Workspaces and outputs that the caller keeps, used again for another call."""
    T, k, E, K, I = 50, 2, 3, 65, 33
    r, order, experts, g = routed(mg, T, k, E, 31)
    n, S = order.size, T * k
    lib = mg.load_library()
    f = mg.PERMUTE_X | mg.GATED_GELU
    ws = torch.empty(lib.moegg_gated_fwd_workspace_bytes(T, k, E, I, K, f), dtype=torch.uint8,
                     device="cuda")
    ws2 = torch.empty(lib.moegg_gated_bwd_workspace_bytes(T, k, E, K, I), dtype=torch.uint8,
                      device="cuda")
    ws3 = torch.empty(mg.dw_packed_workspace_bytes(T, k, E, 2 * I, K, mg.PERMUTE_X), dtype=torch.uint8,
                      device="cuda")
    for seed in range(2):
        x = torch.randn(T, K, generator=g).bfloat16().cuda()
        w = torch.randn(E, 2 * I, K, generator=g).bfloat16().cuda()
        wd = torch.randn(E, K, I, generator=g).bfloat16().cuda()
        dy = torch.randn(S, K, generator=g).bfloat16().cuda()
        a = mg.gated_fwd(x, w, r["m_sizes"], r["gather"], k, f, keep="bf16", workspace=ws)
        b = mg.gated_fwd(x, w, r["m_sizes"], r["gather"], k, f, keep="bf16")
        assert torch.equal(a[0][:n], b[0][:n]) and torch.equal(a[1][:n], b[1][:n])
        d = mg.gated_bwd(dy, wd, a[1], r["m_sizes"], r["gather"], k, mg.GATED_GELU, workspace=ws2)
        d2 = mg.gated_bwd(dy, wd, a[1], r["m_sizes"], r["gather"], k, mg.GATED_GELU)
        assert torch.equal(d[0][:n], d2[0][:n]) and torch.equal(d[1][:n], d2[1][:n])
        xq, xs = mg.pack8(x)
        args = (xq, xs, d[0], r["m_sizes"], r["gather"], k, mg.PERMUTE_X)
        assert torch.equal(mg.grouped_gemm_dW_packed(*args, K=K, workspace=ws3),
                           mg.grouped_gemm_dW_packed(*args, K=K))


@pytest.mark.parametrize("T", [4, 32])
def test_graph_of_few_tokens(mg, T):
    """A serving step of a few rows an expert, replayed for other tokens and other experts:
    nothing of the capture's routing stays."""
    layer = Layer(mg, T=T, E=16 if T > 4 else 4, K=1024, I=256, seed=12)
    layer.serve()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = layer.serve()
    for seed in range(4):
        g = torch.Generator().manual_seed(seed)
        ids = torch.randint(0, layer.E, (T, layer.k), generator=g, dtype=torch.int32)
        if seed == 1:
            ids[:] = 3                                   # one expert for all
        if seed == 2:
            ids[1:] = -1                                 # one token, the others dropped
        layer.ids.copy_(ids)
        layer.x.copy_(torch.randn(T, layer.K, generator=g).bfloat16())
        want = layer.serve()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
        live = ids.reshape(-1).numpy() >= 0
        got = f64(outs[0])
        assert (np.abs(got[live]).max(1) > 0).all() and (got[~live] == 0).all()


def test_few_rows_on_two_streams(mg):
    layers = [Layer(mg, T=4, K=1024, I=256, seed=13), Layer(mg, T=5, K=2048, I=128, seed=14)]
    want = [x.serve() for x in layers]
    torch.cuda.synchronize()
    got = []
    for layer, s in zip(layers, [torch.cuda.Stream(), torch.cuda.Stream()]):
        with torch.cuda.stream(s):
            got.append([layer.serve() for _ in range(3)][-1])
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a[0], b[0])
