"""Measured cases of the feed-forward block around the grouped products: products
of 8-bit integers, the gated block with its backward pass, and activations kept
in 8 bits for that backward pass.

Each case is one pass as a user's program makes it.  With `own` false `run`
computes the operators in their plain form, elementary torch operations in 32
bits (64 for the choice of a code) rounded once at the end; with `own` true it
calls token_routing_amd.  `exact` evaluates the same definitions in 64 bits.

Definitions (T tokens, k choices a token, S = T*k rows in expert order, row p of
expert e comes from slot s(p) of token t(p)):

i8        Xq[i] = round(127 X[i] / m_i), m_i = max |X[i]|, scale x_i = m_i / 127
          (ties to even); W rows were quantised so once, scale w_en.
          y[p, n] = x_i * w_en * sum_k Xq[i, k] Wq[e, n, k], i = t(p).
          gated: (gate, up) pairs of columns, out = act(y_gate) * y_up.
          scattered: out row s(p) = weight_s * y[p], i = p.
ffn       A = X[t(p)] W_e^T, gate and up columns g and u; H = act(g) * u.
ffn_bwd   dH = dY W_e of the down projection W [E, N, I];
          dg = dH * u * act'(g), du = dH * act(g) from the kept g and u, and
          H = act(g) * u again for the down projection's own gradient.
ffn_step  ffn that keeps g and u in 8 bits, then ffn_bwd from them.
packed    blocks of 32 neighbours of a row share a power of two 2^e, the
          smallest with round(max / 2^e) <= 127 (e >= -126); code = round(x / 2^e).
          pack: there and back.  dw: dW_e = dY_e^T X_e from X kept so.
act       silu: g / (1 + e^-g); gelu: g/2 (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))).
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BLOCK = 32


# ---------------------------------------------------------------- cases

def listed():
    return [
        # One token of a small layer in a decode loop, served in 8 bits: latency alone.
        dict(name="i8_one_token", op="i8", T=1, E=8, k=2, K=1024, N=2048, form="gated",
             act="silu", halves=False),
        # A decode step of 64 requests, first projections of a fine-grained layer.
        dict(name="i8_decode", op="i8", T=64, E=128, k=8, K=2048, N=1536, form="gated",
             act="silu", halves=True),
        # The prefill batch of a wide top-2 layer.
        dict(name="i8_batch", op="i8", T=4096, E=8, k=2, K=4096, N=28672, form="gated",
             act="silu", halves=False),
        # Down projection of the fine-grained layer's batch, scattered back to
        # slot order with the routing weights.
        dict(name="i8_down_batch", op="i8", T=8192, E=128, k=8, K=768, N=2048,
             form="scattered", act="silu", halves=False),
        # Training forward of the fine-grained layer, pre-activations kept in 16 bits.
        dict(name="ffn_batch", op="ffn", T=8192, E=128, k=8, K=2048, I=768, act="silu",
             halves=False, kept=True),
        # An odd small layer, gate and up in halves: rows of no whole 16 bytes.
        dict(name="ffn_odd", op="ffn", T=1001, E=9, k=3, K=1003, I=517, act="gelu",
             halves=True, kept=True),
        # Training of the wide layer: forward that keeps 8 bits, and the
        # activation's backward behind the down projection's gradient.
        dict(name="ffn_step_batch", op="ffn_step", T=4096, E=8, k=2, K=4096, I=14336,
             act="silu", halves=False),
        # The fine-grained layer's backward from 8 bits.
        dict(name="ffn_bwd_batch", op="ffn_bwd", T=8192, E=128, k=8, K=2048, I=768,
             act="silu", halves=True, packed=True),
        # A layer's input put by in 8 bits and taken back.
        dict(name="pack_batch", op="pack", T=16384, K=4096, dtype="bf16"),
        # The same of an odd small batch in 32 bits.
        dict(name="pack_odd", op="pack", T=1001, K=1003, dtype="fp32"),
        # Weight gradient of the fine-grained layer's first projections, its
        # input kept in 8 bits.
        dict(name="dw_batch", op="dw", T=8192, E=128, k=8, K=2048, N=1536),
        # The same for a short batch: most experts hold a few rows.
        dict(name="dw_short", op="dw", T=64, E=128, k=8, K=768, N=2048),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi, multiple):
    """A third of the time any size, else a multiple."""
    v = _log_int(rng, lo, hi)
    return v if rng.random() < 0.33 else max(multiple, v // multiple * multiple)


def draw(rng):
    op = rng.choice(["i8", "i8", "ffn", "ffn", "ffn_step", "ffn_bwd", "pack", "dw"])
    if op == "pack":
        c = dict(op=op, T=_log_int(rng, 1, 16384), K=_size(rng, 16, 8192, 64),
                 dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
        limit = work(listed()[8])["bytes"]
        while work(c)["bytes"] > limit:
            c["T"] = max(1, c["T"] * 2 // 3)
        return c
    E = rng.choice([1, 4, 8, 16, 60, 128])
    c = dict(op=op, T=_log_int(rng, 1, 8192), E=E, k=rng.randint(1, min(E, 8)),
             K=_size(rng, 128, 4096, 64))
    act, halves = rng.choice(["silu", "silu", "gelu"]), rng.random() < 0.5
    if op == "i8":
        c["form"] = rng.choice(["gated", "scattered", "plain"])
        n = _size(rng, 128, 8192, 64)
        c.update(N=n + n % 2 if c["form"] == "gated" else n, act=act, halves=halves)
    elif op == "dw":
        c["N"] = _size(rng, 128, 4096, 64)
    else:
        c.update(I=_size(rng, 64, 4096, 32), act=act, halves=halves)
        if op == "ffn":
            c["kept"] = rng.random() < 0.6
        if op == "ffn_bwd":
            c["packed"] = rng.random() < 0.6
    limit = work(listed()[6])
    while work(c)["flops"] > limit["flops"] / 2 or work(c)["bytes"] > limit["bytes"]:
        c["T"] = max(1, c["T"] * 2 // 3)
    return c


def _used(S, E):
    """Experts that S slots reach, evenly spread."""
    return E * (1 - (1 - 1 / E) ** S)


def work(case):
    op, T, K = case["op"], case["T"], case["K"]
    if op == "pack":
        es = {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]]
        return {"bytes": T * K * (2 * es + 2 + 2 / BLOCK), "flops": 4 * T * K}
    E, k = case["E"], case["k"]
    S = T * k
    e = _used(S, E)
    if op == "i8":
        N = case["N"]
        rows, cols = (S, N) if case["form"] == "scattered" else (T, N)
        out = S * (N // 2 if case["form"] == "gated" else cols) * 2
        return {"bytes": rows * K * 2 + e * N * (K + 4) + S * 4 + out,
                "flops": 2 * S * N * K + 3 * rows * K}
    if op == "dw":
        N = case["N"]
        return {"bytes": T * K * (1 + 1 / BLOCK) + S * N * 2 + E * N * K * 2 + S * 4,
                "flops": 2 * S * N * K}
    I = case["I"]
    fwd = {"bytes": T * K * 2 + e * 2 * I * K * 2 + S * I * 2 + S * 4, "flops": 4 * S * I * K}
    kept8 = S * 2 * I * (1 + 1 / BLOCK)
    bwd = {"bytes": S * K * 2 + e * I * K * 2 + S * 3 * I * 2 + S * 4, "flops": 2 * S * I * K}
    if op == "ffn":
        return {"bytes": fwd["bytes"] + (S * 2 * I * 2 if case["kept"] else 0),
                "flops": fwd["flops"]}
    if op == "ffn_bwd":
        return {"bytes": bwd["bytes"] + (kept8 if case["packed"] else S * 2 * I * 2),
                "flops": bwd["flops"]}
    return {"bytes": fwd["bytes"] + bwd["bytes"] + 2 * kept8, "flops": fwd["flops"] + bwd["flops"]}


# ---------------------------------------------------------------- inputs

def _routing(T, E, k, gen, dev):
    """k distinct experts a token, skewed towards the low ones; slots sorted by expert."""
    pref = -torch.log1p(torch.arange(E, device=dev, dtype=torch.float32)) * 0.7
    noise = torch.rand(T, E, generator=gen, device=dev).clamp_(1e-6, 1 - 1e-6)
    flat = (pref - torch.log(-torch.log(noise))).topk(k, dim=1).indices.reshape(-1)
    order = torch.argsort(flat, stable=True)
    return order.to(torch.int32), torch.bincount(flat, minlength=E)


def _round_up(n, m):
    return (n + m - 1) // m * m


def _codes(x):
    """Codes of one scale a row: round(127 x / max), and the scales."""
    m = x.abs().amax(1, keepdim=True)
    safe = torch.where(m > 0, m, torch.ones_like(m)).double()
    return torch.round(x.double() * 127 / safe), m.double().squeeze(1) / 127


def _blocks(x):
    """Rows of x in blocks of 32 (zeros behind the row), and each block's exponent."""
    rows, cols = x.shape
    b = torch.nn.functional.pad(x, (0, _round_up(cols, BLOCK) - cols)).view(rows, -1, BLOCK)
    frac, exp = torch.frexp(b.abs().amax(2))
    return b, (exp - 7 + (frac >= 255 / 256).int()).clamp(min=-126)


def _packed(x):
    """int8 codes [rows, cols in whole blocks] and the exponents' bytes [rows, blocks]."""
    b, e = _blocks(x.float())
    q = torch.round(torch.ldexp(b, -e.unsqueeze(2)))
    return q.view(x.shape[0], -1).to(torch.int8), (e + 127).to(torch.uint8)


def _stack(first, second, halves):
    """Gate and up as neighbours, or as halves, along the last dimension."""
    if halves:
        return torch.cat([first, second], -1)
    return torch.stack([first, second], -1).flatten(-2)


def _planes(a, halves):
    """The inverse of _stack."""
    n = a.shape[-1] // 2
    return (a[..., :n], a[..., n:]) if halves else (a[..., 0::2], a[..., 1::2])


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 6364 + 29)
    op, T, K = case["op"], case["T"], case["K"]

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=gen, device=dev, dtype=dtype).mul_(std)

    st = dict(case)
    if op == "pack":
        # rows of different size, as a residual stream has them
        x = normal(T, K, dtype=DTYPES[case["dtype"]])
        st["X"] = x * torch.exp2(torch.randint(-3, 4, (T, 1), generator=gen, device=dev)).to(x.dtype)
        return st
    E, k = case["E"], case["k"]
    S = T * k
    order, sizes = _routing(T, E, k, gen, dev)
    st["gather"] = order
    st["m_sizes"] = sizes.to(torch.int32)
    st["sizes"] = sizes.tolist()                        # the plain form's host copy
    if op == "i8":
        N, scattered = case["N"], case["form"] == "scattered"
        st["X"] = normal(S if scattered else T, K)
        Kq = _round_up(K, 16)                           # the weights, laid out once
        st["Wq"] = torch.zeros(E, N, Kq, dtype=torch.int8, device=dev)
        st["w_scales"] = torch.empty(E, N, device=dev)
        for e in range(E):
            w = normal(N, K, std=K ** -0.5).float()
            m = w.abs().amax(1, keepdim=True)
            st["Wq"][e, :, :K] = torch.round(w * (127 / m)).to(torch.int8)
            st["w_scales"][e] = m[:, 0] / 127
        st["weights"] = (torch.rand(S, generator=gen, device=dev) + 0.05) if scattered else None
        return st
    if op == "dw":
        st["Xq"], st["Xs"] = _packed(normal(T, K))
        st["dY"] = normal(S, case["N"], std=0.1)
        return st
    I = case["I"]
    if op in ("ffn", "ffn_step"):
        st["X"] = normal(T, K)
        st["W"] = normal(E, 2 * I, K, std=K ** -0.5)
    if op in ("ffn_bwd", "ffn_step"):
        st["dY"] = normal(S, K, std=0.1)                # expert order
        st["Wd"] = normal(E, K, I, std=I ** -0.5)       # down projection [E, N = K, I]
    if op == "ffn_bwd":
        g, u = normal(S, I), normal(S, I)
        if case["packed"]:
            (gq, gs), (uq, us) = _packed(g), _packed(u)
            st["kept"] = (torch.cat([gq, uq], 1), torch.cat([gs, us], 1))
        else:
            st["kept"] = _stack(g, u, case["halves"])
    return st


# ---------------------------------------------------------------- plain forms

def _act(g, name):
    if name == "silu":
        return g / (1 + torch.exp(-g))
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))


def _act_slope(g, name):
    if name == "silu":
        s = 1 / (1 + torch.exp(-g))
        return s * (1 + g * (1 - s))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def _spans(st):
    """(expert, its rows in expert order) of the experts that hold rows."""
    o = 0
    for e, m in enumerate(st["sizes"]):
        if m:
            yield e, slice(o, o + m)
        o += m


def _unpacked(q, s, cols):
    v = q.float().view(q.shape[0], -1, BLOCK)
    return torch.ldexp(v, (s.int() - 127).unsqueeze(2)).view(q.shape[0], -1)[:, :cols]


def _there_and_back(x):
    b, e = _blocks(x)
    e = e.unsqueeze(2)
    return torch.ldexp(torch.round(torch.ldexp(b, -e)), e).view(x.shape[0], -1)[:, :x.shape[1]]


def _plain_i8(st):
    codes, scales = _codes(st["X"])
    codes, scales = codes.float(), scales.float()
    S, N, K = st["T"] * st["k"], st["N"], st["K"]
    order = st["gather"].long()
    gated = st["form"] == "gated"
    out = torch.empty(S, N // 2 if gated else N, dtype=torch.bfloat16, device=codes.device)
    for e, rows in _spans(st):
        src = torch.arange(rows.start, rows.stop, device=codes.device)
        if st["form"] != "scattered":
            src = order[rows] // st["k"]
        y = codes[src] @ st["Wq"][e, :, :K].float().T
        y = y * scales[src].unsqueeze(1) * st["w_scales"][e]
        if gated:
            g, u = _planes(y, st["halves"])
            out[rows] = (_act(g, st["act"]) * u).to(out.dtype)
        elif st["form"] == "scattered":
            out[order[rows]] = (y * st["weights"][order[rows]].unsqueeze(1)).to(out.dtype)
        else:
            out[rows] = y.to(out.dtype)
    return [out]


def _plain_ffn(st):
    """H, and the fp32 gate and up columns [S, I] each."""
    S, I = st["T"] * st["k"], st["I"]
    g = torch.empty(S, I, device=st["X"].device)
    u = torch.empty_like(g)
    for e, rows in _spans(st):
        x = st["X"][st["gather"][rows].long() // st["k"]].float()
        g[rows], u[rows] = _planes(x @ st["W"][e].float().T, st["halves"])
    return (_act(g, st["act"]) * u).to(torch.bfloat16), g, u


def _plain_ffn_bwd(st, g, u):
    dh = torch.empty_like(g)
    for e, rows in _spans(st):
        dh[rows] = st["dY"][rows].float() @ st["Wd"][e].float()
    a = _act(g, st["act"])
    dg = (dh * u * _act_slope(g, st["act"])).to(torch.bfloat16)
    du = (dh * a).to(torch.bfloat16)
    return [_stack(dg, du, st["halves"]), (a * u).to(torch.bfloat16)]


def _plain(st):
    op = st["op"]
    if op == "i8":
        return _plain_i8(st)
    if op == "pack":
        return [_there_and_back(st["X"].float()).to(st["X"].dtype)]
    if op == "dw":
        x = _unpacked(st["Xq"], st["Xs"], st["K"])
        dw = torch.zeros(st["E"], st["N"], st["K"], dtype=torch.bfloat16, device=x.device)
        for e, rows in _spans(st):
            src = x[st["gather"][rows].long() // st["k"]]
            dw[e] = (st["dY"][rows].float().T @ src).to(torch.bfloat16)
        return [dw]
    if op == "ffn_bwd":
        if st["packed"]:
            g, u = (_unpacked(q, s, st["I"]) for q, s in zip(st["kept"][0].chunk(2, 1),
                                                             st["kept"][1].chunk(2, 1)))
        else:
            g, u = (v.float() for v in _planes(st["kept"], st["halves"]))
        return _plain_ffn_bwd(st, g, u)
    h, g, u = _plain_ffn(st)
    if op == "ffn_step":
        return [h] + _plain_ffn_bwd(st, _there_and_back(g), _there_and_back(u))
    if st["kept"]:
        return [h, _stack(g.to(torch.bfloat16), u.to(torch.bfloat16), st["halves"])]
    return [h]


# ---------------------------------------------------------------- the framework's calls

def _own(st):
    import token_routing_amd as mg
    op = st["op"]
    if op == "pack":
        codes, scales = mg.pack8(st["X"])
        return [mg.unpack8(codes, scales, st["K"], st["X"].dtype)]
    if op == "dw":
        return [mg.grouped_gemm_dW_packed(st["Xq"], st["Xs"], st["dY"], st["m_sizes"],
                                          st["gather"], st["k"], mg.PERMUTE_X, K=st["K"])]
    shape = ((mg.GATED_GELU if st["act"] == "gelu" else mg.GATED_SILU)
             | (mg.GATED_HALVES if st["halves"] else 0))
    if op == "i8":
        flags = {"gated": mg.PERMUTE_X | shape, "plain": mg.PERMUTE_X,
                 "scattered": mg.PERMUTE_Y | mg.FUSE_MUL_POST}[st["form"]]
        q, scales = mg.quant_rows(st["X"])
        return [mg.grouped_gemm_i8(q, scales, st["Wq"], st["w_scales"], st["m_sizes"],
                                   st["gather"], st["weights"], st["k"], flags)]
    if op == "ffn_bwd":
        return list(mg.gated_bwd(st["dY"], st["Wd"], st["kept"], st["m_sizes"], st["gather"],
                                 st["k"], shape))
    keep = "packed" if op == "ffn_step" else "bf16" if st["kept"] else None
    h, kept = mg.gated_fwd(st["X"], st["W"], st["m_sizes"], st["gather"], st["k"],
                           mg.PERMUTE_X | shape, keep=keep)
    if op == "ffn_step":
        return [h] + list(mg.gated_bwd(st["dY"], st["Wd"], kept, st["m_sizes"], st["gather"],
                                       st["k"], shape))
    return [h] if kept is None else [h, kept]


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- 64-bit values

def _owners(st):
    return torch.repeat_interleave(torch.arange(st["E"], device=st["gather"].device),
                                   st["m_sizes"].long())


def _by_expert(st, left, right, transposed):
    """left[p] times its expert's matrix, in 64 bits: [out, in] matrices when transposed."""
    owner = _owners(st)
    cols = right.shape[1] if transposed else right.shape[2]
    out = torch.zeros(owner.numel(), cols, dtype=torch.float64, device=left.device)
    for e in torch.unique(owner).tolist():
        at = torch.nonzero(owner == e).flatten()
        w = right[e].double()
        out[at] = torch.mm(left[at].double(), w.t() if transposed else w)
    return out


def _exact_act(g, name):
    """Activation and its derivative."""
    g = g.detach().requires_grad_(True)
    if name == "silu":
        a = g * torch.sigmoid(g)
    else:
        a = g * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))
    slope, = torch.autograd.grad(a.sum(), g)
    return a.detach(), slope


def _exact_packed(x):
    """Values of x in blocks of 32, the exponent found by trying."""
    rows, cols = x.shape
    b = torch.zeros(rows, _round_up(cols, BLOCK), dtype=torch.float64, device=x.device)
    b[:, :cols] = x
    b = b.view(rows, -1, BLOCK)
    top = b.abs().amax(2, keepdim=True).clamp(min=2.0 ** -126)
    e = torch.floor(torch.log2(top)) - 8
    for _ in range(3):
        e = torch.where(torch.round(top / torch.exp2(e)) > 127, e + 1, e)
    step = torch.exp2(e.clamp(min=-126))
    return (torch.round(b / step) * step).view(rows, -1)[:, :cols]


def _exact_bwd(st, g, u):
    dh = _by_expert(st, st["dY"], st["Wd"], False)
    a, slope = _exact_act(g, st["act"])
    return [_stack(dh * u * slope, dh * a, st["halves"]), a * u]


def _values(q, s, cols):
    step = torch.exp2(s.double() - 127).repeat_interleave(BLOCK, 1)
    return (q.double() * step)[:, :cols]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "pack":
        return [_exact_packed(st["X"].double())]
    order = st["gather"].long()
    if op == "i8":
        x = st["X"].double()
        m = x.abs().amax(1, keepdim=True)
        q = torch.round(127 * x / torch.where(m == 0, torch.ones_like(m), m))
        src = (torch.arange(order.numel(), device=x.device) if case["form"] == "scattered"
               else order // st["k"])
        y = _by_expert(st, q[src], st["Wq"][:, :, :st["K"]], True)
        y = y * (m / 127)[src] * st["w_scales"].double()[_owners(st)]
        if case["form"] == "gated":
            g, u = _planes(y, st["halves"])
            return [_exact_act(g, st["act"])[0] * u]
        if case["form"] == "scattered":
            out = torch.empty_like(y)
            out[order] = y * st["weights"].double()[order].unsqueeze(1)
            return [out]
        return [y]
    if op == "dw":
        x = _values(st["Xq"], st["Xs"], st["K"])[order // st["k"]]
        dw = torch.zeros(st["E"], st["N"], st["K"], dtype=torch.float64, device=x.device)
        owner = _owners(st)
        for e in torch.unique(owner).tolist():
            at = torch.nonzero(owner == e).flatten()
            dw[e] = torch.mm(st["dY"][at].double().t(), x[at])
        return [dw]
    if op == "ffn_bwd":
        if st["packed"]:
            q, s = st["kept"]
            half, n = q.shape[1] // 2, s.shape[1] // 2
            g, u = _values(q[:, :half], s[:, :n], st["I"]), _values(q[:, half:], s[:, n:], st["I"])
        else:
            g, u = (v.double() for v in _planes(st["kept"], st["halves"]))
        return _exact_bwd(st, g, u)
    a = _by_expert(st, st["X"][order // st["k"]], st["W"], True)
    g, u = (v.contiguous() for v in _planes(a, st["halves"]))
    h = _exact_act(g, st["act"])[0] * u
    if op == "ffn_step":
        return [h] + _exact_bwd(st, _exact_packed(g), _exact_packed(u))
    return [h, a] if case["kept"] else [h]
