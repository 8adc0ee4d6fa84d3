"""Measured cases of the operators around the experts' products: the gate, the
sort of token rows into expert order and back, and the low-rank adapters of
many requests.

Each case is one call as a user's program makes it.  With `own` false `run`
computes the operator in its plain form, elementary torch operations in 32
bits rounded once at the end; with `own` true it calls token_routing_amd.
`exact` evaluates the same definitions in 64 bits.

Definitions (T tokens, k choices a token, slot s = t*k + j, E experts):

gate      score = softmax(l) or sigmoid(l); key = score + bias; the k experts
          of largest key, inside the chosen groups where there are groups
          (group value: the sum of its two largest keys), ties to the lowest
          index; weight = scale * score, divided by the picked scores' sum
          with renorm.  A logit of -inf masks its expert; a token with fewer
          than k experts left gets id -1 and weight 0 in the places left over.
permute   Xs[row(s)] = w[s] * X[t]; row(s) is the slot's place in expert
          order, with every expert's rows padded to a multiple of block_m by
          zero rows in the padded layout.
          Backward: dX[t] = sum_j w[s] * dXs[row(s)], dw[s] = <X[t], dXs[row(s)]>.
unpermute out[t] = base[t] + sum_j w[s] * Y[row(s)].
          Backward: dY[row(s)] = w[s] * dOut[t], dw[s] = <dOut[t], Y[row(s)]>.
lora      h[t] = X[t] A_a^T, Y[t] = base[t] + scale_a * h[t] B_a^T for the
          adapter a of row t, of rank_a rows of A_a [R, K] and columns of
          B_a [N, R].  Backward: dh = scale_a * dY B_a, dX = base + dh A_a,
          dA_a = dh^T X, dB_a = scale_a * dY^T h over the adapter's rows.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # One token of a small layer in a decode loop: launch latency alone.
        dict(name="gate_one_token", op="gate", T=1, E=8, k=2, dtype="bf16", sigmoid=False,
             renorm=True, bias=False, groups=1, top_groups=1, scores=False, masked=False),
        # The prefill or training batch of a fine-grained layer, with the scores
        # a load-balancing loss reads.
        dict(name="gate_batch", op="gate", T=8192, E=128, k=8, dtype="bf16", sigmoid=False,
             renorm=True, bias=False, groups=1, top_groups=1, scores=True, masked=False),
        # Balanced by a selection bias and limited to groups of experts, an odd
        # token count, some tokens (padding) with every expert masked.
        dict(name="gate_bias_groups", op="gate", T=4099, E=256, k=8, dtype="fp32", sigmoid=True,
             renorm=True, bias=True, groups=8, top_groups=4, scores=False, masked=True),
        # Training: gradients from the combine's weights and from a
        # load-balancing loss on the scores.
        dict(name="gate_bwd_batch", op="gate_bwd", T=8192, E=128, k=8, dtype="bf16",
             sigmoid=False, renorm=True, scores=True),
        # A decode step of 64 tokens, top-8 of 128 experts.
        dict(name="permute_decode", op="permute", T=64, E=128, k=8, K=2048, dtype="bf16",
             weighted=False, block_m=0),
        # The fine-grained layer's batch into the block-padded layout.
        dict(name="permute_padded", op="permute", T=8192, E=128, k=8, K=2048, dtype="bf16",
             weighted=False, block_m=128),
        # Top-2 of 8 wide experts, weights applied on the way in: training.
        dict(name="permute_bwd_weighted", op="permute_bwd", T=4096, E=8, k=2, K=4096,
             dtype="bf16", weighted=True, block_m=0),
        # The fine-grained layer's outputs back to token order, onto the
        # residual or a shared expert's output.
        dict(name="unpermute_batch", op="unpermute", T=8192, E=128, k=8, K=2048, dtype="bf16",
             weighted=True, block_m=0, base=True),
        # An odd small layer in 32 bits, padded: rows of no whole 16 bytes.
        dict(name="unpermute_bwd_odd", op="unpermute_bwd", T=1001, E=9, k=3, K=1003,
             dtype="fp32", weighted=True, block_m=16),
        # A decode step of 64 requests over 32 adapters.
        dict(name="lora_decode", op="lora", T=64, L=32, R=16, K=4096, N=4096, dtype="bf16",
             ragged=False),
        # A prefill batch through a wide projection, eight adapters of different ranks.
        dict(name="lora_batch", op="lora", T=4096, L=8, R=64, K=4096, N=28672, dtype="bf16",
             ragged=True),
        # Fine-tuning four adapters in one batch.
        dict(name="lora_bwd_batch", op="lora_bwd", T=4096, L=4, R=32, K=4096, N=4096,
             dtype="bf16", ragged=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _log_odd(rng, lo, hi, multiple):
    """Half the time any size, half the time a multiple."""
    v = _log_int(rng, lo, hi)
    return v if rng.random() < 0.35 else max(multiple, v // multiple * multiple)


def draw(rng):
    op = rng.choice(["gate", "gate", "gate_bwd", "permute", "permute_bwd", "unpermute",
                     "unpermute_bwd", "lora", "lora", "lora_bwd"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("gate", "gate_bwd"):
        E = rng.choice([4, 8, 16, 60, 64, 128, 160, 256, 511])
        c = dict(op=op, T=_log_int(rng, 1, 8192), E=E, k=rng.randint(1, min(E, 10)), dtype=dtype,
                 sigmoid=rng.random() < 0.4, renorm=rng.random() < 0.6,
                 scores=rng.random() < 0.4)
        if op == "gate":
            c.update(bias=rng.random() < 0.4, groups=1, top_groups=1, masked=rng.random() < 0.3)
            if E % 8 == 0 and E >= 32 and rng.random() < 0.4:
                c.update(groups=8, top_groups=4)
                c["k"] = min(c["k"], E // 8 * 4)
        return c
    if op in ("lora", "lora_bwd"):
        T = _log_int(rng, 1, 4096)
        c = dict(op=op, T=T, L=rng.randint(1, min(T, 48)),
                 R=rng.choice([4, 8, 16, 16, 24, 32, 64, 128]),
                 K=_log_odd(rng, 256, 4096, 64), N=_log_odd(rng, 256, 8192, 64),
                 dtype=rng.choice(["bf16", "bf16", "fp16"]), ragged=rng.random() < 0.5)
        return c
    E = rng.choice([4, 8, 16, 60, 128])
    k = rng.randint(1, min(E, 8))
    c = dict(op=op, T=_log_int(rng, 1, 8192), E=E, k=k, K=_log_odd(rng, 256, 4096, 64),
             dtype=dtype, weighted=rng.random() < 0.6, block_m=rng.choice([0, 0, 16, 128]))
    if op == "unpermute":
        c["base"] = rng.random() < 0.5
    limit = max(work(x)["bytes"] for x in listed() if x["op"].startswith("permute"))
    while work(c)["bytes"] > limit:
        c["T"] = max(1, c["T"] * 2 // 3)
    return c


def work(case):
    T, op = case["T"], case["op"]
    es = {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]]
    if op == "gate":
        E, k = case["E"], case["k"]
        b = T * E * es + T * k * 8 + (T * E * 4 if case["scores"] else 0)
        return {"bytes": b + (E * 4 if case["bias"] else 0), "flops": 6 * T * E}
    if op == "gate_bwd":
        E, k = case["E"], case["k"]
        return {"bytes": 2 * T * E * es + T * k * 8 + (T * E * 4 if case["scores"] else 0),
                "flops": 10 * T * E}
    if op in ("lora", "lora_bwd"):
        L, K, N = case["L"], case["K"], case["N"]
        ranks = _ranks(case)
        rank_sum = sum(ranks)
        # rows are shared out evenly but for the remainder: T * mean rank products
        mean = rank_sum / L
        wts = rank_sum * (K + N) * es
        if op == "lora":
            return {"bytes": T * (K + 2 * N) * es + wts + T * 4 + L * 12,
                    "flops": int(2 * T * mean * (K + N)) + T * N}
        return {"bytes": T * (3 * K + N) * es + 2 * wts + T * case["R"] * 4 + T * 4 + L * 12,
                "flops": int(4 * T * mean * (K + N)) + T * K}
    k, K = case["k"], case["K"]
    S = T * k
    pad = case["E"] * (case["block_m"] - 1) // 2 if case["block_m"] else 0
    b = T * K * es + S * 4 + (S * 4 if case["weighted"] else 0)
    if op == "permute":
        return {"bytes": b + (S + pad) * K * es, "flops": S * K}
    if op == "permute_bwd":
        extra = T * K * es + S * 4 if case["weighted"] else 0
        return {"bytes": b + S * K * es + extra, "flops": (4 if case["weighted"] else 2) * S * K}
    if op == "unpermute":
        return {"bytes": b + S * K * es + (T * K * es if case["base"] else 0),
                "flops": 2 * S * K}
    extra = S * K * es + S * 4 if case["weighted"] else 0
    return {"bytes": b + (S + pad) * K * es + extra,
            "flops": (3 if case["weighted"] else 1) * S * K}


# ---------------------------------------------------------------- inputs

def _ranks(case):
    """Ranks of the adapters: all R, or R, R/2, ... and one of rank 0 (rows without an adapter)."""
    L, R = case["L"], case["R"]
    if not case["ragged"]:
        return [R] * L
    cycle = [R, max(1, R // 2), max(1, R - 3), max(1, R // 4)]
    ranks = [cycle[i % 4] for i in range(L)]
    if L > 2:
        ranks[L // 2] = 0
    return ranks


def _routing(T, E, k, gen, dev):
    """k distinct experts a token, skewed towards the low ones, and the sorted order's metadata."""
    pref = -torch.log1p(torch.arange(E, device=dev, dtype=torch.float32)) * 0.7
    noise = torch.rand(T, E, generator=gen, device=dev).clamp_(1e-6, 1 - 1e-6)
    ids = (pref - torch.log(-torch.log(noise))).topk(k, dim=1).indices.to(torch.int32)
    flat = ids.reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    scatter = torch.empty_like(order)
    scatter[order] = torch.arange(order.numel(), device=dev)
    sizes = torch.bincount(flat, minlength=E)
    return ids, flat, scatter.to(torch.int32), sizes


def _starts(sizes):
    z = torch.zeros(1, dtype=torch.int64, device=sizes.device)
    return torch.cat([z, torch.cumsum(sizes, 0)]).to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 7919 + 17)
    dt = DTYPES[case["dtype"]]
    T, op = case["T"], case["op"]

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device=dev) * std).to(dtype)

    st = dict(case)
    if op in ("gate", "gate_bwd"):
        E, k = case["E"], case["k"]
        st["logits"] = normal(T, E, std=2.0)
        if op == "gate":
            st["bias_t"] = normal(E, std=0.1, dtype=torch.float32) if case["bias"] else None
            if case["masked"]:
                u = torch.rand(T, E, generator=gen, device=dev)
                st["logits"][u < 0.1] = -math.inf       # single experts masked
                st["logits"][16::17] = -math.inf        # padding tokens: every expert
            st["scale"] = 2.5 if case["sigmoid"] else 1.0
        else:
            st["scale"] = 2.5 if case["sigmoid"] else 1.0
            st["ids"] = torch.sort(st["logits"], dim=1, descending=True,
                                   stable=True).indices[:, :k].to(torch.int32).contiguous()
            st["dweights"] = normal(T, k, std=0.1, dtype=torch.float32)
            st["dscores"] = normal(T, E, std=0.01, dtype=torch.float32) if case["scores"] else None
        return st
    if op in ("lora", "lora_bwd"):
        L, R, K, N = case["L"], case["R"], case["K"], case["N"]
        ids = torch.cat([torch.arange(L, device=dev),
                         torch.randint(0, L, (T - L,), generator=gen, device=dev)])
        ids = ids[torch.randperm(T, generator=gen, device=dev)]
        st["gather"] = torch.argsort(ids, stable=True).to(torch.int32)
        st["m_sizes"] = torch.bincount(ids, minlength=L).to(torch.int32)
        st["sizes"] = st["m_sizes"].tolist()            # the plain form's host copy
        st["rank_list"] = _ranks(case)
        st["ranks"] = torch.tensor(st["rank_list"], dtype=torch.int32, device=dev)
        st["scales"] = torch.rand(L, generator=gen, device=dev) * 1.5 + 0.5
        st["X"] = normal(T, K)
        st["A"] = normal(L, R, K, std=K ** -0.5)
        st["B"] = normal(L, N, R, std=0.5 * R ** -0.5)
        if op == "lora":
            st["base"] = normal(T, N)
        else:
            st["dY"] = normal(T, N, std=0.1)
            st["base"] = normal(T, K, std=0.1)
            # what the forward kept: h in the adapters' order, columns past the rank zero
            h = torch.zeros(T, R, device=dev)
            x = st["X"].float()[st["gather"].long()]
            o = 0
            for a, m in enumerate(st["sizes"]):
                r = st["rank_list"][a]
                h[o:o + m, :r] = x[o:o + m] @ st["A"][a, :r].float().T
                o += m
            st["H"] = h
        return st
    E, k, K = case["E"], case["k"], case["K"]
    ids, flat, scatter, sizes = _routing(T, E, k, gen, dev)
    st["scatter"], st["topk"] = scatter, k
    st["weights"] = None
    if case["weighted"]:
        w = torch.rand(T, k, generator=gen, device=dev) + 0.05
        st["weights"] = (w / w.sum(1, keepdim=True)).reshape(-1).contiguous()
    st["offsets"] = st["padded_offsets"] = None
    st["rows"] = T * k
    row_map = scatter
    if case["block_m"]:
        b = case["block_m"]
        st["offsets"] = _starts(sizes)
        st["padded_offsets"] = _starts((sizes + b - 1) // b * b)
        shift = st["padded_offsets"][:-1] - st["offsets"][:-1]
        row_map = scatter + shift[flat]
        st["rows"] = T * k + E * (b - 1)                # what a user sizes without a host sync
    st["map"] = row_map.to(torch.int32)
    if op == "permute":
        st["X"] = normal(T, K)
        st["Xs"] = torch.zeros(st["rows"], K, dtype=dt, device=dev)
    elif op == "permute_bwd":
        st["X"] = normal(T, K)
        st["dXs"] = normal(st["rows"], K, std=0.1)
    elif op == "unpermute":
        st["Y"] = normal(st["rows"], K)
        st["base"] = normal(T, K) if case["base"] else None
    else:
        st["dOut"] = normal(T, K, std=0.1)
        st["Y"] = normal(st["rows"], K)
        st["dY"] = torch.zeros(st["rows"], K, dtype=dt, device=dev)
    return st


# ---------------------------------------------------------------- plain forms

def _gate_pick(l, st, key):
    """Ids in the order of falling key, ties to the lowest index; -1 where none is left."""
    T, E, k = st["T"], st["E"], st["k"]
    ok = l > -math.inf
    if st["groups"] > 1:
        n = st["groups"]
        g = torch.where(ok, key, torch.full_like(key, -math.inf)).view(T, n, E // n)
        top = torch.sort(g, dim=2, descending=True).values[:, :, :2]
        val = torch.where(top > -math.inf, top, torch.zeros_like(top)).sum(2)
        val = torch.where(ok.view(T, n, -1).any(2), val, torch.full_like(val, -math.inf))
        order = torch.sort(val, dim=1, descending=True, stable=True).indices
        keep = torch.zeros_like(val, dtype=torch.bool)
        keep.scatter_(1, order[:, :st["top_groups"]], True)
        ok = ok & keep.repeat_interleave(E // n, dim=1)
    key = torch.where(ok, key, torch.full_like(key, -math.inf))
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    return ids, torch.gather(ok, 1, ids)


def _softmax(l):
    m = l.amax(1, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    e = torch.exp(l - m)
    s = e.sum(1, keepdim=True)
    return e / torch.where(s > 0, s, torch.ones_like(s))


def _plain_gate(st):
    l = st["logits"].float()
    score = 1 / (1 + torch.exp(-l)) if st["sigmoid"] else _softmax(l)
    if st["bias_t"] is None and st["groups"] == 1:
        key = l                                        # both scores rise with the logit
    else:
        # keys next to one another: the choice is made in 64 bits
        d = st["logits"].double()
        key = 1 / (1 + torch.exp(-d)) if st["sigmoid"] else _softmax(d)
        if st["bias_t"] is not None:
            key = key + st["bias_t"].double()
    ids, ok = _gate_pick(l, st, key)
    w = torch.where(ok, torch.gather(score, 1, ids), torch.zeros((), device=l.device))
    if st["renorm"]:
        s = w.sum(1, keepdim=True)
        w = w / torch.where(s > 0, s, torch.ones_like(s))
    w = w * st["scale"]
    ids = torch.where(ok, ids, torch.full_like(ids, -1)).to(torch.int32)
    return [ids, w] + ([score] if st["scores"] else [])


def _plain_gate_bwd(st):
    l = st["logits"].float()
    ids = st["ids"].long()
    g = st["dweights"] * st["scale"]
    score = 1 / (1 + torch.exp(-l)) if st["sigmoid"] else _softmax(l)
    picked = torch.gather(score, 1, ids)
    if st["renorm"]:
        s = picked.sum(1, keepdim=True)
        g = (g - (g * picked).sum(1, keepdim=True) / s) / s
    ds = torch.zeros_like(score) if st["dscores"] is None else st["dscores"].clone()
    ds.scatter_add_(1, ids, g)
    if st["sigmoid"]:
        dl = ds * score * (1 - score)
    else:
        dl = score * (ds - (ds * score).sum(1, keepdim=True))
    return [dl.to(st["logits"].dtype)]


def _plain_spread(src, rows, st, other=None):
    """rows[map[s]] = w[s] * src[t], and <src[t], other[map[s]]>."""
    T, k, K = st["T"], st["topk"], src.shape[1]
    x = src.float().unsqueeze(1).expand(T, k, K).reshape(T * k, K)
    v = x if st["weights"] is None else x * st["weights"].unsqueeze(1)
    out = torch.zeros(rows, K, dtype=src.dtype, device=src.device)
    out[st["map"].long()] = v.to(out.dtype)
    dw = None if other is None else (x * other[st["map"].long()].float()).sum(1)
    return out, dw


def _plain_collect(rows, st, base=None, other=None):
    """sum_j w[s] * rows[map[s]] (+ base), and <other[t], rows[map[s]]>."""
    T, k, K = st["T"], st["topk"], rows.shape[1]
    y = rows[st["map"].long()].float()
    out = (y if st["weights"] is None else y * st["weights"].unsqueeze(1)).view(T, k, K).sum(1)
    if base is not None:
        out = out + base.float()
    dw = None
    if other is not None:
        dw = (y.view(T, k, K) * other.float().unsqueeze(1)).sum(2).reshape(-1)
    return out.to(rows.dtype), dw


def _segments(st):
    o = 0
    g = st["gather"].long()
    for a, m in enumerate(st["sizes"]):
        if m:
            yield a, st["rank_list"][a], g[o:o + m], slice(o, o + m)
        o += m


def _plain_lora(st):
    y = st["base"].float()
    for a, r, rows, _ in _segments(st):
        if r:
            h = st["X"][rows].float() @ st["A"][a, :r].float().T
            y[rows] += st["scales"][a] * (h @ st["B"][a, :, :r].float().T)
    return [y.to(st["base"].dtype)]


def _plain_lora_bwd(st):
    dx = st["base"].float()
    dA = torch.zeros(st["A"].shape, device=dx.device)
    dB = torch.zeros(st["B"].shape, device=dx.device)
    for a, r, rows, seg in _segments(st):
        if r:
            dy = st["dY"][rows].float() * st["scales"][a]
            dh = dy @ st["B"][a, :, :r].float()
            dx[rows] += dh @ st["A"][a, :r].float()
            dA[a, :r] = dh.T @ st["X"][rows].float()
            dB[a, :, :r] = dy.T @ st["H"][seg, :r]
    dt = st["X"].dtype
    return [dx.to(dt), dA.to(dt), dB.to(dt)]


def _plain(st):
    op = st["op"]
    if op == "gate":
        return _plain_gate(st)
    if op == "gate_bwd":
        return _plain_gate_bwd(st)
    if op == "lora":
        return _plain_lora(st)
    if op == "lora_bwd":
        return _plain_lora_bwd(st)
    if op == "permute":
        return [_plain_spread(st["X"], st["rows"], st)[0], st["map"].clone()]
    if op == "unpermute":
        return [_plain_collect(st["Y"], st, base=st["base"])[0]]
    if op == "permute_bwd":
        other = st["X"] if st["weighted"] else None
        out, dw = _plain_collect(st["dXs"], st, other=other)
    else:
        other = st["Y"] if st["weighted"] else None
        out, dw = _plain_spread(st["dOut"], st["rows"], st, other=other)
    return [out] + ([dw] if st["weighted"] else [])


# ---------------------------------------------------------------- the framework's calls

def _own(st):
    import token_routing_amd as mg
    op = st["op"]
    if op == "gate":
        ids, w, scores = mg.moe_gate(
            st["logits"], st["k"], bias=st["bias_t"], n_groups=st["groups"],
            topk_groups=st["top_groups"], scale=st["scale"], sigmoid=st["sigmoid"],
            renorm=st["renorm"], want_scores=st["scores"])
        return [ids, w] + ([scores] if st["scores"] else [])
    if op == "gate_bwd":
        return [mg.moe_gate_bwd(st["logits"], st["ids"], st["dweights"], dscores=st["dscores"],
                                scale=st["scale"], sigmoid=st["sigmoid"], renorm=st["renorm"])]
    if op == "lora":
        y, _ = mg.lora_fwd(st["X"], st["A"], st["B"], st["m_sizes"], st["gather"],
                           ranks=st["ranks"], scales=st["scales"], base=st["base"])
        return [y]
    if op == "lora_bwd":
        return list(mg.lora_bwd(st["X"], st["dY"], st["A"], st["B"], st["H"], st["m_sizes"],
                                st["gather"], ranks=st["ranks"], scales=st["scales"],
                                base=st["base"]))
    if op == "permute":
        xs, row_map = mg.permute(st["X"], st["scatter"], st["topk"], st["weights"],
                                 offsets=st["offsets"], padded_offsets=st["padded_offsets"],
                                 Xs=st["Xs"])
        return [xs, row_map]
    if op == "permute_bwd":
        dx, dw = mg.permute_bwd(st["dXs"], st["X"], st["topk"], st["map"], st["weights"],
                                want_dw=st["weighted"])
        return [dx] + ([dw] if st["weighted"] else [])
    if op == "unpermute":
        return [mg.unpermute(st["Y"], st["topk"], st["map"], st["weights"], base=st["base"])]
    dy, dw = mg.unpermute_bwd(st["dOut"], st["Y"], st["topk"], st["map"], st["weights"],
                              offsets=st["offsets"], padded_offsets=st["padded_offsets"],
                              want_dw=st["weighted"], dY=st["dY"])
    return [dy] + ([dw] if st["weighted"] else [])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- 64-bit values

def _exact_gate(st):
    l = st["logits"].double()
    T, E, k = st["T"], st["E"], st["k"]
    if st["sigmoid"]:
        logscore = -torch.log1p(torch.exp(-l.abs())) + l.clamp(max=0)
    else:
        logscore = l - torch.logsumexp(torch.where(l > -math.inf, l, torch.full_like(l, -1e300)),
                                       1, keepdim=True)
    score = torch.exp(logscore)
    live = torch.isfinite(l)
    key = l if (st["bias_t"] is None and st["groups"] == 1) else score
    if st["bias_t"] is not None:
        key = key + st["bias_t"].double()
    key = key.masked_fill(~live, -math.inf)
    if st["groups"] > 1:
        n, per = st["groups"], E // st["groups"]
        g = key.view(T, n, per)
        first = g.amax(2)
        rest = g.clone().scatter_(2, g.argmax(2, keepdim=True), -math.inf)
        second = rest.amax(2) if per > 1 else torch.full_like(first, -math.inf)
        val = first + torch.where(torch.isfinite(second), second, torch.zeros_like(second))
        for_group = torch.zeros_like(val, dtype=torch.bool)
        for _ in range(st["top_groups"]):
            best = val.amax(1, keepdim=True)
            at = (val == best).int().argmax(1, keepdim=True)
            for_group.scatter_(1, at, True)
            val = val.scatter(1, at, -math.inf)
        key = key.masked_fill(~for_group.repeat_interleave(per, 1), -math.inf)
    ids = torch.full((T, k), -1, dtype=torch.int32, device=l.device)
    pick = torch.full((T, k), -math.inf, dtype=torch.float64, device=l.device)
    for j in range(k):
        best = key.amax(1, keepdim=True)
        at = (key == best).int().argmax(1, keepdim=True)
        has = torch.isfinite(best)
        ids[:, j:j + 1] = torch.where(has, at, torch.full_like(at, -1)).int()
        pick[:, j:j + 1] = torch.where(has, torch.gather(logscore, 1, at), pick[:, j:j + 1])
        key = key.scatter(1, at, -math.inf)
    if st["renorm"]:
        top = pick.amax(1, keepdim=True)
        e = torch.exp(pick - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
        w = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        w = torch.exp(pick)
    out = [ids, w * st["scale"]]
    if st["scores"]:
        out.append(score.masked_fill(~live, 0.0))
    return out


def _exact_gate_bwd(st):
    l = st["logits"].double().requires_grad_(True)
    ids = st["ids"].long()
    score = torch.sigmoid(l) if st["sigmoid"] else torch.exp(l - torch.logsumexp(l, 1, keepdim=True))
    w = torch.gather(score, 1, ids)
    if st["renorm"]:
        w = w / w.sum(1, keepdim=True)
    loss = (w * st["scale"] * st["dweights"].double()).sum()
    if st["dscores"] is not None:
        loss = loss + (score * st["dscores"].double()).sum()
    return [torch.autograd.grad(loss, l)[0]]


def _exact_lora(st, with_grads):
    """One adapter after the other over the whole batch, other adapters' rows at scale zero."""
    x = st["X"].double()
    gather = st["gather"].long()
    owner = torch.empty_like(gather)
    owner[gather] = torch.repeat_interleave(torch.arange(st["L"], device=x.device),
                                            st["m_sizes"].long())
    y = st["base"].double().clone()
    if with_grads:
        dA = torch.zeros(st["A"].shape, dtype=torch.float64, device=x.device)
        dB = torch.zeros(st["B"].shape, dtype=torch.float64, device=x.device)
        h_tok = torch.empty_like(st["H"], dtype=torch.float64)
        h_tok[gather] = st["H"].double()
    for a in range(st["L"]):
        rows = torch.nonzero(owner == a).flatten()
        r = int(st["rank_list"][a])
        if rows.numel() == 0 or r == 0:
            continue
        A, B = st["A"][a, :r].double(), st["B"][a, :, :r].double()
        s = float(st["scales"][a].double())
        if not with_grads:
            y[rows] = y[rows] + torch.matmul(torch.matmul(x[rows], A.T), B.T) * s
        else:
            dy = st["dY"][rows].double()
            dh = torch.matmul(dy, B) * s
            y[rows] = y[rows] + torch.matmul(dh, A)
            dA[a, :r] = torch.matmul(dh.T, x[rows])
            dB[a, :, :r] = torch.matmul(dy.T, h_tok[rows][:, :r]) * s
    return [y, dA, dB] if with_grads else [y]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "gate":
        return _exact_gate(st)
    if op == "gate_bwd":
        return _exact_gate_bwd(st)
    if op == "lora":
        return _exact_lora(st, False)
    if op == "lora_bwd":
        return _exact_lora(st, True)
    T, k = st["T"], st["topk"]
    idx = st["map"].long().view(T, k)
    w = (torch.ones(T, k, dtype=torch.float64, device=idx.device) if st["weights"] is None
         else st["weights"].double().view(T, k))
    if op in ("permute", "unpermute_bwd"):
        src = (st["X"] if op == "permute" else st["dOut"]).double()
        out = torch.zeros(st["rows"], src.shape[1], dtype=torch.float64, device=src.device)
        dw = torch.empty(T, k, dtype=torch.float64, device=src.device)
        for j in range(k):
            out[idx[:, j]] = w[:, j, None] * src
            if op == "unpermute_bwd" and st["weighted"]:
                dw[:, j] = (st["Y"][idx[:, j]].double() * src).sum(1)
        if op == "permute":
            return [out, st["map"]]
        return [out] + ([dw.reshape(-1)] if st["weighted"] else [])
    rows = st["dXs"] if op == "permute_bwd" else st["Y"]
    out = torch.zeros(T, rows.shape[1], dtype=torch.float64, device=rows.device)
    dw = torch.empty(T, k, dtype=torch.float64, device=rows.device)
    for j in range(k):
        picked = rows[idx[:, j]].double()
        out += w[:, j, None] * picked
        if op == "permute_bwd" and st["weighted"]:
            dw[:, j] = (picked * st["X"].double()).sum(1)
    if op == "unpermute":
        return [out if st["base"] is None else out + st["base"].double()]
    return [out] + ([dw.reshape(-1)] if st["weighted"] else [])
