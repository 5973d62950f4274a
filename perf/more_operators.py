"""Integer products and the experts' routing as they are measured: cases, inputs, one pass, its floor, its exact value.

Rows in 8-bit integers hold codes in [-127, 127] and one fp32 scale a row (activations: of a token; weights: of an output
channel): s = max(max|y| / 127, 2^-126), code = rint(y / s).

  linear   Y = (Xq . Wq^T) * Xs * Ws (+ bias) in bf16, from codes, from bf16 rows that the call quantizes first, or from
           [gate | up] rows whose silu(gate) * up it quantizes first
  grouped  the same product for E experts: sorted rows offsets[e] .. offsets[e + 1] meet expert e's weight; the rows are
           read where the router's order points
  route    logits -> experts of each token (softmax or sigmoid scores, a bias for the choice alone, groups, top-k,
           weights renormalised), and the order that sorts all choices by expert
  combine  out = base + sum of each token's choices' rows times their weights, in bf16

With `own` false, run() computes the plain forms (32 or 64 bit torch operations, rounded once); with `own` true it makes
the calls of weight_only_bit_dequant_amd.int8 and weight_only_bit_dequant_amd.experts.
"""

import math

import torch

own = False

TINY = 2.0**-126
DEV = "cuda"
INF = float("inf")


def listed():
    return [
        # one token through a square layer: the weight's stream and the call's latency
        dict(name="linear 1x4096x4096", op="linear", M=1, N=4096, K=4096, bias=True, act="codes"),
        # a mixed serving batch from bf16 rows: an odd width, a depth that ends inside a step
        dict(name="linear 333x5003x2064 bf16", op="linear", M=333, N=5003, K=2064, bias=True, act="bf16"),
        # a prompt's down projection, from the gate and up projections' output
        dict(name="linear 4096x2048x5632 gate", op="linear", M=4096, N=2048, K=5632, bias=False, act="gate"),
        # a long prompt on a wide layer: the matrix cores
        dict(name="linear 8192x8192x8192", op="linear", M=8192, N=8192, K=8192, bias=False, act="codes"),
        # a decode batch over many experts: few rows each, some experts without any
        dict(name="grouped 12x4 of 64", op="grouped", tokens=12, top=4, E=64, N=1408, K=2048),
        # a mixed batch over many experts with uneven loads
        dict(name="grouped 700x4 of 64", op="grouped", tokens=700, top=4, E=64, N=1536, K=2048),
        # a prompt over few wide experts
        dict(name="grouped 4096x2 of 8", op="grouped", tokens=4096, top=2, E=8, N=4096, K=4096),
        # one token's choice: launch latency
        dict(name="route 1 of 128", op="route", M=1, E=128, top=8, score="softmax", bias=False, groups=1, keep=1, pair=False, renorm=True, padded=False, bits=32),
        # a padded serving batch, bf16 logits, a number of experts that fills no vector, weights left as they are
        dict(name="route 900 of 60 bf16", op="route", M=900, E=60, top=4, score="softmax", bias=False, groups=1, keep=1, pair=False, renorm=False, padded=True, bits=16),
        # a long prompt over many experts: sigmoid scores, a balancing bias, the best 4 of 8 groups
        dict(name="route 16384 of 256 grouped", op="route", M=16384, E=256, top=8, score="sigmoid", bias=True, groups=8, keep=4, pair=True, renorm=True, padded=False, bits=32),
        # a decode batch's results on their way back to the tokens
        dict(name="combine 16x4x2048", op="combine", M=16, top=4, N=2048, base=True, padded=False),
        # a long prompt's: the memory stream
        dict(name="combine 8192x8x4096", op="combine", M=8192, top=8, N=4096, base=True, padded=False),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(round(v / step)) * step)


def draw(rng):
    op = rng.choice(["linear", "linear", "grouped", "grouped", "route", "route", "combine"])
    if op == "linear":
        # half the depths are whole steps; widths are whole output vectors but for a fifth of them
        return dict(op=op, M=_log(rng, 1, 8192), N=_log(rng, 512, 8192, 1 if rng.random() < 0.2 else 8),
                    K=_log(rng, 512, 8192, rng.choice([16, 128])), bias=rng.random() < 0.5, act=rng.choice(["codes", "codes", "bf16", "gate"]))
    if op == "grouped":
        E, top = rng.choice([4, 8, 16, 32, 64, 128]), rng.choice([1, 2, 4])
        N, K = _log(rng, 256, 4096, 8), _log(rng, 256, 4096, rng.choice([16, 128]))
        while E * N * K > 1 << 28:
            E //= 2
        return dict(op=op, tokens=_log(rng, 1, 8192 // top * 2), top=min(top, E), E=E, N=N, K=K)
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        E = groups * rng.choice([2, 8, 15, 16, 20, 32]) if groups > 1 else rng.choice([8, 16, 60, 64, 128, 160, 256])
        keep = max(1, groups // 2)
        top = min(rng.choice([1, 2, 4, 6, 8]), E // groups * keep)
        score, bias = rng.choice([("softmax", False), ("softmax", False), ("sigmoid", True), ("sigmoid", False), ("softmax", True)])
        return dict(op=op, M=_log(rng, 1, 16384), E=E, top=top, score=score, bias=bias, groups=groups, keep=keep, pair=groups > 1 and bias,
                    renorm=rng.random() < 0.7, padded=rng.random() < 0.3, bits=rng.choice([32, 32, 16]))
    top = rng.choice([1, 2, 4, 6, 8])
    return dict(op=op, M=_log(rng, 1, 8192), top=top, N=_log(rng, 256, 4096, 1 if rng.random() < 0.2 else 8), base=rng.random() < 0.5, padded=rng.random() < 0.3)


# ---------------------------------------------------------------- inputs


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _acts(g, M, K):
    """bf16 activations as a model's: normal, a few channels several times larger than the rest."""
    x = torch.randn(M, K, generator=g, device=DEV)
    x *= 1 + 7 * (torch.rand(K, generator=g, device=DEV) < 0.01)
    return x.to(torch.bfloat16)


def _codes(y):
    """Codes and scales of fp32 rows y [..., K]."""
    s = (y.abs().amax(-1) / 127).clamp_min(TINY)
    return torch.round(y / s[..., None]).to(torch.int8), s


def _weight(g, E, N, K):
    """E weights [N, K] of normal values in codes, one scale a channel: the library's weight dict."""
    codes = torch.empty(E, N, K, dtype=torch.int8, device=DEV)
    scales = torch.empty(E, N, device=DEV)
    for e in range(E):
        codes[e], scales[e] = _codes(torch.randn(N, K, generator=g, device=DEV) / math.sqrt(K))
    return {"E": E, "N": N, "K": K, "codes": codes, "scales": scales}


def _valid(g, M):
    """A padded batch: some of the rows, the last ones among them, hold no token."""
    v = torch.rand(M, generator=g, device=DEV) < 0.9
    v[M - M // 8 :] = False
    return v


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        st = {"q": _weight(g, 1, N, K), "bias": torch.randn(N, generator=g, device=DEV).to(torch.bfloat16) if case["bias"] else None}
        st["q"]["codes"], st["q"]["scales"] = st["q"]["codes"][0], st["q"]["scales"][0]
        st["act"] = case["act"]
        if case["act"] == "codes":
            st["xq"], st["xs"] = _codes(_acts(g, M, K).float())
        else:
            st["x"] = _acts(g, M, 2 * K if case["act"] == "gate" else K)
            # the codes' buffers, as a serving loop keeps them
            st["out"] = torch.empty(M, K, dtype=torch.int8, device=DEV), torch.empty(M, device=DEV)
        st["Y"] = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    elif op == "grouped":
        M, E, N, K, T = case["tokens"], case["E"], case["N"], case["K"], case["tokens"] * case["top"]
        # a router's choice: some experts are liked more than others
        score = torch.randn(M, E, generator=g, device=DEV) + torch.randn(E, generator=g, device=DEV)
        pick = score.topk(case["top"], dim=1).indices.reshape(-1)
        order = torch.argsort(pick, stable=True)
        count = torch.bincount(pick, minlength=E)
        offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
        offsets[1:] = count.cumsum(0)
        st = {"q": _weight(g, E, N, K), "rows": (order // case["top"]).to(torch.int32), "offsets": offsets,
              "most": int(count.max()), "Y": torch.empty(T, N, dtype=torch.bfloat16, device=DEV)}
        st["xq"], st["xs"] = _codes(_acts(g, M, K).float())
    elif op == "route":
        M, E, top = case["M"], case["E"], case["top"]
        logits = 1.5 * torch.randn(M, E, generator=g, device=DEV) + torch.randn(E, generator=g, device=DEV)
        st = {k: case[k] for k in ("E", "top", "score", "groups", "keep", "pair", "renorm")}
        st["logits"] = logits.to(torch.bfloat16 if case["bits"] == 16 else torch.float32)
        st["bias"] = 0.1 * torch.randn(E, generator=g, device=DEV) if case["bias"] else None
        st["valid"] = _valid(g, M) if case["padded"] else None
        whole = dict(dtype=torch.int32, device=DEV)
        # ids, weights, offsets, rows (those behind the last choice stay as they are), places
        st["out"] = (torch.empty(M, top, **whole), torch.empty(M, top, device=DEV), torch.empty(E + 1, **whole),
                     torch.full((M * top,), -7, **whole), torch.empty(M, top, **whole))
    else:
        M, top, N = case["M"], case["top"], case["N"]
        w = torch.rand(M, top, generator=g, device=DEV) + 0.1
        st = {"y": _acts(g, M * top, N), "weights": w / w.sum(-1, keepdim=True), "base": _acts(g, M, N) if case["base"] else None}
        st["places"] = torch.randperm(M * top, generator=g, device=DEV).to(torch.int32).view(M, top)
        if case["padded"]:
            none = ~_valid(g, M)
            st["places"][none] = -1
            st["weights"][none] = 0
        st["Y"] = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    st["op"] = op
    return st


# ---------------------------------------------------------------- one pass


def _plain_codes(st):
    if st["act"] == "codes":
        return st["xq"], st["xs"]
    y = st["x"].float()
    if st["act"] == "gate":
        gate, up = y.chunk(2, dim=-1)
        y = gate / (1 + torch.exp(-gate)) * up
    return _codes(y)


def _plain_route(st):
    l, E, top, G, bias = st["logits"].double(), st["E"], st["top"], st["groups"], st["bias"]
    M = l.shape[0]
    off = l == -INF
    # scores in 64 bits: sums with the bias that lie next to each other decide whole numbers
    if st["score"] == "softmax":
        e = torch.exp(l - l.amax(-1, keepdim=True)).masked_fill(off, 0)
        score = e / e.sum(-1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-l))
    choice = (l if bias is None and not st["pair"] else score if bias is None else score + bias.double()).masked_fill(off, -INF)
    if G > 1:
        best = choice.view(M, G, E // G).sort(dim=-1, descending=True).values
        value = best[..., 0]
        if st["pair"] and E // G > 1:
            value = value + best[..., 1].masked_fill(best[..., 1] == -INF, 0)
        rank = value.sort(dim=-1, descending=True, stable=True).indices
        kept = torch.zeros(M, G, dtype=torch.bool, device=l.device).scatter(1, rank[:, : st["keep"]], True)
        choice = choice.masked_fill(~kept.repeat_interleave(E // G, dim=1), -INF)
    value, ids = choice.sort(dim=-1, descending=True, stable=True)
    ids, none = ids[:, :top], value[:, :top] == -INF
    if st["valid"] is not None:
        none = none | ~st["valid"][:, None]
    w = score.gather(1, ids).masked_fill(none, 0)
    if st["renorm"]:
        total = w.sum(-1, keepdim=True)
        w = (w / total).masked_fill(total == 0, 0)
    ids = ids.masked_fill(none, -1)
    # the order by expert; what has none goes behind the last
    key = ids.reshape(-1).masked_fill(none.reshape(-1), E)
    order = torch.argsort(key, stable=True)
    t = torch.arange(key.numel(), device=l.device)
    offsets = torch.searchsorted(key[order], torch.arange(E + 1, device=l.device))
    rows = torch.where(t < offsets[E], order // top, st["out"][3])
    places = torch.empty_like(order).index_copy(0, order, t).view(M, top).masked_fill(none, -1)
    whole = torch.int32
    return [ids.to(whole), w.float(), offsets.to(whole), rows.to(whole), places.to(whole)]


def _plain(st):
    op = st["op"]
    if op == "route":
        return _plain_route(st)
    if op == "combine":
        none = st["places"] < 0
        z = st["y"][st["places"].long().clamp_min(0)].float().masked_fill(none[..., None], 0)
        z = (z * st["weights"][..., None]).sum(1)
        return [(z if st["base"] is None else z + st["base"].float()).to(torch.bfloat16)]
    q = st["q"]
    if op == "linear":
        xq, xs = _plain_codes(st)
        y = (xq.float() @ q["codes"].float().t()) * xs[:, None] * q["scales"]
        return [(y if st["bias"] is None else y + st["bias"].float()).to(torch.bfloat16)]
    # sorted row t is row t - offsets[e] of its expert e's padded block; one batched product over the experts
    rows, off = st["rows"].long(), st["offsets"].long()
    t = torch.arange(rows.numel(), device=DEV)
    e = torch.searchsorted(off[1:], t, right=True)
    at = e * st["most"] + t - off[e]
    x = st["xq"][rows].float() * st["xs"][rows][:, None]
    padded = torch.zeros(q["E"] * st["most"], x.shape[1], device=DEV).index_copy(0, at, x)
    y = torch.bmm(padded.view(q["E"], st["most"], -1), q["codes"].float().transpose(1, 2)) * q["scales"][:, None]
    return [y.reshape(-1, y.shape[-1])[at].to(torch.bfloat16)]


def _own(st):
    from weight_only_bit_dequant_amd import experts, int8

    op = st["op"]
    if op == "route":
        return list(experts.route(st["logits"], st["top"], score=st["score"], bias=st["bias"], groups=st["groups"], keep_groups=st["keep"],
                                  group_score="top2" if st["pair"] else "max", renormalize=st["renorm"], valid=st["valid"], out=st["out"]))
    if op == "combine":
        return [experts.combine(st["y"], st["places"], st["weights"], base=st["base"], out=st["Y"])]
    if op == "grouped":
        return [int8.grouped_linear(st["xq"], st["xs"], st["q"], st["offsets"], rows=st["rows"], out=st["Y"])]
    if st["act"] == "codes":
        xq, xs = st["xq"], st["xs"]
    elif st["act"] == "gate":
        xq, xs = int8.silu_mul_quantize(st["x"], out=st["out"])
    else:
        xq, xs = int8.quantize_act(st["x"], out=st["out"])
    return [int8.linear(xq, xs, st["q"], st["bias"], out=st["Y"])]


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- floors and exact values


def work(case):
    op = case["op"]
    if op == "route":
        M, E, top = case["M"], case["E"], case["top"]
        return {"bytes": M * E * case["bits"] // 8 + 16 * M * top + 4 * (E + 1) + 4 * E * case["bias"] + M * case["padded"], "flops": 8 * M * E}
    if op == "combine":
        M, top, N = case["M"], case["top"], case["N"]
        return {"bytes": 2 * M * N * (top + 1 + case["base"]) + 8 * M * top, "flops": 2 * M * top * N}
    N, K = case["N"], case["K"]
    w = N * K + 4 * N
    if op == "linear":
        M = case["M"]
        x = {"codes": M * K + 4 * M, "bf16": 2 * M * K, "gate": 4 * M * K}[case["act"]]
        return {"bytes": x + w + 2 * M * N + 2 * N * case["bias"], "flops": 2 * M * N * K}
    M, E, T = case["tokens"], case["E"], case["tokens"] * case["top"]
    used = E * (1 - (1 - case["top"] / E) ** M)  # experts that an even router would reach
    return {"bytes": M * (K + 4) + used * w + 2 * T * N + 4 * T + 4 * E, "flops": 2 * T * N * K}


def exact(case, seed):
    st = prepare(case, seed)
    op = st["op"]
    if op == "route":
        l, E, top, G = st["logits"].double(), st["E"], st["top"], st["groups"]
        score = torch.softmax(l, -1) if st["score"] == "softmax" else torch.sigmoid(l)
        choice = score if st["bias"] is None else score + st["bias"].double()
        if G > 1:
            value = choice.view(-1, G, E // G).topk(min(2, E // G) if st["pair"] else 1, dim=-1).values.sum(-1)
            kept = torch.zeros_like(value)
            kept.scatter_(1, value.topk(st["keep"], dim=1).indices, 1.0)
            choice = choice.where(kept.view(-1, G, 1).expand(-1, G, E // G).reshape(-1, E) > 0, torch.full_like(choice, -INF))
        w = score.gather(1, choice.topk(top, dim=1).indices)
        if st["renorm"]:
            w = w / torch.linalg.vector_norm(w, ord=1, dim=1, keepdim=True)
        if st["valid"] is not None:
            w = w * st["valid"].double().view(-1, 1)
        return [None, w, None, None, None]
    if op == "combine":
        y = torch.zeros(st["Y"].shape, dtype=torch.float64, device=DEV)
        if st["base"] is not None:
            y += st["base"]
        for j in range(case["top"]):
            at = st["places"][:, j].long()
            has = (at >= 0).nonzero().flatten()
            y.index_add_(0, has, st["y"].double().index_select(0, at[has]) * st["weights"].double()[has, j : j + 1])
        return [y]
    q = st["q"]
    if op == "linear":
        if case["act"] == "codes":
            x = st["xq"].double() * st["xs"].double().view(-1, 1)
        else:
            x = st["x"].double()
            if case["act"] == "gate":
                x = x[:, : case["K"]] * torch.sigmoid(x[:, : case["K"]]) * x[:, case["K"] :]
            step = torch.clamp(torch.linalg.vector_norm(x, ord=INF, dim=1, keepdim=True) / 127.0, min=TINY)
            x = torch.round(x / step) * step
        y = x @ (q["codes"].double() * q["scales"].double().view(-1, 1)).T
        return [y if st["bias"] is None else y + st["bias"].double()]
    y = torch.empty(st["Y"].shape, dtype=torch.float64, device=DEV)
    off = st["offsets"].tolist()
    x = st["xq"].double() * st["xs"].double().view(-1, 1)
    for e in range(case["E"]):
        w = q["codes"][e].double() * q["scales"][e].double().view(-1, 1)
        y[off[e] : off[e + 1]] = x[st["rows"][off[e] : off[e + 1]].long()] @ w.T
    return [y]
