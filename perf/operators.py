"""The block-scaled FP8 operators as they are measured: cases, inputs, one pass, its floor, its exact value.

A block-scaled tensor holds E4M3 codes and one fp32 scale for each 128 codes along K (activations: of one row;
weights: of 128 rows).  Four operators work on it:

  norm     h = x (+ residual); y = h * rsqrt(mean h^2 + eps) * gain; y leaves as codes and scales, the new residual
           (and y itself, where asked) in bf16
  gate     y = silu(gate) * up of one [M, 2 I] tensor; y leaves as codes and scales
  linear   Y = deq(X) . deq(W)^T (+ bias) in bf16, from codes, or from bf16 rows that the call quantizes first
  grouped  the same product for E experts: sorted rows offsets[e] .. offsets[e + 1] meet expert e's weight; the rows are
           read where the router's order points

The quantizer: s = max(max|y| / 448, 2^-126) of each block, code = E4M3(clamp(y / s, +-448)), nearest even.

With `own` false, run() computes the plain forms (fp32 torch operations, rounded once); with `own` true it makes the
calls of weight_only_bit_dequant_amd.block.
"""

import math

import torch

own = False

BLK = 128
EPS = 1e-5
TINY = 2.0**-126
DEV = "cuda"
F8 = torch.float8_e4m3fn


def listed():
    return [
        # one token's residual stream before a decoder layer's projections: launch latency
        dict(name="norm 1x4096", op="norm", M=1, K=4096, residual=True, bf16=False),
        # an odd batch, a width that ends inside a scale block, y kept for a router
        dict(name="norm 777x2896", op="norm", M=777, K=2896, residual=True, bf16=True),
        # a long prompt: the memory stream
        dict(name="norm 16384x8192", op="norm", M=16384, K=8192, residual=True, bf16=False),
        # the gated activation of a decode batch
        dict(name="gate 64x2048", op="gate", M=64, I=2048),
        # the gated activation of a long prompt
        dict(name="gate 8192x8192", op="gate", M=8192, I=8192),
        # this repository's layer, one token: the weight's stream
        dict(name="linear 1x4096x3072", op="linear", M=1, N=4096, K=3072, bias=True, act="codes"),
        # the same layer at its benchmark's 32 rows, from bf16 rows (quantized in the pass)
        dict(name="linear 32x4096x3072 bf16", op="linear", M=32, N=4096, K=3072, bias=True, act="bf16"),
        # a mixed serving batch: rows and columns that end inside a tile
        dict(name="linear 300x6152x4096", op="linear", M=300, N=6152, K=4096, bias=False, act="codes"),
        # a long prompt on a wide layer: the matrix cores
        dict(name="linear 8192x8192x8192", op="linear", M=8192, N=8192, K=8192, bias=False, act="codes"),
        # a decode batch over many experts: few rows each, some experts without any
        dict(name="grouped 16x4 of 32", op="grouped", tokens=16, top=4, E=32, N=2048, K=2048),
        # a mixed batch over many experts with uneven loads
        dict(name="grouped 500x4 of 64", op="grouped", tokens=500, top=4, E=64, N=1536, K=2048),
        # a prompt over few wide experts
        dict(name="grouped 4096x2 of 8", op="grouped", tokens=4096, top=2, E=8, N=4096, K=4096),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(round(v / step)) * step)


def draw(rng):
    op = rng.choice(["norm", "gate", "linear", "linear", "grouped", "grouped"])
    if op == "norm":
        # any width of whole 16-byte rows of codes
        return dict(op=op, M=_log(rng, 1, 16384), K=_log(rng, 512, 8192, 16), residual=rng.random() < 0.7, bf16=rng.random() < 0.3)
    if op == "gate":
        return dict(op=op, M=_log(rng, 1, 8192), I=_log(rng, 256, 8192, 16))
    if op == "linear":
        # half the depths are whole scale blocks; widths are whole output vectors but for a fifth of them
        return dict(op=op, M=_log(rng, 1, 8192), N=_log(rng, 512, 8192, 1 if rng.random() < 0.2 else 8),
                    K=_log(rng, 512, 8192, rng.choice([16, 128])), bias=rng.random() < 0.5, act=rng.choice(["codes", "codes", "bf16"]))
    E, top = rng.choice([4, 8, 16, 32, 64, 128]), rng.choice([1, 2, 4])
    N, K = _log(rng, 256, 4096, 8), _log(rng, 256, 4096, rng.choice([16, 128]))
    while E * N * K > 1 << 28:
        E //= 2
    return dict(op=op, tokens=_log(rng, 1, 8192 // top * 2), top=min(top, E), E=E, N=N, K=K)


# ---------------------------------------------------------------- inputs


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _acts(g, M, K):
    """bf16 activations as a model's: normal, a few channels many times larger than the rest."""
    x = torch.randn(M, K, generator=g, device=DEV)
    x *= 1 + 15 * (torch.rand(K, generator=g, device=DEV) < 0.01)
    return x.to(torch.bfloat16)


def _codes(y):
    """Codes and scales of fp32 rows y: one scale for each 128 along the last dimension."""
    n, K = y.shape
    kb = -(-K // BLK)
    p = torch.nn.functional.pad(y, (0, kb * BLK - K)).view(n, kb, BLK)
    s = (p.abs().amax(-1) / 448).clamp_min(TINY)
    c = (p / s[..., None]).clamp(-448, 448).to(F8)
    return c.view(torch.uint8).view(n, kb * BLK)[:, :K].contiguous(), s


def _weight(g, E, N, K):
    """E weights [N, K] of normal values in codes, one scale for each 128 x 128 block: the library's weight dict."""
    nb, kb = -(-N // BLK), -(-K // BLK)
    codes = torch.empty(E, N, K, dtype=torch.uint8, device=DEV)
    scales = torch.empty(E, nb, kb, device=DEV)
    for e in range(E):
        w = torch.randn(N, K, generator=g, device=DEV) / math.sqrt(K)
        p = torch.nn.functional.pad(w, (0, kb * BLK - K, 0, nb * BLK - N)).view(nb, BLK, kb, BLK)
        scales[e] = (p.abs().amax((1, 3)) / 448).clamp_min(TINY)
        c = (p / scales[e][:, None, :, None]).clamp(-448, 448).to(F8).view(torch.uint8)
        codes[e] = c.view(nb * BLK, kb * BLK)[:N, :K]
    return {"E": E, "N": N, "K": K, "codes": codes, "scales": scales}


def _codes_out(M, K):
    """Output buffers of a quantizing operator, as a serving loop keeps them."""
    return torch.empty(M, K, dtype=torch.uint8, device=DEV), torch.empty(M, -(-K // BLK), device=DEV)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    if op == "norm":
        M, K = case["M"], case["K"]
        st = {"x": _acts(g, M, K), "gain": (1 + 0.2 * torch.randn(K, generator=g, device=DEV)).to(torch.bfloat16),
              "residual": 4 * _acts(g, M, K) if case["residual"] else None, "out": _codes_out(M, K)}
        st["h"] = torch.empty_like(st["x"]) if case["residual"] else None
        st["y"] = torch.empty_like(st["x"]) if case["bf16"] else None
    elif op == "gate":
        st = {"x": _acts(g, case["M"], 2 * case["I"]), "out": _codes_out(case["M"], case["I"])}
    elif op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        st = {"q": _weight(g, 1, N, K), "bias": torch.randn(N, generator=g, device=DEV).to(torch.bfloat16) if case["bias"] else None}
        st["q"]["codes"], st["q"]["scales"] = st["q"]["codes"][0], st["q"]["scales"][0]
        x = _acts(g, M, K)
        if case["act"] == "bf16":
            st["x"], st["out"] = x, _codes_out(M, K)
        else:
            st["xq"], st["xs"] = _codes(x.float())
        st["Y"] = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    else:
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
    st["op"] = op
    return st


# ---------------------------------------------------------------- one pass


def _spread(s, n, dim):
    """Block scales along `dim` as one for each of n elements."""
    return s.repeat_interleave(BLK, dim=dim).narrow(dim, 0, n)


def _deq_rows(xq, xs):
    return xq.view(F8).float() * _spread(xs, xq.shape[-1], -1)


def _deq_weight(q):
    c, s = q["codes"], q["scales"]
    return c.view(F8).float() * _spread(_spread(s, c.shape[-1], -1), c.shape[-2], -2)


def _plain(st):
    op = st["op"]
    if op == "norm":
        h = st["x"].float() if st["residual"] is None else st["x"].float() + st["residual"].float()
        y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * st["gain"].float()
        return [*_codes(y), None if st["residual"] is None else h.to(torch.bfloat16), None if st["y"] is None else y.to(torch.bfloat16)]
    if op == "gate":
        gate, up = st["x"].float().chunk(2, dim=-1)
        return list(_codes(gate / (1 + torch.exp(-gate)) * up))
    xq, xs = _codes(st["x"].float()) if "x" in st else (st["xq"], st["xs"])
    if op == "linear":
        y = _deq_rows(xq, xs) @ _deq_weight(st["q"]).t()
        return [(y if st["bias"] is None else y + st["bias"].float()).to(torch.bfloat16)]
    # sorted row t is row t - offsets[e] of its expert e's padded block; one batched product over the experts
    rows, off = st["rows"].long(), st["offsets"].long()
    t = torch.arange(rows.numel(), device=DEV)
    e = torch.searchsorted(off[1:], t, right=True)
    at = e * st["most"] + t - off[e]
    x = _deq_rows(xq, xs)[rows]
    padded = torch.zeros(st["q"]["E"] * st["most"], x.shape[1], device=DEV).index_copy(0, at, x)
    y = torch.bmm(padded.view(st["q"]["E"], st["most"], -1), _deq_weight(st["q"]).transpose(1, 2))
    return [y.reshape(-1, y.shape[-1])[at].to(torch.bfloat16)]


def _own(st):
    from weight_only_bit_dequant_amd import block

    op = st["op"]
    if op == "norm":
        return list(block.add_rmsnorm_quantize(st["x"], st["gain"], EPS, residual=st["residual"], out=st["out"], residual_out=st["h"], y_out=st["y"]))
    if op == "gate":
        return list(block.silu_mul_quantize(st["x"], out=st["out"]))
    if op == "linear":
        xq, xs = block.quantize_act(st["x"], out=st["out"]) if "x" in st else (st["xq"], st["xs"])
        return [block.linear(xq, xs, st["q"], st["bias"], out=st["Y"])]
    return [block.grouped_linear(st["xq"], st["xs"], st["q"], st["offsets"], rows=st["rows"], out=st["Y"])]


def run(state):
    out = _own(state) if own else _plain(state)
    if state["op"] in ("norm", "gate"):
        out[0] = out[0].view(F8)  # the codes as the E4M3 values that they stand for
    return out


# ---------------------------------------------------------------- floors and exact values


def work(case):
    op = case["op"]
    if op == "norm":
        M, K = case["M"], case["K"]
        per = 2 + 1 + 4 * case["residual"] + 2 * case["bf16"]  # x, codes; residual in and out; y
        return {"bytes": M * K * per + 4 * M * -(-K // BLK) + 2 * K, "flops": 8 * M * K}
    if op == "gate":
        M, K = case["M"], case["I"]
        return {"bytes": M * K * 5 + 4 * M * -(-K // BLK), "flops": 8 * M * K}
    N, K = case["N"], case["K"]
    w = N * K + 4 * -(-N // BLK) * -(-K // BLK)
    if op == "linear":
        M = case["M"]
        x = 2 * M * K if case["act"] == "bf16" else M * K + 4 * M * -(-K // BLK)
        return {"bytes": x + w + 2 * M * N + 2 * N * case["bias"], "flops": 2 * M * N * K}
    M, E, T = case["tokens"], case["E"], case["tokens"] * case["top"]
    used = E * (1 - (1 - case["top"] / E) ** M)  # experts that an even router would reach
    return {"bytes": M * (K + 4 * -(-K // BLK)) + used * w + 2 * T * N + 4 * T + 4 * E, "flops": 2 * T * N * K}


def _round_e4m3(v):
    """float64 values rounded to E4M3, nearest even: steps of 2^(e - 3), e at least -6."""
    step = torch.exp2(torch.frexp(v).exponent.clamp_min(-5).double() - 4)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _exact_codes(y):
    """(code values, scales) of float64 rows y."""
    n, K = y.shape
    kb = -(-K // BLK)
    at = torch.arange(K, device=y.device) // BLK
    top = torch.zeros(n, kb, dtype=torch.float64, device=y.device)
    top.scatter_reduce_(1, at.expand(n, K), y.abs(), "amax")
    s = torch.clamp(top / 448.0, min=TINY)
    return _round_e4m3(y / s[:, at]), s


def exact(case, seed):
    st = prepare(case, seed)
    op = st["op"]
    if op == "norm":
        h = st["x"].double()
        if st["residual"] is not None:
            h += st["residual"].double()
        y = st["gain"].double() * h / torch.sqrt(torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / h.shape[1] + EPS)
        return [*_exact_codes(y), None if st["residual"] is None else h, None if st["y"] is None else y]
    if op == "gate":
        n = st["x"].shape[1] // 2
        gate = st["x"][:, :n].double()
        return list(_exact_codes(gate * torch.sigmoid(gate) * st["x"][:, n:].double()))
    N, K = case["N"], case["K"]
    n_at, k_at = torch.arange(N, device=DEV) // BLK, torch.arange(K, device=DEV) // BLK
    if "x" in st:
        c, s = _exact_codes(st["x"].double())
        x = c * s[:, k_at]
    else:
        x = st["xq"].view(F8).double() * st["xs"].double()[:, k_at]
    q = st["q"]
    if op == "linear":
        y = x @ (q["codes"].view(F8).double() * q["scales"].double()[n_at][:, k_at]).T
        return [y if st["bias"] is None else y + st["bias"].double()]
    y = torch.empty(st["Y"].shape, dtype=torch.float64, device=DEV)
    off = st["offsets"].tolist()
    for e in range(case["E"]):
        w = q["codes"][e].view(F8).double() * q["scales"][e].double()[n_at][:, k_at]
        y[off[e] : off[e + 1]] = x[st["rows"][off[e] : off[e + 1]].long()] @ w.T
    return [y]
