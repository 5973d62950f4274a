"""The 8-bit integer operators and the experts' routing as they are used: the
module swap, the mixture-of-experts example, a layer's run of all of them against
float64 and in a graph with a padded batch."""

import importlib.util
import os

import numpy as np
import pytest
import torch

pytest.importorskip("weight_only_bit_dequant_amd.int8")

from int8_bound import SILU_REL, U, rounded
from oracle import experts as X
from weight_only_bit_dequant_amd import block, experts, int8, modules

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# A code's rounding is off by at most half a step of amax / 127, evenly spread: amax / 127 / sqrt(12) in the mean.  Rows of up
# to 2048 normal values have amax <= 4.6 of their deviation: 0.0105 of it; a product of two quantized operands sqrt(2) times
# that.  A gated row's values are products of normal ones, their largest up to 15 of the deviation: 0.034.  Two products of
# quantized operands and the quantized activation between them: sqrt(2 * 0.0149^2 + 0.034^2) = 0.04; twice that bounds a
# layer of two.
TWO = 0.08


@torch.no_grad()
def test_module_swap():
    print("[case] int8 module swap", flush=True)
    torch.manual_seed(0)
    model = torch.nn.Sequential(torch.nn.Linear(528, 640), torch.nn.ReLU(), torch.nn.Sequential(torch.nn.Linear(640, 200, bias=False)))
    model = model.to(DEV, torch.bfloat16)
    x = torch.randn(3, 7, 528, device=DEV, dtype=torch.bfloat16)
    want = model.double()(x.double()).float()
    model.to(torch.bfloat16)
    modules.quantize_linear_int8(model)
    assert isinstance(model[0], modules.Int8Linear) and isinstance(model[2][0], modules.Int8Linear)
    got = model(x)
    assert got.shape == (3, 7, 200) and got.dtype == torch.bfloat16
    assert float((got.float() - want).norm() / want.norm()) < TWO
    # the module is the two calls
    x2 = x.reshape(-1, 528)
    y = int8.linear(*int8.quantize_act(x2), model[0].q, model[0].bias)
    assert torch.equal(y, model[0](x).reshape(-1, 640))


@pytest.mark.parametrize("tokens,hidden,inner,E,top", [(1, 256, 144, 8, 2), (40, 528, 272, 6, 3), (300, 1024, 512, 4, 2)])
def test_moe_example(tokens, hidden, inner, E, top):
    print(f"[case] int8 moe {tokens} {hidden} {inner} {E} {top}", flush=True)
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    moe = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(moe)
    layer, weights, draw = moe.random_layer(hidden, inner, E, top, seed=tokens, ops=int8)
    x, residual = draw(tokens, hidden), draw(tokens, hidden, scale=4.0)
    out, h = layer(x, residual)
    want, want_h = moe.float_layer(layer, weights, x, residual)
    assert torch.equal(h, want_h.to(torch.bfloat16))
    assert float((out.float() - want).norm() / want.norm()) < TWO
    again, _ = layer(x, residual)
    assert torch.equal(out, again)


def make(M, E, top, hidden, inner, seed):
    g = torch.Generator().manual_seed(seed)

    def draw(*shape, scale=1.0):
        return (scale * torch.randn(*shape, generator=g)).to(torch.bfloat16).to(DEV)

    return {"x": draw(M, hidden), "logits": torch.randn(M, E, generator=g).to(DEV), "bias": 0.1 * torch.randn(E, generator=g).to(DEV),
            "shared": draw(M, hidden), "gu": draw(E, 2 * inner, hidden, scale=hidden**-0.5), "down": draw(E, hidden, inner, scale=inner**-0.5)}


def run(ops, d, q, top, valid):
    r = experts.route(d["logits"], top, score="sigmoid", bias=d["bias"], groups=4, keep_groups=2, group_score="top2", valid=valid)
    xq, xs = ops.quantize_act(d["x"])
    gu = ops.grouped_linear(xq, xs, q[0], r.offsets, rows=r.rows)
    hq, hs = ops.silu_mul_quantize(gu)
    z = ops.grouped_linear(hq, hs, q[1], r.offsets)
    return r, (xq, xs), gu, (hq, hs), z, experts.combine(z, r.places, r.weights, base=d["shared"])


@pytest.mark.parametrize("M,E,top,hidden,inner", [(1, 8, 2, 256, 128), (23, 16, 4, 272, 144), (400, 32, 3, 528, 272)])
def test_layer_step_by_step(M, E, top, hidden, inner):
    """Every operator's output from the one before it, against float64."""
    print(f"[case] int8 layer {M} {E} {top} {hidden} {inner}", flush=True)
    d = make(M, E, top, hidden, inner, M)
    q = int8.quantize_weight(d["gu"]), int8.quantize_weight(d["down"])
    valid = torch.rand(M, generator=torch.Generator().manual_seed(M)) < 0.8
    valid[0] = True
    r, x, gu, h, z, out = run(int8, d, q, top, valid.to(DEV))
    ids, w, off, rows, places = X.route(d["logits"].double().cpu().numpy(), top, valid=valid.numpy(), kind="sigmoid", bias=d["bias"].cpu().numpy(),
                                        groups=4, keep=2, pairs=True)
    n = int(off[-1])
    assert np.array_equal(r.ids.cpu().numpy(), ids) and np.array_equal(r.offsets.cpu().numpy(), off) and np.array_equal(r.places.cpu().numpy(), places)
    assert np.array_equal(r.rows.cpu().numpy()[:n], rows)

    def product(codes, scales, q, src):
        out = torch.empty(n, q["codes"].shape[1], dtype=torch.float64, device=DEV)
        for e in range(E):
            a, b = int(off[e]), int(off[e + 1])
            at = src[a:b]
            out[a:b] = (codes[at].double() @ q["codes"][e].double().T) * scales[at].double()[:, None] * q["scales"][e].double()
        return out.cpu().numpy()

    for got, ref in ((gu, product(*x, q[0], r.rows.long())), (z, product(*h, q[1], torch.arange(n, device=DEV)))):
        assert (np.abs(got[:n].double().cpu().numpy() - ref) <= rounded(ref, 4 * U * np.abs(ref))).all()
    g, u = gu[:n].double().chunk(2, dim=-1)
    y = (g / (1 + torch.exp(-g)) * u).cpu().numpy()
    s = h[1][:n].double().cpu().numpy()[:, None]
    assert (np.abs(h[0][:n].double().cpu().numpy() * s - y) <= s / 2 + (SILU_REL + 8 * U) * np.abs(y)).all()
    ref, size = X.combine(z.double().cpu().numpy(), places, r.weights.double().cpu().numpy(), d["shared"].double().cpu().numpy())
    assert (np.abs(out.double().cpu().numpy() - ref) <= rounded(ref, (top + 1) * U * (1 + 2.0**-14) * size)).all()
    none = torch.from_numpy((ids < 0).all(1)).to(DEV)
    assert torch.equal(out[none], d["shared"][none])


@pytest.mark.parametrize("ops", [int8, block], ids=["int8", "fp8"])
def test_layer_in_a_graph_with_a_padded_batch(ops):
    """One graph, replayed with other inputs and another number of tokens, against eager calls between the replays."""
    M, E, top, hidden, inner = 150, 16, 3, 528, 272
    print(f"[case] layer in a graph {ops.__name__}", flush=True)
    d = make(M, E, top, hidden, inner, 5)
    q = ops.quantize_weight(d["gu"]), ops.quantize_weight(d["down"])
    valid = torch.ones(M, dtype=torch.bool, device=DEV)
    run(ops, d, q, top, valid)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, _, _, _, _, out = run(ops, d, q, top, valid)
    for step, tokens in enumerate((150, 1, 64, 0, 149)):
        other = make(M, E, top, hidden, inner, 10 + step)
        d["x"].copy_(other["x"])
        d["logits"].copy_(other["logits"])
        valid.copy_(torch.arange(M, device=DEV) < tokens)
        out.zero_()
        graph.replay()
        got, ids, total = out.clone(), r.ids.clone(), int(r.offsets[E])
        want = run(ops, d, q, top, valid)
        assert torch.equal(got, want[5]) and torch.equal(ids, want[0].ids) and total == tokens * top
        assert torch.equal(got[tokens:], d["shared"][tokens:])
