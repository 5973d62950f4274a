"""The block-scaled operators as they are used: the module swap and the
mixture-of-experts example, against float layers."""

import importlib.util
import os

import pytest
import torch

pytest.importorskip("weight_only_bit_dequant_amd.block")

from weight_only_bit_dequant_amd import block, modules

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# An E4M3 rounding is off by at most 2^-4 of the value and spread over its step: 0.027 of a normal value in the mean;
# a product of two quantized operands sqrt(2) times that.  Two products and the quantized activation between them make
# three such errors, summed as squares 0.066; twice that bounds a layer of two.
TWO = 0.13


@torch.no_grad()
def test_module_swap():
    print("[case] module swap", flush=True)
    torch.manual_seed(0)
    model = torch.nn.Sequential(torch.nn.Linear(528, 640), torch.nn.ReLU(), torch.nn.Sequential(torch.nn.Linear(640, 200, bias=False)))
    model = model.to(DEV, torch.bfloat16)
    x = torch.randn(3, 7, 528, device=DEV, dtype=torch.bfloat16)
    want = model.double()(x.double()).float()
    model.to(torch.bfloat16)
    modules.quantize_linear_fp8_block(model)
    assert isinstance(model[0], modules.BlockFP8Linear) and isinstance(model[2][0], modules.BlockFP8Linear)
    got = model(x)
    assert got.shape == (3, 7, 200) and got.dtype == torch.bfloat16
    assert float((got.float() - want).norm() / want.norm()) < TWO
    # the module is the two calls
    x2 = x.reshape(-1, 528)
    y = block.linear(*block.quantize_act(x2), model[0].q, model[0].bias)
    assert torch.equal(y, model[0](x).reshape(-1, 640))


@pytest.mark.parametrize("tokens,hidden,inner,experts,top", [(1, 256, 144, 8, 2), (40, 528, 272, 6, 3), (300, 1024, 512, 4, 2)])
def test_moe_example(tokens, hidden, inner, experts, top):
    print(f"[case] moe {tokens} {hidden} {inner} {experts} {top}", flush=True)
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    moe = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(moe)
    layer, weights, draw = moe.random_layer(hidden, inner, experts, top, seed=tokens)
    x, residual = draw(tokens, hidden), draw(tokens, hidden, scale=4.0)
    out, h = layer(x, residual)
    want, want_h = moe.float_layer(layer, weights, x, residual)
    assert torch.equal(h, want_h.to(torch.bfloat16))
    assert float((out.float() - want).norm() / want.norm()) < TWO
    again, _ = layer(x, residual)
    assert torch.equal(out, again)
