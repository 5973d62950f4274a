"""The INT8 gate's precision over all bf16 gates, where int8_bound.py's random gates do not come.

u = 2^-24.  The kernel's silu(g) u for exp(-g) within fp32: the power of two is off by an ulp (2 u), its correction
(1 - g C) by the square that is left out, (88.72 * 4.8885e-6)^2 / 2 < 1.6 u, and one rounding; then 1 + exp(-g) (u), the
reciprocal (an ulp, 2 u), and two products (u each): 9.6 u to first order, GATE_REL with the rest.  Results below 2^-126
are off by half a subnormal step, 2^-150, at each of their roundings.  Beyond fp32's exp (g < -88.72) the result is 0."""

import numpy as np
import pytest
import torch

from int8_bound import U, check_codes
from oracle import codecs as C
from test_gpu_block import case, host, up

int8 = pytest.importorskip("weight_only_bit_dequant_amd.int8")

pytestmark = pytest.mark.gpu

GATE_REL = 10 * U


def gated(g, u):
    """float64 silu(g) u with fp32's range of exp(-g)."""
    with np.errstate(all="ignore"):
        e = np.exp(-g)
        return np.where(e > float(np.finfo(np.float32).max), np.copysign(0.0, g * u), g / (1.0 + e) * u)


@pytest.mark.parametrize("factor", [1.0, -(2.0**60), 2.0**110, 2.0**-40])
def test_gate_every_bf16(factor):
    """Every gate in a row of its own: the row's scale is max(|silu(g) up| / 127, 2^-126)."""
    case(f"int8 gate every bf16, up {factor:g}")
    gu = np.zeros((65536, 32), np.uint16)
    gu[:, 0], gu[:, 16] = np.arange(65536), C.f32_to_bf16(np.float32([factor]))[0]
    xq, xs = (host(t) for t in int8.silu_mul_quantize(up(gu)))
    g = C.bf16_to_f32(gu[:, 0]).astype(np.float64)
    y = gated(g, factor)
    bad = ~np.isfinite(g) | (np.abs(y) >= 2.0**128)
    assert np.isnan(xs[bad]).all() and (xq[bad] == 0).all()
    y, s, q = np.abs(y[~bad]), xs[~bad].astype(np.float64), xq[~bad]
    want = np.maximum(y / 127.0, 2.0**-126)
    # (the silu's half steps grow with the factor)
    off = (GATE_REL + U) * (1 + 2.0**-20) * want + 2.0**-149 * (1 + abs(factor)) / 127
    assert (np.abs(s - want) <= off).all(), (np.abs(s / want - 1) / U).max()
    above = y / 127.0 > 2.0**-125
    assert (np.abs(q[above, 0].astype(int)) == 127).all() and (q[:, 1:] == 0).all()
    assert np.array_equal(np.sign(q[above, 0]), np.sign(g[~bad][above] * factor))


def test_gate_far_negative_gates_with_large_factors():
    """silu(-87.5) 1e37 is a number of ordinary size."""
    case("int8 gate far negative")
    gu = np.zeros((1, 32), np.float32)
    gu[0, :6] = -87.0, -87.5, -88.0, -88.5, -89.0, 1.0
    gu[0, 16:22] = 1e37, 1e37, 1e37, 1e37, 1e37, 4.0
    b = C.f32_to_bf16(gu)
    y = C.bf16_to_f32(b).astype(np.float64)
    xq, xs = (host(t) for t in int8.silu_mul_quantize(up(b)))
    ok, text = check_codes(xq, xs, gated(y[:, :16], y[:, 16:]), GATE_REL)
    assert ok, text
    assert xq[0, 1] != 0 and xq[0, 4] == 0


@pytest.mark.parametrize("M,K", [(4000, 512), (300, 5632), (40, 40000)])
def test_gate_codes_over_all_gates(M, K):
    """Gates from -88.7 to 30 and small ones, factors that bring their products to like sizes."""
    case(f"int8 gate codes {M}x{K}")
    g = torch.Generator().manual_seed(M)
    gate = torch.empty(M, K).uniform_(-88.7, 30.0, generator=g)
    gate = torch.where(torch.rand(M, K, generator=g) < 0.3, torch.randn(M, K, generator=g), gate)
    gate = C.bf16_to_f32(C.f32_to_bf16(gate.numpy())).astype(np.float64)
    factor = np.clip(torch.randn(M, K, generator=g).numpy() / (gated(gate, 1.0) + (gate == 0)), -1e38, 1e38)
    gu = C.f32_to_bf16(np.concatenate([gate, factor], axis=1).astype(np.float32))
    y = C.bf16_to_f32(gu).astype(np.float64)
    xq, xs = (host(t) for t in int8.silu_mul_quantize(up(gu)))
    ok, text = check_codes(xq, xs, gated(y[:, :K], y[:, K:]), GATE_REL)
    assert ok, text
