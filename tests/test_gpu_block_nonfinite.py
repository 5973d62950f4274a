"""Infinities and NaN through the block-scaled quantizing operators: what the
definition gives for them, and nothing for their neighbours."""

import numpy as np
import pytest

from block_bound import SILU_REL, U
from oracle import codecs as C
from test_gpu_block import case, host, rows_bits, up

block = pytest.importorskip("weight_only_bit_dequant_amd.block")

pytestmark = pytest.mark.gpu

INF, NAN = np.inf, np.nan


# (gate, up): what silu(gate) * up = gate / (1 + exp(-gate)) * up is
GATES = [(INF, 2.0, INF), (INF, -2.0, -INF), (INF, INF, INF), (INF, 0.0, NAN), (-INF, 2.0, NAN), (-INF, 0.0, NAN),
         (-INF, INF, NAN), (NAN, 1.0, NAN), (1.0, INF, INF), (1.0, -INF, -INF), (-1.0, INF, -INF), (0.0, INF, NAN),
         (1.0, NAN, NAN), (NAN, INF, NAN), (89.0, -INF, -INF)]


def test_gate_nonfinite_pairs():
    case("gate non-finite pairs")
    M, K = len(GATES), 384
    gu = rows_bits(M, 2 * K, 3)
    xq, xs = block.silu_mul_quantize(up(gu))
    want_q, want_s = host(xq), host(xs)
    y = C.bf16_to_f32(gu).copy()
    for m, (g, u, _) in enumerate(GATES):
        at = 128 + 8 * m % 128 + m % 8  # in the second block, in different lanes and elements
        y[m, at], y[m, K + at] = g, u
    xq, xs = block.silu_mul_quantize(up(C.f32_to_bf16(y)))
    codes, scales = host(xq), host(xs)
    for m, (g, u, v) in enumerate(GATES):
        assert np.isnan(scales[m, 1]) if np.isnan(v) else scales[m, 1] == INF, (g, u, scales[m, 1])
    # the other blocks of the rows
    keep = np.r_[0:128, 256:384]
    assert np.array_equal(codes[:, keep], want_q[:, keep]) and np.array_equal(scales[:, [0, 2]], want_s[:, [0, 2]])


def test_gate_every_bf16():
    """silu of every bf16 value in a block of its own, up = 1: the block's scale is |silu| / 448."""
    case("gate every bf16")
    gu = np.zeros((65536, 32), np.uint16)
    gu[:, 0], gu[:, 16] = np.arange(65536), C.f32_to_bf16(np.ones(1, np.float32))[0]
    xs = host(block.silu_mul_quantize(up(gu))[1])[:, 0].astype(np.float64)
    g = C.bf16_to_f32(gu[:, 0]).astype(np.float64)
    with np.errstate(all="ignore"):
        y = g / (1.0 + np.exp(-g))
    want = np.abs(y) / 448.0
    assert np.array_equal(np.isnan(xs), np.isnan(want)) and np.array_equal(np.isinf(xs), np.isinf(want))
    ok = np.isfinite(want)
    want = np.maximum(want[ok], 2.0**-126)
    assert (np.abs(xs[ok] - want) <= (SILU_REL + 4 * U) * want).all()


def check_infinite_block(codes, scale, y):
    """A block with infinities in y: finite values over an infinite scale are zeros of their sign, the infinities NaN."""
    assert scale == INF
    inf = np.isinf(y)
    assert inf.any() and (codes[inf] & 0x7F == 0x7F).all()
    assert np.array_equal(codes[~inf], np.where(np.signbit(y[~inf]), 0x80, 0))


def test_codes_of_infinite_and_nan_blocks():
    case("codes of infinite and NaN blocks")
    M, K = 6, 400
    x = C.bf16_to_f32(rows_bits(M, K, 8, spread=True)).copy()
    x[1, 5], x[2, [130, 200, 255]], x[3, 399], x[4, 300] = INF, [-INF, 0.0, INF], -INF, NAN
    x[2, 131] = -0.0
    b = C.f32_to_bf16(x)
    x = C.bf16_to_f32(b)
    # rows
    codes, scales = [host(t) for t in block.quantize_act(up(b))]
    for m, kb in ((1, 0), (2, 1), (3, 3)):
        at = slice(128 * kb, min(K, 128 * kb + 128))
        check_infinite_block(codes[m, at], scales[m, kb], x[m, at])
    assert np.isnan(scales[4, 2]) and (codes[4, 256:384] & 0x7F == 0x7F).all()
    # a weight: one scale for all rows of a block
    q = block.quantize_weight(up(np.delete(b, 4, axis=0)))
    w, codes, scales = np.delete(x, 4, axis=0), host(q["codes"]), host(q["scales"])
    for kb in (0, 1, 3):
        at = slice(128 * kb, min(K, 128 * kb + 128))
        check_infinite_block(codes[:, at].ravel(), scales[0, kb], w[:, at].ravel())
    # gate: gate * up leaves fp32
    gu = np.concatenate([np.full((1, 16), 3e38), np.r_[1e10, -1e10, np.linspace(-0.9, 0.9, 14)][None]], axis=1)
    gu = C.f32_to_bf16(gu.astype(np.float32))
    f = C.bf16_to_f32(gu)
    with np.errstate(over="ignore"):
        y = f[0, :16] * f[0, 16:]  # silu(3e38) = 3e38
    codes, scales = [host(t) for t in block.silu_mul_quantize(up(gu))]
    check_infinite_block(codes[0], scales[0, 0], y)
    # norm: an infinite gain
    g = C.bf16_to_f32(rows_bits(1, K, 9)).copy()
    g[0, 140] = -INF
    x = rows_bits(M, K, 10)
    codes, scales = [host(t) for t in block.add_rmsnorm_quantize(up(x), up(C.f32_to_bf16(g)[0]))[:2]]
    y = np.sign(C.bf16_to_f32(x)) * g
    for m in range(M):
        check_infinite_block(codes[m, 128:256], scales[m, 1], y[m, 128:256])
        assert np.isfinite(scales[m, [0, 2, 3]]).all()
