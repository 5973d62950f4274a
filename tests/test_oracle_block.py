"""Pins of the block-scaled FP8 oracle (no GPU): closed forms, round trips and
planted mistakes."""

import numpy as np
import pytest

from oracle import block as B
from oracle import codecs as C


def bits(x):
    return C.f32_to_bf16(np.asarray(x, np.float32))


def test_quantizer_closed_forms():
    # one block whose largest magnitude is 448 * 2^-3: scale 2^-3, codes the E4M3 values of y * 8
    y = np.zeros((1, 128), np.float32)
    y[0, :4] = [56.0, -1.0, 0.125, -0.0]
    codes, s = B.quantize_rows(y)
    assert s.shape == (1, 1) and s[0, 0] == np.float32(0.125)
    assert C.e4m3_decode(codes)[0, :3].tolist() == [448.0, -8.0, 1.0] and codes[0, 3] == 0x80
    # an all-zero block: the floor scale, zero codes
    codes, s = B.quantize_rows(np.zeros((2, 32), np.float32))
    assert (codes == 0).all() and (s == np.float32(2.0**-126)).all()


def test_quantizer_error_is_half_a_step():
    rng = np.random.default_rng(1)
    y = (rng.standard_normal((5, 400)) * np.exp2(rng.integers(-30, 30, (5, 1)))).astype(np.float32)
    codes, s = B.quantize_rows(y)
    assert codes.shape == (5, 400) and s.shape == (5, 4)
    se = np.repeat(s.astype(np.float64), 128, axis=1)[:, :400]
    err = np.abs(B.dequant_rows(codes, s) - y)
    assert (err <= se * np.maximum(2.0**-10, 2.0**-4 * np.abs(y / se)) * (1 + 2.0**-20)).all()


def test_nonfinite_blocks():
    y = np.ones((2, 256), np.float32)
    assert np.isnan(B._scale(np.float32("nan"))) and np.isinf(B._scale(np.float32("inf")))
    _, s = B.quantize_rows(y)
    assert (s == np.float32(1) / np.float32(448)).all()


def test_weight_blocks_are_128_by_128():
    rng = np.random.default_rng(2)
    w = rng.standard_normal((130, 144)).astype(np.float32)
    w[129, 140] = 100.0
    codes, s = B.quantize_weight(bits(w))
    assert s.shape == (2, 2)
    w16 = C.bf16_to_f32(bits(w))
    for i, j in [(0, 0), (0, 1), (1, 0), (1, 1)]:
        part = np.abs(w16[128 * i : 128 * i + 128, 128 * j : 128 * j + 128]).max()
        assert s[i, j] == np.float32(part) / np.float32(448)
    assert C.e4m3_decode(codes[129, 140]) == 448.0


def test_norm_and_gate_closed_forms():
    x = bits(np.full((1, 16), 3.0))
    h, y = B.add_rmsnorm(x, bits(np.full((1, 16), 1.0)), bits(np.full(16, 0.5)), 0.0)
    assert (h == 4.0).all() and np.allclose(y, 0.5, rtol=1e-15)
    gu = bits(np.concatenate([np.zeros((1, 16)), np.ones((1, 16))], axis=1))
    assert (B.silu_mul(gu) == 0.0).all()
    big = B.silu_mul(bits(np.concatenate([np.full((1, 16), 64.0), np.full((1, 16), 2.0)], axis=1)))
    assert np.allclose(big, 128.0, rtol=1e-15)


def test_grouped_is_the_linear_of_each_expert():
    rng = np.random.default_rng(3)
    E, N, K, M = 3, 20, 160, 7
    xq, xs = B.quantize_rows(rng.standard_normal((M, K)).astype(np.float32))
    w = [B.quantize_weight(bits(rng.standard_normal((N, K)))) for _ in range(E)]
    wq, ws = np.stack([c for c, _ in w]), np.stack([s for _, s in w])
    rows, offsets = np.array([6, 0, 1, 1, 5]), np.array([0, 2, 2, 4])
    y = B.grouped_linear(xq, xs, wq, ws, offsets, rows)
    assert np.array_equal(y[:2], B.linear(xq[[6, 0]], xs[[6, 0]], wq[0], ws[0]))
    assert np.array_equal(y[2:4], B.linear(xq[[1, 1]], xs[[1, 1]], wq[2], ws[2]))
    assert np.isnan(y[4]).all()


@pytest.mark.parametrize("plant", ["scale", "code", "expert"])
def test_planted_mistakes_exceed_the_product_bound(plant):
    from block_bound import product_bound

    rng = np.random.default_rng(4)
    N, K, M = 40, 272, 6
    xq, xs = B.quantize_rows(rng.standard_normal((M, K)).astype(np.float32))
    wq, ws = B.quantize_weight(bits(rng.standard_normal((N, K))))
    ref = B.linear(xq, xs, wq, ws)
    bound = product_bound(xq, xs, wq, ws, None, ref)
    if plant == "scale":  # a block's scale of the neighbouring K block
        bad = B.linear(xq, xs[:, [1, 0, 2]], wq, ws)
    elif plant == "code":  # one code one step up
        w2 = wq.copy()
        w2[7, 200] ^= 8
        bad = B.linear(xq, xs, w2, ws)
    else:
        bad = B.linear(xq, xs, wq[::-1], ws)
    assert (np.abs(bad - ref) > bound).any()


def test_matrix_core_reference():
    from block_bound import matrix_core_linear

    # small codes: nothing is cut, the plain product
    rng = np.random.default_rng(5)
    xq, wq = rng.integers(0, 0x20, (5, 272)).astype(np.uint8), rng.integers(0, 0x20, (7, 272)).astype(np.uint8)
    xs, ws = rng.random((5, 3), np.float32), rng.random((1, 3), np.float32)
    assert np.allclose(matrix_core_linear(xq, xs, wq, ws), B.linear(xq, xs, wq, ws), rtol=1e-13)
    # 256 * 256 beside 2 * 2 in the same eight (lost), in another eight (kept), and 2.5 * 4 = 10 in it (8 kept)
    enc = lambda *v: C.e4m3_encode(np.array(v, np.float64))  # noqa: E731
    x, w = np.zeros((1, 16), np.uint8), np.zeros((1, 16), np.uint8)
    one = np.ones((1, 1), np.float32)
    x[0, [0, 3]], w[0, [0, 3]] = enc(256, 2), enc(256, 2)
    assert matrix_core_linear(x, one, w, one)[0, 0] == 65536
    x[0, [0, 3, 9]], w[0, [0, 3, 9]] = enc(256, 2.5, 2), enc(256, 4, 2)
    assert matrix_core_linear(x, one, w, one)[0, 0] == 65536 + 8 + 4
