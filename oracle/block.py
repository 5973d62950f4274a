"""Oracle of the block-scaled FP8 operators (numpy).

Quantizers follow the definition step by step in fp32, so that codes and
scales can be compared bit for bit where the kernel's input is exact; norms,
activations and products are in float64.
"""

import numpy as np

from .codecs import bf16_to_f32, e4m3_decode, e4m3_encode

BLOCK = 128
TINY = np.float32(2.0**-126)


def blocks(n):
    return -(-n // BLOCK)


def _scale(amax):
    """max(amax / 448, 2^-126) in fp32; NaN and infinity stay."""
    with np.errstate(invalid="ignore", over="ignore"):
        s = np.asarray(amax, np.float32) / np.float32(448)
        return np.where(s < TINY, TINY, s).astype(np.float32)


def quantize_rows(y):
    """fp32 rows [M, K] -> (codes uint8 [M, K], scales fp32 [M, KB])."""
    y = np.asarray(y, np.float32)
    M, K = y.shape
    codes, scales = np.zeros((M, K), np.uint8), np.zeros((M, blocks(K)), np.float32)
    for b in range(blocks(K)):
        part = y[:, BLOCK * b : BLOCK * (b + 1)]
        scales[:, b] = _scale(np.abs(part).max(axis=1))
        v = (part / scales[:, b, None]).astype(np.float32)
        codes[:, BLOCK * b : BLOCK * (b + 1)] = e4m3_encode(np.clip(v, np.float32(-448), np.float32(448)))
    return codes, scales


def quantize_weight(W_bits):
    """bf16 bits [N, K] -> (codes uint8 [N, K], scales fp32 [NB, KB])."""
    w = bf16_to_f32(W_bits)
    N, K = w.shape
    codes, scales = np.zeros((N, K), np.uint8), np.zeros((blocks(N), blocks(K)), np.float32)
    for i in range(blocks(N)):
        for b in range(blocks(K)):
            at = np.s_[BLOCK * i : BLOCK * (i + 1), BLOCK * b : BLOCK * (b + 1)]
            scales[i, b] = _scale(np.abs(w[at]).max())
            v = (w[at] / scales[i, b]).astype(np.float32)
            codes[at] = e4m3_encode(np.clip(v, np.float32(-448), np.float32(448)))
    return codes, scales


def dequant_rows(codes, scales):
    """float64 values of activation codes."""
    K = codes.shape[1]
    return e4m3_decode(codes).astype(np.float64) * np.repeat(scales.astype(np.float64), BLOCK, axis=1)[:, :K]


def dequant_weight(codes, scales):
    """float64 values of weight codes [N, K]."""
    N, K = codes.shape
    s = np.repeat(np.repeat(scales.astype(np.float64), BLOCK, axis=0)[:N], BLOCK, axis=1)[:, :K]
    return e4m3_decode(codes).astype(np.float64) * s


def add_rmsnorm(x_bits, residual_bits, gain_bits, eps):
    """(h, y) in float64."""
    h = bf16_to_f32(x_bits).astype(np.float64)
    if residual_bits is not None:
        h = h + bf16_to_f32(residual_bits).astype(np.float64)
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)
    return h, h * rstd * bf16_to_f32(gain_bits).astype(np.float64)


def silu_mul(gu_bits):
    gu = bf16_to_f32(gu_bits).astype(np.float64)
    K = gu.shape[1] // 2
    g, u = gu[:, :K], gu[:, K:]
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def linear(xq, xs, wq, ws, bias_bits=None):
    y = dequant_rows(xq, xs) @ dequant_weight(wq, ws).T
    return y if bias_bits is None else y + bf16_to_f32(bias_bits).astype(np.float64)


def grouped_linear(xq, xs, wq, ws, offsets, rows=None):
    """float64 [T, N]; NaN in rows that no expert has."""
    T = xq.shape[0] if rows is None else len(rows)
    x = dequant_rows(xq, xs)
    y = np.full((T, wq.shape[1]), np.nan)
    for e in range(wq.shape[0]):
        t = np.arange(offsets[e], offsets[e + 1])
        src = t if rows is None else np.asarray(rows)[t]
        y[t] = x[src] @ dequant_weight(wq[e], ws[e]).T
    return y
