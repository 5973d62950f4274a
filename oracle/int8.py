"""Oracle of the 8-bit integer operators (numpy): one scale a row.

The quantizer follows the definition step by step in fp32; products sum in
int64 and scale in float64.
"""

import numpy as np

from .codecs import bf16_to_f32

TINY = np.float32(2.0**-126)


def quantize_rows(y):
    """fp32 rows [..., K] -> (codes int8 [..., K], scales fp32 [...], quotients fp32)."""
    y = np.asarray(y, np.float32)
    amax = np.abs(y).max(axis=-1)
    bad = ~np.isfinite(amax)
    s = np.maximum(np.where(bad, np.float32(0), amax) / np.float32(127), TINY).astype(np.float32)
    with np.errstate(invalid="ignore"):
        v = (np.where(bad[..., None], np.float32(0), y) / s[..., None]).astype(np.float32)
    return np.rint(v).astype(np.int8), np.where(bad, np.float32("nan"), s), v


def dequant(codes, scales):
    return codes.astype(np.float64) * scales.astype(np.float64)[..., None]


def linear(xq, xs, wq, ws, bias_bits=None):
    """float64 product before its rounding, and the sum's and the bias's magnitude."""
    # (fp64 holds every sum of K < 2^17 products of codes exactly, and multiplies fast)
    p = (xq.astype(np.float64) @ wq.astype(np.float64).T) * xs.astype(np.float64)[:, None] * ws.astype(np.float64)
    if bias_bits is None:
        return p, np.abs(p)
    b = bf16_to_f32(bias_bits).astype(np.float64)
    return p + b, np.abs(p) + np.abs(b)
