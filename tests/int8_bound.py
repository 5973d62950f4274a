"""Per-element bounds of the 8-bit integer operators and of the experts' sum
against the oracle; u = 2^-24.

Products: the int32 sum is exact; it is rounded to 24 bits (u), multiplied by
two scales (u each), the bias is added (u of the sum): |fp32 - ref| <= 4 u S (1 + u)^4,
S = |product| + |bias|.  The rounding to bf16 takes at most 2^-8 of that value, or
half the smallest subnormal, 2^-134.

Sums: each of `top` fused multiply-adds and the base's addition is off by at most
u of the partial sum's magnitude: (top + 1) u S (1 + u)^(top + 1).

Codes of a gated row: the kernel's y is off by SILU_REL |y| (block_bound.py), the
scale by that and 2 u, the quotient by 4 u more; the code is its nearest whole
number: |code s - y| <= s / 2 + (SILU_REL + 8 u) |y|.
"""

import numpy as np

from block_bound import SILU_REL, U


def rounded(ref, off):
    """Bound of bf16(fp32) where |fp32 - ref| <= off."""
    return off + 2.0**-8 * (np.abs(ref) + off) + 2.0**-134


def product_bound(ref, size):
    return rounded(ref, 4 * U * (1 + 2.0**-20) * size + 2.0**-149)


def sum_bound(ref, size, top):
    return rounded(ref, (top + 1) * U * (1 + 2.0**-14) * size + 2.0**-149 * (top + 1))


def check_codes(codes, scales, y, rel):
    """(ok, text): codes/scales quantize float64 rows y that the kernel has within `rel`."""
    want = np.maximum(np.abs(y).max(axis=1) / 127.0, 2.0**-126)
    if not (np.abs(scales - want) <= want * (rel + 2 * U)).all():
        return False, "scales off by %g" % np.abs(scales / want - 1).max()
    s = scales.astype(np.float64)[:, None]
    ratio = np.abs(codes.astype(np.float64) * s - y) / (s / 2 + (rel + 8 * U) * np.abs(y))
    return bool(ratio.max() <= 1), "codes off by %g of the bound" % ratio.max()


__all__ = ["SILU_REL", "U", "check_codes", "product_bound", "rounded", "sum_bound"]
