"""The integer products' bits: every kernel form gives what the definition's operations give, each rounded by itself,

    bf16(float(sum) * Xs * Ws + bias),

so that no row's bits go by how many rows are beside it.  The reference makes these operations one by one in torch (the
sums exact in float64).  The bias nearly cancels the product of half of the rows, so that a product that was not
rounded before it shows up; some columns' scales take the outputs to subnormal numbers and zeros of either sign."""

import pytest
import torch

import int8_forms as F
from test_gpu_block import DEV, case, groups
from test_gpu_int8 import codes_of, weight

int8 = pytest.importorskip("weight_only_bit_dequant_amd.int8")

pytestmark = pytest.mark.gpu


def operands(M, N, K, seed, E=None):
    """Rows of which every second one has row 0's codes, weights with tiny scales in some columns."""
    xq, xs = codes_of(M, K, seed)
    xq[::2] = xq[0].clone()
    q = weight(N, K, seed + 1, E)
    q["scales"][..., 3::11] *= 2.0**-128
    q["scales"][..., 5::17] *= 2.0**-140
    return xq, xs, q


def product(xq, xs, w, ws):
    return (xq.double() @ w.double().T).float() * xs[:, None] * ws


def cancelling(p):
    """A bias that leaves little of product row 0, zeros of either sign among its values."""
    b = -p[0].to(torch.bfloat16)
    b[1::13], b[2::13] = 0.0, -0.0
    return b


def same_bits(y, want):
    y, want = y.view(torch.int16), want.to(torch.bfloat16).view(torch.int16)
    bad = (y != want).nonzero()
    assert len(bad) == 0, (len(bad), bad[0].tolist())


def check_linear(M, N, K):
    xq, xs, q = operands(M, N, K, M + 3 * K)
    p = product(xq, xs, q["codes"], q["scales"])
    same_bits(int8.linear(xq, xs, q), p)
    b = cancelling(p)
    same_bits(int8.linear(xq, xs, q, b), p + b.float())


@pytest.mark.parametrize("form,M,N,K", F.PLAIN + F.PLAIN_SPLIT)
def test_linear_bits(form, M, N, K):
    case(f"int8 linear bits {form}: {M}x{N}x{K}")
    check_linear(M, N, K)


def check_grouped(counts, N, K, M):
    E = len(counts)
    off, rows = groups(counts, 7, M)
    T = int(off[-1])
    rows = None if rows is None else torch.from_numpy(rows).to(DEV)
    xq, xs, q = operands(T if rows is None else M, N, K, T + K, E)
    y = int8.grouped_linear(xq, xs, q, torch.from_numpy(off).to(DEV), rows=rows)
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        if lo < hi:
            src = torch.arange(lo, hi, device=DEV) if rows is None else rows[lo:hi].long()
            same_bits(y[lo:hi], product(xq[src], xs[src], q["codes"][e], q["scales"][e]))


@pytest.mark.parametrize("form,counts,N,K,M,spare", F.GROUPED + F.GROUPED_SPLIT)
def test_grouped_bits(form, counts, N, K, M, spare):
    case(f"int8 grouped bits {form}: {sum(counts)} of {len(counts)} {N}x{K}")
    check_grouped(counts, N, K, M)


@pytest.mark.parametrize("N,K", [(4096, 4096), (1200, 2064), (4200, 6240), (1096, 144), (8190, 528), (250, 1536)])
def test_a_row_alone_and_among_others(N, K):
    """The same 16 rows again and again, at a number of rows for each form that they reach."""
    case(f"int8 linear rows among others {N}x{K}")
    forms = {}
    for M in (*range(1, 160), *range(160, 2000, 37), *range(2000, 9000, 500)):
        forms.setdefault(F.form(M, N, K), M)
    assert len(forms) >= 6
    xq, xs, q = operands(16, N, K, K)
    b = cancelling(product(xq, xs, q["codes"], q["scales"]))
    want = torch.cat([int8.linear(xq[i : i + 1], xs[i : i + 1], q, b) for i in range(16)])
    for M in forms.values():
        y = int8.linear(xq.repeat(M // 16 + 1, 1)[:M].contiguous(), xs.repeat(M // 16 + 1)[:M].contiguous(), q, b)
        same_bits(y, want.repeat(M // 16 + 1, 1)[:M])
