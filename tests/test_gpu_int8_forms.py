"""Whole outputs of every kernel form of the integer products, each at sizes that
are asserted to take it (int8_forms.py)."""

import pytest

import int8_forms as F
from test_gpu_block import case
from test_gpu_int8 import check_grouped, check_linear

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form,M,N,K", F.PLAIN)
def test_linear_form(form, M, N, K):
    case(f"int8 linear {form}: {M}x{N}x{K}")
    assert F.form(M, N, K) == form
    check_linear(M, N, K)


@pytest.mark.parametrize("form,counts,N,K,M,spare", F.GROUPED)
def test_grouped_form(form, counts, N, K, M, spare):
    case(f"int8 grouped {form}: {sum(counts)} of {len(counts)} {N}x{K}")
    assert F.form(sum(counts) + spare, N, K, len(counts)) == form
    check_grouped(counts, N, K, M, 31, spare=spare)


@pytest.mark.parametrize("form,M,N,K", F.PLAIN_SPLIT)
def test_linear_split_round(form, M, N, K):
    """A few tiles more than whole rounds of the chip: those in 128 x 128 pieces, every output compared."""
    case(f"int8 linear split {form}: {M}x{N}x{K}")
    assert F.form(M, N, K) == form and F.rest(form, [M], N) > 0
    check_linear(M, N, K)


@pytest.mark.parametrize("form,counts,N,K,M,spare", F.GROUPED_SPLIT)
def test_grouped_split_round(form, counts, N, K, M, spare):
    case(f"int8 grouped split {form}: {sum(counts)} of {len(counts)} {N}x{K}")
    assert F.form(sum(counts) + spare, N, K, len(counts)) == form and F.rest(form, counts, N) > 0
    check_grouped(counts, N, K, M, 32, spare=spare)
