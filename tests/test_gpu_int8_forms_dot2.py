"""Whole outputs of the grouped products' form "dot 2", within the products' bound and bit for bit."""

import pytest

import int8_forms as F
import int8_forms_dot2 as D
from test_gpu_block import case
from test_gpu_int8 import check_grouped
from test_gpu_int8_bits import check_grouped as check_bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form,counts,N,K,M,spare", D.GROUPED)
def test_grouped_form(form, counts, N, K, M, spare):
    case(f"int8 grouped {form}: {sum(counts)} of {len(counts)} {N}x{K}")
    assert F.form(sum(counts) + spare, N, K, len(counts)) == form
    check_grouped(counts, N, K, M, 31, spare=spare)
    if not spare:
        check_bits(counts, N, K, M)
