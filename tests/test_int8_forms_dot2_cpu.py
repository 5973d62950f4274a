"""With the sizes of int8_forms_dot2.py grouped products reach every kernel form, with whole and with short last steps
of K, odd widths and gathered rows (no GPU)."""

import os

import pytest

import int8_forms as F
import int8_forms_dot2 as D
from weight_only_bit_dequant_amd import wq

if not os.path.exists(wq.LIB_PATH):  # pragma: no cover
    pytest.skip("libwq.so not built", allow_module_level=True)


def test_sizes_take_the_form():
    for f, counts, N, K, M, spare in D.GROUPED:
        assert F.form(sum(counts) + spare, N, K, len(counts)) == f, (len(counts), N, K)


def test_grouped_sizes_reach_every_form():
    every = F.GROUPED + D.GROUPED
    assert {(f, K % 128 == 0) for f, _, _, K, _, _ in every} == {(f, whole) for f in F.FORMS for whole in (True, False)}
    assert {f for f, _, N, _, _, _ in D.GROUPED if N % 8} == {"dot 2"}
    assert {M is None for _, _, _, _, M, _ in D.GROUPED} == {spare > 0 for *_, spare in D.GROUPED} == {True, False}
