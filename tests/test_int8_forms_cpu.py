"""The integer products' sizes together reach every kernel form, with whole and
with short last steps of K (no GPU)."""

import os

import pytest

import int8_forms as F
from weight_only_bit_dequant_amd import wq

if not os.path.exists(wq.LIB_PATH):  # pragma: no cover
    pytest.skip("libwq.so not built", allow_module_level=True)


def test_plain_sizes_take_their_forms_and_reach_all():
    for f, M, N, K in F.PLAIN + F.PLAIN_SPLIT:
        assert F.form(M, N, K) == f, (f, M, N, K)
    assert {(f, K % 128 == 0) for f, _, _, K in F.PLAIN} == {(f, whole) for f in F.FORMS for whole in (True, False)}
    assert {f for f, M, N, K in F.PLAIN if N % 8} == set(F.FORMS)


def test_grouped_sizes_take_their_forms_and_reach_all():
    for f, counts, N, K, M, spare in F.GROUPED + F.GROUPED_SPLIT:
        assert F.form(sum(counts) + spare, N, K, len(counts)) == f, (f, len(counts), N, K)
    assert {(f, K % 128 == 0) for f, _, _, K, _, _ in F.GROUPED} == {(f, whole) for f in F.FORMS[1:] for whole in (True, False)}


def test_split_rounds():
    for f, M, N, K in F.PLAIN_SPLIT:
        assert F.rest(f, [M], N) > 0, (f, M, N, K)
    for f, counts, N, K, M, spare in F.GROUPED_SPLIT:
        assert F.rest(f, counts, N) > 0, (f, len(counts), N, K)


def test_no_rows_no_form():
    assert F.form(0, 64, 64) == ""
