"""The sizes that the GPU tests run take the forms that they are meant for, and
together every form (host code: no GPU needed)."""

import os
import re

import pytest

import block_forms as F

wq = pytest.importorskip("weight_only_bit_dequant_amd.wq")

if not os.path.exists(wq.LIB_PATH):  # pragma: no cover
    pytest.skip("libwq.so not built", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_sizes_take_their_form():
    for want, M, N, K in F.PLAIN:
        assert F.form(M, N, K) == want, (want, M, N, K, F.form(M, N, K))
    for want, counts, N, K, _, spare in F.GROUPED:
        got = F.form(sum(counts) + spare, N, K, len(counts))
        assert got == want, (want, sum(counts), len(counts), N, K, got)


def test_every_form_has_sizes():
    text = open(os.path.join(ROOT, "weight_only_bit_dequant_amd", "csrc", "wq_block_plan.cpp")).read()
    names = re.findall(r'"([^"]+)"', re.search(r"kNames\[\] = \{(.*?)\};", text, re.S).group(1))
    assert len(names) == 12
    plain = {(f, K % 128 == 0) for f, _, _, K in F.PLAIN}
    grouped = {(f, K % 128 == 0) for f, _, _, K, _, _ in F.GROUPED}
    for name in names:
        if name != "stream 64x16":  # experts only
            assert {(name, True), (name, False)} <= plain, name
        if name not in ("stream 32x16 eight",):  # plain only
            assert {(name, True), (name, False)} <= grouped, name
    # both parities of the number of blocks where groups of waves share them; tiles of more experts than a wave has lanes
    for name in ("tile 64x64", "tile 128x64"):
        assert len({(K % 128 == 0, -(-K // 128) % 2) for f, _, _, K in F.PLAIN if f == name}) == 4, name
    assert {f for f, c, *_ in F.GROUPED if len(c) > 64 and f.startswith("tile")} == {n for n in names if n.startswith("tile")}


def test_sizes_that_split_a_round():
    text = open(os.path.join(ROOT, "weight_only_bit_dequant_amd", "csrc", "wq_block_internal.hpp")).read()
    assert "kRound = %d, kMostRest = kRound / %d" % (F.ROUND, F.ROUND // F.MOST_REST) in text
    for form, M, N, K in F.PLAIN_SPLIT:
        assert F.form(M, N, K) == form and F.rest(form, [M], N) > 0, (form, M, N, K)
    for form, counts, N, K, _, spare in F.GROUPED_SPLIT:
        assert F.form(sum(counts) + spare, N, K, len(counts)) == form and F.rest(form, counts, N) > 0, (form, counts, N)
    for sizes in (F.PLAIN_SPLIT, F.GROUPED_SPLIT):  # both forms that split, with and without a short last block
        assert {(s[0], s[3] % 128 == 0) for s in sizes} == {(f, w) for f in F._SPLIT_TILES for w in (True, False)}
    # and the others leave their tiles whole
    assert not any(F.rest(f, [M], N) for f, M, N, _ in F.PLAIN) and not any(F.rest(s[0], s[1], s[2]) for s in F.GROUPED)


@pytest.mark.parametrize("T,E,N,K", [(1, 0, 4096, 3072), (32, 0, 4096, 3072), (300, 0, 6152, 4096), (8192, 0, 8192, 8192),
                                     (64, 32, 2048, 2048), (2000, 64, 1536, 2048), (8192, 8, 4096, 4096)])
def test_measured_sizes_take_a_tested_kernel(T, E, N, K):
    have = {(f, k % 128 == 0) for f, *_, k in F.PLAIN} if E == 0 else {(f, k % 128 == 0) for f, _, _, k, _, _ in F.GROUPED}
    assert (F.form(T, N, K, E), K % 128 == 0) in have
