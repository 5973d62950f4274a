"""Whole outputs of every kernel form of the block-scaled products, each at
sizes that are asserted to take it (block_forms.py)."""

import numpy as np
import pytest
import torch

import block_forms as F
from oracle import codecs as C
from test_gpu_block import DEV, case, check_grouped, check_product, host, rows_bits, up, weight

block = pytest.importorskip("weight_only_bit_dequant_amd.block")

pytestmark = pytest.mark.gpu


def check_linear(M, N, K):
    xq, xs = block.quantize_act(up(rows_bits(M, K, M + K, spread=True)))
    q = weight(N, K, N + K)
    bias = rows_bits(1, N, N)[0] if (M + N) % 2 else None
    out = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    y = C.bf16_to_f32(host(block.linear(xq, xs, q, None if bias is None else up(bias), out=out))).astype(np.float64)
    check_product(y, (host(xq), host(xs), host(q["codes"]), host(q["scales"])), bias)


@pytest.mark.parametrize("form,M,N,K", F.PLAIN)
def test_linear_form(form, M, N, K):
    case(f"linear {form}: {M}x{N}x{K}")
    assert F.form(M, N, K) == form
    check_linear(M, N, K)


@pytest.mark.parametrize("form,counts,N,K,M,spare", F.GROUPED)
def test_grouped_form(form, counts, N, K, M, spare):
    case(f"grouped {form}: {sum(counts)} of {len(counts)} {N}x{K}")
    assert F.form(sum(counts) + spare, N, K, len(counts)) == form
    check_grouped(counts, N, K, M, 31, spare=spare)


@pytest.mark.parametrize("form,M,N,K", F.PLAIN_SPLIT)
def test_linear_split_round(form, M, N, K):
    """A few tiles more than whole rounds of the chip: those in 128 x 128 pieces, every output compared."""
    case(f"linear split {form}: {M}x{N}x{K}")
    assert F.form(M, N, K) == form and F.rest(form, [M], N) > 0
    check_linear(M, N, K)


@pytest.mark.parametrize("form,counts,N,K,M,spare", F.GROUPED_SPLIT)
def test_grouped_split_round(form, counts, N, K, M, spare):
    case(f"grouped split {form}: {sum(counts)} of {len(counts)} {N}x{K}")
    assert F.form(sum(counts) + spare, N, K, len(counts)) == form and F.rest(form, counts, N) > 0
    check_grouped(counts, N, K, M, 32, spare=spare)


def test_tiled_weights_past_32_bit_offsets():
    """The last of nine experts' weights start at byte 2^32; its rows go through a tiled form."""
    E, N, K, T = 9, 16384, 32768, 160
    case(f"grouped {E}x{N}x{K}")
    assert F.form(T, N, K, E).startswith("tile")
    gen = torch.Generator(device=DEV).manual_seed(3)
    codes = torch.randint(0, 256, (E, N, K), dtype=torch.uint8, device=DEV, generator=gen)
    codes[codes & 0x7F == 0x7F] = 0x31  # no NaN
    scales = torch.rand(E, N // 128, K // 128, device=DEV, generator=gen) + 0.5
    xq, xs = block.quantize_act(up(rows_bits(T, K, 4)))
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[E:] = T
    y = block.grouped_linear(xq, xs, {"E": E, "N": N, "K": K, "codes": codes, "scales": scales}, off)
    for n in (0, N - 128):  # the first and the last 128 columns
        at = slice(n, n + 128)
        check_product(C.bf16_to_f32(host(y[:, at].contiguous())).astype(np.float64),
                      (host(xq), host(xs), host(codes[E - 1, at]), host(scales[E - 1, n // 128 : n // 128 + 1])))


@pytest.mark.parametrize("T,E,N,K", [(40, 64, 136, 272), (300, 9, 1040, 400), (2000, 40, 1000, 144)])
def test_offsets_out_of_order_stay_inside(T, E, N, K):
    """Decreasing offsets count more tiles than are launched: the rows after Y's stay as they were."""
    case(f"grouped offsets out of order {T} {E} {N}x{K} {F.form(T, N, K, E)}")
    xq, xs = block.quantize_act(up(rows_bits(T, K, 1)))
    q = weight(N, K, 2, E)
    off = torch.tensor([0 if e % 2 == 0 else T for e in range(E + 1)], dtype=torch.int32, device=DEV)
    buf = torch.full((T + 300, N), 7.0, dtype=torch.bfloat16, device=DEV)
    y = block.grouped_linear(xq, xs, q, off, out=buf[:T])
    assert y.data_ptr() == buf.data_ptr()
    assert bool((buf[T:] == 7.0).all()) and bool(torch.isfinite(y.float()).all())
