"""The 8-bit integer operators and the experts' routing at sizes that pass 32 bits, in every row
form of the quantizers, and as two calls at once on two streams."""

import numpy as np
import pytest
import torch

pytest.importorskip("weight_only_bit_dequant_amd.int8")

from int8_bound import SILU_REL, check_codes
from oracle import block as B
from oracle import codecs as C
from test_gpu_block import DEV, case, host, rows_bits, up
from test_gpu_int8 import check_product, codes_of, exact, same_codes, weight
from weight_only_bit_dequant_amd import experts, int8

pytestmark = pytest.mark.gpu

# a row of each number of waves and chunks to a lane: 1 to 16 waves of 64 chunks of 8, one, two or four to a lane, or read twice
WIDTHS = [512, 1024, 1536, 2048, 2896, 4096, 5904, 8192, 16384, 32768, 32784]


@pytest.mark.parametrize("K", WIDTHS)
def test_every_row_form(K):
    case(f"int8 rows of {K}")
    x = rows_bits(5, K, K)
    xq, xs = int8.quantize_act(up(x))
    same_codes(host(xq), host(xs), C.bf16_to_f32(x))
    gu = rows_bits(3, 2 * K, K + 1)
    ok, text = check_codes(*(host(t) for t in int8.silu_mul_quantize(up(gu))), B.silu_mul(gu), SILU_REL)
    assert ok, text


@pytest.fixture
def room():
    """Large tensors go back before and after."""
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def test_rows_past_32_bit_offsets(room):
    """Rows from byte 2^32 on: quantized, gated, and read by the products with and without an order."""
    case("int8 rows past 2^32 bytes")
    M, K = 2_100_000, 2064
    q = weight(24, K, 1)
    x = torch.zeros(M, K, dtype=torch.bfloat16, device=DEV)
    last = up(rows_bits(40, K, 2))
    x[-40:] = last
    xq, xs = int8.quantize_act(x)
    want = int8.quantize_act(last)
    assert torch.equal(xq[-40:], want[0]) and torch.equal(xs[-40:], want[1]) and not bool(xq[:-40].any())
    wide = x.view(M // 2, 2 * K)
    hq, hs = int8.silu_mul_quantize(wide)
    want = int8.silu_mul_quantize(last.view(20, 2 * K))
    assert torch.equal(hq[-20:], want[0]) and torch.equal(hs[-20:], want[1])
    del x, wide, hq, hs
    y = int8.linear(xq, xs, q)
    check_product(y[-40:], *exact(xq[-40:], xs[-40:], q["codes"], q["scales"]))
    assert not bool(y[:-40].any())
    # with an order, codes up to byte 2^32 - 16
    M = (1 << 32) // K
    xq, xs = xq[-M:].contiguous(), xs[-M:].contiguous()
    qe = weight(24, K, 3, 2)
    rows = torch.tensor([M - 1, 0, M - 40, M - 1, M, M - 7], dtype=torch.int32, device=DEV)
    off = torch.tensor([0, 2, 6], dtype=torch.int32, device=DEV)
    y = int8.grouped_linear(xq, xs, qe, off, rows=rows)
    for e, (a, b) in enumerate(((0, 2), (2, 6))):
        src = rows[a:b].long()
        has = src < M
        src = src.clamp_max(M - 1)
        check_product(y[a:b][has], *exact(xq[src][has], xs[src][has], qe["codes"][e], qe["scales"][e]))
    assert not bool(y[4].any())


def test_outputs_past_32_bit_offsets(room):
    """Elements of Y from 2^31 on, plain and grouped."""
    case("int8 outputs past 2^31 elements")
    M, N, K = 1_100_000, 2000, 16
    xq, xs = codes_of(M, K, 5)
    q = weight(N, K, 6, 2)
    out = torch.zeros(M, N, dtype=torch.bfloat16, device=DEV)
    int8.linear(xq, xs, {"codes": q["codes"][1], "scales": q["scales"][1]}, out=out)
    check_product(out[-300:], *exact(xq[-300:], xs[-300:], q["codes"][1], q["scales"][1]))
    check_product(out[:300], *exact(xq[:300], xs[:300], q["codes"][1], q["scales"][1]))
    out.zero_()
    off = torch.tensor([0, 1000, M - 5], dtype=torch.int32, device=DEV)
    int8.grouped_linear(xq, xs, q, off, out=out)
    check_product(out[-305:-5], *exact(xq[-305:-5], xs[-305:-5], q["codes"][1], q["scales"][1]))
    check_product(out[:1000], *exact(xq[:1000], xs[:1000], q["codes"][0], q["scales"][0]))
    assert not bool(out[-5:].any())


def test_logits_past_32_bit_offsets(room):
    """Rows of strided logits from byte 2^32 on are those of a copy."""
    case("route past 2^32 bytes")
    M, E, ld = 70_000, 200, 16384
    wide = torch.zeros(M, ld, device=DEV)
    wide[:, :E] = torch.randn(M, E, generator=torch.Generator().manual_seed(1)).to(DEV)
    for kw in (dict(), dict(score="sigmoid", bias=torch.linspace(-0.1, 0.1, E, device=DEV), groups=8, keep_groups=3)):
        got, want = experts.route(wide[:, :E], 6, **kw), experts.route(wide[:, :E].contiguous(), 6, **kw)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert int(got.offsets[E]) == 6 * M


def test_two_calls_at_once():
    """Two streams, one layer's calls on each at the same time, again and again: each its own result."""
    case("two calls at once")
    M, E, top, hidden, inner = 600, 16, 3, 528, 272
    gen = torch.Generator().manual_seed(1)
    q = weight(2 * inner, hidden, 1, E), weight(hidden, inner, 2, E)
    x = [torch.randn(M, hidden, generator=gen).to(torch.bfloat16).to(DEV) for _ in range(2)]
    logits = [torch.randn(M, E, generator=gen).to(DEV) for _ in range(2)]
    bias = 0.1 * torch.randn(E, generator=gen).to(DEV)

    def layer(i):
        r = experts.route(logits[i], top, score="sigmoid", bias=bias, groups=4, keep_groups=2)
        gu = int8.grouped_linear(*int8.quantize_act(x[i]), q[0], r.offsets, rows=r.rows)
        z = int8.grouped_linear(*int8.silu_mul_quantize(gu), q[1], r.offsets)
        return experts.combine(z, r.places, r.weights, base=x[i])

    want = [layer(i).clone() for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(layer(i))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])
    assert not np.array_equal(host(want[0]), host(want[1]))
