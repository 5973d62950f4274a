"""Block-scaled FP8 operators on the GPU against the oracle.

Quantizers of bf16 inputs are compared bit for bit; norm, gate and products
element by element with the bounds derived in block_bound.py, products also with
the plain float64 product at the framework's bar (relative Frobenius error
1e-2)."""

import numpy as np
import pytest
import torch

from block_bound import NORM_REL, SILU_REL, check_codes, matrix_core_linear, product_bound
from elementwise_bound import ulp_bf16
from oracle import block as B
from oracle import codecs as C
from weight_only_bit_dequant_amd import synth

block = pytest.importorskip("weight_only_bit_dequant_amd.block")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def rows_bits(M, K, seed, spread=False):
    """bf16 bits [M, K]: normal; `spread`: block magnitudes over 2^-12 .. 2^12."""
    g = torch.Generator().manual_seed(seed)
    t = torch.randn(M, K, generator=g)
    if spread:
        e = torch.randint(-12, 13, (M, B.blocks(K)), generator=g).float()
        t = t * torch.exp2(e).repeat_interleave(128, dim=1)[:, :K]
    return synth.from_torch_bf16(t.to(torch.bfloat16))


def up(bits):
    return synth.as_torch_bf16(bits, DEV)


def host(t):
    torch.cuda.synchronize()
    return synth.from_torch_bf16(t) if t.dtype == torch.bfloat16 else t.cpu().numpy()


def strided(bits, pad=24):
    """The same rows with `pad` more elements between them."""
    t = torch.full((bits.shape[0], bits.shape[1] + pad), float("nan"), dtype=torch.bfloat16, device=DEV)
    t[:, : bits.shape[1]] = up(bits)
    return t[:, : bits.shape[1]]


def case(text):
    print("[case] " + text, flush=True)


# ---------------------------------------------------------------- quantizers


@pytest.mark.parametrize("M,K", [(1, 16), (1, 128), (3, 144), (17, 2048), (5, 2896), (130, 528), (2, 40000)])
@pytest.mark.parametrize("stride", [False, True])
def test_quantize_act_bits(M, K, stride):
    case(f"quantize_act {M}x{K} strided={stride}")
    x = rows_bits(M, K, M * 7 + K, spread=True)
    xq, xs = block.quantize_act(strided(x) if stride else up(x))
    codes, scales = B.quantize_rows(C.bf16_to_f32(x))
    assert np.array_equal(host(xq), codes) and np.array_equal(host(xs), scales)


def test_quantize_act_extreme_blocks():
    case("quantize_act extreme blocks")
    x = np.zeros((6, 384), np.float32)
    x[1, 5], x[1, 200] = 3.3e38, 1e-38          # the largest bf16 values; below 2^-126 * 448
    x[2, :128] = np.linspace(-1e-40, 1e-40, 128)  # subnormal in bf16
    x[3, 130:140] = -0.0
    b = C.f32_to_bf16(x)
    codes, scales = B.quantize_rows(C.bf16_to_f32(b))
    xq, xs = block.quantize_act(up(b))
    assert np.array_equal(host(xq), codes) and np.array_equal(host(xs), scales)
    # non-finite: the block's scale says so, its neighbours are untouched
    y = C.bf16_to_f32(b).copy()
    y[4, 7], y[5, 300] = np.nan, -np.inf
    xq, xs = block.quantize_act(up(C.f32_to_bf16(y)))
    xs = host(xs)
    assert np.isnan(xs[4, 0]) and np.isinf(xs[5, 2])
    ok = np.ones_like(xs, bool)
    ok[4, 0] = ok[5, 2] = False
    assert np.array_equal(xs[ok], scales[ok])


@pytest.mark.parametrize("shape", [(1, 16), (128, 128), (130, 144), (300, 512), (3, 40, 272)])
def test_quantize_weight_bits(shape):
    case(f"quantize_weight {shape}")
    w = rows_bits(int(np.prod(shape[:-1])), shape[-1], sum(shape), spread=True).reshape(shape)
    q = block.quantize_weight(up(w))
    for e in range(q["E"]):
        codes, scales = B.quantize_weight(w if len(shape) == 2 else w[e])
        got = [host(q[k]) if len(shape) == 2 else host(q[k])[e] for k in ("codes", "scales")]
        assert np.array_equal(got[0], codes) and np.array_equal(got[1], scales)


# ---------------------------------------------------------------- norm


NORM_SIZES = [(1, 16), (3, 128), (9, 512), (2, 528), (5, 1024), (3, 1040), (7, 2048), (1, 2896), (6, 4096), (4, 4112),
              (2, 8192), (3, 8208), (2, 16384), (1, 20000), (2, 32768), (300, 1536), (5000, 144)]


@pytest.mark.parametrize("M,K", NORM_SIZES)
@pytest.mark.parametrize("form", ["plain", "residual", "all"])
def test_add_rmsnorm_quantize(M, K, form):
    case(f"norm {M}x{K} {form}")
    x, g = rows_bits(M, K, M + 3 * K), rows_bits(1, K, K)[0]
    r = None if form == "plain" else rows_bits(M, K, M + K + 1, spread=True)
    y_out = torch.full((M, K), float("nan"), dtype=torch.bfloat16, device=DEV) if form == "all" else None
    xt = strided(x) if form == "all" else up(x)
    xq, xs, ro, yo = block.add_rmsnorm_quantize(xt, up(g), 1e-5, residual=None if r is None else up(r), y_out=y_out)
    h, y = B.add_rmsnorm(x, r, g, float(np.float32(1e-5)))
    ok, text = check_codes(host(xq), host(xs), y, NORM_REL)
    assert ok, text
    if r is None:
        assert ro is None
    else:  # bf16 of one fp32 addition
        assert np.array_equal(host(ro), C.f32_to_bf16(C.bf16_to_f32(x) + C.bf16_to_f32(r)))
    if yo is not None:
        got = C.bf16_to_f32(host(yo)).astype(np.float64)
        assert (np.abs(got - y) <= ulp_bf16(y) + NORM_REL * np.abs(y)).all()


def test_norm_in_place_and_zero_rows():
    case("norm in place, zero rows")
    x, r, g = rows_bits(12, 1040, 1), rows_bits(12, 1040, 2), rows_bits(1, 1040, 3)[0]
    x[3], r[3] = 0, 0
    xt, rt = up(x), up(r)
    want = block.add_rmsnorm_quantize(xt, up(g), 1e-6, residual=rt)
    for name in ("residual", "x"):
        xc, rc = xt.clone(), rt.clone()
        got = block.add_rmsnorm_quantize(xc, up(g), 1e-6, residual=rc, residual_out=rc if name == "residual" else xc)
        for a, b in zip(want[:3], got[:3]):
            assert np.array_equal(host(a), host(b))
    assert (host(want[0])[3] & 0x7F == 0).all() and (host(want[1])[3] == np.float32(2.0**-126)).all()
    # eps = 0 on a zero row is 0 * inf: NaN in that row's scales, no other row
    q = block.add_rmsnorm_quantize(xt, up(g), 0.0, residual=rt)
    assert np.isnan(host(q[1])[3]).all() and np.isfinite(np.delete(host(q[1]), 3, axis=0)).all()


def test_norm_nonfinite_rows_stay_alone():
    case("norm non-finite rows")
    x, g = rows_bits(9, 656, 5), rows_bits(1, 656, 6)[0]
    want = [host(t) for t in block.add_rmsnorm_quantize(up(x), up(g))[:2]]
    y = C.bf16_to_f32(x).copy()
    y[2, 650], y[6, 3] = np.nan, np.inf
    got = [host(t) for t in block.add_rmsnorm_quantize(up(C.f32_to_bf16(y)), up(g))[:2]]
    keep = [0, 1, 3, 4, 5, 7, 8]
    assert all(np.array_equal(a[keep], b[keep]) for a, b in zip(want, got))
    assert np.isnan(got[1][2]).all() and np.isnan(got[1][6, 0])


# ---------------------------------------------------------------- gate


@pytest.mark.parametrize("M,K", [(1, 16), (1, 2048), (3, 144), (64, 1040), (17, 2896), (700, 272)])
@pytest.mark.parametrize("stride", [False, True])
def test_silu_mul_quantize(M, K, stride):
    case(f"gate {M}x{K} strided={stride}")
    gu = rows_bits(M, 2 * K, M * K, spread=True)
    xq, xs = block.silu_mul_quantize(strided(gu) if stride else up(gu))
    ok, text = check_codes(host(xq), host(xs), B.silu_mul(gu), SILU_REL)
    assert ok, text


def test_silu_far_values():
    case("gate far values")
    g = np.array([0.0, -0.0, 80.0, -80.0, 88.5, -88.5, 100.0, -100.0, 3e38, -3e38, 1e-30, -1e-30, 1.0, -1.0, 20.0, -20.0])
    gu = C.f32_to_bf16(np.concatenate([g, np.ones(16)])[None].astype(np.float32))
    xq, xs = block.silu_mul_quantize(up(gu))
    y = B.silu_mul(gu)
    # one block whose scale is the 3e38's: the rest, at most 1e2, are below half a step
    assert host(xs)[0, 0] == np.float32(C.bf16_to_f32(gu)[0, 8]) / np.float32(448)
    want = np.zeros(16)
    want[8] = 448
    assert np.array_equal(C.e4m3_decode(host(xq))[0], want) and np.isfinite(y).all()
    # and each value in a block of its own (-3e38 gives -0)
    each = np.zeros((16, 256), np.uint16)
    each[:, 0], each[:, 128] = gu[0, :16], gu[0, 16:]
    xq, xs = block.silu_mul_quantize(up(each))
    ok, text = check_codes(host(xq), host(xs), B.silu_mul(each), SILU_REL)
    assert ok, text


# ---------------------------------------------------------------- products


def weight(N, K, seed, E=None):
    w = rows_bits(N * (E or 1), K, seed, spread=True)
    w = w.reshape((N, K) if E is None else (E, N, K))
    return block.quantize_weight(up(w))


def check_product(y, args, bias=None):
    """`y` (float64) is the product of args = (xq, xs, wq, ws) (numpy)."""
    plain = B.linear(*args, bias)
    ref = matrix_core_linear(*args, bias, device=DEV)
    ratio = np.abs(y - ref) / product_bound(*args, bias, ref)
    assert ratio.max() <= 1, (ratio.max(), np.unravel_index(ratio.argmax(), ratio.shape))
    assert np.linalg.norm(y - plain) <= 1e-2 * np.linalg.norm(plain)


LINEAR_SIZES = [
    # rows: every row tile and one past it; depth: whole blocks, a tail of 16, one short block; widths: odd, narrow
    (1, 16, 16), (1, 1, 128), (1, 300, 272), (2, 128, 4096), (5, 129, 400), (15, 64, 1024), (16, 1000, 2048),
    (17, 520, 656), (31, 257, 1152), (32, 4096, 512), (33, 640, 2064), (48, 200, 3712), (64, 384, 1536), (65, 130, 384),
    (96, 264, 896), (128, 512, 2560), (129, 1032, 528), (200, 96, 4096), (255, 255, 640), (256, 768, 1024),
    (257, 640, 144), (400, 1544, 272), (513, 520, 1280), (1000, 1000, 256), (1500, 2056, 400), (1024, 3000, 640),
]


@pytest.mark.parametrize("M,N,K", LINEAR_SIZES)
def test_linear(M, N, K):
    case(f"linear {M}x{N}x{K}")
    xq, xs = block.quantize_act(up(rows_bits(M, K, M + K, spread=True)))
    q = weight(N, K, N + K)
    bias = rows_bits(1, N, N)[0] if (M + N) % 2 else None
    out = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    y = C.bf16_to_f32(host(block.linear(xq, xs, q, None if bias is None else up(bias), out=out))).astype(np.float64)
    check_product(y, (host(xq), host(xs), host(q["codes"]), host(q["scales"])), bias)


@pytest.mark.parametrize("M,N,K", [(1, 200, 5632), (3, 2500, 6160), (30, 1000, 7424), (64, 136, 16400)])
def test_linear_long_and_narrow(M, N, K):
    """Two blocks of a wave under way; runs of blocks that end in the middle of a wave's share."""
    test_linear(M, N, K)


@pytest.mark.parametrize("M,N,K", [(2048, 2304, 1280), (1900, 4000, 272), (4096, 2048, 2048), (3000, 2500, 1040)])
def test_linear_large(M, N, K):
    """Whole outputs of the large-tile forms."""
    case(f"linear large {M}x{N}x{K}")
    xq, xs = block.quantize_act(up(rows_bits(M, K, M + K, spread=True)))
    q = weight(N, K, N + K)
    y = C.bf16_to_f32(host(block.linear(xq, xs, q))).astype(np.float64)
    check_product(y, (host(xq), host(xs), host(q["codes"]), host(q["scales"])))


@pytest.mark.parametrize("M,N,K", [(4300, 4096, 528), (1025, 8190, 528)])
def test_linear_rest_of_a_round(M, N, K):
    """A few tiles more than the chip holds at once, of each form that splits those: every output row and column piece."""
    case(f"linear rest {M}x{N}x{K}")
    xq, xs = block.quantize_act(up(rows_bits(M, K, M + K, spread=True)))
    q = weight(N, K, N + K)
    out = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    y = C.bf16_to_f32(host(block.linear(xq, xs, q, out=out))).astype(np.float64)
    assert np.isfinite(y).all()
    hx, hs, hw, hv = host(xq), host(xs), host(q["codes"]), host(q["scales"])
    rows = np.unique(np.concatenate([np.arange(0, M, 16), np.arange(max(0, M - 140), M)]))
    check_product(y[rows], (hx[rows], hs[rows], hw, hv))


@pytest.mark.parametrize("counts,N,K", [([1, 0, 2], 1000, 2064), ([17, 0, 5, 1] * 5, 392, 528), ([1, 0, 2], 600, 5776),
                                        ([16, 0, 40, 3, 1] * 26, 648, 272)])
def test_grouped_few_rows(counts, N, K):
    """16, 32 and 64 columns to a workgroup, by the number of tiles."""
    case(f"grouped few rows {len(counts)} {N}x{K}")
    check_grouped(counts, N, K, 70, 5, spare=3)


@pytest.mark.parametrize("counts,N", [([1000, 0, 1300, 2000], 4000), ([40, 700, 0, 290], 8192), ([100] * 17, 4096)])
def test_grouped_rest_of_a_round(counts, N):
    case(f"grouped rest {counts} {N}")
    check_grouped(counts, N, 400, 900, 3)


def test_linear_nan_codes_reach_their_row_and_column_only():
    case("linear NaN codes")
    M, N, K = 70, 200, 272
    xq, xs = block.quantize_act(up(rows_bits(M, K, 1)))
    q = weight(N, K, 2)
    want = host(block.linear(xq, xs, q))
    xq2, w2 = xq.clone(), q["codes"].clone()
    xq2[5, 3], w2[77, 271] = 0x7F, 0xFF
    y = C.bf16_to_f32(host(block.linear(xq2, xs, dict(q, codes=w2))))
    bad = np.zeros((M, N), bool)
    bad[5], bad[:, 77] = True, True
    assert np.isnan(y[bad]).all() and np.array_equal(C.f32_to_bf16(y)[~bad], want[~bad])


def groups(counts, seed, M=None):
    """(offsets, rows) of the counts, rows drawn from M source rows."""
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows = None if M is None else np.random.default_rng(seed).integers(0, M, off[-1]).astype(np.int32)
    return off, rows


def check_grouped(counts, N, K, M, seed, spare=0):
    E = len(counts)
    off, rows = groups(counts, seed, M)
    T = int(off[-1]) + spare
    if rows is None:
        M = T
    else:
        rows = np.concatenate([rows, np.zeros(spare, np.int32)])
    xq, xs = block.quantize_act(up(rows_bits(M, K, seed, spread=True)))
    q = weight(N, K, seed + 1, E)
    out = torch.full((T, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    y = block.grouped_linear(xq, xs, q, torch.from_numpy(off).to(DEV),
                             rows=None if rows is None else torch.from_numpy(rows).to(DEV), out=out)
    y = C.bf16_to_f32(host(y)).astype(np.float64)
    hx, hs, hw, hv = host(xq), host(xs), host(q["codes"]), host(q["scales"])
    assert np.isnan(y[off[-1]:]).all(), "rows past the last expert were written"
    for e in range(E):
        at = np.arange(off[e], off[e + 1])
        if not at.size:
            continue
        src = at if rows is None else rows[at]
        check_product(y[at], (hx[src], hs[src], hw[e], hv[e]))


GROUPS = {
    "one row": [1],
    "empty ends": [0, 3, 0, 0, 17, 0],
    "ragged": [5, 16, 0, 33, 1, 64, 15, 2],
    "one takes all": [0, 0, 150, 0],
    "many experts": [i % 5 for i in range(150)],
    "tiles": [127, 128, 129, 255, 256, 257, 1],
    "large": [700, 0, 1300, 48],
}


@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("N,K", [(64, 128), (200, 400), (520, 656)])
def test_grouped_linear(name, N, K):
    counts = GROUPS[name]
    case(f"grouped {name} {N}x{K}")
    check_grouped(counts, N, K, None, 11)
    check_grouped(counts, N, K, 40, 12, spare=5)


def test_grouped_edges():
    case("grouped edges")
    N, K, E = 136, 272, 4
    xq, xs = block.quantize_act(up(rows_bits(9, K, 1)))
    q = weight(N, K, 2, E)
    # no rows at all; every expert empty: nothing is written
    assert block.grouped_linear(xq[:0], xs[:0], q, torch.zeros(E + 1, dtype=torch.int32, device=DEV)).shape == (0, N)
    out = torch.full((9, N), 7.0, dtype=torch.bfloat16, device=DEV)
    block.grouped_linear(xq, xs, q, torch.zeros(E + 1, dtype=torch.int32, device=DEV), out=out)
    assert bool((out == 7.0).all())
    # offsets outside [0, T] are clamped, rows outside [0, M) read as zeros
    off = torch.tensor([0, 4, 4, 9, 1000], dtype=torch.int32, device=DEV)
    rows = torch.tensor([0, -1, 8, 9, 1, 2, 1 << 30, 3, 4], dtype=torch.int32, device=DEV)
    y = host(block.grouped_linear(xq, xs, q, off, rows=rows, out=out))
    zero = [1, 3, 6]
    assert (y[zero] & 0x7FFF == 0).all()
    good = torch.tensor([0, 0, 8, 0, 1, 2, 0, 3, 4], dtype=torch.int32, device=DEV)
    want = host(block.grouped_linear(xq, xs, q, off, rows=good))
    keep = [0, 2, 4, 5, 7, 8]
    assert np.array_equal(y[keep], want[keep])


@pytest.mark.parametrize("counts", [[3, 4], [40, 30, 0, 60]])
def test_rows_without_a_source_are_zero_beside_nan(counts):
    """A row index outside the source reads zeros, whatever scales row 0 has."""
    case(f"grouped rows without a source {counts}")
    N, K, E = 136, 272, len(counts)
    off, rows = groups(counts, 1, 9)
    rows[rows == 0] = 1
    rows[::3] = np.resize([-1, 9, 1 << 30], rows[::3].shape)
    xq, xs = block.quantize_act(up(rows_bits(9, K, 1)))
    q = weight(N, K, 2, E)
    xs[0] = float("nan")
    y = host(block.grouped_linear(xq, xs, q, torch.from_numpy(off).to(DEV), rows=torch.from_numpy(rows).to(DEV)))
    assert (y[::3] & 0x7FFF == 0).all() and np.isfinite(C.bf16_to_f32(y)).all()


def test_grouped_over_many_experts():
    """More experts than a wave's 64 lanes, the last ones in reach of every row tile."""
    case("grouped over 1000 experts")
    E, N, K = 1000, 40, 144
    counts = np.zeros(E, np.int64)
    counts[[0, 63, 64, 127, 500, 998, 999]] = [3, 1, 20, 2, 17, 1, 5]
    check_grouped(list(counts), N, K, 12, 21)


def test_weights_past_32_bit_offsets():
    """More than 2^32 bytes of weights: the last expert's product."""
    E, N, K = 67, 2048, 32768
    case(f"grouped {E}x{N}x{K}")
    gen = torch.Generator(device=DEV).manual_seed(3)
    codes = torch.randint(0, 0x60, (E, N, K), dtype=torch.uint8, device=DEV, generator=gen)  # finite, nonnegative
    scales = torch.rand(E, N // 128, K // 128, device=DEV, generator=gen) + 0.5
    q = {"E": E, "N": N, "K": K, "codes": codes, "scales": scales}
    xq, xs = block.quantize_act(up(rows_bits(20, K, 4)))
    for T, e in ((20, E - 1), (7, E - 2)):
        off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
        off[e + 1:] = T
        y = block.grouped_linear(xq[:T].contiguous(), xs[:T].contiguous(), q, off).double()
        f8 = torch.float8_e4m3fn
        x = xq[:T].view(f8).double() * xs[:T].double().repeat_interleave(128, 1)
        w = codes[e].view(f8).double() * scales[e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
        ref, S = x @ w.T, x.abs() @ w.abs().T
        bound = ref.abs() * 2.0**-7 + (256 + K // 128 + 20) * 2.0**-24 * S * (1 + 2.0**-7)
        assert bool(((y - ref).abs() <= bound).all())


# ---------------------------------------------------------------- use


def test_same_bits_again_on_other_streams_and_in_a_graph():
    case("repeat, stream, graph")
    M, N, K, E = 37, 272, 656, 5
    x, r, g = up(rows_bits(M, K, 1)), up(rows_bits(M, K, 2)), up(rows_bits(1, K, 3)[0])
    q1 = weight(2 * N, K, 4, E)
    off = torch.tensor([0, 5, 5, 20, 36, 37], dtype=torch.int32, device=DEV)
    bufs = {"a": (torch.empty(M, K, dtype=torch.uint8, device=DEV), torch.empty(M, 6, device=DEV)),
            "h": torch.empty_like(x), "gu": torch.empty(M, 2 * N, dtype=torch.bfloat16, device=DEV)}
    bufs["c"] = torch.empty(M, N, dtype=torch.uint8, device=DEV), torch.empty(M, 3, device=DEV)

    def step():
        xq, xs, h, _ = block.add_rmsnorm_quantize(x, g, residual=r, out=bufs["a"], residual_out=bufs["h"])
        gu = block.grouped_linear(xq, xs, q1, off, out=bufs["gu"])
        return [xq, xs, h, gu, *block.silu_mul_quantize(gu, out=bufs["c"])]

    want = [host(t).copy() for t in step()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = step()
    torch.cuda.current_stream().wait_stream(s)
    assert all(np.array_equal(a, host(b)) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        assert all(np.array_equal(a, host(b)) for a, b in zip(want, out))
        assert all(np.array_equal(a, host(b)) for a, b in zip(want, step()))


def test_refusals():
    case("refusals")
    M, N, K = 4, 40, 144
    x = up(rows_bits(M, K, 1))
    xq, xs = block.quantize_act(x)
    q = weight(N, K, 2)
    g = up(rows_bits(1, K, 3)[0])
    bad = [
        lambda: block.quantize_act(x.float()),
        lambda: block.quantize_act(x.cpu()),
        lambda: block.quantize_act(x[:, :136].contiguous()),      # K % 16
        lambda: block.quantize_act(x.t()),                        # strided elements
        lambda: block.quantize_act(x, out=(xq[:3], xs)),
        lambda: block.quantize_act(x, out=(xq, xs.double())),
        lambda: block.silu_mul_quantize(x[:, :16].contiguous()),  # 8 values: K % 16
        lambda: block.add_rmsnorm_quantize(x, g[:128]),
        lambda: block.add_rmsnorm_quantize(x, g, eps=-1.0),
        lambda: block.add_rmsnorm_quantize(x, g, eps=float("nan")),
        lambda: block.add_rmsnorm_quantize(x, g, residual=x.float()),
        lambda: block.add_rmsnorm_quantize(x, g, residual=x[:, ::2]),
        lambda: block.linear(xq, xs[:, :1].contiguous(), q),
        lambda: block.linear(xq.view(torch.int8), xs, q),
        lambda: block.linear(xq, xs, q, bias=g[:N].float()),
        lambda: block.linear(xq[:, :128].contiguous(), xs, q),
        lambda: block.linear(xq, xs, q, out=torch.empty(M, N, device=DEV)),
        lambda: block.grouped_linear(xq, xs, q, torch.zeros(2, dtype=torch.int32, device=DEV)),
        lambda: block.grouped_linear(xq, xs, weight(N, K, 2, 3), torch.zeros(4, device=DEV)),
        lambda: block.grouped_linear(xq, xs, weight(N, K, 2, 3), torch.zeros(3, dtype=torch.int32, device=DEV)),
        lambda: block.grouped_linear(xq, xs, weight(N, K, 2, 3), torch.zeros(4, dtype=torch.int32, device=DEV),
                                     rows=torch.zeros(4, dtype=torch.int64, device=DEV)),
        lambda: block.quantize_weight(x.float()),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            print("not refused:", i)
    # empty calls are valid
    assert block.linear(xq[:0], xs[:0], q).shape == (0, N)
    assert block.quantize_act(x[:0])[0].shape == (0, K)
