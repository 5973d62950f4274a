"""8-bit integer operators on the GPU against the oracle: quantizers of bf16
inputs bit for bit, the gate and the products element by element with the bounds
derived in int8_bound.py."""

import numpy as np
import pytest
import torch

from int8_bound import SILU_REL, check_codes, product_bound
from oracle import block as B
from oracle import codecs as C
from oracle import int8 as I
from test_gpu_block import DEV, GROUPS, LINEAR_SIZES, case, groups, host, rows_bits, strided, up

int8 = pytest.importorskip("weight_only_bit_dequant_amd.int8")

pytestmark = pytest.mark.gpu


def same_codes(got, scales, y):
    """Codes and scales are the definition's, but that a quotient within an ulp of a tie may go either way."""
    codes, s, v = I.quantize_rows(y)
    assert np.array_equal(scales, s, equal_nan=True)
    near = np.abs(np.abs(v - np.trunc(v)) - 0.5) <= np.abs(v) * 2.0**-23
    differ = got != codes
    assert not (differ & ~near).any() and (np.abs(got.astype(int) - codes) <= 1).all()
    assert differ.sum() <= max(2, near.sum() // 2), (differ.sum(), near.sum())


# ---------------------------------------------------------------- quantizers


@pytest.mark.parametrize("M,K", [(1, 16), (1, 512), (3, 144), (9, 528), (17, 2048), (5, 2896), (130, 656), (2, 4112), (3, 8192),
                                 (2, 8208), (1, 16400), (2, 32768), (2, 40000), (1, 131056), (3000, 272)])
@pytest.mark.parametrize("stride", [False, True])
def test_quantize_act(M, K, stride):
    case(f"int8 quantize_act {M}x{K} strided={stride}")
    x = rows_bits(M, K, M * 7 + K)
    x[M // 2] = rows_bits(1, K, 3, spread=True)[0]
    xq, xs = int8.quantize_act(strided(x) if stride else up(x))
    same_codes(host(xq), host(xs), C.bf16_to_f32(x))


def test_quantize_act_extremes():
    case("int8 quantize_act extremes")
    y = np.zeros((9, 272), np.float32)
    y[1, :2] = 3.38e38, -1e38
    y[2, :3] = 1e-38, -3e-39, 1e-40      # below 127 * 2^-126
    y[3] = -0.0
    y[4, 3], y[5, 271], y[6, 0] = np.nan, np.inf, -np.inf
    y[7] = np.arange(272) - 127.5        # ties where the largest is 144.5
    y[8, :254] = (np.arange(254) - 127) / 2 + 0.0
    y[8, 0] = 127
    x = C.f32_to_bf16(y)
    xq, xs = int8.quantize_act(up(x))
    same_codes(host(xq), host(xs), C.bf16_to_f32(x))
    # exact ties go to even: the last row's scale is 1
    assert host(xs)[8] == 1.0 and np.array_equal(host(xq)[8, :254], np.rint(C.bf16_to_f32(x)[8, :254]).astype(np.int8))
    assert np.isnan(host(xs)[4:7]).all() and (host(xq)[4:7] == 0).all()


@pytest.mark.parametrize("shape", [(1, 16), (130, 144), (3, 40, 272), (2, 5, 33024)])
def test_quantize_weight(shape):
    case(f"int8 quantize_weight {shape}")
    w = rows_bits(int(np.prod(shape[:-1])), shape[-1], sum(shape)).reshape(shape)
    q = int8.quantize_weight(up(w))
    assert (q["E"], q["N"], q["K"]) == ((1,) + shape)[-3:]
    assert q["codes"].shape == shape and q["scales"].shape == shape[:-1]
    same_codes(host(q["codes"]), host(q["scales"]), C.bf16_to_f32(w))


@pytest.mark.parametrize("M,K", [(1, 16), (1, 2048), (3, 144), (64, 1040), (17, 2896), (700, 272), (2, 5632), (1, 8192), (2, 12304), (1, 40000)])
@pytest.mark.parametrize("stride", [False, True])
def test_silu_mul_quantize(M, K, stride):
    case(f"int8 gate {M}x{K} strided={stride}")
    gu = rows_bits(M, 2 * K, M * K)
    xq, xs = int8.silu_mul_quantize(strided(gu) if stride else up(gu))
    ok, text = check_codes(host(xq), host(xs), B.silu_mul(gu), SILU_REL)
    assert ok, text


def test_silu_nonfinite():
    """+inf * 1 and anything times NaN spoil their row; -inf is NaN, a far negative gate is 0."""
    case("int8 gate non-finite")
    gu = np.ones((6, 64), np.float32)
    gu[1, 3], gu[2, 3], gu[3, 40], gu[4, 5] = np.inf, -np.inf, np.nan, -3e38
    gu[5, :32] = -3e38
    xq, xs = int8.silu_mul_quantize(up(C.f32_to_bf16(gu)))
    xq, xs = host(xq), host(xs)
    assert np.isnan(xs[1:4]).all() and (xq[1:4] == 0).all()
    assert np.isfinite(xs[[0, 4, 5]]).all() and (xq[0] == 127).all() and xq[4, 5] == 0 and xq[4, 6] == 127
    assert xs[5] == np.float32(2.0**-126) and (xq[5] == 0).all()


# ---------------------------------------------------------------- products


def codes_of(M, K, seed, E=None, full=False):
    """Random codes and scales; `full`: of +-127 (and -128, which a caller may have) alone, the largest sums."""
    g = torch.Generator().manual_seed(seed)
    shape = (M, K) if E is None else (E, M, K)
    c = torch.randint(-127, 128, shape, generator=g, dtype=torch.int8)
    if full:
        c = torch.where(c < 0, torch.tensor(-128, dtype=torch.int8), torch.tensor(127, dtype=torch.int8))
    s = torch.rand(shape[:-1], generator=g) + 0.25
    return c.to(DEV), s.to(DEV)


def weight(N, K, seed, E=None, full=False):
    c, s = codes_of(N, K, seed, E, full)
    return {"E": E or 1, "N": N, "K": K, "codes": c, "scales": s * 2.0**-12}


def exact(x, xs, w, ws, bias=None):
    """(float64 product, its and the bias's magnitude), on the device: fp64 holds the sums exactly."""
    p = (x.double() @ w.double().T) * xs.double()[:, None] * ws.double()
    b = 0.0 if bias is None else bias.double()
    ref, size = p + b, p.abs() + (0.0 if bias is None else b.abs())
    return ref.cpu().numpy(), size.cpu().numpy()


def check_product(y, ref, size):
    y = C.bf16_to_f32(host(y)).astype(np.float64)
    ratio = np.abs(y - ref) / product_bound(ref, size)
    assert ratio.max() <= 1, (ratio.max(), np.unravel_index(ratio.argmax(), ratio.shape))


def check_linear(M, N, K, full=False):
    xq, xs = codes_of(M, K, M + K, full=full)
    q = weight(N, K, N + K, full=full)
    bias = up(rows_bits(1, N, N)[0]) if (M + N) % 2 else None
    out = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    y = int8.linear(xq, xs, q, bias, out=out)
    check_product(y, *exact(xq, xs, q["codes"], q["scales"], bias))


def test_small_product_against_the_oracle():
    """The device's float64 reference of the other tests is the oracle's."""
    case("int8 linear 5x7x48 oracle")
    x, w, b = rows_bits(5, 48, 1), rows_bits(7, 48, 2), rows_bits(1, 7, 3)[0]
    xq, xs = int8.quantize_act(up(x))
    q = int8.quantize_weight(up(w))
    ref, size = I.linear(host(xq), host(xs), host(q["codes"]), host(q["scales"]), b)
    r2, s2 = exact(xq, xs, q["codes"], q["scales"], up(b))
    assert np.allclose(ref, r2, rtol=1e-14) and np.allclose(size, s2, rtol=1e-14)
    check_product(int8.linear(xq, xs, q, up(b)), ref, size)


@pytest.mark.parametrize("M,N,K", LINEAR_SIZES + [(1, 200, 5632), (3, 2500, 6160), (30, 1000, 7424), (64, 136, 16400), (17, 80, 131056)])
def test_linear(M, N, K):
    case(f"int8 linear {M}x{N}x{K}")
    check_linear(M, N, K)


@pytest.mark.parametrize("M,N,K", [(2048, 2304, 1280), (1900, 4000, 272), (3000, 2500, 1040), (4300, 4096, 528), (1025, 8190, 528)])
def test_linear_large(M, N, K):
    case(f"int8 linear large {M}x{N}x{K}")
    check_linear(M, N, K)


@pytest.mark.parametrize("M,N,K", [(1, 64, 131056), (70, 160, 131056), (300, 512, 65536)])
def test_largest_sums(M, N, K):
    """Codes of -128 and 127 throughout, and all of one sign: sums up to 2^31 - 2^18."""
    case(f"int8 linear largest sums {M}x{N}x{K}")
    check_linear(M, N, K, full=True)
    xq, xs = torch.full((M, K), -128, dtype=torch.int8, device=DEV), torch.ones(M, device=DEV)
    q = {"codes": torch.full((N, K), -128, dtype=torch.int8, device=DEV), "scales": torch.ones(N, device=DEV)}
    y = int8.linear(xq, xs, q)
    assert bool((y == torch.tensor(float(K) * 16384, dtype=torch.float64).to(torch.bfloat16).to(DEV)).all())


def test_nan_scales_reach_their_row_and_column_only():
    case("int8 linear NaN scales")
    M, N, K = 70, 200, 272
    xq, xs = codes_of(M, K, 1)
    q = weight(N, K, 2)
    want = host(int8.linear(xq, xs, q))
    xs2, w2 = xs.clone(), q["scales"].clone()
    xs2[5], w2[77] = float("nan"), float("nan")
    y = C.bf16_to_f32(host(int8.linear(xq, xs2, dict(q, scales=w2))))
    bad = np.zeros((M, N), bool)
    bad[5], bad[:, 77] = True, True
    assert np.isnan(y[bad]).all() and np.array_equal(C.f32_to_bf16(y)[~bad], want[~bad])


def check_grouped(counts, N, K, M, seed, spare=0):
    E = len(counts)
    off, rows = groups(counts, seed, M)
    T = int(off[-1]) + spare
    if rows is None:
        M = T
    else:
        rows = torch.from_numpy(np.concatenate([rows, np.zeros(spare, np.int32)])).to(DEV)
    xq, xs = codes_of(M, K, seed)
    q = weight(N, K, seed + 1, E)
    out = torch.full((T, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    y = int8.grouped_linear(xq, xs, q, torch.from_numpy(off).to(DEV), rows=rows, out=out)
    assert bool(y[int(off[-1]):].isnan().all()), "rows past the last expert were written"
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        if lo < hi:
            src = torch.arange(lo, hi, device=DEV) if rows is None else rows[lo:hi].long()
            check_product(y[lo:hi], *exact(xq[src], xs[src], q["codes"][e], q["scales"][e]))


@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("N,K", [(64, 128), (200, 400), (520, 656)])
def test_grouped_linear(name, N, K):
    case(f"int8 grouped {name} {N}x{K}")
    check_grouped(GROUPS[name], N, K, None, 11)
    check_grouped(GROUPS[name], N, K, 40, 12, spare=5)


@pytest.mark.parametrize("counts,N,K", [([1, 0, 2], 1000, 2064), ([17, 0, 5, 1] * 5, 392, 528), ([1, 0, 2], 600, 5776),
                                        ([16, 0, 40, 3, 1] * 26, 648, 272), ([1000, 0, 1300, 2000], 4000, 400),
                                        ([40, 700, 0, 290], 8192, 400), ([100] * 17, 4096, 400), ([31] * 64, 1536, 2048)])
def test_grouped_shapes(counts, N, K):
    case(f"int8 grouped shapes {sum(counts)} of {len(counts)} {N}x{K}")
    check_grouped(counts, N, K, 900, 5, spare=3)


def test_grouped_over_many_experts():
    """More experts than a wave's 64 lanes, the last ones in reach of every row tile."""
    case("int8 grouped over 1000 experts")
    counts = np.zeros(1000, np.int64)
    counts[[0, 63, 64, 127, 500, 998, 999]] = [3, 1, 20, 2, 17, 1, 5]
    check_grouped(list(counts), 40, 144, 12, 21)


def test_grouped_edges():
    case("int8 grouped edges")
    N, K, E = 136, 272, 4
    xq, xs = codes_of(9, K, 1)
    q = weight(N, K, 2, E)
    none = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    assert int8.grouped_linear(xq[:0], xs[:0], q, none).shape == (0, N)
    out = torch.full((9, N), 7.0, dtype=torch.bfloat16, device=DEV)
    int8.grouped_linear(xq, xs, q, none, out=out)
    assert bool((out == 7.0).all())
    # offsets outside [0, T] are clamped, rows outside [0, M) read as zeros whatever row 0's scale
    off = torch.tensor([0, 4, 4, 9, 1000], dtype=torch.int32, device=DEV)
    rows = torch.tensor([1, -1, 8, 9, 1, 2, 1 << 30, 3, 4], dtype=torch.int32, device=DEV)
    nan0 = xs.clone()
    nan0[0] = float("nan")
    y = host(int8.grouped_linear(xq, nan0, q, off, rows=rows, out=out))
    assert (y[[1, 3, 6]] & 0x7FFF == 0).all()
    good = torch.tensor([1, 1, 8, 1, 1, 2, 1, 3, 4], dtype=torch.int32, device=DEV)
    want = host(int8.grouped_linear(xq, nan0, q, off, rows=good))
    keep = [0, 2, 4, 5, 7, 8]
    assert np.array_equal(y[keep], want[keep])


@pytest.mark.parametrize("T,N,K,E", [(20, 2048, 32768, 67), (160, 16384, 32768, 9)])
def test_weights_past_32_bit_offsets(T, N, K, E):
    """More than 2^32 bytes of weights: the last expert's product."""
    case(f"int8 grouped {E}x{N}x{K}")
    gen = torch.Generator(device=DEV).manual_seed(3)
    codes = torch.randint(-127, 128, (E, N, K), dtype=torch.int8, device=DEV, generator=gen)
    q = {"codes": codes, "scales": torch.rand(E, N, device=DEV, generator=gen) + 0.5}
    xq, xs = codes_of(T, K, 4)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[E:] = T
    check_product(int8.grouped_linear(xq, xs, q, off), *exact(xq, xs, codes[E - 1], q["scales"][E - 1]))


# ---------------------------------------------------------------- use


def test_same_bits_again_on_other_streams_and_in_a_graph():
    case("int8 repeat, stream, graph")
    M, N, K, E = 37, 272, 656, 5
    x = up(rows_bits(M, K, 1))
    q1, q2 = weight(2 * N, K, 4, E), weight(200, N, 5)
    off = torch.tensor([0, 5, 5, 20, 36, 37], dtype=torch.int32, device=DEV)
    a = torch.empty(M, K, dtype=torch.int8, device=DEV), torch.empty(M, device=DEV)
    c = torch.empty(M, N, dtype=torch.int8, device=DEV), torch.empty(M, device=DEV)
    gu_out, y_out = (torch.empty(M, n, dtype=torch.bfloat16, device=DEV) for n in (2 * N, 200))

    def step():
        xq, xs = int8.quantize_act(x, out=a)
        gu = int8.grouped_linear(xq, xs, q1, off, out=gu_out)
        hq, hs = int8.silu_mul_quantize(gu, out=c)
        return [xq, xs, gu, hq, hs, int8.linear(hq, hs, q2, out=y_out)]

    want = [host(t).copy() for t in step()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = step()
    torch.cuda.current_stream().wait_stream(s)
    assert all(np.array_equal(u, host(v)) for u, v in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        assert all(np.array_equal(u, host(v)) for u, v in zip(want, out))
        assert all(np.array_equal(u, host(v)) for u, v in zip(want, step()))


def test_refusals():
    case("int8 refusals")
    M, N, K = 4, 40, 144
    x = up(rows_bits(M, K, 1))
    xq, xs = int8.quantize_act(x)
    q, qe = weight(N, K, 2), weight(N, K, 2, 3)
    i32 = dict(dtype=torch.int32, device=DEV)
    long = torch.zeros(1, 1 << 17, dtype=torch.bfloat16, device=DEV)
    bad = [
        lambda: int8.quantize_act(x.float()),
        lambda: int8.quantize_act(x.cpu()),
        lambda: int8.quantize_act(x[:, :136].contiguous()),      # K % 16
        lambda: int8.quantize_act(x.t()),                        # strided elements
        lambda: int8.quantize_act(x[:1].expand(M, K)),           # rows on top of each other
        lambda: int8.quantize_act(long),                         # K of 2^17
        lambda: int8.quantize_act(x, out=(xq[:3], xs)),
        lambda: int8.quantize_act(x, out=(xq, xs.double())),
        lambda: int8.quantize_act(x, out=(xq.view(torch.uint8), xs)),
        lambda: int8.silu_mul_quantize(x[:, :16].contiguous()),  # 8 values: K % 16
        lambda: int8.silu_mul_quantize(x[:, :17].contiguous()),
        lambda: int8.linear(xq, xs[:3], q),
        lambda: int8.linear(xq.view(torch.uint8), xs, q),
        lambda: int8.linear(xq, xs, q, bias=torch.zeros(N, device=DEV)),
        lambda: int8.linear(xq[:, :128].contiguous(), xs, q),
        lambda: int8.linear(xq, xs, q, out=torch.empty(M, N, device=DEV)),
        lambda: int8.linear(xq, xs, dict(q, scales=q["scales"][:3])),
        lambda: int8.linear(xq, xs, qe),
        lambda: int8.grouped_linear(xq, xs, q, torch.zeros(2, **i32)),
        lambda: int8.grouped_linear(xq, xs, qe, torch.zeros(4, device=DEV)),
        lambda: int8.grouped_linear(xq, xs, qe, torch.zeros(3, **i32)),
        lambda: int8.grouped_linear(xq, xs, qe, torch.zeros(4, **i32), rows=torch.zeros(4, dtype=torch.int64, device=DEV)),
        lambda: int8.quantize_weight(x.float()),
        lambda: int8.quantize_weight(x[:, ::2]),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            print("not refused:", i)
    # empty calls are valid
    assert int8.linear(xq[:0], xs[:0], q).shape == (0, N)
    assert int8.quantize_act(x[:0])[0].shape == (0, K)
    assert int8.quantize_weight(x[:0])["codes"].shape == (0, K)
