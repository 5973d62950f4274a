"""The C ABI of the 8-bit integer operators and of the experts' routing rejects
bad arguments on the host before touching HIP, and exports every symbol its
headers declare (no GPU needed)."""

import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

wq = pytest.importorskip("weight_only_bit_dequant_amd.wq")
int8 = pytest.importorskip("weight_only_bit_dequant_amd.int8")
experts = pytest.importorskip("weight_only_bit_dequant_amd.experts")

if not os.path.exists(wq.LIB_PATH):  # pragma: no cover
    pytest.skip("libwq.so not built", allow_module_level=True)

V = ctypes.c_void_p


@pytest.mark.parametrize("header,prefix,count", [("wq_int8.h", "wq_int8_", 5), ("wq_experts.h", "wq_experts_", 3)])
def test_every_declared_symbol_is_exported(header, prefix, count):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(%s[a-z0-9_]+)\s*\(" % prefix, text)))
    assert len(names) == count
    for n in names:
        assert hasattr(wq.lib(), n), n


def act(X=16, ldx=144, M=4, K=144, Xq=16, Xs=4):
    return int8._lib().wq_int8_quantize_act(V(X), ldx, M, K, V(Xq), V(Xs), None)


def gate(X=16, ldx=288, M=4, K=144, Xq=16, Xs=4):
    return int8._lib().wq_int8_silu_mul_quantize(V(X), ldx, M, K, V(Xq), V(Xs), None)


def weight(W=16, E=1, N=4, K=144, C=16, S=4):
    return int8._lib().wq_int8_quantize_weight(V(W), E, N, K, V(C), V(S), None)


def linear(X=16, Xs=4, M=4, K=144, W=16, Ws=4, B=2, N=24, Y=16):
    return int8._lib().wq_int8_linear(V(X), V(Xs), M, K, V(W), V(Ws), V(B), N, V(Y), None)


def grouped(X=16, Xs=4, M=4, K=144, R=4, O=4, T=8, E=3, W=16, Ws=4, N=24, Y=16):
    return int8._lib().wq_int8_grouped_linear(V(X), V(Xs), M, K, V(R), V(O), T, E, V(W), V(Ws), N, V(Y), None)


def route(L=4, bits=32, ld=12, M=6, E=12, top=2, score=0, B=4, G=3, keep=2, pairs=0, renorm=1, scale=1.0, valid=1, I=4, W=4, O=4, R=4,
          P=4, WS=None, ws=0):
    return experts._lib().wq_experts_route(V(L), bits, ld, M, E, top, score, V(B), G, keep, pairs, renorm, scale, V(valid), V(I), V(W), V(O),
                                           V(R), V(P), V(WS), ws, None)


def combine(Y=16, T=5, N=24, P=4, W=4, M=6, top=2, B=16, O=16):
    return experts._lib().wq_experts_combine(V(Y), T, N, V(P), V(W), M, top, V(B), V(O), None)


@pytest.mark.parametrize("call", [act, gate])
def test_row_operators(call):
    assert call(M=-1) == wq.EINVAL
    assert call(K=-16) == wq.EINVAL
    assert call(K=136) == wq.ESHAPE
    assert call(K=1 << 17) == wq.EUNSUPPORTED
    assert call(X=None) == wq.EINVAL
    assert call(Xq=None) == wq.EINVAL
    assert call(Xs=None) == wq.EINVAL
    assert call(ldx=136) == wq.EINVAL       # shorter than a row
    assert call(ldx=292) == wq.EALIGN
    assert call(X=8) == wq.EALIGN
    assert call(Xq=24) == wq.EALIGN
    assert call(Xs=2) == wq.EALIGN
    assert call(M=(1 << 30) + 1) == wq.EUNSUPPORTED
    assert call(M=0, X=None) == wq.OK
    assert call(K=0, X=None) == wq.OK
    assert b"" == wq.lib().wq_last_error()


def test_weight():
    assert weight(E=-1) == wq.EINVAL
    assert weight(N=-1) == wq.EINVAL
    assert weight(K=100) == wq.ESHAPE
    assert weight(W=None) == wq.EINVAL
    assert weight(C=8) == wq.EALIGN
    assert weight(S=1) == wq.EALIGN
    assert weight(E=1 << 20, N=1 << 20) == wq.EUNSUPPORTED
    assert weight(E=1 << 62, N=1 << 30) == wq.EUNSUPPORTED
    assert weight(E=0, W=None) == wq.OK
    assert weight(N=0, W=None) == wq.OK


@pytest.mark.parametrize("call", [linear, grouped])
def test_products(call):
    assert call(M=-1) == wq.EINVAL
    assert call(N=-1) == wq.EINVAL
    assert call(K=24) == wq.ESHAPE
    assert call(K=0) == wq.EUNSUPPORTED
    assert call(K=1 << 17) == wq.EUNSUPPORTED
    assert call(N=(1 << 30) + 1) == wq.EUNSUPPORTED
    for p in ("X", "Xs", "W", "Ws", "Y"):
        assert call(**{p: None}) == wq.EINVAL
    for p in ("X", "W", "Y"):
        assert call(**{p: 8}) == wq.EALIGN
    for p in ("Xs", "Ws"):
        assert call(**{p: 2}) == wq.EALIGN
    assert call(N=0, W=None) == wq.OK


def test_linear_alone():
    assert linear(B=1) == wq.EALIGN
    assert linear(M=0, X=None) == wq.OK


def test_grouped_alone():
    assert grouped(O=None) == wq.EINVAL
    assert grouped(O=2) == wq.EALIGN
    assert grouped(R=2) == wq.EALIGN
    assert grouped(T=-1) == wq.EINVAL
    assert grouped(E=-1) == wq.EINVAL
    assert grouped(R=None) == wq.EINVAL             # M != T without rows
    assert grouped(M=0) == wq.EINVAL                # rows of no source
    assert grouped(M=1 << 20, K=4096) == wq.EUNSUPPORTED
    assert grouped(E=(1 << 20) + 1) == wq.EUNSUPPORTED
    assert grouped(T=0, O=None) == wq.OK
    assert grouped(E=0, O=None) == wq.OK


def test_route():
    for p in ("L", "I", "W", "O", "R", "P"):
        assert route(**{p: None}) == wq.EINVAL
        assert route(**{p: 2}) == wq.EALIGN
    assert route(L=2, bits=16) != wq.EALIGN
    assert route(L=1, bits=16) == wq.EALIGN
    assert route(B=2) == wq.EALIGN
    assert route(M=-1) == wq.EINVAL
    assert route(E=0) == wq.EINVAL
    assert route(top=0) == wq.EINVAL
    assert route(top=13) == wq.EINVAL
    assert route(bits=8) == wq.EINVAL
    assert route(score=2) == wq.EINVAL
    assert route(G=0) == wq.EINVAL
    assert route(keep=0) == wq.EINVAL
    assert route(keep=4) == wq.EINVAL
    assert route(G=5) == wq.ESHAPE
    assert route(ld=11) == wq.EINVAL
    assert route(E=1025, ld=1025, G=1, keep=1) == wq.EUNSUPPORTED
    assert route(E=64, ld=64, top=33, G=1, keep=1) == wq.EUNSUPPORTED
    assert route(E=130, ld=130, G=65, keep=1) == wq.EUNSUPPORTED
    assert route(M=1 << 29) == wq.EUNSUPPORTED
    assert route(M=1 << 62) == wq.EUNSUPPORTED
    need = experts._lib().wq_experts_route_workspace(65, 12)
    assert need == 17 * 12 * 2  # stretches of four tokens
    assert route(M=65) == wq.EWORKSPACE
    assert route(M=65, WS=4, ws=need - 1) == wq.EWORKSPACE
    assert route(M=65, WS=2, ws=need) == wq.EALIGN


def test_route_workspace():
    size = experts._lib().wq_experts_route_workspace
    assert size(0, 8) == size(-5, 8) == size(16, 8) == size(1000, 0) == size(1000, 2000) == size(1 << 40, 8) == 0
    assert size(64 * 256, 8) == 256 * 8 * 2
    # what serves many tokens and experts serves fewer
    sizes = [size(M, 60) for M in (*range(1, 5000), 16384, 16385, 65536, 65537, 1 << 20, 1 << 24, 1 << 25, 1 << 29)]
    assert sizes == sorted(sizes)
    assert all(size(700, E) <= size(700, E + 1) for E in range(1, 1024))
    for M in (65, 1000, 16384, 16385, 100000, 1 << 24):
        assert 0 < size(M, 1024) <= 257 * 1024 * 2


def test_combine():
    for p in ("Y", "P", "W", "O"):
        assert combine(**{p: None}) == wq.EINVAL
    for p in ("Y", "B", "O"):
        assert combine(**{p: 8}) == wq.EALIGN
        assert combine(N=25, **{p: 1}) == wq.EALIGN
    for p in ("P", "W"):
        assert combine(**{p: 2}) == wq.EALIGN
    for p in ("T", "N", "M", "top"):
        assert combine(**{p: -1}) == wq.EINVAL
    assert combine(M=(1 << 30) + 1) == wq.EUNSUPPORTED
    assert combine(top=1025) == wq.EUNSUPPORTED
    assert combine(M=0, Y=None) == wq.OK
    assert combine(N=0, Y=None) == wq.OK


def test_python_checks_need_no_gpu():
    import torch

    x = torch.zeros(2, 16, dtype=torch.bfloat16)
    i32 = dict(dtype=torch.int32)
    q = {"E": 1, "N": 4, "K": 16, "codes": torch.zeros(4, 16, dtype=torch.int8), "scales": torch.zeros(4)}
    for f in (lambda: int8.quantize_act(x), lambda: int8.silu_mul_quantize(x), lambda: int8.quantize_weight(x),
              lambda: int8.linear(torch.zeros(2, 16, dtype=torch.int8), torch.zeros(2), q),
              lambda: experts.route(torch.zeros(2, 8), 2), lambda: experts.route(torch.zeros(2, 8), 9),
              lambda: experts.route([1.0], 1),
              lambda: experts.combine(x, torch.zeros(2, 2, **i32), torch.zeros(2, 2))):
        with pytest.raises(ValueError):
            f()
