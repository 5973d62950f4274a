"""The block-scaled operators' C ABI rejects bad arguments on the host before
touching HIP, and exports every symbol its header declares (no GPU needed)."""

import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "wq_block.h")

wq = pytest.importorskip("weight_only_bit_dequant_amd.wq")
block = pytest.importorskip("weight_only_bit_dequant_amd.block")

if not os.path.exists(wq.LIB_PATH):  # pragma: no cover
    pytest.skip("libwq.so not built", allow_module_level=True)

V = ctypes.c_void_p


def test_every_declared_symbol_is_exported():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(wq_block_[a-z0-9_]+)\s*\(", text)))
    assert len(names) == 6
    for n in names:
        assert hasattr(block._lib(), n), n


def act(X=16, ldx=144, M=4, K=144, Xq=16, Xs=4):
    return block._lib().wq_block_quantize_act(V(X), ldx, M, K, V(Xq), V(Xs), None)


def gate(X=16, ldx=288, M=4, K=144, Xq=16, Xs=4):
    return block._lib().wq_block_silu_mul_quantize(V(X), ldx, M, K, V(Xq), V(Xs), None)


def norm(X=16, ldx=144, R=16, G=16, eps=1e-5, M=4, K=144, Xq=16, Xs=4, Ro=16, Yo=16):
    return block._lib().wq_block_add_rmsnorm_quantize(V(X), ldx, V(R), V(G), eps, M, K, V(Xq), V(Xs), V(Ro), V(Yo), None)


def weight(W=16, E=1, N=4, K=144, C=16, S=4):
    return block._lib().wq_block_quantize_weight(V(W), E, N, K, V(C), V(S), None)


def linear(X=16, Xs=4, M=4, K=144, W=16, Ws=4, B=2, N=24, Y=16):
    return block._lib().wq_block_linear(V(X), V(Xs), M, K, V(W), V(Ws), V(B), N, V(Y), None)


def grouped(X=16, Xs=4, M=4, K=144, R=4, O=4, T=8, E=3, W=16, Ws=4, N=24, Y=16):
    return block._lib().wq_block_grouped_linear(V(X), V(Xs), M, K, V(R), V(O), T, E, V(W), V(Ws), N, V(Y), None)


@pytest.mark.parametrize("call", [act, gate, norm])
def test_row_operators(call):
    assert call(M=-1) == wq.EINVAL
    assert call(K=-16) == wq.EINVAL
    assert call(K=136) == wq.ESHAPE
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


def test_too_many_blocks():
    assert act(M=1 << 30, K=256, ldx=256) == wq.EUNSUPPORTED
    assert gate(M=1 << 30, K=256, ldx=512) == wq.EUNSUPPORTED
    assert act(M=1 << 27, K=128, ldx=128) == wq.EUNSUPPORTED
    assert norm(M=1 << 26, K=128, ldx=128) == wq.EUNSUPPORTED


def test_norm():
    assert norm(G=None) == wq.EINVAL
    assert norm(G=8) == wq.EALIGN
    assert norm(R=8) == wq.EALIGN
    assert norm(Ro=8) == wq.EALIGN
    assert norm(Yo=8) == wq.EALIGN
    assert norm(eps=-1e-5) == wq.EINVAL
    assert norm(eps=float("inf")) == wq.EINVAL
    assert norm(eps=float("nan")) == wq.EINVAL
    assert norm(K=32784, ldx=32784) == wq.EUNSUPPORTED
    assert norm(X=32, Ro=32, ldx=160) == wq.EINVAL  # in place over strided rows
    assert b"contiguous" in wq.lib().wq_last_error()


def test_weight():
    assert weight(E=-1) == wq.EINVAL
    assert weight(N=-1) == wq.EINVAL
    assert weight(K=100) == wq.ESHAPE
    assert weight(W=None) == wq.EINVAL
    assert weight(C=8) == wq.EALIGN
    assert weight(S=1) == wq.EALIGN
    assert weight(E=65536) == wq.EUNSUPPORTED
    assert weight(N=1 << 24) == wq.EUNSUPPORTED
    assert weight(E=0, W=None) == wq.OK
    assert weight(N=0, W=None) == wq.OK


@pytest.mark.parametrize("call", [linear, grouped])
def test_products(call):
    assert call(M=-1) == wq.EINVAL
    assert call(N=-1) == wq.EINVAL
    assert call(K=24) == wq.ESHAPE
    assert call(K=0) == wq.EUNSUPPORTED
    assert call(K=1 << 22) == wq.EUNSUPPORTED
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


def test_python_checks_need_no_library():
    import torch

    x = torch.zeros(2, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        block.quantize_act(x)
    with pytest.raises(ValueError):
        block.quantize_weight(x)
    q = {"E": 1, "N": 4, "K": 16, "codes": torch.zeros(4, 16, dtype=torch.uint8), "scales": torch.zeros(1, 1)}
    with pytest.raises(ValueError):
        block.linear(torch.zeros(2, 16, dtype=torch.uint8), torch.zeros(2, 1), q)
