"""Routing of 1025 to 4096 tokens, in stretches of 16 over several workgroups, against the oracle: every number of
experts to a lane, with and without a bias, groups that lie over the lanes, padded batches; and each token's experts at
numbers of tokens on both sides of every change of stretches."""

import pytest
import torch

from test_gpu_block import DEV, case
from test_gpu_experts import check_route, logits_of

experts = pytest.importorskip("weight_only_bit_dequant_amd.experts")

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("M,E,top,G,keep,half", [(1025, 8, 2, 1, 1, False), (1025, 60, 4, 1, 1, True), (2000, 64, 6, 8, 3, False), (4096, 64, 1, 1, 1, True),
                                                 (1025, 128, 8, 4, 2, True), (2000, 100, 5, 1, 1, False), (4096, 128, 8, 1, 1, False),
                                                 (1025, 256, 8, 8, 4, False), (2000, 250, 11, 2, 1, True), (4096, 160, 6, 8, 3, False),
                                                 (1025, 1024, 8, 16, 5, False), (2000, 512, 32, 1, 1, True), (4096, 300, 3, 4, 2, False)])
def test_route_in_stretches_of_16(M, E, top, G, keep, half, biased):
    case(f"route stretches {M} of {E} top {top} {keep} of {G} biased={biased}")
    bias = 0.2 * torch.randn(E, generator=torch.Generator().manual_seed(E)) if biased else None
    valid = torch.rand(M, generator=torch.Generator().manual_seed(M)) < 0.9
    valid[M - M // 8:] = False
    check_route(logits_of(M, E, M + E, half), top, valid=valid if M != 2000 else None, bias=bias, groups=G, keep_groups=keep,
                group_score="top2" if G > 4 else "max", score="sigmoid" if E % 3 else "softmax", renormalize=M != 1025)


@pytest.mark.parametrize("E,top,G", [(8, 2, 1), (60, 4, 1), (128, 8, 4), (256, 8, 8), (500, 6, 1), (1024, 16, 8)])
@pytest.mark.parametrize("biased", [False, True])
def test_a_token_alone_and_among_others(E, top, G, biased):
    case(f"route a token among others, {E} top {top} biased={biased}")
    l = logits_of(4200, E, E).to(DEV)
    kw = dict(groups=G, keep_groups=max(1, G // 2), bias=0.1 * torch.randn(E, generator=torch.Generator().manual_seed(1)).to(DEV) if biased else None)
    want = experts.route(l, top, score="sigmoid", **kw)
    for M in (1, 4, 5, 16, 17, 64, 65, 1024, 1025, 4096, 4097):
        r = experts.route(l[:M], top, score="sigmoid", **kw)
        assert torch.equal(r.ids, want.ids[:M])
        assert torch.allclose(r.weights, want.weights[:M], rtol=2.0**-22, atol=0)
