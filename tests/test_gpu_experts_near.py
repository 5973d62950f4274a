"""Routing of choices that lie next to each other in 64 bits: a token's experts are the oracle's, and the same
however many tokens are routed with it (up to 4096 tokens and more of them take different kernels)."""

import numpy as np
import pytest
import torch

from test_gpu_block import DEV, case, host
from test_gpu_experts import check_route

experts = pytest.importorskip("weight_only_bit_dequant_amd.experts")

pytestmark = pytest.mark.gpu

STEP = 2.0**-49  # sixteen steps of fp64 below 1


def both_sides(l, top, **kw):
    """The oracle's experts for few tokens, and the same for those tokens among 4097 and 4352."""
    n = l.shape[0]
    few = check_route(l, top, **kw)
    gpu = {k: v.to(DEV) if isinstance(v, torch.Tensor) else v for k, v in kw.items()}
    for M in (4096, 4097, 4352):
        r = experts.route(l.to(DEV).repeat(-(-M // n), 1)[:M].contiguous(), top, **gpu)
        at = torch.arange(M, device=DEV) % n
        assert torch.equal(r.ids, few.ids[at]), (M, (r.ids != few.ids[at]).any(1).nonzero()[:4].tolist())
        assert torch.equal(r.weights.isnan(), few.weights[at].isnan())
        assert torch.allclose(r.weights, few.weights[at], rtol=2.0**-22, atol=0, equal_nan=True)


def test_saturated_sigmoids():
    """Scores just below 1: logits of 26 to 33 are some 2^-37 to 2^-48 from it."""
    case("route saturated sigmoids")
    g = torch.Generator().manual_seed(1)
    l = torch.empty(64, 256).uniform_(-3, 3, generator=g)
    at = torch.rand(64, 256, generator=g).argsort(1)
    for j, v in enumerate((33.0, 32.0, 31.0, 30.0, 29.5, 29.0, 28.5, 28.0, 27.5, 27.0, 26.5, 26.0)):
        l.scatter_(1, at[:, j : j + 1], v)
    both_sides(l, 8, score="sigmoid", bias=torch.zeros(256))
    both_sides(l, 3, score="sigmoid", bias=torch.zeros(256))
    both_sides(l, 2, score="sigmoid", bias=torch.zeros(256), groups=8, keep_groups=2, group_score="top2")
    both_sides(l, 4, score="sigmoid", groups=8, keep_groups=2, group_score="top2")


@pytest.mark.parametrize("E,top", [(40, 4), (60, 9), (128, 3), (128, 8), (256, 4), (256, 8), (250, 11), (512, 4), (510, 8), (512, 17)])
def test_order_and_border(E, top):
    """All scores alike, biases a few steps from each other, in many orders: the picks' order, the last pick and what
    lies beyond it, all nearest ones in one lane's experts, more of them than a lane orders."""
    case(f"route near order and border, {E} top {top}")
    g = torch.Generator().manual_seed(E + top)
    l = torch.full((40, E), 0.75)
    for spread in range(6):
        bias = torch.randperm(E, generator=g).double() * STEP
        if spread == 1:
            bias = -torch.arange(E).double() * STEP
        if spread == 2:
            bias = torch.arange(E).double() * STEP
        if spread == 3:  # the nearest ones next to each other, the best last
            bias = torch.where((torch.arange(E) >= 17) & (torch.arange(E) < 33), torch.arange(E) * STEP, -0.125)
        if spread == 4:  # pairs of equal ones
            bias = (torch.randperm(E, generator=g) // 2).double() * STEP
        if spread == 5:  # a few near ones about the border, far ones before
            bias = torch.where(torch.arange(E) % 5 == 0, torch.arange(E) * STEP, -0.25 * torch.rand(E, generator=g).double().round(decimals=2))
            bias[torch.randperm(E, generator=g)[: top - 1]] = 0.5
        both_sides(l, top, score="sigmoid", bias=bias.float())
        both_sides(l[:, : E // 2 * 2], top, score="sigmoid", bias=bias[: E // 2 * 2].float(), groups=2, keep_groups=1)


@pytest.mark.parametrize("E,G,keep,top", [(64, 8, 3, 4), (128, 16, 5, 8), (256, 8, 4, 8), (256, 16, 3, 4), (256, 2, 1, 8), (512, 32, 9, 6), (496, 8, 4, 8)])
@pytest.mark.parametrize("group_score", ["max", "top2"])
def test_groups_at_the_border(E, G, keep, top, group_score):
    """Groups whose values differ by few steps: their largest, and sums whose parts are of either sign."""
    case(f"route near groups, {E} in {G}")
    g = torch.Generator().manual_seed(E + G)
    per = E // G
    for kind in range(4):
        bias = torch.zeros(E, dtype=torch.float64)
        best = torch.stack([torch.randperm(per, generator=g)[:2] + per * i for i in range(G)])
        order = torch.randperm(G, generator=g).double()
        l = torch.full((30, E), 0.75)
        l[:, ::3] = 0.5
        l[:, best.flatten()] = 0.75
        if kind == 0:  # the largest by steps
            bias[best[:, 0]] = order * STEP
        if kind == 1:  # both
            bias[best[:, 0]], bias[best[:, 1]] = order * STEP, -order * STEP / 2
        if kind == 2:  # equal values, but for one group
            bias[best[:, 0]] = STEP
            bias[best[G // 2, 0]] = 2 * STEP
        if kind == 3:  # sums near zero
            bias -= 8.0
            bias[best[:, 0]], bias[best[:, 1]] = 1.0, -2.0 - 0.679178699175393 * 2 + 1
            bias[best[:, 0]] += order * 2.0**-22
        both_sides(l, min(top, keep * per), score="sigmoid", bias=bias.float(), groups=G, keep_groups=keep, group_score=group_score)


def test_equal_choices_of_narrow_logits():
    """bf16 logits and a bias of few values: many equal choices, the lowest index first."""
    case("route equal choices")
    g = torch.Generator().manual_seed(3)
    for E, top, kw in ((256, 8, {}), (256, 8, dict(groups=8, keep_groups=4, group_score="top2")), (250, 6, {}), (512, 16, {}), (64, 6, dict(groups=4, keep_groups=2)),
                       (100, 4, {})):
        l = (1.5 * torch.randn(100, E, generator=g)).to(torch.bfloat16)
        for bias in (torch.zeros(E), torch.randint(-2, 3, (E,), generator=g) * 2.0**-10):
            for score in ("sigmoid", "softmax"):
                both_sides(l, top, score=score, bias=bias, **kw)
        both_sides(torch.zeros(5, E), top, score="sigmoid", bias=torch.zeros(E), **kw)
        both_sides(torch.full((5, E), 60.0) + torch.arange(E), top, score="sigmoid", bias=torch.zeros(E), **kw)


def test_masked_and_padded_tokens_with_near_choices():
    case("route near choices, masks")
    g = torch.Generator().manual_seed(5)
    l = torch.full((64, 256), 0.75)
    l[::3] = torch.where(torch.rand(22, 256, generator=g) < 0.97, -float("inf"), 0.75)
    l[5, 40] = float("nan")
    l[6, 7:9] = float("inf")
    bias = (torch.randperm(256, generator=g) * STEP).float()
    for kw in (dict(), dict(groups=8, keep_groups=3), dict(groups=8, keep_groups=3, group_score="top2")):
        both_sides(l, 8, score="sigmoid", bias=bias, **kw)
    valid = torch.rand(4100, generator=g) < 0.5
    gpu = torch.cat([l] * 65)[:4100].to(DEV)
    r = experts.route(gpu, 8, score="sigmoid", bias=bias.to(DEV), valid=valid.to(DEV))
    want = experts.route(gpu[:64].contiguous(), 8, score="sigmoid", bias=bias.to(DEV))
    ids = want.ids[torch.arange(4100, device=DEV) % 64]
    assert np.array_equal(host(r.ids), np.where(valid.numpy()[:, None], host(ids), -1))
