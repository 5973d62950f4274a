"""Weights of a softmax that is not renormalized, of choices by logits: fp64 throughout and rounded once to fp32.

The terms are within a few 2^-52 of themselves and at most 1024 of them added in chains of 16 and trees of 6, all
positive: the sum is within 2^-48, the weight within 2^-47 before its rounding, u = 2^-24."""

import numpy as np
import pytest
import torch

from int8_bound import U
from oracle import experts as X
from test_gpu_block import DEV, case, host
from test_gpu_experts import logits_of

experts = pytest.importorskip("weight_only_bit_dequant_amd.experts")

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("spread", [0.01, 1.0, 30.0])
@pytest.mark.parametrize("M,E,top,G", [(1, 128, 8, 1), (5, 1000, 9, 1), (40, 60, 4, 1), (64, 128, 8, 1), (300, 256, 8, 1), (900, 60, 4, 1), (1100, 256, 8, 8),
                                       (1500, 512, 6, 1), (4100, 16, 2, 1), (4100, 60, 4, 1), (4100, 128, 8, 4), (4100, 256, 8, 1), (4100, 500, 3, 1),
                                       (4100, 1024, 8, 1), (200, 60, 4, 6)])
def test_softmax_weights_as_they_are(M, E, top, G, spread, half):
    case(f"route weights {M} of {E} x {spread} half={half}")
    l = spread * logits_of(M, E, M + E)
    l[M // 2, :: 3] = -float("inf")
    l = l.to(torch.bfloat16) if half else l
    kw = dict(groups=G, keep_groups=max(1, G // 2))
    r = experts.route(l.to(DEV), top, renormalize=False, scale=1.5, **kw)
    at = sorted({0, M // 2, M - 1, *range(0, M, max(1, M // 100))})
    got, ids = host(r.weights)[at].astype(np.float64), host(r.ids)[at]
    for i, m in enumerate(at):
        want_ids, want = X.route_token(l[m].double().numpy(), top, groups=G, keep=kw["keep_groups"], renormalize=False, scale=1.5)
        assert np.array_equal(ids[i], want_ids)
        off = np.abs(got[i] - want)
        assert (off <= (U + 2.0**-46) * want + 2.0**-149).all(), (off / want / U).max()
