"""Rows of no elements have no scale that a quantizer could leave: they are refused, no rows at all are not."""

import pytest
import torch

from test_gpu_block import DEV, case

int8 = pytest.importorskip("weight_only_bit_dequant_amd.int8")

pytestmark = pytest.mark.gpu


def test_rows_without_elements():
    case("int8 rows without elements")
    bf = dict(dtype=torch.bfloat16, device=DEV)
    for f, shape in ((int8.quantize_act, (3, 0)), (int8.silu_mul_quantize, (3, 0)), (int8.quantize_weight, (3, 0)), (int8.quantize_weight, (2, 3, 0))):
        with pytest.raises(ValueError, match="must have columns"):
            f(torch.empty(shape, **bf))
    for f in (int8.quantize_act, int8.silu_mul_quantize):
        codes, scales = f(torch.empty(0, 0, **bf))
        assert codes.shape == (0, 0) and scales.shape == (0,)
    assert int8.quantize_weight(torch.empty(0, 16, **bf))["scales"].shape == (0,)
