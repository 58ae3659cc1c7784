"""Refusals of the serving calls' binding (no GPU): arguments that the C entry points
cannot see are wrong."""
import pytest
import torch

import block_scaled_fp4_amax_amd as fq


@pytest.mark.parametrize("codes,scales", [(torch.int32, torch.uint8), (torch.uint8, torch.int32),
                                          (torch.uint8, torch.float32), (torch.int16, torch.int16)])
def test_linear_refuses_wider_codes_and_scales(codes, scales):
    """A wider type of the same shape is large enough and would be read as bytes."""
    w = {"codes": torch.zeros(4, 16, dtype=codes), "scales": torch.zeros(4, 2, dtype=scales), "outer": None}
    with pytest.raises(ValueError, match="bytes"):
        fq.fp4_linear(torch.zeros(2, 32, dtype=torch.bfloat16), w, fq.make_cfg())
