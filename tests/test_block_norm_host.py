"""Refusals of the block norm's binding that need no GPU: they come before a tensor is looked at."""
import pytest
import torch

from moe_linear_layers_b200 import q4

X, W = torch.zeros((4, 64)), torch.ones(64)
CODES, SCALES = torch.zeros((4, 64), dtype=torch.int8), torch.zeros(4)


@pytest.mark.parametrize("given", [
    dict(xq=CODES), dict(scale_a=SCALES), dict(xq=CODES, scale_a=SCALES),           # codes are not asked for
    dict(y=X, want_y=False, quant=True), dict(residual_out=X, want_residual=False),
])
def test_an_output_that_is_not_written_is_refused(given):
    with pytest.raises(ValueError, match="would not write"):
        q4.block_norm(X, X, W, **given)


@pytest.mark.parametrize("given", [dict(xq=CODES, scale_a=SCALES, quant=True), dict(y=X), dict(residual_out=X), dict(want_y=False, quant=True)])
def test_outputs_that_are_written_pass_on(given):
    with pytest.raises(TypeError, match="CUDA tensor"):   # (the host tensors are refused next)
        q4.block_norm(X, X, W, **given)
