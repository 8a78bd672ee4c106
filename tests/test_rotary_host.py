"""Rotary positions, differentiable: what is refused before a device is asked for (CPU only)."""
import pytest
import torch

from memory_efficient_biased_gb300.autograd import rotary


def test_frequencies_that_require_a_gradient_are_refused():
    """They would get none, without a word."""
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16, requires_grad=True)
    pos, f = torch.zeros(4, dtype=torch.int32), torch.ones(8, dtype=torch.float64, requires_grad=True)
    with pytest.raises(ValueError, match="gradient"):
        rotary(q, None, pos, f)
    with pytest.raises(ValueError, match="CUDA"):  # (as any call without a GPU)
        rotary(q, None, pos, f.detach())
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):  # no gradients are asked for
        rotary(q, None, pos, f)
