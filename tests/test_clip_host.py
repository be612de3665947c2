"""Gradient clipping without a GPU: what the binding does with the largest norm it is given."""

import pytest


@pytest.mark.parametrize("max_norm", [1e39, 3.5e38, 1e308])
def test_a_largest_norm_beyond_float32_is_not_taken_for_infinity(max_norm):
    # Infinity asks for the norm alone and leaves gradients that are not finite; a finite bound, however
    # large, makes them zeros.  One that float32 does not hold is refused.
    import torch
    from torch._subclasses.fake_tensor import FakeTensorMode

    import differentiable_gaussian_splatting_gb300 as gs

    with FakeTensorMode():
        norm = torch.empty(1, device="cuda")
        ws = torch.empty(1 << 13, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="max_norm: .* is beyond float32"):
        gs.gs_clip_grad_norm([], max_norm, norm, ws, stream=0)
