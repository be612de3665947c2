"""Gradient clipping with the largest bounds: infinity asks for the norm alone and leaves gradients that
are not finite, a finite bound makes them zeros, however large it is."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("max_norm", [3.4e38, 3.5e38, 1e39, 1e308])
def test_a_finite_bound_beyond_float32_is_not_infinity(max_norm):
    import torch

    import differentiable_gaussian_splatting_gb300 as gs

    norm = torch.zeros(1, device="cuda")
    ws = torch.empty(gs.gs_clip_grad_norm_workspace_bytes(2), dtype=torch.uint8, device="cuda")
    g = [torch.randn(20000, device="cuda"), torch.randn(7, device="cuda").bfloat16()]
    kept = [t.clone() for t in g]
    gs.gs_clip_grad_norm(g, max_norm, norm, ws)
    assert all(torch.equal(a, b) for a, b in zip(g, kept)) and np.isfinite(norm.item())
    for value in (float("inf"), float("nan")):
        for bound, zero in ((max_norm, True), (float("inf"), False)):
            g = [t.clone() for t in kept]
            g[0][12345] = value
            gs.gs_clip_grad_norm(g, bound, norm, ws)
            assert not np.isfinite(norm.item())
            if zero:
                assert all((t == 0).all() for t in g)
            else:
                assert torch.equal(g[1], kept[1]) and torch.equal(g[0][:12345], kept[0][:12345])
    with pytest.raises(gs.GSError):
        gs.gs_clip_grad_norm(kept, -1e39, norm, ws)
