"""Tensors of another device than the current one are refused by the token operators: a kernel on this
device would fault on them.  The tensors here are fakes of no tokens."""

import pytest

pytestmark = pytest.mark.gpu


def test_tensors_of_another_device_are_refused(monkeypatch):
    import torch
    from torch._subclasses import fake_tensor
    from torch._subclasses.fake_tensor import FakeTensorMode

    import differentiable_gaussian_splatting_gb300 as gs

    # (fakes else begin with a real tensor on their device, which may not be there)
    monkeypatch.setattr(fake_tensor, "init_gpu_context", lambda *a: None, raising=False)
    other = f"cuda:{torch.cuda.current_device() + 1}"

    def on(device):
        with FakeTensorMode():
            new = lambda *shape, dtype=torch.bfloat16: torch.empty(shape, dtype=dtype, device=device)
            return (new(0, 2, 64), new(0, 64), new(0, dtype=torch.uint8), new(2, 0, dtype=torch.float32))

    h, r, ws, lse = on(other)
    refused = [
        lambda: gs.gs_qk_norm_rope(h, h, None, None, None, None, h, h),
        lambda: gs.gs_qk_norm_rope_bwd(h, h, None, None, None, None, h, h, h, h, None, None, ws),
        lambda: gs.gs_attention_fwd(h, h, h, h, lse, ws),
        lambda: gs.gs_attention_bwd(h, h, h, h, lse, h, h, h, h, ws),
        lambda: gs.gs_attention_window_fwd(h, h, h, h, lse, ws, 1),
        lambda: gs.gs_attention_window_bwd(h, h, h, h, lse, h, h, h, h, ws, 1),
        lambda: gs.gs_residual_norm(r, r, r, r),
        lambda: gs.gs_residual_norm_bwd(r, r, r, r, r, r, ws),
        lambda: gs.gs_dropout_add(r, r, r, r, 0.0),
        lambda: gs.gs_dropout_add_bwd(r, r, r, 0.0),
        lambda: gs.gs_clip_grad_norm([r], 1.0, lse, ws),
    ]
    for call in refused:
        with pytest.raises(ValueError, match=f"is on {other}, the current device is cuda:"):
            call()
    # one of them among others of this device
    here, rows, here_ws, here_lse = on(f"cuda:{torch.cuda.current_device()}")
    for args in ((h, here, here, here, here_lse), (here, here, h, here, here_lse),
                 (here, here, here, h, here_lse), (here, here, here, here, lse)):
        with pytest.raises(ValueError, match="the current device is"):
            gs.gs_attention_window_fwd(*args, here_ws, 1)
    with pytest.raises(ValueError, match="workspace: is on"):
        gs.gs_residual_norm_bwd(rows, rows, rows, rows, rows, rows, ws)
    # all of this device: nothing to do
    gs.gs_residual_norm(rows, rows, rows, rows)
    gs.gs_attention_window_fwd(here, here, here, here, here_lse, here_ws, 1)
