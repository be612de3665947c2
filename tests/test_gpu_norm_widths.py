"""Residual norms value by value: odd widths, rows that start off a word and strides of no whole words,
in both types and with and without biases and layer norms, against the float64 definition of
tests/block_ref.py with its bounds; for bfloat16 outputs half a unit in their last place, H of the
value, more."""

import numpy as np
import pytest

import block_ref as ref
from test_gpu_blocks import _close, _gs, _inputs, _params
from token_ref import H

pytestmark = pytest.mark.gpu

CASES = [  # lens, width, dtype, pre, post, gate, bias, stride, elements before the first row
    (300, 1001, "f32", "rms", "none", False, False, 1001, 0),
    (300, 1001, "f32", "rms", "rms", True, False, 1001, 0),
    (300, 1001, "f32", "none", "rms", True, False, 1002, 3),
    ([140, 0, 700, 3], 1001, "f32", "rms", "rms", True, False, 1001, 0),
    (300, 1001, "f32", "rms", "layer", True, True, 1001, 0),
    (9, 2047, "f32", "layer", "none", False, False, 2047, 1),
    (9, 2049, "f32", "layer", "layer", True, True, 2049, 0),
    (700, 2049, "f32", "rms", "rms", False, False, 2050, 0),
    (7, 4095, "f32", "rms", "rms", True, False, 4095, 0),
    (7, 4099, "f32", "rms", "rms", True, False, 4099, 0),
    (5, 8191, "f32", "layer", "rms", False, False, 8191, 0),
    (5, 8192, "f32", "layer", "layer", True, True, 8195, 2),
    (300, 1001, "bf16", "rms", "rms", True, False, 1001, 0),
    (700, 1001, "bf16", "rms", "none", False, False, 1003, 5),
    ([90, 300, 0, 7], 2049, "bf16", "layer", "layer", True, True, 2049, 0),
    (700, 2049, "bf16", "none", "rms", True, False, 2049, 0),
    (7, 4099, "bf16", "rms", "rms", True, False, 4099, 0),
    # widths of whole words in rows that are none: off a word, or of an odd stride
    (300, 1024, "f32", "rms", "rms", True, False, 1024, 1),
    (300, 1024, "bf16", "rms", "rms", True, True, 1024, 1),
    (300, 1000, "f32", "rms", "rms", False, False, 1001, 0),
    (130, 2048, "bf16", "layer", "layer", True, True, 2052, 4),
    (130, 4096, "bf16", "rms", "rms", False, False, 4097, 0),
    # ends of a lane's, a warp's and a row's values
    *[(40, w, "f32", "rms", "rms", False, False, w, 0)
      for w in (2, 7, 9, 31, 33, 255, 257, 511, 513, 769, 1023)],
    *[(40, w, "f32", "layer", "layer", True, True, w, 0) for w in (3, 127, 129, 383)],
    *[(40, w, "bf16", "rms", "layer", True, False, w, 0) for w in (1, 33, 255, 257, 1025)],
]


def _rows(values, dtype, stride, shift):
    """(the whole buffer of NaN, the rows in it)"""
    import torch

    T, width = values.shape
    flat = torch.full((shift + T * stride + 8,), float("nan"), device="cuda",
                      dtype=torch.bfloat16 if dtype == "bf16" else torch.float32)
    rows = flat[shift:].as_strided((T, width), (stride, 1))
    rows.copy_(torch.from_numpy(np.ascontiguousarray(values, np.float32)).cuda())
    return flat, rows


@pytest.mark.parametrize("case", range(len(CASES)))
def test_residual_norm_value_by_value(case):
    import torch

    gs = _gs()
    lens, width, dtype, pre, post, gate, bias, stride, shift = CASES[case]
    x, y, p, cu, dr, dh = _inputs(lens, width, dtype, pre, post, gate, bias, seed=case)
    (T, _), (alpha, beta, eps) = x.shape, (0.75, 1.5, 1e-5)
    want = ref.residual_norm(x, y, **p, cu=cu, pre=pre, post=post, alpha=alpha, beta=beta,
                             eps=float(np.float32(eps)), dr=dr, dh=dh)
    h_ = H if dtype == "bf16" else 0.0
    kw = dict(**_params(p, cu), pre=pre, post=post, alpha=alpha, beta=beta, eps=eps)
    put = lambda a: None if a is None else _rows(a, dtype, stride, shift)[1]
    new = lambda: _rows(np.full((T, width), np.nan), dtype, stride, shift)
    tx, ty, tdr, tdh = (put(a) for a in (x, y, dr, dh))
    (rf, r), (xf, gx), (yf, gy) = new(), new(), new()
    hf, h = new() if pre != "none" else (None, None)
    gs.gs_residual_norm(tx, ty, r, h, **kw)
    for n, got in (("r", r), ("h", h)):
        if got is not None:
            v, e = want[n]
            _close(got, v, h_ * (np.abs(v) + e) + e, n)
    grads = {"d" + n: torch.full_like(kw[n], float("nan")) for n in
             ("pre_weight", "pre_bias", "post_weight", "post_bias", "gate") if kw[n] is not None}
    batch = 1 if cu is None else len(cu) - 1
    size = gs.gs_residual_norm_workspace_bytes(T, width, batch)
    ws = torch.full((size + 64,), 255, dtype=torch.uint8, device="cuda")
    gs.gs_residual_norm_bwd(tx, ty, tdr, tdh, gx, gy, ws[:size], **kw, **grads)
    assert (ws[size:] == 255).all()
    for n, got in (("x", gx), ("y", gy)):
        v, e = want[n]
        _close(got, v, h_ * (np.abs(v) + e) + e, "d" + n)
    for n, got in grads.items():
        v, e = want[n[1:]]
        _close(got.view(v.shape), v, e, n)
    # what lies before, between and behind the rows stays
    for flat in (rf, hf, xf, yf):
        if flat is not None:
            outside = torch.ones_like(flat, dtype=torch.bool)
            outside[shift:].as_strided((T, width), (stride, 1)).fill_(False)
            assert torch.isnan(flat[outside]).all()
