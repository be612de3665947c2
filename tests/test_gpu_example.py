"""The example that predicts Gaussians: its blocks' gradients against plain torch, and training."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location(
        "predict_gaussians", os.path.join(ROOT, "examples", "predict_gaussians.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _plain_heads(torch, qkv, qw, kw, table, hk):
    """HeadAttention in plain fp32 torch"""
    T, heads, D = qkv.shape
    hq, half = heads - 2 * hk, D // 2
    c, s = table[:, None, :half], table[:, None, half:]

    def side(x, w):
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
        a, b = x[..., :half], x[..., half:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    q, k, v = side(qkv[:, :hq], qw), side(qkv[:, hq:hq + hk], kw), qkv[:, hq + hk:]
    k, v = (x.repeat_interleave(hq // hk, 1) for x in (k, v))
    prob = torch.softmax(torch.einsum("ihd,jhd->hij", q, k) * D ** -0.5, -1)
    return torch.einsum("hij,jhd->ihd", prob, v)


def test_head_attention_gradients_match_plain_torch(ex):
    import torch

    torch.manual_seed(3)
    T, hq, hk, D = 77, 4, 2, 64
    table = ex.axial_table(7, 11, D)
    qkv = torch.randn(T, hq + 2 * hk, D, device="cuda").bfloat16()
    qw, kw = (1 + 0.1 * torch.randn(D, device="cuda") for _ in range(2))
    dout = torch.randn(T, hq, D, device="cuda").bfloat16()
    ours = [x.clone().requires_grad_() for x in (qkv, qw, kw)]
    out = ex.HeadAttention.apply(*ours, table, hk, None)
    out.backward(dout)
    plain = [x.clone().float().requires_grad_() for x in (qkv, qw, kw)]
    ref = _plain_heads(torch, *plain, table, hk)
    ref.backward(dout.float())
    # bfloat16 queries, keys, probabilities and outputs: 2^-8 each on the way, by norms
    for a, b in ((out, ref), *((x.grad, y.grad) for x, y in zip(ours, plain))):
        a, b = a.detach().float(), b.detach()
        assert ((a - b).norm() / b.norm()).item() < 4 * 2.0 ** -8


def test_training_falls_and_repeats(ex):
    a = ex.train(steps=200, size=96, seed=1)
    assert a[-1] < 0.6 * a[0], (a[0], a[-1])
    # the rasterizer's backward adds with atomics in the order they come: close, not equal
    b = ex.train(steps=3, size=96, seed=1)
    assert b[0] == a[0] and abs(b[2] - a[2]) < 1e-3
