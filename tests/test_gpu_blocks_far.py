"""The operators around the blocks where offsets pass 32 bits, and long windows at sampled rows, against
their float64 definitions (tests/block_ref.py), with the tolerances of tests/test_gpu_window.py and
tests/test_gpu_blocks.py."""

import numpy as np
import pytest

import block_ref as ref
from token_ref import H, U, bf16

pytestmark = pytest.mark.gpu

ROWS, STRIDE = 70000, 32768  # 2.3e9 elements


@pytest.fixture(scope="module")
def wide():
    """an array of 4.6 GB whose last rows lie beyond 2^31 elements"""
    import torch

    w = torch.empty((ROWS, STRIDE), dtype=torch.bfloat16, device="cuda")
    yield w
    del w
    torch.cuda.empty_cache()


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _close(got, want, bound, what):
    err = np.abs(_np(got) - want)
    worst = np.unravel_index(np.argmax(err - bound), err.shape)
    assert (err <= bound).all(), (what, worst, err[worst], bound[worst])


def test_residual_norm_of_far_rows(wide):
    import torch

    import differentiable_gaussian_splatting_gb300 as gs

    C = 256
    x, y, r, h, dx, dy = (wide[:, i * C:(i + 1) * C] for i in range(6))
    dr, dh = (torch.randn((ROWS, C), device="cuda").bfloat16() for _ in range(2))
    x.copy_(torch.randn((ROWS, C), device="cuda"))
    y.copy_(torch.randn((ROWS, C), device="cuda"))
    w, q = (1 + 0.1 * torch.randn(C, device="cuda") for _ in range(2))
    kw = dict(pre_weight=w, post_weight=q, post="rms")
    ws = torch.empty(gs.gs_residual_norm_workspace_bytes(ROWS, C), dtype=torch.uint8, device="cuda")
    gs.gs_residual_norm(x, y, r, h, **kw)
    gs.gs_residual_norm_bwd(x, y, dr, dh, dx, dy, ws, **kw)
    at = [0, 1, 65535, 65536, ROWS - 1]
    take = lambda t: t[at].float().cpu().numpy()
    want = ref.residual_norm(take(x), take(y), pw=take_all(w), qw=take_all(q), post="rms",
                             eps=float(np.float32(1e-6)), dr=take(dr), dh=take(dh))
    for n, got in (("r", r), ("h", h), ("x", dx), ("y", dy)):
        v, e = want[n]
        _close(got[at], v, H * (np.abs(v) + e) + e, n)


def take_all(t):
    return t.float().cpu().numpy()


@pytest.mark.parametrize("n", [1, 600])
def test_window_attention_of_far_keys(wide, n):
    # single tokens and a prompt at the end of a long cache
    import torch

    import differentiable_gaussian_splatting_gb300 as gs

    hq, hk, D, left, sinks = 4, 2, 64, 700, 4
    k = wide[:, :hk * D].view(ROWS, hk, D)
    v = wide[:, 4096:4096 + hk * D].view(ROWS, hk, D)
    k.copy_(torch.randn((ROWS, hk, D), device="cuda"))
    v.copy_(torch.randn((ROWS, hk, D), device="cuda"))
    q, do = (torch.randn((n, hq, D), device="cuda").bfloat16() for _ in range(2))
    out, lse = torch.empty_like(q), torch.empty((hq, n), device="cuda")
    ws = torch.empty(gs.gs_attention_window_workspace_bytes(n, ROWS, 1, hq, hk, D, left, 0, sinks),
                     dtype=torch.uint8, device="cuda")
    gs.gs_attention_window_fwd(q, k, v, out, lse, ws, left, 0, sinks, causal=True)
    # the same for keys that are seen alone: the sinks and the last n + left
    far = list(range(sinks)) + list(range(ROWS - n - left, ROWS))
    kk, vv = take_all(k[far]), take_all(v[far])
    o, l, mag, smag = ref.window_attention(take_all(q), kk, vv, D ** -0.5, left, 0, sinks, True)
    _close(out, o, (2 * H + 2.0 ** -12) * mag, "out")
    _close(lse, l, D * U * smag + 4 * U * (1 + np.abs(l)) + 2.0 ** -20, "lse")
    if n == 1:
        return
    dq = torch.empty_like(q)
    dk = wide[:, 8192:8192 + hk * D].view(ROWS, hk, D)
    dv = wide[:, 12288:12288 + hk * D].view(ROWS, hk, D)
    gs.gs_attention_window_bwd(q, k, v, out, lse, do, dq, dk, dv, ws, left, 0, sinks, causal=True)
    want = ref.window_attention_bwd(take_all(q), kk, vv, _np(out), _np(lse), take_all(do), D ** -0.5,
                                    left, 0, sinks, True)
    for name, t in (("q", dq), ("k", dk[far]), ("v", dv[far])):
        w, b = want[name]
        _close(t, w, b + H * np.abs(w) + 1e-30, "d" + name)
    assert (dk[sinks:ROWS - n - left] == 0).all() and (dv[sinks:ROWS - n - left] == 0).all()
    gs.gs_attention_status()


def test_clip_of_an_array_beyond_32_bits(wide):
    import torch

    import differentiable_gaussian_splatting_gb300 as gs

    flat = wide.view(-1)
    flat.zero_()
    flat[:1000], flat[-1000:] = 3.0, 4.0
    flat[2 ** 31 - 3:2 ** 31 + 3] = 12.0
    norm = torch.empty(1, device="cuda")
    ws = torch.empty(gs.gs_clip_grad_norm_workspace_bytes(1), dtype=torch.uint8, device="cuda")
    want = float(np.sqrt(1000 * 9 + 1000 * 16 + 6 * 144))
    gs.gs_clip_grad_norm([flat], want / 4, norm, ws)
    assert abs(norm.item() - want) <= 12 * U * want
    assert (flat[:1000] == 0.75).all() and (flat[-1000:] == 1.0).all()
    assert (flat[2 ** 31 - 3:2 ** 31 + 3] == 3.0).all() and (flat[1000:4000] == 0).all()


@pytest.mark.parametrize("T,hq,hk,D,left,right,causal", [
    (16320, 4, 1, 128, 1023, 0, True), (8160, 4, 2, 64, 256, 256, False), (8160, 2, 1, 72, 8160, 0, True)])
def test_long_windows_at_sampled_rows(T, hq, hk, D, left, right, causal):
    import torch

    import differentiable_gaussian_splatting_gb300 as gs

    torch.manual_seed(T + D)
    sinks = 4
    q, do = (torch.randn((T, hq, D), device="cuda").bfloat16() for _ in range(2))
    k, v = (torch.randn((T, hk, D), device="cuda").bfloat16() for _ in range(2))
    out, lse = torch.empty_like(q), torch.empty((hq, T), device="cuda")
    ws = torch.empty(gs.gs_attention_window_workspace_bytes(T, T, 1, hq, hk, D, left, right, sinks),
                     dtype=torch.uint8, device="cuda")
    gs.gs_attention_window_fwd(q, k, v, out, lse, ws, left, right, sinks, causal=causal)
    g = [torch.empty_like(t) for t in (q, k, v)]
    gs.gs_attention_window_bwd(q, k, v, out, lse, do, *g, ws, left, right, sinks, causal=causal)
    nq, nk, nv, ndo = (take_all(t).astype(np.float64) for t in (q, k, v, do))
    no, nl, scale = _np(out), _np(lse), D ** -0.5
    group, E = hq // hk, 2.0 ** -12
    rows = sorted({0, 1, 127, 128, 129, left, T // 2, T - 2, T - 1} & set(range(T)))
    for i in rows:
        seen = np.flatnonzero(ref.seen(1, i + 1, left, 0, sinks, True)[0])  # keys up to the query
        if not causal:
            seen = np.unique(np.concatenate([seen, np.arange(i, min(T, i + right + 1)), np.arange(sinks)]))
        for h in range(hq):
            kk, vv = nk[seen, h // group], nv[seen, h // group]
            s = scale * kk @ nq[i, h]
            p = np.exp(s - s.max())
            l = s.max() + np.log(p.sum())
            p /= p.sum()
            assert np.all(np.abs(no[i, h] - p @ vv) <= (2 * H + E) * (p @ np.abs(vv))), (i, h)
            size = scale * (np.abs(kk) @ np.abs(nq[i, h])).max()
            assert abs(nl[h, i] - l) <= D * U * size + 4 * U * (1 + abs(l)) + 2.0 ** -20, (i, h)
            p = np.exp(s - nl[h, i])
            delta = no[i, h] @ ndo[i, h]
            ds = p * (vv @ ndo[i, h] - delta)
            err = H * np.abs(ds) + E * p * (np.abs(vv) @ np.abs(ndo[i, h])
                                            + np.abs(no[i, h]) @ np.abs(ndo[i, h]))
            w = scale * ds @ kk
            assert np.all(np.abs(_np(g[0][i, h]) - w) <= abs(scale) * err @ np.abs(kk)
                          + H * np.abs(w) + 1e-30), (i, h)
    for j in sorted({0, sinks - 1, sinks, 127, 128, T // 3, T - 1}):
        i = np.arange(T)
        near = (j >= i - left) & (j <= i + right) | (j < sinks)
        i = i[near & (j <= i)] if causal else i[near]
        for h in range(hk):
            dk, dv, bk, bv = (np.zeros(D) for _ in range(4))
            for e in range(h * group, (h + 1) * group):
                p = np.exp(scale * nq[i, e] @ nk[j, h] - nl[e, i])
                delta, size = (no[i, e] * ndo[i, e]).sum(-1), np.abs(no[i, e] * ndo[i, e]).sum(-1)
                ds = p * (ndo[i, e] @ nv[j, h] - delta)
                err = H * np.abs(ds) + E * p * (np.abs(ndo[i, e]) @ np.abs(nv[j, h]) + size)
                dk += scale * ds @ nq[i, e]
                bk += abs(scale) * err @ np.abs(nq[i, e])
                dv += p @ ndo[i, e]
                bv += (H + E) * (p @ np.abs(ndo[i, e]))
            assert np.all(np.abs(_np(g[1][j, h]) - dk) <= bk + H * np.abs(dk) + 1e-30), ("dk", j, h)
            assert np.all(np.abs(_np(g[2][j, h]) - dv) <= bv + H * np.abs(dv) + 1e-30), ("dv", j, h)
    gs.gs_attention_status()
