"""Window attention without a GPU: the plain definition that the GPU tests compare with is pinned, and
the host's checks refuse bad calls before anything is enqueued."""

import ctypes as C
import os
import re

import numpy as np
import pytest

import block_ref as ref
import token_ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P, MIS = 0x100000, 0x100004  # addresses that are never read


@pytest.fixture(scope="module")
def lib():
    from differentiable_gaussian_splatting_gb300 import build

    build.build()
    import differentiable_gaussian_splatting_gb300 as gs

    return gs.library()


def test_what_a_window_sees():
    # five queries at the last five of seven keys
    s = ref.seen(5, 7, 1, 1, 1, False).astype(int)
    assert s.tolist() == [[1, 1, 1, 1, 0, 0, 0], [1, 0, 1, 1, 1, 0, 0], [1, 0, 0, 1, 1, 1, 0],
                          [1, 0, 0, 0, 1, 1, 1], [1, 0, 0, 0, 0, 1, 1]]
    s = ref.seen(3, 2, 0, 5, 1, True).astype(int)  # the first query stands before the first key
    assert s.tolist() == [[0, 0], [1, 0], [1, 1]]
    assert ref.seen(3, 2, 0, 0, 2, False).all()
    full = ref.seen(6, 9, 9, 9, 0, True)
    assert (full == (np.arange(9)[None] <= np.arange(6)[:, None] + 3)).all()


@pytest.mark.parametrize("causal", [False, True])
def test_wide_windows_are_full_attention(causal):
    rng = np.random.default_rng(1)
    q, k, v = rng.normal(size=(8, 4, 8)), rng.normal(size=(9, 2, 8)), rng.normal(size=(9, 2, 8))
    cu_q, cu_k = np.array([0, 3, 3, 8]), np.array([0, 4, 6, 9])
    a = ref.window_attention(q, k, v, 0.4, 20, 20, 0, causal, cu_q, cu_k)
    b = token_ref.attention(q, k, v, 0.4, causal, cu_q, cu_k)
    for x, y in zip(a[:2], b[:2]):
        np.testing.assert_allclose(x, y, rtol=1e-12)


@pytest.mark.parametrize("window,causal", [((1, 0, 1), True), ((1, 2, 0), False), ((0, 0, 2), False)])
def test_window_gradient_equals_differences(window, causal):
    rng = np.random.default_rng(2)
    cu_q, cu_k = np.array([0, 5, 5, 9]), np.array([0, 4, 6, 11])
    q, k, v = rng.normal(size=(9, 4, 8)), rng.normal(size=(11, 2, 8)), rng.normal(size=(11, 2, 8))
    do = rng.normal(size=q.shape)
    run = lambda q, k, v: ref.window_attention(q, k, v, 0.4, *window, causal, cu_q, cu_k)
    f = lambda *a: (run(*a)[0] * do).sum()
    out, lse, _, _ = run(q, k, v)
    g = ref.window_attention_bwd(q, k, v, out, lse, do, 0.4, *window, causal, cu_q, cu_k)
    h = 1e-6
    for n, (name, arr) in enumerate((("q", q), ("k", k), ("v", v))):
        num = np.zeros_like(arr)
        for i in np.ndindex(*arr.shape):
            a, b = [q, k, v], [q, k, v]
            a[n], b[n] = arr.copy(), arr.copy()
            a[n][i] += h
            b[n][i] -= h
            num[i] = (f(*a) - f(*b)) / (2 * h)
        np.testing.assert_allclose(g[name][0], num, rtol=1e-5, atol=1e-8, err_msg=name)


def test_window_arguments_are_checked_on_the_host(lib):
    import differentiable_gaussian_splatting_gb300 as gs

    ok = dict(tokens_q=10, tokens_k=20, batch=1, heads_q=8, heads_k=2, head_dim=64, causal=0,
              scale=0.125)

    def shape(**kw):
        s = {**ok, **kw}
        return C.byref(gs.AttentionShape(*[s[f] for f, _ in gs.AttentionShape._fields_]))

    h = lambda p=P, ts=512: C.byref(gs.Heads(p, ts, 64))

    def both(w=(5, 0, 4), q=None, k=None, wsb=1 << 40, cu=(None, None), null=False, **kw):
        w = None if null else C.byref(gs.Window(*w))
        s, q, k = shape(**kw), q or h(), k or h(ts=128)
        a = lib.gs_attention_window_fwd(s, w, q, k, h(ts=128), *cu, h(), P, P, wsb, None)
        b = lib.gs_attention_window_bwd(s, w, q, k, h(ts=128), *cu, h(), P, h(), h(), h(ts=128),
                                        h(ts=128), P, wsb, None)
        assert a == b
        return a

    for kw in (dict(null=True), dict(w=(-1, 0, 0)), dict(w=(0, -1, 0)), dict(w=(0, 0, -1)),
               dict(w=(0, 0, 129)), dict(tokens_q=-1), dict(heads_q=7), dict(head_dim=136),
               dict(causal=2), dict(scale=float("nan")), dict(batch=2), dict(cu=(P, None)),
               dict(cu=(P, MIS)), dict(q=h(None)), dict(q=h(MIS)), dict(k=h(ts=124))):
        assert both(**kw) == 1, kw
    assert both(tokens_q=0, tokens_k=0) == 0
    window = gs.Window(5, 0, 4)
    need = lib.gs_attention_window_workspace_bytes(shape(), C.byref(window))
    assert need > 0 and both(wsb=need - 1) == 5
    assert need == gs.gs_attention_window_workspace_bytes(10, 20, 1, 8, 2, 64, 5, 0, 4)
    assert lib.gs_attention_window_workspace_bytes(shape(), C.byref(gs.Window(5, 0, 200))) == 0
    assert lib.gs_attention_window_workspace_bytes(shape(head_dim=4), C.byref(window)) == 0


def test_window_workspace_of_extreme_shapes(lib):
    # sizes stay in range, whatever the window, and do not divide by empty sides
    import differentiable_gaussian_splatting_gb300 as gs

    for shape in ((1 << 30, 1 << 30, 1 << 20, 1024, 1, 128), (0, 5, 1, 4, 2, 64), (5, 0, 2, 4, 2, 64),
                  (0, 0, 2, 4, 4, 8), (8160, 8160, 1, 16, 4, 128), (40, 500000, 40, 16, 4, 128)):
        for window in ((0, 0, 0), (1023, 0, 4), (2 ** 40, 2 ** 40, 128), (0, 1 << 30, 1)):
            n = gs.gs_attention_window_workspace_bytes(*shape, *window)
            tq, tk, batch, hq, hk, D = shape
            dp = 64 if D <= 64 else 128
            # the gradient's two rows, a quarter of a GB of pieces, the sinks' sums: two slots for
            # every 256 queries at most
            sinks = (2 * tq // 256 + 2) * hk * 2 * window[2] * dp * 4
            assert 8 * tq * hq <= n <= 8 * tq * hq + (1 << 28) + sinks, (shape, window)


def test_binding_refuses_bad_windows():
    import torch
    from torch._subclasses.fake_tensor import FakeTensorMode

    import differentiable_gaussian_splatting_gb300 as gs

    with FakeTensorMode():
        x = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
        lse, ws = torch.empty((2, 0), device="cuda"), torch.empty(1, dtype=torch.uint8, device="cuda")
    for bad in ((-1, 0, 0), (0, -3, 0), (0, 0, -1)):
        with pytest.raises(ValueError, match="expected a number from 0 on"):
            gs.gs_attention_window_fwd(x, x, x, x, lse, ws, *bad, stream=0)
        with pytest.raises(ValueError):
            gs.gs_attention_window_bwd(x, x, x, x, lse, x, x, x, x, ws, *bad, stream=0)
    with pytest.raises(gs.GSError):
        gs.gs_attention_window_fwd(x, x, x, x, lse, ws, 1, 0, 129, stream=0)
    with pytest.raises(TypeError):
        gs.gs_attention_window_fwd(x, x, x, x, lse, ws, "wide", stream=0)
    with pytest.raises(TypeError):
        gs.gs_attention_window_fwd(x, x, x, x, lse, ws, 1.5, stream=0)
    gs.gs_attention_window_fwd(x, x, x, x, lse, ws, 2 ** 40, 0, 4, stream=0)  # no tokens: nothing to do


def _source(name):
    path = os.path.join(ROOT, "differentiable_gaussian_splatting_gb300", "csrc", name)
    with open(path) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("file,drain,rings,once", [
    ("gs_attention_window_fwd.cu", "bar_drain", {"bar_full"}, {"bar_q[t]"}),
    ("gs_attention_window_dq.cuh", "bar_all", {"full_k", "full_v"}, {"bar_q", "bar_d"}),
    ("gs_attention_window_dkv.cuh", "sh.bar_all", {"full_q", "full_d"}, {"sh.bar_k", "sh.bar_v"})])
def test_no_copy_or_product_outlives_a_cta(file, drain, rings, once):
    # Whoever issued asynchronous work waits for it last of all, whether or not a wait has given up.
    # (What such a CTA does cannot be run: here the sources are held to it.)
    text = _source(file)
    assert len(re.findall(rf"mma_commit\(smem_u32\(&{drain}\)\);\s*"
                          rf"mbar_drain\(smem_u32\(&{drain}\), 0\);", text)) == 1
    assert set(re.findall(r"drain_ring<Sh::\w+>\((\w+), \w+\)", text)) == rings
    assert once <= set(re.findall(r"mbar_drain\(smem_u32\(&([\w.\[\]]+)\)", text))
    # a copy that is mended before it counts is waited for where that wait gives up
    assert re.search(r"mbar_wait\(bar, parity, &?dead\);\s*if \(!ok\) \{\s*mbar_drain\(bar, parity\);",
                     text)
    # every wait is one of the bounded ones
    assert not re.search(r"while\s*\(\s*!?\s*mbar_try", text)


def test_shares_of_registers_add_up():
    # a share that the launch does not have would be waited for without end: the sources' shares are
    # those of the launch, which the host checks against the kernel's own count
    for file, first in (("gs_attention_window_fwd.cu", "kSoftmaxRegisters"),
                        ("gs_attention_window_dq.cuh", "kMathRegisters")):
        text = _source(file)
        a, b = re.search(rf"{first} = (\d+), kOtherRegisters = (\d+);", text).groups()
        assert 2 * int(a) + int(b) == 3 * 168 and int(a) % 8 == 0 and int(b) % 8 == 0
        assert f"2 * {first} + kOtherRegisters == 3 * kLaunchRegisters" in text
    assert "kLaunchRegisters = 168;" in _source("gs_attention.cuh")
    assert "launch_registers_ok" in _source("gs_attention_window_fwd.cu")
    assert "launch_registers_ok" in _source("gs_attention_bwd.cu")
