"""Residual norms and gradient clipping without a GPU: the plain definitions that the GPU tests
compare with are pinned, and the host's checks refuse bad calls before anything is enqueued."""

import ctypes as C

import numpy as np
import pytest

import block_ref as ref

P, MIS = 0x100000, 0x100004  # addresses that are never read: 16-byte aligned, and not


@pytest.fixture(scope="module")
def lib():
    from differentiable_gaussian_splatting_gb300 import build

    build.build()
    import differentiable_gaussian_splatting_gb300 as gs

    return gs.library()


@pytest.fixture
def fake():
    import torch
    from torch._subclasses.fake_tensor import FakeTensorMode

    def make(*shape, dtype=torch.float32):
        with FakeTensorMode():
            return torch.empty(shape, dtype=dtype, device="cuda")

    return make


# ---------------------------------------------------------------------------
# the definitions
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("pre,post", [("rms", "none"), ("layer", "rms"), ("rms", "layer"),
                                      ("none", "layer"), ("layer", "none")])
def test_residual_norm_gradient_equals_differences(pre, post):
    rng = np.random.default_rng(3)
    T, C_, cu = 7, 6, np.array([0, 2, 2, 7])
    a = {n: rng.normal(size=s) for n, s in (("x", (T, C_)), ("y", (T, C_)), ("gate", (3, C_)))}
    if pre != "none":
        a["pw"], a["pb"] = rng.normal(1, 0.3, C_), rng.normal(size=C_)
    if post != "none":
        a["qw"], a["qb"] = rng.normal(1, 0.3, C_), rng.normal(size=C_)
    dr, dh = rng.normal(size=(T, C_)), rng.normal(size=(T, C_))
    kw = dict(cu=cu, pre=pre, post=post, alpha=1.3, beta=-0.7, eps=1e-2)

    def f(a):
        out = ref.residual_norm(**a, **kw)
        return (out["r"][0] * dr).sum() + ((out["h"][0] * dh).sum() if pre != "none" else 0.0)

    g = ref.residual_norm(**a, **kw, dr=dr, dh=dh)
    names = {"x": "x", "y": "y", "gate": "gate", "pw": "pre_weight", "pb": "pre_bias",
             "qw": "post_weight", "qb": "post_bias"}
    step = 1e-5
    for n in a:
        num = np.zeros_like(a[n])
        for i in np.ndindex(*num.shape):
            up, down = (dict(a, **{n: a[n].copy()}) for _ in range(2))
            up[n][i] += step
            down[n][i] -= step
            num[i] = (f(up) - f(down)) / (2 * step)
        np.testing.assert_allclose(g[names[n]][0], num, rtol=1e-5, atol=1e-7, err_msg=n)
    # rows of a norm without weights have root mean square 1, a layer norm's no mean
    v, _, _, _ = ref.norm(a["x"], 0 * a["x"], "layer", 0.0)
    np.testing.assert_allclose((v * v).mean(-1), 1.0, rtol=1e-12)
    np.testing.assert_allclose(v.mean(-1), 0.0, atol=1e-12)


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_bounds_hold_for_the_formulas_in_32_bits(kind):
    # numpy's fp32 arithmetic, whose sums take fewer roundings than the bound counts
    rng = np.random.default_rng(4)
    x = rng.normal(rng.normal(0, 5, (40, 1)), 1.0, (40, 96)).astype(np.float32)
    v = x - x.mean(-1, keepdims=True, dtype=np.float32) if kind == "layer" else x
    got = v / np.sqrt((v * v).mean(-1, keepdims=True, dtype=np.float32) + np.float32(1e-6))
    want, e, _, _ = ref.norm(x.astype(np.float64), np.zeros(x.shape), kind, float(np.float32(1e-6)))
    err = np.abs(got - want)
    assert got.dtype == np.float32 and (err <= e).all() and (err > e / 300).any()


def test_clip_definition():
    g = [np.array([3.0, 0.0]), np.array([[4.0]])]
    norm, out = ref.clip_grad_norm(g, 10.0)
    assert norm == 5.0 and out[0].tolist() == [3.0, 0.0]
    norm, out = ref.clip_grad_norm(g, 1.0)
    np.testing.assert_allclose(np.sqrt(sum((o ** 2).sum() for o in out)), 1.0, rtol=1e-15)
    norm, out = ref.clip_grad_norm([np.array([np.inf, 1.0])], 1.0)
    assert norm == np.inf and out[0].tolist() == [0.0, 0.0]
    assert ref.clip_grad_norm([], 1.0) == (0.0, [])


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------
def test_residual_norm_arguments_are_checked_on_the_host(lib):
    import differentiable_gaussian_splatting_gb300 as gs

    none = C.byref(gs.Rows(None, 64))
    R = lambda p=P, s=64: C.byref(gs.Rows(p, s))
    base = dict(type=1, pre=1, post=1, batch=1, alpha=1.0, beta=1.0, eps=1e-6)

    def norm(**kw):
        return C.byref(gs.BlockNorm(*[{**base, **kw}[n] for n, _ in gs.BlockNorm._fields_]))

    def params(**kw):
        return C.byref(gs.NormParams(*[kw.get(n) for n, _ in gs.NormParams._fields_]))

    def fwd(T=10, C_=64, x=None, y=None, r=None, h=None, w=None, cu=None, **kw):
        return lib.gs_residual_norm(T, C_, norm(**kw), x or R(), y or R(), w or params(), cu, r or R(),
                                    h or R(), None)

    assert fwd(T=0) == 0 and fwd(T=0, cu=P, w=params(gate=P), batch=3) == 0
    for kw in (dict(T=-1), dict(T=(1 << 30) + 1), dict(C_=0), dict(C_=8193), dict(type=2),
               dict(pre=3), dict(post=-1), dict(eps=0.0), dict(eps=float("nan")),
               dict(alpha=float("inf")), dict(beta=float("nan")), dict(batch=0), dict(batch=2),
               dict(cu=P), dict(cu=MIS, w=params(gate=P)), dict(cu=P, w=params(gate=P), batch=1 << 21),
               dict(pre=0, w=params(pre_weight=P)), dict(pre=0), dict(post=0, w=params(post_bias=P)),
               dict(w=params(post_weight=MIS)), dict(w=params(gate=MIS)), dict(w=params(pre_bias=MIS)),
               dict(x=none), dict(x=R(P + 1)), dict(x=R(s=63)), dict(y=none), dict(y=R(s=(1 << 29) + 1)),
               dict(y=none, post=0, w=params(gate=P)), dict(r=R(s=8)), dict(h=none), dict(h=R(P + 1)),
               dict(type=0, x=R(P + 2))):
        assert fwd(**kw) == 1, kw
    ws = lib.gs_residual_norm_workspace_bytes(10, 64, 1)
    assert ws > 0 and ws == gs.gs_residual_norm_workspace_bytes(10, 64)
    for a in ((-1, 64, 1), (10, 0, 1), (10, 8193, 1), (10, 64, 0), (10, 64, (1 << 20) + 1)):
        assert lib.gs_residual_norm_workspace_bytes(*a) == 0

    def bwd(T=10, x=None, y=None, dr=None, dh=None, dx=None, dy=None, w=None, g=None, wsp=P, wsb=ws,
            **kw):
        return lib.gs_residual_norm_bwd(T, 64, norm(**kw), x or R(), y or R(), w or params(), None,
                                        dr or none, dh or R(), dx or R(), dy or R(), g or params(),
                                        wsp, wsb, None)

    for kw in (dict(dh=none), dict(pre=0), dict(dx=none), dict(dy=none), dict(y=none, post=0),
               dict(dr=R(P + 1)), dict(g=params(gate=P)), dict(pre=0, dh=none, g=params(pre_bias=P)),
               dict(post=0, g=params(post_weight=P)), dict(g=params(pre_weight=MIS)), dict(wsp=None),
               dict(wsp=MIS), dict(T=-5)):
        assert bwd(**kw) == 1, kw
    assert bwd(wsb=ws - 1) == 5


def test_clip_arguments_are_checked_on_the_host(lib):
    import differentiable_gaussian_splatting_gb300 as gs

    def arrays(*a):
        return (gs.Array * len(a))(*[gs.Array(*x) for x in a])

    one, huge = arrays((P, 10, 0)), 1 << 60

    def call(n=1, g=one, o=None, top=1.0, norm=P, ws=P, wsb=huge):
        return lib.gs_clip_grad_norm(n, g, o, top, norm, ws, wsb, None)

    big = arrays(*[(P, 1 << 40, 0)] * 5)
    for kw in (dict(n=-1), dict(n=65537), dict(g=None), dict(top=-1.0), dict(top=float("nan")),
               dict(norm=None), dict(norm=P + 2), dict(ws=None), dict(ws=MIS),
               dict(g=arrays((None, 10, 0))), dict(g=arrays((P, -1, 0))), dict(g=arrays((P, 10, 2))),
               dict(g=arrays((P + 2, 10, 0))), dict(g=arrays((P + 1, 10, 1))),
               dict(g=arrays((P, (1 << 40) + 1, 0))), dict(n=5, g=big),
               dict(o=arrays((P, 11, 0))), dict(o=arrays((P, 10, 1))), dict(o=arrays((None, 10, 0)))):
        assert call(**kw) == 1, kw
    need = lib.gs_clip_grad_norm_workspace_bytes(1)
    assert need > 0 and call(wsb=need - 1) == 5
    assert lib.gs_clip_grad_norm_workspace_bytes(-1) == 0
    assert lib.gs_clip_grad_norm_workspace_bytes(65537) == 0
    # every table of arrays keeps its blocks' sums
    assert lib.gs_clip_grad_norm_workspace_bytes(65536) >= 64 * need


def test_binding_refuses_other_shapes(lib, fake):
    import torch

    import differentiable_gaussian_splatting_gb300 as gs

    x, w, cu = fake(0, 64), fake(64), fake(3, dtype=torch.int32)
    for bad, name in ((fake(0, 32), "y"), (fake(64), "y"), (fake(0, 64, dtype=torch.bfloat16), "y")):
        with pytest.raises(ValueError, match=name):
            gs.gs_residual_norm(x, bad, x, x, stream=0)
    with pytest.raises(ValueError, match="r_out"):
        gs.gs_residual_norm(x, x, fake(1, 64), x, stream=0)
    with pytest.raises(ValueError, match="x"):
        gs.gs_residual_norm(None, x, x, x, stream=0)
    with pytest.raises(ValueError, match="contiguous"):
        gs.gs_residual_norm(fake(64, 4).t(), None, None, fake(4, 64), stream=0)
    for kw in (dict(pre_weight=fake(63)), dict(pre_bias=fake(128)), dict(gate=fake(2, 64)),
               dict(gate=w, cu=cu), dict(cu=cu)):
        with pytest.raises(ValueError, match=list(kw)[0]):
            gs.gs_residual_norm(x, x, x, x, stream=0, **kw)
    with pytest.raises(ValueError, match="post"):
        gs.gs_residual_norm(x, x, x, x, post="batch", stream=0)
    with pytest.raises(gs.GSError):
        gs.gs_residual_norm(x, x, x, x, eps=-1.0, stream=0)
    with pytest.raises(ValueError, match="too large"):
        gs.gs_residual_norm(fake(0, 2 ** 32 + 64), None, None, None, stream=0)
    ws = fake(1, dtype=torch.uint8)
    with pytest.raises(ValueError, match="dgate"):
        gs.gs_residual_norm_bwd(x, x, x, x, x, x, ws, gate=w, dgate=fake(63), stream=0)
    with pytest.raises(gs.GSError):  # workspace too small
        gs.gs_residual_norm_bwd(x, x, x, x, x, x, ws, stream=0)
    gs.gs_residual_norm(x, x, x, x, pre_weight=w, post="layer", stream=0)  # no tokens: nothing to do

    norm = fake(1)
    for g, kw in ((x, {}), ([x, fake(4, dtype=torch.int32)], {}), ([fake(8, 4).t()], {}),
                  ([x], dict(outs=[])), ([x], dict(outs=[fake(4)])),
                  ([x], dict(outs=[fake(0, dtype=torch.bfloat16)])), ([torch.zeros(3)], {}),
                  ([None], {})):
        with pytest.raises((TypeError, ValueError)):
            gs.gs_clip_grad_norm(g, 1.0, norm, ws, stream=0, **kw)
    with pytest.raises(gs.GSError):
        gs.gs_clip_grad_norm([x], 1.0, norm, ws, stream=0)
    with pytest.raises(ValueError, match="norm"):
        gs.gs_clip_grad_norm([x], 1.0, None, ws, stream=0)


def test_clip_outputs_that_meet_are_refused(lib):
    import differentiable_gaussian_splatting_gb300 as gs

    def call(grads, outs=None):
        n = len(grads)
        g = (gs.Array * n)(*[gs.Array(*x) for x in grads])
        o = (gs.Array * n)(*[gs.Array(*x) for x in outs]) if outs else None
        # no workspace is that small: what the arrays pass, this refuses
        return lib.gs_clip_grad_norm(n, g, o, 1.0, P, P, 8, None)

    a, b, c = (P, 100, 0), (P + 400, 50, 1), (P + 8192, 7, 0)
    apart = [(P + (1 << 20), 100, 0), (P + (2 << 20), 50, 1), (P + (3 << 20), 7, 0)]
    assert call([a, b, c]) == 5 and call([c, a, b]) == 5
    assert call([a, b, c], apart) == 5
    assert call([a, (None, 0, 0), (P, 0, 0)]) == 5       # nothing in an empty array
    assert call([a, a], [apart[0], (P + (4 << 20), 100, 0)]) == 5  # only read twice
    assert call([a, a], [a, apart[0]]) == 1              # read while it is written
    assert call([a, b, a]) == 1                          # in place twice
    assert call([a, (P + 396, 50, 1)]) == 1              # by its last element
    assert call([(P + 396, 50, 1), a]) == 1
    assert call([a, b, c], [apart[0], apart[1], (P + (1 << 20) + 396, 7, 0)]) == 1
    assert call([a, b, c], [apart[0], apart[1], (P + 4, 7, 0)]) == 1   # over a's gradient
    assert call([a, b, c], [(P + 4, 100, 0), apart[1], apart[2]]) == 1  # over its own, moved
