"""Residual norms and gradient clipping against their float64 definitions (tests/block_ref.py).

Tolerances: the definitions' own bounds on fp32 arithmetic, and for bfloat16 outputs half a unit in
their last place, H = 2^-8 of the value.  Clipping: a thread sums at most 64 squares in fp32 (19
roundings; the rest is fp64), which the root halves: the norm is off by at most 12 U of itself, an
output by 14 U (norm, factor, product) and H in bfloat16; below fp32's normal range by half of
its smallest value too.
"""

import numpy as np
import pytest

import block_ref as ref
from token_ref import H, U, bf16

pytestmark = pytest.mark.gpu


def _gs():
    import differentiable_gaussian_splatting_gb300 as gs

    return gs


def _round(x, dtype):
    x = np.asarray(x, np.float32)
    return bf16(x) if dtype == "bf16" else x


def _dev(x, dtype="f32", stride=None):
    """on the device, as rows of a wider array of NaN where a stride is given"""
    import torch

    if x is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda()
    t = t.to(torch.bfloat16) if dtype == "bf16" else t
    if stride is None:
        return t
    wide = torch.full((t.shape[0], stride), float("nan"), dtype=t.dtype, device="cuda")
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _close(got, want, bound, what):
    got = _np(got)
    err = np.where(got == want, 0.0, np.abs(got - want))
    assert np.isfinite(got).all() or np.isnan(want).any(), what
    worst = np.unravel_index(np.argmax(err - bound), err.shape) if err.size else None
    assert (err <= bound).all(), (what, worst, got[worst], want[worst], bound[worst])


# ---------------------------------------------------------------------------
# residual norms
# ---------------------------------------------------------------------------
CASES = [  # lens (of the gate's sequences, or one number of tokens), width, dtype, pre, post, gate, bias, stride
    (1, 1, "f32", "rms", "none", False, False, None),
    (1, 8, "bf16", "layer", "layer", True, True, None),
    (64, 256, "bf16", "layer", "none", False, True, None),
    (33, 264, "bf16", "rms", "rms", True, False, 280),      # two warps a row, a wider array
    (700, 1024, "bf16", "rms", "rms", True, True, None),    # several blocks a sequence
    (130, 515, "f32", "layer", "layer", True, True, None),  # odd width
    (130, 515, "bf16", "rms", "layer", False, True, 517),
    (9, 4096, "bf16", "layer", "rms", True, False, None),
    (7, 8192, "f32", "rms", "rms", True, True, None),
    (5, 8191, "bf16", "layer", "layer", True, True, None),
    (40, 72, "f32", "none", "rms", True, False, None),      # no norm behind the residual
    (40, 72, "bf16", "none", "none", True, False, 73),
    ([0, 5, 0, 300, 1, 2000, 0], 128, "bf16", "rms", "rms", True, True, None),
    ([2600, 3, 900], 40, "f32", "layer", "layer", True, True, 44),
    ([1] * 500, 96, "f32", "rms", "none", True, False, None),  # a gate a token
    ([700, 1500], 1000, "f32", "rms", "rms", True, False, None),
    # several rows of a block behind each other, on their way ahead of it
    (1700, 2048, "bf16", "rms", "rms", True, False, None),
    ([900, 0, 1100], 2048, "bf16", "layer", "layer", True, True, 2056),
    (1300, 4096, "bf16", "none", "rms", False, False, None),
    (1300, 4096, "bf16", "layer", "none", True, False, None),
]


def _inputs(lens, width, dtype, pre, post, gate, bias, seed=0):
    rng = np.random.default_rng(seed)
    T = int(np.sum(lens))
    vec = lambda on, mean: rng.normal(mean, 0.3, width).astype(np.float32) if on else None
    cu = None if np.isscalar(lens) else np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    batch = 1 if cu is None else len(lens)
    x = _round(rng.normal(rng.normal(0, 3, (T, 1)), 2.0, (T, width)), dtype)
    y = _round(rng.normal(1.0, rng.uniform(0.1, 4.0, (T, 1)), (T, width)), dtype)
    p = dict(pw=vec(pre != "none", 1.0), pb=vec(bias and pre != "none", 0.0),
             qw=vec(post != "none", 1.0), qb=vec(bias and post != "none", 0.0),
             gate=rng.normal(0, 0.7, (batch, width)).astype(np.float32) if gate else None)
    dr, dh = (_round(rng.normal(size=(T, width)), dtype) for _ in range(2))
    return x, y, p, cu, dr, dh if pre != "none" else None


def _params(p, cu):
    import torch

    names = {"pw": "pre_weight", "pb": "pre_bias", "qw": "post_weight", "qb": "post_bias",
             "gate": "gate"}
    kw = {names[n]: _dev(v) for n, v in p.items()}
    kw["cu"] = None if cu is None else torch.from_numpy(cu).cuda()
    return kw


@pytest.mark.parametrize("case", range(len(CASES)))
def test_residual_norm(case):
    import torch

    gs = _gs()
    lens, width, dtype, pre, post, gate, bias, stride = CASES[case]
    x, y, p, cu, dr, dh = _inputs(lens, width, dtype, pre, post, gate, bias, seed=case)
    T, (alpha, beta, eps) = x.shape[0], (1.25, 0.5, 1e-5)
    want = ref.residual_norm(x, y, **p, cu=cu, pre=pre, post=post, alpha=alpha, beta=beta,
                             eps=float(np.float32(eps)), dr=dr, dh=dh)
    h_ = H if dtype == "bf16" else 0.0
    kw = dict(**_params(p, cu), pre=pre, post=post, alpha=alpha, beta=beta, eps=eps)
    dx_, dy_, ddr, ddh = (_dev(a, dtype, stride) for a in (x, y, dr, dh))
    new = lambda: _dev(np.full((T, width), np.nan), dtype, stride)
    r, h = new(), new() if pre != "none" else None
    gs.gs_residual_norm(dx_, dy_, r, h, **kw)
    for n, got in (("r", r), ("h", h)):
        if got is not None:
            v, e = want[n]
            _close(got, v, h_ * (np.abs(v) + e) + e, n)
    gx, gy = new(), new()
    grads = {"d" + n: torch.full_like(kw[n], float("nan")) for n in
             ("pre_weight", "pre_bias", "post_weight", "post_bias", "gate") if kw[n] is not None}
    batch = 1 if cu is None else len(cu) - 1
    ws = torch.full((gs.gs_residual_norm_workspace_bytes(T, width, batch),), 255, dtype=torch.uint8,
                    device="cuda")
    call = lambda: gs.gs_residual_norm_bwd(dx_, dy_, ddr, ddh, gx, gy, ws, **kw, **grads)
    call()
    for n, got in (("x", gx), ("y", gy)):
        v, e = want[n]
        _close(got, v, h_ * (np.abs(v) + e) + e, "d" + n)
    for n, got in grads.items():
        v, e = want[n[1:]]
        _close(got.view(v.shape), v, e, n)
    first = [t.clone() for t in (gx, gy, *grads.values())]
    ws.random_()
    call()
    assert all(torch.equal(a, b) for a, b in zip(first, (gx, gy, *grads.values())))
    # what lies between the rows stays
    if stride is not None:
        for t in (r, gx, gy):
            assert torch.isnan(torch.as_strided(t, (T, stride - width), (stride, 1), width)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_residual_norm_without_a_block(dtype):
    # the first norm of a stack: h = pre(x), its gradient with the stream's
    gs = _gs()
    import torch

    x, _, p, _, dr, dh = _inputs(77, 320, dtype, "layer", "none", False, True)
    want = ref.residual_norm(x, None, **p, pre="layer", eps=float(np.float32(1e-6)), dr=dr, dh=dh)
    h_ = H if dtype == "bf16" else 0.0
    kw = dict(**_params(p, None), pre="layer")
    tx, h, gx = _dev(x, dtype), _dev(x * 0, dtype), _dev(x * 0, dtype)
    gs.gs_residual_norm(tx, None, None, h, **kw)
    _close(h, want["h"][0], h_ * np.abs(want["h"][0]) + 2 * want["h"][1], "h")
    ws = torch.empty(gs.gs_residual_norm_workspace_bytes(77, 320), dtype=torch.uint8, device="cuda")
    gw = torch.empty(320, device="cuda")
    gs.gs_residual_norm_bwd(tx, None, _dev(dr, dtype), _dev(dh, dtype), gx, None, ws, **kw,
                            dpre_weight=gw)
    _close(gx, want["x"][0], h_ * np.abs(want["x"][0]) + 2 * want["x"][1], "dx")
    _close(gw, *want["pre_weight"], "dpre_weight")


def test_residual_norm_in_place_and_rows_of_no_sequence():
    import torch

    gs = _gs()
    x, y, p, _, dr, dh = _inputs([30, 0, 50, 20], 136, "bf16", "rms", "rms", True, False)
    cu = torch.tensor([0, 30, 30, 80], dtype=torch.int32, device="cuda")  # 20 rows behind the last
    kw = dict(**_params({**p, "gate": p["gate"][:3]}, None), post="rms")
    kw["cu"] = cu
    arrays = [_dev(a, "bf16") for a in (x, y, dr, dh)]
    out = [torch.zeros_like(a) for a in arrays]
    grads = {n: torch.empty_like(kw[n[1:]]) for n in ("dpre_weight", "dpost_weight", "dgate")}
    ws = torch.empty(gs.gs_residual_norm_workspace_bytes(100, 136, 3), dtype=torch.uint8, device="cuda")
    gs.gs_residual_norm(*arrays[:2], *out[:2], **kw)
    gs.gs_residual_norm_bwd(*arrays, *out[2:], ws, **kw, **grads)
    kept = [g.clone() for g in grads.values()]
    assert all((o[80:] == 0).all() for o in out)
    assert (grads["dgate"][1] == 0).all()
    want = ref.residual_norm(x[:80], y[:80], **{**p, "gate": p["gate"][:3]},
                             cu=np.array([0, 30, 30, 80]), pre="rms", post="rms",
                             eps=float(np.float32(1e-6)), dr=dr[:80], dh=dh[:80])
    for n, g in grads.items():
        _close(g, *want[n[1:]], n)
    # outputs over their inputs
    a, b = [t.clone() for t in arrays], [t.clone() for t in arrays]
    gs.gs_residual_norm(a[0], a[1], a[0], a[1], **kw)
    gs.gs_residual_norm_bwd(b[0], b[1], b[2], b[3], b[2], b[1], ws, **kw, **grads)
    assert torch.equal(a[0][:80], out[0][:80]) and torch.equal(a[1][:80], out[1][:80])
    assert torch.equal(b[2][:80], out[2][:80]) and torch.equal(b[1][:80], out[3][:80])
    assert all(torch.equal(g, k) for g, k in zip(grads.values(), kept))
    for t, s in ((a[0], arrays[0]), (b[2], arrays[2])):
        assert torch.equal(t[80:], s[80:])


def test_residual_norm_without_tokens():
    import torch

    gs = _gs()
    x = torch.empty((0, 64), device="cuda")
    gate, grads = torch.ones((2, 64), device="cuda"), [torch.ones(64, device="cuda") for _ in range(2)]
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    dg = torch.ones_like(gate)
    ws = torch.empty(gs.gs_residual_norm_workspace_bytes(0, 64, 2), dtype=torch.uint8, device="cuda")
    gs.gs_residual_norm(x, x, x, x, gate=gate, cu=cu, post="rms")
    gs.gs_residual_norm_bwd(x, x, x, x, x, x, ws, gate=gate, cu=cu, post="rms", dgate=dg,
                            pre_weight=grads[0], dpre_weight=grads[1])
    assert (dg == 0).all() and (grads[1] == 0).all()


# ---------------------------------------------------------------------------
# gradient norm and clipping
# ---------------------------------------------------------------------------
def _clip(grads, dtypes, max_norm, outs=True, shift=0):
    """(norm, outs) of the call; shift: elements by which the arrays lie behind a 16-byte word"""
    import torch

    gs = _gs()

    def put(g, dtype):
        t = _dev(np.concatenate([np.zeros(shift), np.ravel(g)]), dtype)
        return t[shift:]

    tg = [put(g, d) for g, d in zip(grads, dtypes)]
    to = [torch.full_like(t, 3.0) for t in tg] if outs else None
    norm = torch.full((1,), -1.0, device="cuda")
    ws = torch.full((gs.gs_clip_grad_norm_workspace_bytes(len(tg)),), 255, dtype=torch.uint8,
                    device="cuda")
    gs.gs_clip_grad_norm(tg, max_norm, norm, ws, outs=to)
    return norm.item(), to if outs else tg


def _check_clip(grads, dtypes, max_norm, **kw):
    grads = [_round(g, d) for g, d in zip(grads, dtypes)]
    max_norm = float(np.float32(max_norm))
    norm, want = ref.clip_grad_norm(grads, max_norm)
    got, outs = _clip(grads, dtypes, max_norm, **kw)
    assert abs(got - norm) <= 12 * U * norm + 2.0 ** -150, (got, norm)
    for o, w, d in zip(outs, want, dtypes):
        _close(o, w.ravel(), (14 * U + (H if d == "bf16" else 0.0)) * np.abs(w.ravel()) + 2.0 ** -134
               if d == "bf16" else 14 * U * np.abs(w.ravel()) + 2.0 ** -150, d)


SIZES = [[1], [7, 1, 0, 300], [4096, 4097, 8191, 8192, 8193], [100000, 3, 12288, 1, 1, 70001],
         [17] * 95 + [0] * 10, [33] * 97, [5] * 2600 + [40000], []]


@pytest.mark.parametrize("sizes", range(len(SIZES)))
@pytest.mark.parametrize("dtype", ["f32", "bf16", "both"])
@pytest.mark.parametrize("ratio,outs,shift", [(3.0, True, 0), (0.5, True, 0), (3.0, False, 1),
                                              (0.5, False, 0)])
def test_clip_grad_norm(sizes, dtype, ratio, outs, shift):
    rng = np.random.default_rng(sizes)
    sizes = SIZES[sizes]
    dtypes = [("f32", "bf16")[i % 2] if dtype == "both" else dtype for i in range(len(sizes))]
    grads = [rng.normal(size=n) * 10.0 ** rng.uniform(-3, 1) for n in sizes]
    norm = float(np.sqrt(sum((g ** 2).sum() for g in grads))) or 1.0
    _check_clip(grads, dtypes, norm / ratio, outs=outs, shift=shift)


@pytest.mark.parametrize("scale", [1e-44, 1e-30, 1e-22, 1e18, 1e25, 3e37])
@pytest.mark.parametrize("n", [1, 5000, 40000])
@pytest.mark.parametrize("max_norm", [0.0, 1e-30, 1.0, 1e30])
def test_clip_grad_norm_of_small_and_large_values(scale, n, max_norm):
    # squares leave fp32's range, norms and factors stay
    rng = np.random.default_rng(1)
    g = (np.clip(rng.normal(size=n), -3, 3) * scale).astype(np.float32)
    g[::3] = 0.0
    norm, _ = ref.clip_grad_norm([g], 1.0)
    got, outs = _clip([g], ["f32"], max_norm)
    m = float(np.float32(max_norm))
    if norm < 3.4e38:
        assert abs(got - norm) <= 12 * U * norm + 2.0 ** -150
    else:
        assert got == np.inf
    _, want = ref.clip_grad_norm([g], m)
    _close(outs[0], want[0], 14 * U * np.abs(want[0]) + 2.0 ** -150, "out")


@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("outs", [True, False])
def test_clip_grad_norm_that_is_not_finite(value, outs):
    rng = np.random.default_rng(2)
    for at in (0, 4095, 12000):
        g = [rng.normal(size=n).astype(np.float32) for n in (12001, 50, 16384)]
        g[0][at] = value
        norm, out = _clip(g, ["f32", "bf16", "bf16"], 1.0, outs=outs)
        assert np.isnan(norm) if np.isnan(value) else norm == np.inf
        assert all((o == 0).all() for o in out)


def test_norm_alone_and_untouched_gradients():
    import torch

    gs = _gs()
    g = [torch.randn(n, device="cuda") for n in (5, 100000)]
    kept, norm = [x.clone() for x in g], torch.empty(1, device="cuda")
    ws = torch.empty(gs.gs_clip_grad_norm_workspace_bytes(2), dtype=torch.uint8, device="cuda")
    gs.gs_clip_grad_norm(g, float("inf"), norm, ws)
    want = float(torch.cat(g).double().norm())
    assert abs(norm.item() - want) <= 12 * U * want
    assert all(torch.equal(a, b) for a, b in zip(g, kept))
    a = norm.clone()
    gs.gs_clip_grad_norm(tuple(g), want / 2, norm, ws)
    assert torch.equal(a, norm)  # the same bits again
    gs.gs_clip_grad_norm(g, float("inf"), norm, ws)
    assert abs(norm.item() - want / 2) <= 32 * U * want


def test_norm_alone_leaves_what_is_not_finite():
    import torch

    gs = _gs()
    g = [torch.randn(n, device="cuda") for n in (40000, 3)]
    g[0][7], g[1][2] = float("nan"), float("inf")
    kept, norm = [x.clone() for x in g], torch.zeros(1, device="cuda")
    ws = torch.empty(gs.gs_clip_grad_norm_workspace_bytes(2), dtype=torch.uint8, device="cuda")
    outs = [torch.zeros_like(x) for x in g]
    for o in (None, outs):
        gs.gs_clip_grad_norm(g, float("inf"), norm, ws, outs=o)
        assert norm.isnan().item()
        for a in (g, outs if o else g):
            assert all(torch.equal(x.nan_to_num(5.0), y.nan_to_num(5.0)) for x, y in zip(a, kept))


def test_clip_grad_norm_within_its_bound_beside_outs_of_their_own():
    # some gradients in place, some not: those in place are neither read again nor written
    import torch

    gs = _gs()
    sizes = (3, 100000, 16384, 5, 70000)
    g = [torch.randn(n, device="cuda") for n in sizes]
    kept = [x.clone() for x in g]
    outs = [x if i % 2 else torch.zeros_like(x) for i, x in enumerate(g)]
    norm = torch.zeros(1, device="cuda")
    ws = torch.empty(gs.gs_clip_grad_norm_workspace_bytes(len(g)), dtype=torch.uint8, device="cuda")
    gs.gs_clip_grad_norm(g, 1e6, norm, ws, outs=outs)
    want = float(torch.cat(g).double().norm())
    assert abs(norm.item() - want) <= 12 * U * want
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(kept, g, outs))


@pytest.mark.parametrize("pre,post,with_y,with_dr", [("rms", "rms", True, True), ("layer", "layer", True, False),
                                                     ("rms", "none", False, True), ("none", "rms", True, True)])
@pytest.mark.parametrize("tokens,width", [(2100, 2048), (6, 4096), (900, 8192), (3000, 256)])
def test_residual_norm_in_place_of_rows_that_are_read_ahead(pre, post, with_y, with_dr, tokens, width):
    import torch

    gs = _gs()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(width)
    n = lambda on=True: (torch.randn((tokens, width), generator=gen, device="cuda").bfloat16()
                         if on else None)
    x, y, dr, dh = n(), n(with_y), n(with_dr or pre == "none"), n(pre != "none")
    kw = dict(pre=pre, post=post, alpha=0.75, beta=1.5)
    r, h = torch.empty_like(x), torch.empty_like(x) if pre != "none" else None
    gs.gs_residual_norm(x, y, r, h, **kw)
    a, b = x.clone(), None if y is None else y.clone()
    out = b if b is not None and h is not None else None
    gs.gs_residual_norm(a, b, a, out if out is not None else (h if h is None else torch.empty_like(x)), **kw)
    assert torch.equal(a, r) and (out is None or torch.equal(out, h))
    ws = torch.empty(gs.gs_residual_norm_workspace_bytes(tokens, width), dtype=torch.uint8, device="cuda")
    dx, dy = torch.empty_like(x), None if y is None else torch.empty_like(x)
    gs.gs_residual_norm_bwd(x, y, dr, dh, dx, dy, ws, **kw)
    to_x = dr if dr is not None else dh
    to_y = None if y is None else y
    gs.gs_residual_norm_bwd(x, y, dr, dh, to_x, to_y, ws, **kw)
    assert torch.equal(to_x, dx) and (dy is None or torch.equal(to_y, dy))
