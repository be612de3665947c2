"""The token operators without a GPU: the plain definitions the GPU tests compare with are
pinned (finite differences, closed forms, published generator answers), and the library's host
checks refuse bad calls before anything is enqueued."""

import ctypes as C

import numpy as np
import pytest

import token_ref as ref


# ---------------------------------------------------------------------------
# the definitions
# ---------------------------------------------------------------------------
def test_bf16_rounding():
    x = np.array([1.0, 1.00390625, 1.001953125, -1.005859375, 3.4e38, 0.0], np.float32)
    # 1 + 2^-8 is a tie (to even: 1), 1 + 3 2^-9 rounds up to 1 + 2^-7
    np.testing.assert_array_equal(ref.bf16(x)[:4], np.array([1.0, 1.0, 1.0, -1.0078125], np.float32))
    assert np.isinf(ref.bf16(x)[4]) and ref.bf16(x)[5] == 0


@pytest.mark.parametrize("interleaved", [False, True])
def test_head_norm_gradient_equals_differences(interleaved):
    rng = np.random.default_rng(1)
    T, H, D, rot = 3, 2, 16, 12
    x, w, dy = rng.normal(size=(T, H, D)), rng.normal(size=D), rng.normal(size=(T, H, D))
    ang = rng.uniform(0, 6, (4, rot // 2))
    table, pos = np.concatenate([np.cos(ang), np.sin(ang)], 1), np.array([2, -1, 0])
    f = lambda x, w: (ref.head_norm(x, w, table, pos, 1e-3, interleaved)[0] * dy).sum()
    dx, _, dw, _ = ref.head_norm_bwd(x, w, table, pos, 1e-3, interleaved, dy)
    h = 1e-6
    for got, arr, which in ((dx, x, 0), (dw, w, 1)):
        num = np.zeros_like(arr)
        for i in np.ndindex(*arr.shape):
            d = np.zeros_like(arr)
            d[i] = h
            a = (x + d, w) if which == 0 else (x, w + d)
            b = (x - d, w) if which == 0 else (x, w - d)
            num[i] = (f(*a) - f(*b)) / (2 * h)
        np.testing.assert_allclose(got, num, rtol=1e-6, atol=1e-8)
    # a turn keeps lengths, and without one the row has root mean square |w| = 1
    y, _ = ref.head_norm(x, None, table, pos, 0.0, interleaved)
    np.testing.assert_allclose((y * y).mean(-1), 1.0, rtol=1e-12)


@pytest.mark.parametrize("causal", [False, True])
def test_attention_gradient_equals_differences(causal):
    rng = np.random.default_rng(2)
    cu_q, cu_k = np.array([0, 3, 3, 7]), np.array([0, 4, 6, 8])
    q, k, v = rng.normal(size=(7, 4, 8)), rng.normal(size=(8, 2, 8)), rng.normal(size=(8, 2, 8))
    do = rng.normal(size=q.shape)
    f = lambda q, k, v: (ref.attention(q, k, v, 0.4, causal, cu_q, cu_k)[0] * do).sum()
    out, lse, _, _ = ref.attention(q, k, v, 0.4, causal, cu_q, cu_k)
    g = ref.attention_bwd(q, k, v, out, lse, do, 0.4, causal, cu_q, cu_k)
    h = 1e-6
    for n, arr in (("q", q), ("k", k), ("v", v)):
        num = np.zeros_like(arr)
        for i in np.ndindex(*arr.shape):
            d = np.zeros_like(arr)
            d[i] = h
            args = {"q": q, "k": k, "v": v}
            num[i] = (f(**{**args, n: arr + d}) - f(**{**args, n: arr - d})) / (2 * h)
        np.testing.assert_allclose(g[n][0], num, rtol=1e-6, atol=1e-8)


def test_attention_closed_forms():
    rng = np.random.default_rng(3)
    v = rng.normal(size=(5, 1, 8))
    q, k = np.zeros((3, 1, 8)), rng.normal(size=(5, 1, 8))
    out, lse, _, _ = ref.attention(q, k, v, 1.0)      # equal scores: the mean
    np.testing.assert_allclose(out, np.broadcast_to(v.mean(0), out.shape))
    np.testing.assert_allclose(lse, np.log(5))
    out, lse, _, _ = ref.attention(np.zeros((7, 1, 8)), k, v, 1.0, causal=True)
    assert (out[:2] == 0).all() and np.isneginf(lse[0, :2]).all()   # see no key
    np.testing.assert_allclose(out[2], v[0])                         # sees the first key alone
    np.testing.assert_allclose(out[6], v.mean(0))


def test_generator_published_answers():
    # Random123's known-answer vectors of philox4x32-10
    z = ref.philox4x32_10([0, 0, 0, 0], [0, 0])
    assert [int(x) for x in z] == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    f = 0xFFFFFFFF
    o = ref.philox4x32_10([f, f, f, f], [f, f])
    assert [int(x) for x in o] == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    keep, factor = ref.kept(200_000, 7, 9, 0.25)
    assert abs(keep.mean() - 0.75) < 5 * (0.25 * 0.75 / 200_000) ** 0.5
    assert factor == 4 / 3


# ---------------------------------------------------------------------------
# the host's checks
# ---------------------------------------------------------------------------
@pytest.fixture(scope="module")
def lib():
    from differentiable_gaussian_splatting_gb300 import build

    build.build()
    import differentiable_gaussian_splatting_gb300 as gs

    return gs.library()


P, MIS = 0x100000, 0x100004  # never dereferenced: the checks fail first


def _h(data=P, ts=512, hs=64):
    import differentiable_gaussian_splatting_gb300 as gs

    return C.byref(gs.Heads(data, ts, hs))


def test_head_norm_arguments_are_checked_on_the_host(lib):
    import differentiable_gaussian_splatting_gb300 as gs

    def call(T=10, hq=8, hk=8, D=64, norm=(1, 64, 0, 1e-6, 100), q=None, w=P, table=P, pos=None,
             out=None):
        n = C.byref(gs.HeadNorm(*norm)) if norm else None
        return lib.gs_qk_norm_rope(T, hq, hk, D, n, q or _h(), _h(), w, w, table, pos, out or _h(),
                                   _h(), None)

    assert call(T=0) == 0
    assert call(T=-1) == 1 and call(hq=0) == 1 and call(hk=1025) == 1 and call(norm=None) == 1
    assert call(D=60) == 1 and call(D=0) == 1 and call(D=264) == 1
    for bad in ((2, 64, 0, 1e-6, 100), (1, 65, 0, 1e-6, 100), (1, 66, 0, 1e-6, 100),
                (1, -2, 0, 1e-6, 100), (1, 64, 0, 0.0, 100), (1, 64, 0, float("nan"), 100),
                (1, 64, 0, 1e-6, 0)):
        assert call(norm=bad) == 1, bad
    assert call(table=None) == 1 and call(table=MIS) == 1 and call(w=MIS) == 1
    assert call(norm=(1, 64, 0, 1e-6, 9)) == 1       # ten tokens, nine rows, no positions
    assert call(pos=MIS) == 1
    for bad in (_h(None), _h(MIS), _h(ts=508), _h(hs=60), _h(hs=32), _h(ts=448), _h(ts=520)):
        assert call(q=bad) == 1 and call(out=bad) == 1
    ws = lib.gs_qk_norm_rope_workspace_bytes(10, 8, 8, 64)
    assert ws > 0 and lib.gs_qk_norm_rope_workspace_bytes(10, 8, 8, 7) == 0

    def bwd(w=P, dw=P, wsp=P, wsb=ws, dq=None):
        n = C.byref(gs.HeadNorm(1, 64, 0, 1e-6, 100))
        return lib.gs_qk_norm_rope_bwd(10, 8, 8, 64, n, _h(), _h(), w, w, P, None, _h(), _h(),
                                       dq or _h(), _h(), dw, dw, wsp, wsb, None)

    assert bwd(dw=MIS) == 1 and bwd(wsp=None) == 1 and bwd(dq=_h(MIS)) == 1
    assert bwd(wsb=ws - 1) == 5


def test_attention_arguments_are_checked_on_the_host(lib):
    import differentiable_gaussian_splatting_gb300 as gs

    ok = dict(tokens_q=10, tokens_k=20, batch=1, heads_q=8, heads_k=2, head_dim=64, causal=0,
              scale=0.125)

    def shape(**kw):
        s = {**ok, **kw}
        return gs.AttentionShape(*[s[f] for f, _ in gs.AttentionShape._fields_])

    ws = lib.gs_attention_workspace_bytes(C.byref(shape()))
    assert ws > 0

    def call(s=None, q=None, k=None, cu=(None, None), lse=P, wsp=P, wsb=1 << 40, **kw):
        a = C.byref(shape(**kw)) if s is None else s
        return lib.gs_attention_fwd(a, q or _h(), k or _h(ts=128), _h(ts=128), *cu, _h(), lse, wsp,
                                    wsb, None)

    bad = [dict(tokens_q=-1), dict(tokens_k=(1 << 30) + 1), dict(batch=0), dict(heads_q=0),
           dict(heads_q=7), dict(heads_k=0), dict(heads_q=2048, heads_k=1), dict(head_dim=60),
           dict(head_dim=136), dict(head_dim=0), dict(causal=2), dict(scale=float("inf")),
           dict(batch=2)]  # two sequences without offsets
    for kw in bad:
        assert call(**kw) == 1, kw
        if "batch" not in kw or kw["batch"] < 1:
            assert lib.gs_attention_workspace_bytes(C.byref(shape(**kw))) == 0, kw
    assert call(tokens_q=0) == 0
    assert call(cu=(P, None)) == 1 and call(cu=(P, MIS)) == 1
    assert call(lse=None) == 1 and call(lse=MIS) == 1 and call(wsp=None) == 1
    assert call(q=_h(None)) == 1 and call(q=_h(hs=48)) == 1 and call(k=_h(ts=124)) == 1
    assert call(wsb=ws - 1) == 5

    def bwd(dq=None, dk=None, lse=P, wsb=1 << 40):
        k = _h(ts=128)
        return lib.gs_attention_bwd(C.byref(shape()), _h(), k, k, None, None, _h(), lse, _h(),
                                    dq or _h(), dk or k, k, P, wsb, None)

    assert bwd(dq=_h(MIS)) == 1 and bwd(dk=_h(None)) == 1 and bwd(lse=None) == 1
    assert bwd(wsb=ws - 1) == 5


def test_attention_workspace_covers_every_mask(lib):
    # one size for a shape, whatever the mask and scale
    import differentiable_gaussian_splatting_gb300 as gs

    for tq, tk, b, hq, hk, d in ((1, 40000, 1, 16, 16, 64), (8160, 8160, 1, 16, 4, 128),
                                 (2500, 2500, 1, 8, 8, 64), (3330, 3339, 3, 8, 2, 16),
                                 (1 << 30, 1 << 30, 1 << 20, 1024, 1, 128)):
        sizes = {lib.gs_attention_workspace_bytes(C.byref(gs.AttentionShape(tq, tk, b, hq, hk, d, c, s)))
                 for c in (0, 1) for s in (0.1, -3.0)}
        assert len(sizes) == 1
        n = sizes.pop()
        assert n == gs.gs_attention_workspace_bytes(tq, tk, b, hq, hk, d)
        # the gradient's two rows of lse and delta, and at most a quarter of a GB of pieces
        assert 8 * tq * hq <= n <= 8 * tq * hq + (1 << 28)


def test_dropout_arguments_are_checked_on_the_host(lib):
    def call(n=100, ty=1, x=P, res=None, out=P, rng=P, p=0.1):
        return lib.gs_dropout_add(n, ty, x, res, out, rng, p, None)

    assert call(n=0) == 0
    assert call(n=-1) == 1 and call(ty=2) == 1 and call(x=None) == 1 and call(x=MIS) == 1
    assert call(out=MIS) == 1 and call(rng=None) == 1 and call(res=MIS) == 1
    for p in (-0.1, 1.0, 1.5, float("nan"), 1 - 2.0 ** -20):
        assert call(p=p) == 1, p
    assert lib.gs_dropout_add_bwd(100, 1, None, P, P, 0.1, None) == 1
    assert lib.gs_dropout_add_bwd(0, 0, None, None, None, 0.1, None) == 0


def test_binding_refuses_wrong_tensors():
    import torch

    import differentiable_gaussian_splatting_gb300 as gs

    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)  # on the CPU
    with pytest.raises(ValueError, match="CUDA"):
        gs.gs_attention_fwd(x, x, x, x, None, None)
    with pytest.raises(ValueError, match="CUDA"):
        gs.gs_qk_norm_rope(x, x, None, None, None, None, x, x)
    with pytest.raises(ValueError):
        gs.gs_dropout_add(x.half(), None, x, None, 0.1)
