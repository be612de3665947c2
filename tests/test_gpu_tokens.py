"""The token operators' kernels against their float64 definitions (tests/token_ref.py).

Tolerances, with u = 2^-24 (fp32) and h = 2^-8 (bfloat16), derived from the formulas:

head norm   an output is r (A x + B x'): the sum of squares over at most 256 values in lanes
            and shuffles (8 + 5 roundings, halved by the root), the reciprocal root (2 u) and
            five products and sums: below 32 u of its terms' magnitude.  The gradient's two
            sums and its longer chain: 64 u.  bfloat16 outputs carry h of the value besides.
            dw sums one term per row: rows u + 64 u of the sum of magnitudes.
attention   the probabilities are rounded to bfloat16 once, relative to their own size, for
            the second product, and the output once: 2 h of sum p |v|, which bounds |out|;
            scores (D products, exponent below 32) and the rest in fp32: 2^-12 of it.
            lse: the scores' D u of their terms, and 4 u (1 + |lse|) + 2^-20 for the fp32 sum
            and the exponential.
            gradients: token_ref.attention_bwd's bound and h of the value for the output.
dropout     the mask is exact; a kept value is one fused multiply-add with a rounded factor:
            2 u of the terms' magnitudes, and h of the value in bfloat16.
"""

import numpy as np
import pytest

import token_ref as ref
from token_ref import H, U

pytestmark = pytest.mark.gpu

NAMES = {"f32": np.float32, "bf16": None}


def _torch():
    import torch

    return torch


def _dev(x, dtype="f32"):
    torch = _torch()
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda()
    return t.to(torch.bfloat16) if dtype == "bf16" else t


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _round(x, dtype):
    x = np.asarray(x, np.float32)
    return ref.bf16(x) if dtype == "bf16" else x


def _close(got, want, bound, what):
    got = _np(got) if not isinstance(got, np.ndarray) else got
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    err = np.where(same, 0.0, np.abs(got - want))
    worst = np.unravel_index(np.argmax(err - bound), err.shape) if err.size else None
    assert (err <= bound).all(), (what, worst, got[worst], want[worst], bound[worst])


# ---------------------------------------------------------------------------
# head norm + rotation
# ---------------------------------------------------------------------------
CASES = [  # tokens, hq, hk, dim, rot, interleaved, dtype, positions, weights
    (1, 1, 1, 8, 8, False, "bf16", "given", True),
    (1, 8, 8, 64, 64, False, "bf16", None, True),
    (37, 5, 3, 40, 20, False, "bf16", "given", True),     # pairs that no 8 columns hold
    (64, 8, 8, 64, 32, True, "bf16", "given", True),
    (33, 16, 4, 128, 128, False, "bf16", "given", False),
    (300, 3, 1, 96, 48, False, "f32", "given", True),
    (17, 2, 2, 256, 256, False, "f32", None, True),
    (17, 20, 1, 256, 254, True, "bf16", "given", True),
    (5, 1, 9, 16, 2, False, "f32", "given", True),
    (9, 4, 4, 64, 0, False, "bf16", None, True),           # no rotation
    (2500, 2, 1, 24, 24, True, "f32", None, False),
]


def _norm_inputs(T, hq, hk, D, rot, dtype, positions, weights, seed=0):
    rng = np.random.default_rng(seed)
    q, k = (_round(rng.normal(size=(T, h, D)) * rng.uniform(0.3, 3, (T, h, 1)), dtype)
            for h in (hq, hk))
    qw, kw = ((rng.normal(1, 0.2, D).astype(np.float32) for _ in range(2)) if weights
              else (None, None))
    P = T if positions is None else max(1, T // 2)
    ang = rng.uniform(-4, 4, (P, rot // 2))
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32) if rot else None
    pos = rng.integers(-1, P, T).astype(np.int32) if positions else None
    return rng, q, k, qw, kw, table, pos


@pytest.mark.parametrize("T,hq,hk,D,rot,inter,dtype,positions,weights", CASES)
@pytest.mark.parametrize("packed", [False, True])
def test_head_norm(T, hq, hk, D, rot, inter, dtype, positions, weights, packed):
    import differentiable_gaussian_splatting_gb300 as gs

    torch = _torch()
    rng, q, k, qw, kw, table, pos = _norm_inputs(T, hq, hk, D, rot, dtype, positions, weights)
    opt = lambda x: None if x is None else torch.from_numpy(x).cuda()
    if packed:  # queries, keys and values side by side; outputs in [heads, tokens, dim] order
        both = torch.full((T, hq + hk + 2, D), float("nan"), device="cuda")
        both[:, :hq], both[:, hq:hq + hk] = _dev(q), _dev(k)
        both = both.to(_dev(q[:1], dtype).dtype)
        tq, tk = both[:, :hq], both[:, hq:hq + hk]
        qo = torch.full((hq, T, D), float("nan"), device="cuda", dtype=both.dtype).transpose(0, 1)
    else:
        tq, tk = _dev(q, dtype), _dev(k, dtype)
        qo = torch.full_like(tq, float("nan"))
    ko = torch.full((T, hk, D), float("nan"), device="cuda", dtype=tq.dtype)
    args = (opt(qw), opt(kw), opt(table), opt(pos))
    gs.gs_qk_norm_rope(tq, tk, *args, qo, ko, eps=1e-5, interleaved=inter)
    eps = float(np.float32(1e-5))
    h = H if dtype == "bf16" else 0.0
    for x, w, got, n in ((q, qw, qo, "q"), (k, kw, ko, "k")):
        y, m = ref.head_norm(x, w, table, pos, eps, inter)
        _close(got, y, h * np.abs(y) + 32 * U * m, n)
    # the gradient
    dq, dk = (_round(rng.normal(size=x.shape), dtype) for x in (q, k))
    gq, gk = torch.full_like(qo, float("nan")), torch.full_like(ko, float("nan"))
    gqw, gkw = (torch.full((D,), float("nan"), device="cuda") for _ in range(2))
    ws = torch.empty(gs.gs_qk_norm_rope_workspace_bytes(T, hq, hk, D), dtype=torch.uint8,
                     device="cuda")
    gs.gs_qk_norm_rope_bwd(tq, tk, *args, _dev(dq, dtype), _dev(dk, dtype), gq, gk, gqw, gkw, ws,
                           eps=1e-5, interleaved=inter)
    for x, w, dy, got, gw, n in ((q, qw, dq, gq, gqw, "dq"), (k, kw, dk, gk, gkw, "dk")):
        dx, dxm, dw, dwm = ref.head_norm_bwd(x, w, table, pos, eps, inter, dy)
        _close(got, dx, h * np.abs(dx) + 64 * U * dxm, n)
        rows = x.shape[0] * x.shape[1]
        _close(gw, dw, (rows + 64) * U * dwm, n + " weight")
    first = gqw.clone(), gq.clone()
    gs.gs_qk_norm_rope_bwd(tq, tk, *args, _dev(dq, dtype), _dev(dk, dtype), gq, gk, gqw, gkw, ws,
                           eps=1e-5, interleaved=inter)
    assert torch.equal(first[0], gqw) and torch.equal(first[1], gq)


@pytest.mark.parametrize("dtype,rot", [("bf16", 64), ("bf16", 24), ("f32", 48)])
def test_head_norm_in_place(dtype, rot):
    import differentiable_gaussian_splatting_gb300 as gs

    torch = _torch()
    rng, q, k, qw, kw, table, pos = _norm_inputs(50, 6, 2, 64, rot, dtype, "given", True, 5)
    args = [torch.from_numpy(x).cuda() for x in (qw, kw, table, pos)]
    tq, tk = _dev(q, dtype), _dev(k, dtype)
    qo, ko = torch.empty_like(tq), torch.empty_like(tk)
    gs.gs_qk_norm_rope(tq, tk, *args, qo, ko)
    a, b = tq.clone(), tk.clone()
    gs.gs_qk_norm_rope(a, b, *args, a, b)
    assert torch.equal(a, qo) and torch.equal(b, ko)
    ws = torch.empty(gs.gs_qk_norm_rope_workspace_bytes(50, 6, 2, 64), dtype=torch.uint8,
                     device="cuda")
    dw = [torch.empty(64, device="cuda") for _ in range(4)]
    dq, dk = torch.randn_like(tq), torch.randn_like(tk)
    gq, gk = torch.empty_like(dq), torch.empty_like(dk)
    gs.gs_qk_norm_rope_bwd(tq, tk, *args, dq, dk, gq, gk, dw[0], dw[1], ws)
    a, b = dq.clone(), dk.clone()
    gs.gs_qk_norm_rope_bwd(tq, tk, *args, a, b, a, b, dw[2], dw[3], ws)  # over the gradients
    assert torch.equal(a, gq) and torch.equal(b, gk) and torch.equal(dw[0], dw[2])
    a, b = tq.clone(), tk.clone()
    gs.gs_qk_norm_rope_bwd(a, b, *args, dq, dk, a, b, dw[2], None, ws)   # over the inputs
    assert torch.equal(a, gq) and torch.equal(b, gk) and torch.equal(dw[0], dw[2])


def test_head_norm_edges():
    import differentiable_gaussian_splatting_gb300 as gs

    torch = _torch()
    T, D = 6, 64
    q = torch.randn((T, 2, D), device="cuda")
    q[0] = 0.0                      # a zero row stays zero
    q[1, 0, 3] = float("inf")       # its row alone is not finite
    table = torch.cat([torch.ones(4, 32), torch.zeros(4, 32)], 1).cuda()
    pos = torch.tensor([0, 1, 2, 3, 4, -7], dtype=torch.int32, device="cuda")
    out, ko = torch.empty_like(q), torch.empty_like(q)
    gs.gs_qk_norm_rope(q, q, None, None, table, pos, out, ko)
    assert (out[0] == 0).all() and torch.isfinite(out[1, 1]).all()
    assert torch.isfinite(out[2:4]).all() and torch.isnan(out[4]).all()  # beyond the table
    assert torch.isfinite(out[5]).all()
    empty = q[:0]
    gs.gs_qk_norm_rope(empty, empty, None, None, table, None, empty, empty)
    dw = torch.full((D,), 5.0, device="cuda")
    ws = torch.empty(gs.gs_qk_norm_rope_workspace_bytes(0, 2, 2, D), dtype=torch.uint8, device="cuda")
    gs.gs_qk_norm_rope_bwd(empty, empty, None, None, table, None, empty, empty, empty, empty, dw,
                           None, ws)
    assert (dw == 0).all()          # no tokens: a zero gradient


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def _attention_inputs(Tq, Tk, hq, hk, D, seed=0, spread=1.0):
    rng = np.random.default_rng(seed)
    q, k = (ref.bf16(rng.normal(size=(T, h, D)) * spread) for T, h in ((Tq, hq), (Tk, hk)))
    return rng, q, k, ref.bf16(rng.normal(size=(Tk, hk, D)))


def _run_attention(q, k, v, scale, causal, lens_q=None, lens_k=None, dout=None, poison=False):
    """out, lse and, with dout, the gradients; poison: q, k, v and dout lie in larger arrays of
    NaN, behind which the library must not look"""
    import differentiable_gaussian_splatting_gb300 as gs

    torch = _torch()
    Tq, hq, D = q.shape
    Tk, hk = k.shape[:2]
    cu = [None if n is None else torch.tensor(np.concatenate([[0], np.cumsum(n)]),
                                              dtype=torch.int32, device="cuda")
          for n in (lens_q, lens_k)]

    def put(x):
        if not poison:
            return _dev(x, "bf16")
        big = torch.full((x.shape[0] + 3, x.shape[1] + 1, D + 8), float("nan"), device="cuda",
                         dtype=torch.bfloat16)
        view = big[1:1 + x.shape[0], :x.shape[1], :D]
        view.copy_(_dev(x))
        return view

    batch = 1 if lens_q is None else len(lens_q)
    ws = torch.full((gs.gs_attention_workspace_bytes(Tq, Tk, batch, hq, hk, D),), 255,
                    dtype=torch.uint8, device="cuda")
    tq, tk, tv = put(q), put(k), put(v)
    nan = lambda t: torch.full(t.shape, float("nan"), device="cuda", dtype=torch.bfloat16)
    out, lse = nan(tq), torch.full((hq, Tq), float("nan"), device="cuda")
    kw = dict(cu_q=cu[0], cu_k=cu[1], causal=causal, scale=scale)
    gs.gs_attention_fwd(tq, tk, tv, out, lse, ws, **kw)
    if dout is None:
        return out, lse
    g = nan(tq), nan(tk), nan(tv)
    ws.fill_(255)
    gs.gs_attention_bwd(tq, tk, tv, out, lse, put(dout), *g, ws, **kw)
    return out, lse, g


def _check_attention(q, k, v, scale, causal, lens_q=None, lens_k=None, dout=None, poison=False):
    cu = [None if n is None else np.concatenate([[0], np.cumsum(n)]) for n in (lens_q, lens_k)]
    D = q.shape[2]
    got = _run_attention(q, k, v, scale, causal, lens_q, lens_k, dout, poison)
    out, lse, mag, smag = ref.attention(q, k, v, scale, causal, *cu)
    _close(got[0], out, (2 * H + 2.0 ** -12) * mag, "out")
    fin = np.isfinite(lse)
    l = _np(got[1])
    assert np.array_equal(np.isneginf(l), ~fin) and not np.isnan(l).any()
    _close(l[fin], lse[fin], (D * U * smag + 4 * U * (1 + np.abs(lse)) + 2.0 ** -20)[fin], "lse")
    if dout is not None:
        want = ref.attention_bwd(q, k, v, _np(got[0]), l, dout, scale, causal, *cu)
        for n, t in zip("qkv", got[2]):
            w, b = want[n]
            _close(t, w, b + H * np.abs(w) + 1e-30, "d" + n)
    return got


LENGTHS = [1, 2, 7, 63, 64, 65, 127, 128, 129, 200, 255, 256, 257, 513]


@pytest.mark.parametrize("n", LENGTHS)
@pytest.mark.parametrize("causal", [False, True])
def test_attention_lengths(n, causal):
    rng, q, k, v = _attention_inputs(n, n, 2, 2, 64, seed=n)
    _check_attention(q, k, v, 0.125, causal, dout=ref.bf16(rng.normal(size=q.shape)))


@pytest.mark.parametrize("n,m", [(1, 300), (1, 2500), (3, 129), (130, 1), (257, 100), (100, 257),
                                 (5, 1000), (700, 64), (129, 640)])
@pytest.mark.parametrize("causal", [False, True])
def test_attention_other_lengths_of_keys(n, m, causal):
    # causal with more queries than keys leaves the first rows empty
    rng, q, k, v = _attention_inputs(n, m, 4, 2, 64, seed=n + m)
    _check_attention(q, k, v, 0.125, causal, dout=ref.bf16(rng.normal(size=q.shape)))


@pytest.mark.parametrize("D", [8, 16, 40, 64, 72, 96, 120, 128])
@pytest.mark.parametrize("hq,hk", [(1, 1), (6, 2), (8, 1)])
def test_attention_head_layouts(D, hq, hk):
    rng, q, k, v = _attention_inputs(150, 150, hq, hk, D, seed=D)
    _check_attention(q, k, v, D ** -0.5, True, dout=ref.bf16(rng.normal(size=q.shape)))


@pytest.mark.parametrize("lens_q,lens_k", [
    ([5], [5]), ([0, 1, 130, 0, 64], [0, 1, 130, 0, 64]), ([100, 0, 40], [0, 30, 200]),
    ([1] * 40, [3] * 40), ([300, 129, 1, 128], [10, 260, 128, 1]), ([0, 0], [7, 0]),
    ([0, 0], [0, 0]), ([5, 0], [0, 0]),
])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_ragged(lens_q, lens_k, causal, D):
    rng, q, k, v = _attention_inputs(sum(lens_q), sum(lens_k), 4, 2, D, seed=len(lens_q))
    _check_attention(q, k, v, D ** -0.5, causal, lens_q, lens_k,
                     dout=ref.bf16(rng.normal(size=q.shape)))


@pytest.mark.parametrize("D", [40, 64, 128])
def test_attention_reads_nothing_outside(D):
    # views into arrays that hold NaN everywhere else, and neighbours in the batch that hold
    # NaN and infinities: the other sequences' results are as without them
    lens = [70, 33, 130]
    rng, q, k, v = _attention_inputs(sum(lens), sum(lens), 3, 3, D, seed=4)
    do = ref.bf16(rng.normal(size=q.shape))
    _check_attention(q, k, v, D ** -0.5, False, lens, lens, dout=do, poison=True)
    clean = _run_attention(q, k, v, D ** -0.5, True, lens, lens, do)
    bad = [x.copy() for x in (q, k, v, do)]
    for x, val in zip(bad, (np.nan, np.inf, np.nan, -np.inf)):
        x[70:103] = val
    dirty = _run_attention(*bad[:3], D ** -0.5, True, lens, lens, bad[3])
    torch = _torch()
    rest = torch.tensor([i for i in range(233) if not 70 <= i < 103], device="cuda")
    for a, b in ((clean[0], dirty[0]), (clean[1].t(), dirty[1].t()), *zip(clean[2], dirty[2])):
        assert torch.equal(a[rest], b[rest])
    assert torch.isnan(dirty[0][70:103]).all()


def test_attention_large_scores():
    # scores far apart: rows whose maximum rises late, by much and by little, and rows that
    # one key takes whole
    rng, q, k, v = _attention_inputs(260, 700, 2, 2, 64, seed=9)
    ramp = np.linspace(0.05, 1.0, 700)[:, None, None]
    _check_attention(q, ref.bf16(k * ramp * 1.9), v, 0.125, False,
                     dout=ref.bf16(rng.normal(size=q.shape)))
    q2 = q.copy()
    q2[3] = 0.0                                   # equal scores
    got = _check_attention(q2, k, v, 0.125, False)
    _close(got[0][3], v.astype(np.float64).mean(0), 2 * H * np.abs(v).mean(0) + 1e-6, "mean")
    # scores of some thousands: the softmax picks the largest
    q3, k3 = np.zeros((5, 1, 64), np.float32), np.zeros((300, 1, 64), np.float32)
    q3[:, 0, 0], k3[:, 0, 0] = 64.0, np.arange(300)
    v3 = ref.bf16(rng.normal(size=(300, 1, 64)))
    out, lse = _run_attention(q3, k3, v3, 1.0, False)
    k3b = ref.bf16(k3)[:, 0, 0]
    best = np.flatnonzero(k3b == k3b.max())
    want = np.broadcast_to(v3[best].astype(np.float64).mean(0), (5, 1, 64))
    _close(out, want, 2 * H * np.abs(v3[best]).mean(0) + 0 * want, "largest")
    assert np.allclose(_np(lse), 64.0 * k3b.max() + np.log(len(best)), rtol=1e-6)


def test_attention_negative_and_zero_scale():
    rng, q, k, v = _attention_inputs(140, 150, 2, 1, 64, seed=12)
    do = ref.bf16(rng.normal(size=q.shape))
    _check_attention(q, k, v, -0.125, False, dout=do)
    _check_attention(q, k, v, 0.0, True, dout=do)


def test_attention_gradient_against_differences():
    # the definition's own change along a direction, against the kernels' gradients
    rng, q, k, v = _attention_inputs(90, 140, 4, 2, 64, seed=20)
    do = ref.bf16(rng.normal(size=q.shape))
    out, lse, g = _run_attention(q, k, v, 0.125, True, dout=do)
    want = ref.attention_bwd(q, k, v, _np(out), _np(lse), do, 0.125, True)
    args = dict(q=q.astype(np.float64), k=k.astype(np.float64), v=v.astype(np.float64))
    f = lambda a: (ref.attention(a["q"], a["k"], a["v"], 0.125, True)[0] * do).sum()
    exact = ref.attention_bwd(args["q"], args["k"], args["v"], *ref.attention(**args, scale=0.125,
                              causal=True)[:2], do, 0.125, True)
    for n, t in zip("qkv", g):
        d = rng.normal(size=args[n].shape)
        h = 1e-5
        num = (f({**args, n: args[n] + h * d}) - f({**args, n: args[n] - h * d})) / (2 * h)
        w, b = want[n]
        # the kernel's own bound, and what the rounded out moves delta by
        tol = ((b + H * np.abs(w) + np.abs(w - exact[n][0])) * np.abs(d)).sum() + 1e-6 * abs(num)
        assert abs((_np(t) * d).sum() - num) <= tol, n


@pytest.mark.parametrize("n,m,D,causal", [(300, 300, 64, True), (1, 5000, 64, False),
                                          (700, 520, 128, False)])
def test_attention_same_bits_again_and_on_another_stream(n, m, D, causal):
    import differentiable_gaussian_splatting_gb300 as gs

    torch = _torch()
    rng, q, k, v = _attention_inputs(n, m, 4, 2, D, seed=30)
    do = ref.bf16(rng.normal(size=q.shape))
    a = _run_attention(q, k, v, D ** -0.5, causal, dout=do)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = _run_attention(q, k, v, D ** -0.5, causal, dout=do)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for x, y in zip(a[2], b[2]):
        assert torch.equal(x, y)


def test_attention_offsets_out_of_order_stay_inside():
    # offsets beyond the arrays or descending are cut; nothing outside is touched
    import differentiable_gaussian_splatting_gb300 as gs

    torch = _torch()
    rng, q, k, v = _attention_inputs(100, 100, 2, 2, 64, seed=40)
    t = [_dev(x, "bf16") for x in (q, k, v)]
    out = torch.zeros_like(t[0])
    lse = torch.zeros((2, 100), device="cuda")
    ws = torch.empty(gs.gs_attention_workspace_bytes(100, 100, 3, 2, 2, 64), dtype=torch.uint8,
                     device="cuda")
    cu = torch.tensor([0, 60, 40, 1000], dtype=torch.int32, device="cuda")
    gs.gs_attention_fwd(*t, out, lse, ws, cu_q=cu, cu_k=cu)
    g = [torch.zeros_like(x) for x in t]
    gs.gs_attention_bwd(*t, out, lse, t[0], *g, ws, cu_q=cu, cu_k=cu)
    torch.cuda.synchronize()
    want = ref.attention(q[:40], k[:40], v[:40], 0.125)[0]  # ends at 60, yet inside the first
    assert want.shape == (40, 2, 64)


@pytest.mark.parametrize("lens_q,lens_k,hq,hk,D,causal", [
    ([1115, 2215, 0], [1115, 2215, 9], 8, 2, 16, True),   # few blocks: keys in pieces
    ([3, 700, 1], [4000, 1500, 33], 4, 4, 64, False),
    ([3, 700, 1], [4000, 1500, 33], 4, 1, 128, True),
    ([2300], [2300], 17, 1, 64, False),                   # a last wave of 1 block of 153
    ([1, 1, 1], [6000, 90, 2500], 8, 8, 128, False),
])
def test_attention_keys_in_pieces(lens_q, lens_k, hq, hk, D, causal):
    # scores whose maximum keeps rising, so that rows are rescaled while products are in flight
    rng, q, k, v = _attention_inputs(sum(lens_q), sum(lens_k), hq, hk, D, seed=77)
    ramp = np.concatenate([np.linspace(0.1, 1.0, max(n, 1))[:n] for n in lens_k])
    k = ref.bf16(k * ramp[:, None, None] * 1.9)
    do = ref.bf16(rng.normal(size=q.shape))
    got = _check_attention(q, k, v, D ** -0.5, causal, lens_q, lens_k, dout=do)
    for _ in range(3):
        again = _run_attention(q, k, v, D ** -0.5, causal, lens_q, lens_k, do)
        for a, b in ((got[0], again[0]), (got[1], again[1]), *zip(got[2], again[2])):
            assert bool((a == b).all())


def test_attention_strided_heads():
    # [heads, tokens, dim] arrays and a packed projection, gradients into a packed one
    import differentiable_gaussian_splatting_gb300 as gs

    torch = _torch()
    T, hq, hk, D = 170, 4, 2, 64
    rng, q, k, v = _attention_inputs(T, T, hq, hk, D, seed=50)
    do = ref.bf16(rng.normal(size=q.shape))
    plain = _run_attention(q, k, v, 0.125, True, dout=do)
    packed = torch.cat([_dev(x, "bf16") for x in (q, k, v)], 1)
    tq, tk, tv = packed[:, :hq], packed[:, hq:hq + hk], packed[:, hq + hk:]
    out = torch.empty((hq, T, D), device="cuda", dtype=torch.bfloat16).transpose(0, 1)
    lse = torch.empty((hq, T), device="cuda")
    ws = torch.empty(gs.gs_attention_workspace_bytes(T, T, 1, hq, hk, D), dtype=torch.uint8,
                     device="cuda")
    gs.gs_attention_fwd(tq, tk.transpose(0, 1).contiguous().transpose(0, 1), tv, out, lse, ws,
                        causal=True)
    assert torch.equal(out, plain[0]) and torch.equal(lse, plain[1])
    dp = torch.full_like(packed, float("nan"))
    gs.gs_attention_bwd(tq, tk, tv, out, lse, _dev(do, "bf16"), dp[:, :hq], dp[:, hq:hq + hk],
                        dp[:, hq + hk:], ws, causal=True)
    assert torch.equal(dp, torch.cat(plain[2], 1))


def test_attention_long_rows():
    # 4,346 and 8,160 tokens, sampled heads and rows against the definition
    for T, D in ((4346, 128), (8160, 64)):
        rng, q, k, v = _attention_inputs(T, T, 2, 1, D, seed=T)
        out, lse = _run_attention(q, k, v, D ** -0.5, False)
        rows = np.sort(rng.choice(T, 64, replace=False))
        want, l, mag, smag = ref.attention(q[rows], k, v, D ** -0.5)
        _close(_np(out)[rows], want, (2 * H + 2.0 ** -12) * mag, "out")
        _close(_np(lse)[:, rows], l, D * U * smag + 4 * U * (1 + np.abs(l)) + 2.0 ** -20, "lse")


def test_attention_status_reports_a_wait_that_gave_up():
    # the kernels' own bounded wait, on a barrier at which nothing arrives (a test-only
    # launcher): it ends, is reported once, and the context goes on
    import ctypes as C

    import differentiable_gaussian_splatting_gb300 as gs

    torch = _torch()
    gs.gs_attention_status()
    lib = gs.library()
    lib.gs_test_attention_wait.restype = C.c_int
    lib.gs_test_attention_wait.argtypes = [C.c_void_p]
    assert lib.gs_test_attention_wait(torch.cuda.current_stream().cuda_stream) == 0
    with pytest.raises(gs.GSError) as e:
        gs.gs_attention_status()
    assert e.value.status == 4
    gs.gs_attention_status()
    rng, q, k, v = _attention_inputs(200, 200, 2, 2, 64, seed=60)
    _check_attention(q, k, v, 0.125, True)


# ---------------------------------------------------------------------------
# dropout-add
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("n", [1, 7, 8, 9, 2047, 2048, 2049, 100_003])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("p,with_residual", [(0.1, True), (0.5, False), (0.0, True), (0.9, False)])
def test_dropout_add(n, dtype, p, with_residual):
    import differentiable_gaussian_splatting_gb300 as gs

    torch = _torch()
    rng = np.random.default_rng(n)
    x, y = (_round(rng.normal(size=n), dtype) for _ in range(2))
    seed, offset = -(2 ** 62) + 12345, 2 ** 40 + n
    state = torch.tensor([seed, offset], dtype=torch.int64, device="cuda")
    out = torch.full((n,), float("nan"), device="cuda", dtype=_dev(x[:1], dtype).dtype)
    res = _dev(y, dtype) if with_residual else None
    gs.gs_dropout_add(_dev(x, dtype), res, out, state, p)
    keep, f = ref.kept(n, seed, offset, p)
    part = np.where(keep, x.astype(np.float64) * f, 0.0)
    want = part + (y if with_residual else 0.0)
    mag = np.abs(part) + (np.abs(y) if with_residual else 0.0)
    h = H if dtype == "bf16" else 0.0
    _close(out, want, h * np.abs(want) + 2 * U * mag, "out")
    if not with_residual:
        assert np.array_equal(_np(out) == 0, ~keep | (x == 0))
    dx = torch.full_like(out, float("nan"))
    gs.gs_dropout_add_bwd(_dev(y, dtype), dx, state, p)
    want = np.where(keep, y.astype(np.float64) * f, 0.0)
    _close(dx, want, h * np.abs(want) + 2 * U * np.abs(want), "dx")
    # over its own input, over the residual
    a = _dev(x, dtype)
    gs.gs_dropout_add(a, res, a, state, p)
    assert torch.equal(a, out)
    if with_residual:
        b = res.clone()
        gs.gs_dropout_add(_dev(x, dtype), b, b, state, p)
        assert torch.equal(b, out)


def test_dropout_drops_what_is_not_finite():
    import differentiable_gaussian_splatting_gb300 as gs

    torch = _torch()
    x = torch.full((4096,), float("nan"), device="cuda")
    x[::2] = float("inf")
    state = torch.tensor([3, 4], dtype=torch.int64, device="cuda")
    out, r = torch.empty_like(x), torch.ones_like(x)
    gs.gs_dropout_add(x, r, out, state, 0.5)
    keep, _ = ref.kept(4096, 3, 4, 0.5)
    assert np.array_equal(np.isfinite(_np(out)), ~keep) and (_np(out)[~keep] == 1.0).all()


def test_dropout_in_a_captured_graph_takes_the_new_state():
    import differentiable_gaussian_splatting_gb300 as gs

    torch = _torch()
    x = torch.ones(1000, device="cuda")
    out, state = torch.empty_like(x), torch.tensor([1, 0], dtype=torch.int64, device="cuda")
    gs.gs_dropout_add(x, None, out, state, 0.5)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gs.gs_dropout_add(x, None, out, state, 0.5)
    for offset in (5, 6):
        state[1] = offset
        g.replay()
        assert np.array_equal(_np(out) != 0, ref.kept(1000, 1, offset, 0.5)[0])


def test_calls_refuse_bad_tensors():
    import differentiable_gaussian_splatting_gb300 as gs

    torch = _torch()
    x = torch.zeros((8, 2, 64), device="cuda", dtype=torch.bfloat16)
    lse = torch.zeros((2, 8), device="cuda")
    ws = torch.empty(gs.gs_attention_workspace_bytes(8, 8, 1, 2, 2, 64), dtype=torch.uint8,
                     device="cuda")
    with pytest.raises(ValueError):
        gs.gs_attention_fwd(x.half(), x, x, x, lse, ws)
    with pytest.raises(ValueError):
        gs.gs_attention_fwd(x, x, x[:, :1], x, lse, ws)
    with pytest.raises(gs.GSError):
        gs.gs_attention_fwd(x, x, x, x.clone(), lse, ws[:16])
    with pytest.raises(gs.GSError):  # rows that overlap
        gs.gs_attention_fwd(x[:1].expand(8, 2, 64), x, x, x.clone(), lse, ws)
    with pytest.raises(gs.GSError):  # a stride that is not whole 16-byte words
        odd = torch.zeros((8, 2, 66), device="cuda", dtype=torch.bfloat16)[..., :64]
        gs.gs_attention_fwd(odd, x, x, x.clone(), lse, ws)
    with pytest.raises(ValueError):
        gs.gs_qk_norm_rope(x, x[:4], None, None, None, None, x, x)
    with pytest.raises(gs.GSError):
        gs.gs_dropout_add(x, None, x, torch.zeros(2, dtype=torch.int64, device="cuda"), 1.0)
