"""Window attention against its float64 definition (tests/block_ref.py).

Tolerances as those of full attention, with u = 2^-24 and h = 2^-8: the probabilities are rounded to
bfloat16 once and so is the output, 2 h of sum p |v|; scores (D <= 128 products, exponents below 32)
and the rest in fp32, 2^-12 of it.  lse: the scores' D u of their terms, and 4 u (1 + |lse|) + 2^-20.
Gradients: the definition's bound, and h of the value for the output."""

import numpy as np
import pytest

import block_ref as ref
from token_ref import H, U, bf16

pytestmark = pytest.mark.gpu


def _inputs(Tq, Tk, hq, hk, D, seed=0):
    rng = np.random.default_rng(seed)
    q, k = (bf16(rng.normal(size=(T, h, D))) for T, h in ((Tq, hq), (Tk, hk)))
    return rng, q, k, bf16(rng.normal(size=(Tk, hk, D)))


def _dev(x):
    import torch

    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda().bfloat16()


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _run(q, k, v, scale, window, causal, lens_q=None, lens_k=None, dout=None, poison=False, gs_out=None):
    """out, lse and, with dout, the gradients; poison: inputs lie in larger arrays of NaN"""
    import torch

    import differentiable_gaussian_splatting_gb300 as gs

    Tq, hq, D = q.shape
    Tk, hk = k.shape[:2]
    cu = [None if n is None else torch.tensor(np.concatenate([[0], np.cumsum(n)]),
                                              dtype=torch.int32, device="cuda")
          for n in (lens_q, lens_k)]

    def put(x):
        if not poison:
            return _dev(x)
        big = torch.full((x.shape[0] + 3, x.shape[1] + 1, D + 8), float("nan"), device="cuda",
                         dtype=torch.bfloat16)
        view = big[1:1 + x.shape[0], :x.shape[1], :D]
        view.copy_(_dev(x))
        return view

    batch = 1 if lens_q is None else len(lens_q)
    size = gs.gs_attention_window_workspace_bytes(Tq, Tk, batch, hq, hk, D, *window)
    ws = torch.full((size + 64,), 255, dtype=torch.uint8, device="cuda")
    tq, tk, tv = put(q), put(k), put(v)
    nan = lambda t: torch.full(t.shape, float("nan"), device="cuda", dtype=torch.bfloat16)
    out, lse = nan(tq), torch.full((hq, Tq), float("nan"), device="cuda")
    kw = dict(cu_q=cu[0], cu_k=cu[1], causal=causal, scale=scale)
    gs.gs_attention_window_fwd(tq, tk, tv, out, lse, ws[:size], *window, **kw)
    assert (ws[size:] == 255).all()
    if dout is None:
        return out, lse
    g = nan(tq), nan(tk), nan(tv)
    ws.fill_(255)
    gs.gs_attention_window_bwd(tq, tk, tv, out, lse, put(dout), *g, ws[:size], *window, **kw)
    assert (ws[size:] == 255).all()
    return out, lse, g


def _close(got, want, bound, what):
    got = _np(got) if not isinstance(got, np.ndarray) else got
    err = np.where(got == want, 0.0, np.abs(got - want))
    worst = np.unravel_index(np.argmax(err - bound), err.shape) if err.size else None
    assert (err <= bound).all(), (what, worst, got[worst], want[worst], bound[worst])


def _check(q, k, v, scale, window, causal, lens_q=None, lens_k=None, dout=None, poison=False):
    cu = [None if n is None else np.concatenate([[0], np.cumsum(n)]) for n in (lens_q, lens_k)]
    D = q.shape[2]
    got = _run(q, k, v, scale, window, causal, lens_q, lens_k, dout, poison)
    out, lse, mag, smag = ref.window_attention(q, k, v, scale, *window, causal, *cu)
    fin = np.isfinite(lse)
    l = _np(got[1])
    assert np.array_equal(np.isneginf(l), ~fin) and not np.isnan(l).any()
    _close(got[0], out, (2 * H + 2.0 ** -12) * mag, "out")
    _close(l[fin], lse[fin], (D * U * smag + 4 * U * (1 + np.abs(lse)) + 2.0 ** -20)[fin], "lse")
    if dout is not None:
        want = ref.window_attention_bwd(q, k, v, _np(got[0]), l, dout, scale, *window, causal, *cu)
        for n, t in zip("qkv", got[2]):
            w, b = want[n]
            _close(t, w, b + H * np.abs(w) + 1e-30, "d" + n)
    return got


WINDOWS = [(0, 0, 0), (0, 0, 1), (1, 0, 4), (5, 3, 0), (127, 0, 4), (128, 0, 128), (64, 200, 16),
           (300, 300, 4), (129, 0, 0), (2 ** 31 - 1, 0, 0), (0, 2 ** 31 - 1, 3),
           (2 ** 31 - 1, 2 ** 31 - 1, 128)]


@pytest.mark.parametrize("n", [1, 2, 127, 128, 129, 257, 640, 1000])
@pytest.mark.parametrize("window", range(len(WINDOWS)))
@pytest.mark.parametrize("causal", [False, True])
def test_window_lengths(n, window, causal):
    rng, q, k, v = _inputs(n, n, 2, 1, 64, seed=n)
    _check(q, k, v, 0.125, WINDOWS[window], causal, dout=bf16(rng.normal(size=q.shape)))


@pytest.mark.parametrize("n,m", [(1, 300), (1, 2500), (3, 129), (130, 1), (257, 100), (700, 257),
                                 (5, 1000), (700, 64), (640, 700), (900, 3), (4, 0), (0, 4)])
@pytest.mark.parametrize("window", [0, 1, 3, 4, 6, 9])
@pytest.mark.parametrize("causal", [False, True])
def test_window_other_lengths_of_keys(n, m, window, causal):
    # more queries than keys: the first rows stand before the first key
    rng, q, k, v = _inputs(n, m, 4, 2, 128, seed=n + m)
    _check(q, k, v, 0.09, WINDOWS[window], causal, dout=bf16(rng.normal(size=q.shape)))


@pytest.mark.parametrize("D", [8, 40, 64, 72, 128])
@pytest.mark.parametrize("hq,hk", [(1, 1), (6, 2), (8, 1), (17, 1), (12, 4)])
def test_window_head_layouts(D, hq, hk):
    rng, q, k, v = _inputs(300, 300, hq, hk, D, seed=D)
    _check(q, k, v, D ** -0.5, (100, 0, 4), True, dout=bf16(rng.normal(size=q.shape)))
    _check(q, k, v, D ** -0.5, (30, 40, 0), False, dout=bf16(rng.normal(size=q.shape)))


@pytest.mark.parametrize("lens_q,lens_k", [
    ([5], [5]), ([0, 1, 130, 0, 700], [0, 1, 130, 0, 700]), ([100, 0, 400], [0, 30, 200]),
    ([1] * 40, [3] * 40), ([300, 129, 1, 128], [10, 260, 128, 1]), ([0, 0], [7, 0]),
    ([0, 0], [0, 0]), ([5, 0], [0, 0]), ([1] * 7, [0, 1, 5, 1000, 129, 0, 2222]),
    ([1, 0, 2, 1], [700, 5, 900, 1]),
])
@pytest.mark.parametrize("window", [(50, 0, 4), (200, 100, 128), (0, 0, 0)])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_window_ragged(lens_q, lens_k, window, causal, D):
    rng, q, k, v = _inputs(sum(lens_q), sum(lens_k), 4, 2, D, seed=len(lens_q))
    _check(q, k, v, D ** -0.5, window, causal, lens_q, lens_k, dout=bf16(rng.normal(size=q.shape)))


@pytest.mark.parametrize("lens,hq,hk,D,window", [
    ([1115, 2215, 0], 8, 2, 16, (700, 0, 4)),       # few blocks: keys in pieces
    ([2300], 17, 1, 64, (1000, 1000, 16)),
    ([3000, 1], 4, 1, 128, (100, 0, 4)),            # sinks' queries in pieces
    ([2000, 40, 1300], 2, 2, 64, (127, 128, 128)),
    ([600] * 5 + [0, 1] * 20, 4, 2, 64, (90, 0, 4)),  # more sequences than a warp has lanes
])
@pytest.mark.parametrize("causal", [False, True])
def test_window_long_and_many(lens, hq, hk, D, window, causal):
    # scores whose maximum keeps rising, so that rows are rescaled while products are in flight
    rng, q, k, v = _inputs(sum(lens), sum(lens), hq, hk, D, seed=77)
    ramp = np.concatenate([np.linspace(0.1, 1.0, max(n, 1))[:n] for n in lens])
    k = bf16(k * ramp[:, None, None] * 1.9)
    do = bf16(rng.normal(size=q.shape))
    got = _check(q, k, v, D ** -0.5, window, causal, lens, lens, dout=do)
    for _ in range(2):
        again = _run(q, k, v, D ** -0.5, window, causal, lens, lens, do)
        for a, b in ((got[0], again[0]), (got[1], again[1]), *zip(got[2], again[2])):
            assert bool((a == b).all())


@pytest.mark.parametrize("D", [8, 24, 32, 40, 64, 72, 96, 104, 128])
@pytest.mark.parametrize("hq,hk", [(1, 1), (6, 2), (8, 1), (17, 1), (12, 4), (9, 9)])
def test_window_of_single_tokens(D, hq, hk):
    # one or two queries a sequence; keys none, few, and several steps of every warp
    lens_q, lens_k = [1, 1, 0, 2, 1, 1, 2, 1], [700, 1, 50, 333, 0, 17, 1, 4100]
    rng, q, k, v = _inputs(sum(lens_q), sum(lens_k), hq, hk, D, seed=D + hq)
    ramp = np.concatenate([np.linspace(0.1, 1.0, max(n, 1))[:n] for n in lens_k])
    k = bf16(k * ramp[:, None, None] * 1.9)  # maxima that keep rising
    for window, causal in (((255, 0, 4), True), ((4096, 0, 0), True), ((0, 0, 128), False),
                           ((130, 7, 16), False)):
        _check(q, k, v, D ** -0.5, window, causal, lens_q, lens_k)
    _check(q, k, v, -0.3 * D ** -0.5, (1000, 0, 4), True, lens_q, lens_k, poison=True)


@pytest.mark.parametrize("batch", [1, 2, 31, 33, 1100])
def test_window_of_single_tokens_in_many_sequences(batch):
    # the search for a token's sequence, sequences without queries among them
    rng = np.random.default_rng(batch)
    lens_q, lens_k = list(rng.integers(0, 3, batch)), list(rng.integers(0, 40, batch))
    lens_q[-1] = 1
    while sum(lens_q) > 2 * batch:
        lens_q[int(np.argmax(lens_q))] -= 1
    _, q, k, v = _inputs(sum(lens_q), sum(lens_k), 4, 2, 64, seed=batch)
    _check(q, k, v, 0.125, (9, 0, 2), True, lens_q, lens_k)


def test_window_as_wide_as_all_equals_full_attention():
    import torch

    import differentiable_gaussian_splatting_gb300 as gs

    rng, q, k, v = _inputs(500, 500, 4, 2, 64, seed=3)
    do = bf16(rng.normal(size=q.shape))
    for causal in (False, True):
        out, lse, g = _run(q, k, v, 0.125, (500, 500, 0), causal, dout=do)
        t = [_dev(x) for x in (q, k, v)]
        ws = torch.empty(gs.gs_attention_workspace_bytes(500, 500, 1, 4, 2, 64), dtype=torch.uint8,
                         device="cuda")
        o, l = torch.empty_like(out), torch.empty_like(lse)
        gs.gs_attention_fwd(*t, o, l, ws, causal=causal, scale=0.125)
        assert (o.float() - out.float()).norm() < 2 * H * out.float().norm()
        assert (l - lse).abs().max() < 1e-5


@pytest.mark.parametrize("D", [40, 64, 128])
def test_window_reads_nothing_outside(D):
    import torch

    lens = [170, 33, 330]
    rng, q, k, v = _inputs(sum(lens), sum(lens), 3, 3, D, seed=4)
    do = bf16(rng.normal(size=q.shape))
    for window in ((60, 0, 4), (40, 40, 100)):
        _check(q, k, v, D ** -0.5, window, False, lens, lens, dout=do, poison=True)
        clean = _run(q, k, v, D ** -0.5, window, True, lens, lens, do)
        bad = [x.copy() for x in (q, k, v, do)]
        for x, val in zip(bad, (np.nan, np.inf, np.nan, -np.inf)):
            x[170:203] = val
        dirty = _run(*bad[:3], D ** -0.5, window, True, lens, lens, bad[3])
        rest = torch.tensor([i for i in range(533) if not 170 <= i < 203], device="cuda")
        for a, b in ((clean[0], dirty[0]), (clean[1].t(), dirty[1].t()), *zip(clean[2], dirty[2])):
            assert torch.equal(a[rest], b[rest])


def test_window_offsets_out_of_order_stay_inside():
    import torch

    import differentiable_gaussian_splatting_gb300 as gs

    rng, q, k, v = _inputs(400, 400, 2, 2, 64, seed=40)
    t = [_dev(x) for x in (q, k, v)]
    window = (30, 0, 4)
    size = gs.gs_attention_window_workspace_bytes(400, 400, 4, 2, 2, 64, *window)
    ws = torch.full((size + 4096,), 7, dtype=torch.uint8, device="cuda")
    wide = [torch.full((600, 2, 64), 3.0, device="cuda", dtype=torch.bfloat16) for _ in range(4)]
    out, *g = [w[100:500] for w in wide]
    lse = torch.zeros((2, 400), device="cuda")
    for offsets in ([0, 260, 140, 390, 4000], [-5, 300, 300, 200, 380], [390, 0, 390, 0, 390]):
        cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        gs.gs_attention_window_fwd(*t, out, lse, ws[:size], *window, cu_q=cu, cu_k=cu, causal=True)
        gs.gs_attention_window_bwd(*t, out, lse, t[0], *g, ws[:size], *window, cu_q=cu, cu_k=cu,
                                   causal=True)
    torch.cuda.synchronize()
    assert (ws[size:] == 7).all()
    assert all((w[:100] == 3).all() and (w[500:] == 3).all() for w in wide)
    gs.gs_attention_status()


def test_window_gradient_against_differences():
    # the definition's own change along a direction, against the kernels' gradients
    rng, q, k, v = _inputs(190, 240, 4, 2, 64, seed=20)
    do = bf16(rng.normal(size=q.shape))
    window, causal = (60, 0, 4), True
    out, lse, g = _run(q, k, v, 0.125, window, causal, dout=do)
    want = ref.window_attention_bwd(q, k, v, _np(out), _np(lse), do, 0.125, *window, causal)
    args = dict(q=q.astype(np.float64), k=k.astype(np.float64), v=v.astype(np.float64))
    f = lambda a: (ref.window_attention(a["q"], a["k"], a["v"], 0.125, *window, causal)[0] * do).sum()
    o, l, _, _ = ref.window_attention(**args, scale=0.125, left=60, right=0, sinks=4, causal=True)
    exact = ref.window_attention_bwd(args["q"], args["k"], args["v"], o, l, do, 0.125, *window, causal)
    for n, t in zip("qkv", g):
        d = rng.normal(size=args[n].shape)
        h = 1e-5
        num = (f({**args, n: args[n] + h * d}) - f({**args, n: args[n] - h * d})) / (2 * h)
        w, b = want[n]
        tol = ((b + H * np.abs(w) + np.abs(w - exact[n][0])) * np.abs(d)).sum() + 1e-6 * abs(num)
        assert abs((_np(t) * d).sum() - num) <= tol, n


def test_window_strided_heads_and_another_stream():
    # a packed projection, gradients into a packed one, [heads, tokens, dim] outputs
    import torch

    import differentiable_gaussian_splatting_gb300 as gs

    rng, q, k, v = _inputs(350, 350, 4, 2, 64, seed=8)
    do = bf16(rng.normal(size=q.shape))
    want = _run(q, k, v, 0.125, (70, 0, 4), True, dout=do)
    packed = torch.cat([_dev(q), _dev(k), _dev(v)], 1)
    out = torch.empty((4, 350, 64), device="cuda", dtype=torch.bfloat16).transpose(0, 1)
    lse, dout = torch.empty((4, 350), device="cuda"), _dev(do)
    g = torch.empty_like(packed)
    ws = torch.empty(gs.gs_attention_window_workspace_bytes(350, 350, 1, 4, 2, 64, 70, 0, 4),
                     dtype=torch.uint8, device="cuda")
    part = lambda t: (t[:, :4], t[:, 4:6], t[:, 6:])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gs.gs_attention_window_fwd(*part(packed), out, lse, ws, 70, 0, 4, causal=True, scale=0.125)
        gs.gs_attention_window_bwd(*part(packed), out, lse, dout, *part(g), ws, 70, 0, 4, causal=True,
                                   scale=0.125)
    torch.cuda.synchronize()
    for a, b in ((out, want[0]), (lse, want[1]), *zip(part(g), want[2])):
        assert torch.equal(a, b)


@pytest.mark.parametrize("lens_q,lens_k", [([1, 2, 1], [300, 40, 1500]), ([300], [900])])
def test_queries_that_are_not_finite_say_so(lens_q, lens_k):
    # NaN for the rows of such a query's head, as their softmax is; no other row's
    import torch

    rng, q, k, v = _inputs(sum(lens_q), sum(lens_k), 4, 2, 64, seed=9)
    clean = _run(q, k, v, 0.125, (200, 0, 4), True, lens_q, lens_k)
    bad = q.copy()
    bad[1, 2, 5], bad[0, 0, 0] = np.nan, np.nan
    out, lse = _run(bad, k, v, 0.125, (200, 0, 4), True, lens_q, lens_k)
    hit = torch.zeros(out.shape[:2], dtype=torch.bool, device="cuda")
    hit[1, 2] = hit[0, 0] = True
    assert out[hit].isnan().all() and lse.t()[hit].isnan().all()
    assert torch.equal(out[~hit], clean[0][~hit])
    assert torch.equal(lse.t()[~hit], clean[1].t()[~hit])


@pytest.mark.parametrize("hq,hk,D", [(8, 2, 128), (4, 2, 64), (10, 1, 40), (2, 2, 64)])
@pytest.mark.parametrize("window,causal", [((90, 0, 4), True), ((40, 3, 100), False), ((0, 0, 0), True)])
def test_some_queries_of_every_sequence(hq, hk, D, window, causal):
    # by the kernel of few queries or by tiles, as the heads on a key head decide
    rng, q, k, v = _inputs(15, 1161, hq, hk, D, seed=12)
    _check(q, k, v, D ** -0.5, window, causal, [3, 5, 1, 4, 2], [300, 4, 0, 857, 0])


@pytest.mark.parametrize("lens_q,lens_k", [([1, 0, 2], [200, 10, 90]), ([270, 0, 33], [300, 9, 33]),
                                           ([0, 0, 0], [50, 0, 2]), ([5, 0, 300], [0, 0, 0])])
@pytest.mark.parametrize("more", [4, 300])
def test_rows_behind_the_last_sequence_stay(lens_q, lens_k, more):
    import torch

    import differentiable_gaussian_splatting_gb300 as gs

    nq, nk, window = sum(lens_q), sum(lens_k), (60, 5, 4)
    Tq, Tk = nq + more, nk + 140
    rng, q, k, v = _inputs(Tq, Tk, 2, 1, 64, seed=3)
    t = [_dev(x) for x in (q, k, v)]
    cu = [torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda")
          for n in (lens_q, lens_k)]
    ws = torch.full((gs.gs_attention_window_workspace_bytes(Tq, Tk, 3, 2, 1, 64, *window),), 255,
                    dtype=torch.uint8, device="cuda")
    out, lse = torch.full_like(t[0], 7.0), torch.full((2, Tq), 7.0, device="cuda")
    g = [torch.full_like(x, 7.0) for x in t]
    kw = dict(cu_q=cu[0], cu_k=cu[1])
    gs.gs_attention_window_fwd(*t, out, lse, ws, *window, **kw)
    gs.gs_attention_window_bwd(*t, out, lse, t[0], *g, ws, *window, **kw)
    for x, n in ((out, nq), (lse.t(), nq), (g[0], nq), (g[1], nk), (g[2], nk)):
        assert (x[n:] == 7.0).all() and not x[:n].float().isnan().any()
        assert not (x[:n] == 7.0).all(1).any()
