"""Edges of the token operators on the GPU: waits that run out, arrays' surroundings, batches of
many sequences, long gradients.  Tolerances as derived in test_gpu_tokens.py."""

import numpy as np
import pytest

import token_ref as ref
from test_gpu_tokens import _attention_inputs, _check_attention, _close, _dev, _np, _torch
from token_ref import H, U

pytestmark = pytest.mark.gpu


def _let_a_wait_run_out():
    """A warp's wait in which one lane's phase never comes and the other lanes' are done"""
    import ctypes as C

    import differentiable_gaussian_splatting_gb300 as gs

    lib = gs.library()
    lib.gs_test_attention_wait.restype = C.c_int
    lib.gs_test_attention_wait.argtypes = [C.c_void_p]
    assert lib.gs_test_attention_wait(_torch().cuda.current_stream().cuda_stream) == 0


def test_a_warp_gives_up_as_one():
    # reported by the first lane, whose own phase was done: it has to give up with the last one
    import differentiable_gaussian_splatting_gb300 as gs

    gs.gs_attention_status()
    _let_a_wait_run_out()
    with pytest.raises(gs.GSError) as e:
        gs.gs_attention_status()
    assert e.value.status == 4
    gs.gs_attention_status()


def test_every_thread_is_told_of_a_wait_that_gave_up():
    import threading

    import differentiable_gaussian_splatting_gb300 as gs

    torch = _torch()

    def ask(told):
        with torch.cuda.stream(torch.cuda.Stream()):
            try:
                gs.gs_attention_status()
                told.append(0)
            except gs.GSError as e:
                told.append(e.status)

    asked, may_ask = threading.Event(), threading.Event()
    first, second, main = [], [], []

    def early():  # asks before and after
        ask(first)
        asked.set()
        may_ask.wait(60)
        ask(first)
        ask(first)

    ask(main)
    t = threading.Thread(target=early)
    t.start()
    assert asked.wait(60)
    _let_a_wait_run_out()
    torch.cuda.synchronize()
    ask(main)
    may_ask.set()
    t.join()
    ask(main)
    u = threading.Thread(target=ask, args=(second,))  # a thread that never asked before
    u.start()
    u.join()
    # what happened before this test may be told to the new threads as well
    assert main[1:] == [4, 0] and first[1:] == [4, 0] and second == [4]


# ---------------------------------------------------------------------------
# batches of many sequences
# ---------------------------------------------------------------------------
MIXED = [0, 129, 1, 300, 64, 0, 600, 127, 128, 5, 0, 257, 33, 1, 256, 2, 90, 0, 400, 7]


@pytest.mark.parametrize("lens_q,lens_k,hq,hk", [
    ((MIXED * 4)[:70], (MIXED * 4)[:70], 2, 1),
    ((MIXED * 4)[:70], (MIXED * 4)[3:73], 2, 2),        # other numbers of keys, empty sides
    ([0] * 20 + [1] * 12 + [500], [0] * 20 + [1] * 12 + [700], 4, 1),  # few blocks: cut in pieces
    ([3] * 33, [0] * 32 + [200], 1, 1),
])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_more_than_32_sequences(lens_q, lens_k, hq, hk, causal, D):
    rng, q, k, v = _attention_inputs(sum(lens_q), sum(lens_k), hq, hk, D, seed=len(lens_q) + D)
    _check_attention(q, k, v, D ** -0.5, causal, lens_q, lens_k,
                     dout=ref.bf16(rng.normal(size=q.shape)))


def test_attention_of_many_lone_tokens():
    # One key per query: out is its value and dV its dout to the bit, dS is rounding noise.  A
    # block finds its sequence without a walk over the others: both calls take 15 ms (with a
    # walk in every block they took 900).
    import differentiable_gaussian_splatting_gb300 as gs

    torch = _torch()
    n, h, D = 65536, 2, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v, do = (torch.randn((n, h, D), generator=g, device="cuda").bfloat16() for _ in range(4))
    cu = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    out, dq, dk, dv = (torch.full_like(q, float("nan")) for _ in range(4))
    lse = torch.empty((h, n), device="cuda")
    ws = torch.empty(gs.gs_attention_workspace_bytes(n, n, n, h, h, D), dtype=torch.uint8,
                     device="cuda")
    times = []
    for _ in range(2):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        gs.gs_attention_fwd(q, k, v, out, lse, ws, cu_q=cu, cu_k=cu, causal=True, scale=0.25)
        gs.gs_attention_bwd(q, k, v, out, lse, do, dq, dk, dv, ws, cu_q=cu, cu_k=cu, causal=True,
                            scale=0.25)
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    assert torch.equal(out, v) and torch.equal(dv, do)
    s = 0.25 * (q.double() * k.double()).sum(-1).t()
    m = 0.25 * (q.double() * k.double()).abs().sum(-1).t()
    assert ((lse - s).abs() <= D * U * m + 4 * U * (1 + s.abs()) + 2.0 ** -20).all()
    noise = 2.0 ** -12 * 2 * (do.double() * v.double()).abs().sum(-1, keepdim=True) * 0.25
    assert ((dq.double()).abs() <= noise * k.double().abs()).all()
    assert ((dk.double()).abs() <= noise * q.double().abs()).all()
    assert times[1] < 200.0, times


# ---------------------------------------------------------------------------
# what lies around the arrays
# ---------------------------------------------------------------------------
class Guarded:
    """A tensor inside a larger one of known bytes, with gaps between its rows where it has
    three dimensions; `intact` tells whether the call left them as they were."""

    def __init__(self, shape, dtype, gaps=True):
        torch = _torch()
        size = torch.empty((), dtype=dtype).element_size()
        self.shape, self.dtype, self.gaps = tuple(shape), dtype, gaps and len(shape) == 3
        full = self.shape
        if self.gaps:
            full = (full[0], full[1] + 1, full[2] + 16 // size)
        self.full, self.bytes = full, int(np.prod(full)) * size
        self.all = (torch.arange(self.bytes + 8192, device="cuda") * 37 % 251 + 1).to(torch.uint8)
        self.before = self.all.clone()
        self.t = self._view(self.all)

    def _view(self, raw):
        t = raw[4096:4096 + self.bytes].view(self.dtype).view(self.full)
        return t[:, :self.shape[1], :self.shape[2]] if self.gaps else t

    def rest(self):
        """the bytes around the tensor: as they are, and as they were"""
        after, before = self.all.clone(), self.before.clone()
        self._view(after).zero_()
        self._view(before).zero_()
        return after, before

    def intact(self):
        return _torch().equal(*self.rest())

    def kept(self, rows):
        """whether these rows of t are as before the call"""
        torch = _torch()
        return torch.equal(self.t[rows].contiguous().view(torch.uint8),
                           self._view(self.before)[rows].contiguous().view(torch.uint8))


def _guarded_attention(q, k, v, do, cu_q, cu_k, causal, scale):
    """({name: Guarded}) of both calls"""
    import differentiable_gaussian_splatting_gb300 as gs

    torch = _torch()
    (Tq, hq, D), (Tk, hk, _) = q.shape, k.shape
    bf = torch.bfloat16
    n = gs.gs_attention_workspace_bytes(Tq, Tk, len(cu_q) - 1, hq, hk, D)
    g = {"out": Guarded(q.shape, bf), "dq": Guarded(q.shape, bf), "dk": Guarded(k.shape, bf),
         "dv": Guarded(v.shape, bf), "lse": Guarded((hq, Tq), torch.float32),
         "ws": Guarded((n,), torch.uint8)}
    t = {name: x.t for name, x in g.items()}
    qkv = [_dev(x, "bf16") for x in (q, k, v)]
    cu = dict(cu_q=torch.tensor(cu_q, dtype=torch.int32, device="cuda"),
              cu_k=torch.tensor(cu_k, dtype=torch.int32, device="cuda"))
    gs.gs_attention_fwd(*qkv, t["out"], t["lse"], t["ws"], causal=causal, scale=scale, **cu)
    gs.gs_attention_bwd(*qkv, t["out"], t["lse"], _dev(do, "bf16"), t["dq"], t["dk"], t["dv"],
                        t["ws"], causal=causal, scale=scale, **cu)
    torch.cuda.synchronize()
    for name, x in g.items():
        assert x.intact(), name
    return g


@pytest.mark.parametrize("D", [40, 64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("cu_q,cu_k", [
    ([0, 60, 1000], [0, 70, 2 ** 31 - 1]),       # beyond the arrays: cut
    ([0, 0, 30, 150], [0, 40, 40, 90]),          # short of their end: the rest is left
    ([10, 150, 160], [30, 200, 300]),            # from behind their start
    ([-5, 64, 200], [-2 ** 31, 128, 256]),
    ([0] * 38 + [7, 200], [0] * 38 + [200, 333]),  # more than 32 sequences
    ([13] + [20] * 37 + [190], [5] + [9] * 37 + [290]),
])
def test_attention_touches_nothing_else(D, causal, cu_q, cu_k):
    Tq, Tk, hq, hk = 200, 333, 4, 2
    rng, q, k, v = _attention_inputs(Tq, Tk, hq, hk, D, seed=len(cu_q))
    do = ref.bf16(rng.normal(size=q.shape))
    scale = D ** -0.5
    g = _guarded_attention(q, k, v, do, cu_q, cu_k, causal, scale)
    cq, ck = np.clip(cu_q, 0, Tq), np.clip(cu_k, 0, Tk)
    torch = _torch()
    for names, c, T in ((("out", "dq"), cq, Tq), (("dk", "dv"), ck, Tk)):
        free = torch.tensor([i for i in range(T) if not c[0] <= i < c[-1]], device="cuda",
                            dtype=torch.long)
        for name in names:
            assert g[name].kept(free), name
    lse = g["lse"]
    free = [i for i in range(Tq) if not cq[0] <= i < cq[-1]]
    assert torch.equal(lse.t[:, free].view(torch.int32), lse._view(lse.before)[:, free].view(torch.int32))
    # and what the sequences hold is right
    q_rows, k_rows = slice(cq[0], cq[-1]), slice(ck[0], ck[-1])
    out, l, mag, smag = ref.attention(q, k, v, scale, causal, cq, ck)
    got = _np(g["out"].t)
    _close(got[q_rows], out[q_rows], ((2 * H + 2.0 ** -12) * mag)[q_rows], "out")
    got_l, l, smag = (x[:, q_rows] for x in (_np(lse.t), l, smag))
    fin = np.isfinite(l)
    assert np.array_equal(np.isneginf(got_l), ~fin)
    _close(got_l[fin], l[fin], (D * U * smag + 4 * U * (1 + np.abs(l)) + 2.0 ** -20)[fin], "lse")
    safe = np.zeros((hq, Tq))
    safe[:, q_rows] = got_l
    want = ref.attention_bwd(q, k, v, got, safe, do, scale, causal, cq, ck)
    for n, name, rows in (("q", "dq", q_rows), ("k", "dk", k_rows), ("v", "dv", k_rows)):
        w, b = want[n]
        _close(_np(g[name].t)[rows], w[rows], (b + H * np.abs(w) + 1e-30)[rows], name)


@pytest.mark.parametrize("D", [64, 128])
def test_attention_offsets_that_fall(D):
    # no sequence of the batch has a defined result where two of them overlap, but nothing
    # outside is touched, a negative length is none, and rows of one sequence alone are right
    T, h = 100, 2
    rng, q, k, v = _attention_inputs(T, T, h, h, D, seed=40)
    do = ref.bf16(rng.normal(size=q.shape))
    cu = [0, 60, 40, 1000]                      # 0..59, none, 40..99
    g = _guarded_attention(q, k, v, do, cu, cu, False, 0.125)
    got = _np(g["out"].t)
    for rows, keys in ((slice(0, 40), slice(0, 60)), (slice(60, 100), slice(40, 100))):
        want, _, mag, _ = ref.attention(q[rows], k[keys], v[keys], 0.125)
        _close(got[rows], want, (2 * H + 2.0 ** -12) * mag, "out")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,hq,hk,D,rot,inter", [(5, 3, 1, 40, 20, False), (33, 2, 2, 72, 36, False),
                                                 (129, 5, 3, 64, 48, True), (1, 1, 1, 8, 0, False),
                                                 (700, 16, 4, 128, 128, False)])
def test_head_norm_touches_nothing_else(T, hq, hk, D, rot, inter, dtype):
    import differentiable_gaussian_splatting_gb300 as gs

    torch = _torch()
    ty = torch.bfloat16 if dtype == "bf16" else torch.float32
    q, k, dq, dk = (torch.randn((T, h, D), device="cuda").to(ty) for h in (hq, hk, hq, hk))
    w = torch.randn(D, device="cuda")
    table = torch.randn((T, rot), device="cuda") if rot else None
    n = gs.gs_qk_norm_rope_workspace_bytes(T, hq, hk, D)
    g = {name: Guarded((T, h, D), ty) for name, h in (("qo", hq), ("ko", hk), ("gq", hq), ("gk", hk))}
    g |= {"dqw": Guarded((D,), torch.float32), "dkw": Guarded((D,), torch.float32),
          "ws": Guarded((n,), torch.uint8)}
    t = {name: x.t for name, x in g.items()}
    gs.gs_qk_norm_rope(q, k, w, w, table, None, t["qo"], t["ko"], interleaved=inter)
    gs.gs_qk_norm_rope_bwd(q, k, w, w, table, None, dq, dk, t["gq"], t["gk"], t["dqw"], t["dkw"],
                           t["ws"], interleaved=inter)
    for name, x in g.items():
        assert x.intact(), name
    plain = torch.empty_like(q), torch.empty_like(k)
    gs.gs_qk_norm_rope(q, k, w, w, table, None, *plain, interleaved=inter)
    assert torch.equal(plain[0], t["qo"]) and torch.equal(plain[1], t["ko"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 7, 8, 9, 2049, 4095])
def test_dropout_touches_nothing_else(n, dtype):
    import differentiable_gaussian_splatting_gb300 as gs

    torch = _torch()
    ty = torch.bfloat16 if dtype == "bf16" else torch.float32
    x, r = (torch.randn(n, device="cuda").to(ty) for _ in range(2))
    state = torch.tensor([5, 6], dtype=torch.int64, device="cuda")
    out, dx = Guarded((n,), ty), Guarded((n,), ty)
    gs.gs_dropout_add(x, r, out.t, state, 0.3)
    gs.gs_dropout_add_bwd(x, dx.t, state, 0.3)
    assert out.intact() and dx.intact()
    keep, _ = ref.kept(n, 5, 6, 0.3)
    assert np.array_equal(_np(dx.t) != 0, keep & (_np(x) != 0))


# ---------------------------------------------------------------------------
# long sequences: sampled rows of the outputs and of every gradient
# ---------------------------------------------------------------------------
def _sample(rng, n):
    edge = [0, 1, 63, 127, 128, n // 2, n - 129, n - 2, n - 1]
    return np.unique(np.concatenate([edge, rng.choice(n, 32, replace=False)]))


@pytest.mark.parametrize("n,m,hq,hk,D,causal", [
    (8160, 8160, 2, 1, 64, False), (8160, 8160, 2, 1, 64, True), (8160, 8160, 2, 1, 128, False),
    (8160, 8160, 2, 1, 128, True), (4346, 8160, 2, 2, 72, True), (16320, 16320, 1, 1, 128, False),
])
def test_attention_long_gradients(n, m, hq, hk, D, causal):
    # As test_gpu_tokens.py's bounds; the sums run over up to n rows here, in fp32: n u of their
    # terms' magnitudes besides.
    from test_gpu_tokens import _run_attention

    rng, q, k, v = _attention_inputs(n, m, hq, hk, D, seed=n + D)
    do = ref.bf16(rng.normal(size=q.shape))
    scale, E = D ** -0.5, 2.0 ** -12
    out, lse, (dq, dk, dv) = _run_attention(q, k, v, scale, causal, dout=do)
    out, lse, dq, dk, dv = (_np(x) for x in (out, lse, dq, dk, dv))
    q, k, v, do = (x.astype(np.float64) for x in (q, k, v, do))
    delta, delta_m = (do * out).sum(-1), np.abs(do * out).sum(-1)
    A = max(n, m) * U

    def parts(h, rows, keys):
        """p, dS and the bound of dS's error, of these queries and keys"""
        i, j = np.arange(n)[rows][:, None], np.arange(m)[keys][None]
        kk, vv = k[keys, h // (hq // hk)], v[keys, h // (hq // hk)]
        s = scale * q[rows, h] @ kk.T
        p = np.exp(s - lse[h, rows][:, None]) * ((j <= i + m - n) if causal else 1.0)
        ds = p * (do[rows, h] @ vv.T - delta[rows, h][:, None])
        err = (H + A) * np.abs(ds) + E * p * (np.abs(do[rows, h]) @ np.abs(vv).T +
                                              delta_m[rows, h][:, None])
        return p, ds, err

    rows, keys, every = _sample(rng, n), _sample(rng, m), slice(None)
    for h in range(hq):
        kk, vv = k[:, h // (hq // hk)], v[:, h // (hq // hk)]
        p, ds, err = parts(h, rows, every)
        w = scale * ds @ kk
        _close(dq[rows, h], w, scale * err @ np.abs(kk) + H * np.abs(w) + 1e-30, "dq")
        # the forward's rows: probabilities by its own lse
        s = scale * q[rows, h] @ kk.T
        if causal:
            s = np.where(np.arange(m)[None] <= rows[:, None] + m - n, s, -np.inf)
        top = s.max(-1, keepdims=True)
        e = np.exp(s - top)
        true_lse = (top + np.log(e.sum(-1, keepdims=True)))[:, 0]
        smag = scale * (np.abs(q[rows, h]) @ np.abs(kk).T).max(-1)
        _close(lse[h, rows], true_lse,
               D * U * smag + 4 * U * (1 + np.abs(true_lse)) + 2.0 ** -20, "lse")
        e /= e.sum(-1, keepdims=True)
        _close(out[rows, h], e @ vv, (2 * H + E + A) * (e @ np.abs(vv)), "out")
    for g in range(hk):
        wk = wv = bk = bv = 0.0
        for h in range(g * (hq // hk), (g + 1) * (hq // hk)):
            p, ds, err = parts(h, every, keys)
            wk, bk = wk + scale * ds.T @ q[:, h], bk + scale * err.T @ np.abs(q[:, h])
            wv, bv = wv + p.T @ do[:, h], bv + (H + E + A) * (p.T @ np.abs(do[:, h]))
        _close(dk[keys, g], wk, bk + H * np.abs(wk) + 1e-30, "dk")
        _close(dv[keys, g], wv, bv + H * np.abs(wv) + 1e-30, "dv")


@pytest.mark.parametrize("n,m,D,causal", [(300, 300, 64, True), (700, 520, 128, False),
                                          (1, 5000, 64, False)])
def test_attention_in_a_captured_graph(n, m, D, causal):
    # the chain of dependent launches replayed, on new inputs: the bits of the calls one by one
    import differentiable_gaussian_splatting_gb300 as gs

    torch = _torch()
    hq, hk = 4, 2
    new = lambda t, h: torch.empty((t, h, D), dtype=torch.bfloat16, device="cuda")
    q, k, v, do = new(n, hq), new(m, hk), new(m, hk), new(n, hq)
    out, dq, dk, dv = new(n, hq), new(n, hq), new(m, hk), new(m, hk)
    lse = torch.empty((hq, n), device="cuda")
    ws = torch.empty(gs.gs_attention_workspace_bytes(n, m, 1, hq, hk, D), dtype=torch.uint8,
                     device="cuda")

    def calls():
        gs.gs_attention_fwd(q, k, v, out, lse, ws, causal=causal)
        gs.gs_attention_bwd(q, k, v, out, lse, do, dq, dk, dv, ws, causal=causal)

    for t in (q, k, v, do):
        t.normal_()
    calls()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    for _ in range(3):
        for t in (q, k, v, do):
            t.normal_()
        results = []
        for run in (calls, g.replay):
            ws.fill_(255)
            for t in (out, lse, dq, dk, dv):
                t.fill_(float("nan"))
            run()
            results.append([t.clone() for t in (out, lse, dq, dk, dv)])
        assert all(torch.equal(a, b) for a, b in zip(*results))
        assert all(torch.isfinite(t).all() for t in results[0])
