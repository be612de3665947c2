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
