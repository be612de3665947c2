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
