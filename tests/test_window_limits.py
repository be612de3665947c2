"""Window attention of more sequences and heads than its blocks can be found among in time: a CTA looks
through the tiles' places one after the other, about 1 us each, while its other warps wait with a bound of
two seconds.  Such calls are refused before anything is enqueued."""

import ctypes as C

import pytest

P = 0x100000  # an address that is never read


@pytest.fixture(scope="module")
def lib():
    from differentiable_gaussian_splatting_gb300 import build

    build.build()
    import differentiable_gaussian_splatting_gb300 as gs

    return gs.library()


@pytest.mark.parametrize("batch,heads", [(1 << 20, 64), ((1 << 20) - 1, 33), (1 << 17, 512), (40000, 1024)])
def test_places_beyond_the_limit_are_refused(lib, batch, heads):
    import differentiable_gaussian_splatting_gb300 as gs

    tokens = 8 * batch
    shape = C.byref(gs.AttentionShape(tokens, tokens, batch, heads, heads, 8, 0, 0.125))
    window = C.byref(gs.Window(5, 0, 4))
    h = C.byref(gs.Heads(P, 8 * heads, 8))
    assert lib.gs_attention_window_fwd(shape, window, h, h, h, P, P, h, P, P, 1 << 62, None) == 1
    assert lib.gs_attention_window_bwd(shape, window, h, h, h, P, P, h, P, h, h, h, h, P, 1 << 62,
                                       None) == 1
    # the sizes stay in range all the same
    assert lib.gs_attention_window_workspace_bytes(shape, window) > 0


def test_places_up_to_the_limit_are_not(lib):
    # (refused for their workspace alone, which is looked at last)
    import differentiable_gaussian_splatting_gb300 as gs

    window = C.byref(gs.Window(5, 0, 4))
    for batch, heads, tokens, forward_too in ((1 << 20, 32, 8 << 20, True), (1 << 15, 1024, 8 << 15, True),
                                              (1 << 20, 128, 1 << 20, False)):
        shape = C.byref(gs.AttentionShape(tokens, tokens, batch, heads, heads, 8, 0, 0.125))
        h = C.byref(gs.Heads(P, 8 * heads, 8))
        assert lib.gs_attention_window_fwd(shape, window, h, h, h, P, P, h, P, P, 0, None) == 5
        assert lib.gs_attention_window_bwd(shape, window, h, h, h, P, P, h, P, h, h, h, h, P, 0,
                                           None) == (5 if forward_too else 1)
