"""Window attention where seen keys and values are infinite: what no query's mask hides may be, and the
result is the definition's.  A key is seen by all queries of its sequence here; scores are moderate, so
that its probability is no zero."""

import numpy as np
import pytest

from test_gpu_window import _inputs, _run
from token_ref import H

pytestmark = pytest.mark.gpu

# one query a sequence (the kernel of few queries) whose keys end inside a step of 16, inside a warp's
# second step and at a step's end; with shared and unshared heads; and many queries, by tiles
LENS = [1, 2, 9, 15, 16, 17, 31, 32, 33, 127, 128, 129, 255, 300, 1000, 1601]


def _check(q, k, v, window, causal, lens_q, lens_k, bad):
    """bad: (key, key head, column, value) of v that all queries of the key's sequence see"""
    import torch

    clean = _run(q, k, v, 0.125, window, causal, lens_q, lens_k)
    dirty = v.copy()
    for key, head, column, value in bad:
        dirty[key, head, column] = value
    out, lse = _run(q, k, dirty, 0.125, window, causal, lens_q, lens_k)
    want = clean[0].clone()
    ends_q = np.concatenate([[0], np.cumsum(lens_q)])
    ends_k = np.concatenate([[0], np.cumsum(lens_k)])
    group = q.shape[1] // k.shape[1]
    for key, head, column, value in bad:
        b = int(np.searchsorted(ends_k, key, side="right")) - 1
        want[ends_q[b]:ends_q[b + 1], head * group:(head + 1) * group, column] = value
    assert torch.equal(out, want)
    assert torch.equal(lse, clean[1])


@pytest.mark.parametrize("hq,hk,D", [(8, 2, 128), (2, 2, 64), (12, 1, 40)])
@pytest.mark.parametrize("value", [np.inf, -np.inf])
def test_infinite_values_of_last_keys(hq, hk, D, value):
    lens_q, lens_k = [1] * len(LENS), LENS
    rng, q, k, v = _inputs(len(LENS), sum(LENS), hq, hk, D, seed=D)
    last = np.cumsum(LENS) - 1
    bad = [(int(i), int(rng.integers(hk)), int(rng.integers(D)), value) for i in last]
    _check(q, k, v, (2000, 0, 0), True, lens_q, lens_k, bad)
    _check(q, k, v, (2000, 5, 4), False, lens_q, lens_k, bad)


@pytest.mark.parametrize("hq,hk,D", [(8, 2, 128), (2, 2, 64)])
def test_infinite_values_of_last_sinks(hq, hk, D):
    # the window holds the query's own key alone, the sinks' last one lies inside a step
    lens_q, lens_k = [1, 1, 1], [300, 40, 700]
    rng, q, k, v = _inputs(3, 1040, hq, hk, D, seed=D)
    for sinks in (1, 4, 15, 16, 17, 100):
        bad = [(a + min(sinks, n) - 1, hk - 1, 3, np.inf) for a, n in ((0, 300), (300, 40), (340, 700))]
        _check(q, k, v, (0, 0, sinks), True, lens_q, lens_k, bad)


@pytest.mark.parametrize("hq,hk,D", [(8, 2, 128), (2, 2, 64)])
def test_infinite_values_by_tiles(hq, hk, D):
    lens_q, lens_k = [40, 200], [150, 300]
    rng, q, k, v = _inputs(240, 450, hq, hk, D, seed=D)
    bad = [(149, 0, 3, np.inf), (449, hk - 1, D - 1, -np.inf), (150, 0, 0, np.inf)]
    _check(q, k, v, (400, 400, 0), False, lens_q, lens_k, bad)
