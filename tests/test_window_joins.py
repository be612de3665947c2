"""The sinks' sums of window attention's gradient, which the blocks of a long sequence leave in the
workspace and the last one joins: the warps wait for each other with bounds, and a CTA joins many."""

import os
import re

import numpy as np
import pytest

from token_ref import H

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "differentiable_gaussian_splatting_gb300", "csrc")


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _body(text, head):
    """The braces' content behind the first place where `head` is found."""
    at = text.index("{", text.index(head))
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at + 1:i]
    raise AssertionError(head)


def test_no_barrier_of_the_hardware_between_warps_that_may_leave():
    # A warp leaves its loop where a wait has given up; those that then came to a barrier which counts
    # its threads would stay there for ever.  (This cannot be run: the sources are held to it.)  So the
    # roles' loops have bounded waits alone, and barriers of all threads stand before and behind them.
    counted = r"\bbar\.(sync|red|arrive)|\bbarrier\.(cta|sync|red)|__syncthreads"
    assert not re.search(counted, _source("gs_attention_window_dkv.cuh"))
    for file, setup, between in (("gs_attention_window_fwd.cu", 1, 0),
                                 ("gs_attention_window_dq.cuh", 1, 1)):
        text = _source(file)
        assert not re.search(counted.replace(r"|__syncthreads", ""), text)
        assert len(re.findall("__syncthreads", text)) == setup + between + 1
        # the loops of the roles lie between the branch on the warp and the last barrier
        roles = text[text.index("setmaxnreg.inc"):text.rindex("__syncthreads")]
        assert "__syncthreads" not in roles
    # what lies between the kinds of blocks is met by every warp, whatever its loop's end was: it
    # follows the first kind's part and stands under no condition but the warp's role
    text = _source("gs_attention_window_dq.cuh")
    for part in ("dkv_math<DP>(", "dkv_plan<DP>(", "dkv_bring<DP>(", "dkv_multiply<DP>("):
        after = text[text.index(part):text.index(part) + 420]
        assert re.match(r"[^;]*;\s*((__syncwarp\(\)|int [^;]*);\s*)*(const )?(bool \w+ = |if \()next_kind\(\)",
                        after), part
    # a join's own waits are bounded, and a warp whose wait gave up leaves the loop too
    join = _body(_source("gs_attention_window_dkv.cuh"), "bool join_sinks(")
    assert len(re.findall(r"if \(!mbar_wait\([^;]*dead\)\) return false;", join)) == 2
    assert re.search(r"!join_sinks<DP>\([^;]*\)\) break;",
                     _source("gs_attention_window_dkv.cuh"))


@pytest.mark.gpu
@pytest.mark.parametrize("lens,sinks", [([8192], 16), ([2500, 40, 4700, 300], 128), ([256, 257, 8000], 3)])
def test_ctas_that_join_many_blocks(lens, sinks):
    # A window of the query's own key alone: blocks of the sinks take 256 queries, 480 of them and more
    # for 152 CTAs.  Against the definition in 64 bits over the pairs seen, with the bounds of
    # tests/block_ref.py; three runs alike.
    import torch

    import differentiable_gaussian_splatting_gb300 as gs

    T, heads, D, scale = sum(lens), 16, 8, 8 ** -0.5
    torch.manual_seed(sinks)
    q, k, v, do = (torch.randn((T, heads, D), device="cuda").bfloat16() for _ in range(4))
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((heads, T), device="cuda")
    size = gs.gs_attention_window_workspace_bytes(T, T, len(lens), heads, heads, D, 0, 0, sinks)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    kw = dict(cu_q=cu, cu_k=cu, causal=True, scale=scale)
    gs.gs_attention_window_fwd(q, k, v, out, lse, ws, 0, 0, sinks, **kw)
    runs = []
    for _ in range(3):
        ws.fill_(255)
        g = [torch.full_like(t, float("nan")) for t in (q, k, v)]
        gs.gs_attention_window_bwd(q, k, v, out, lse, do, *g, ws, 0, 0, sinks, **kw)
        runs.append(g)
    gs.gs_attention_status()
    assert all(torch.equal(a, b) for g in runs[1:] for a, b in zip(runs[0], g))
    E = 2.0 ** -12
    ends = np.concatenate([[0], np.cumsum(lens)])
    for a, b in zip(ends[:-1], ends[1:]):
        n = b - a
        qq, kk, vv, dd, oo = (t[a:b].double() for t in (q, k, v, do, out))
        keys = torch.arange(n, device="cuda")
        # columns: the sinks, then the query's own key where it is none of them
        at = torch.cat([torch.arange(min(sinks, n), device="cuda").expand(n, -1), keys[:, None]], 1)
        seen = at <= keys[:, None]
        seen[:, -1] &= keys >= sinks
        s = scale * torch.einsum("nhd,njhd->nhj", qq, kk[at])
        p = torch.exp(s - lse[:, a:b].t().double()[..., None]) * seen[:, None]
        delta, size = (oo * dd).sum(-1, keepdim=True), (oo * dd).abs().sum(-1, keepdim=True)
        ds = p * (torch.einsum("nhd,njhd->nhj", dd, vv[at]) - delta)
        err = H * ds.abs() + E * p * (torch.einsum("nhd,njhd->nhj", dd.abs(), vv[at].abs()) + size)

        def keys_of(w, x):  # sum over queries, by key
            t = torch.zeros((n, heads, D), dtype=torch.float64, device="cuda")
            return t.index_add_(0, at.reshape(-1), (w[..., None] * x[:, :, None]).transpose(1, 2)
                                .reshape(-1, heads, D))

        want = [(scale * torch.einsum("nhj,njhd->nhd", ds, kk[at]),
                 scale * torch.einsum("nhj,njhd->nhd", err, kk[at].abs())),
                (scale * keys_of(ds, qq), scale * keys_of(err, qq.abs())),
                (keys_of(p, dd), (H + E) * keys_of(p, dd.abs()))]
        for name, got, (w, bound) in zip("qkv", runs[0], want):
            off = (got[a:b].double() - w).abs() - (bound + H * w.abs() + 1e-30)
            assert bool((off <= 0).all()), (name, a, off.max().item())
