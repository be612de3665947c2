"""Residual norms of several widths at once: from threads of the host, whose calls meet in one kernel's
state, and in one captured graph.  What a call answers does not depend on the others: the same bits."""

import threading

import pytest

pytestmark = pytest.mark.gpu

# widths that one instance of the forward or of the gradient serves, in bfloat16
FORWARD, GRADIENT = (1032, 2048, 4096, 8192), (72, 256, 1032, 4096)


def _calls(width, tokens=6):
    """(forward, gradient): each makes its call on the current stream and returns its outputs"""
    import torch

    import differentiable_gaussian_splatting_gb300 as gs

    torch.manual_seed(width)
    x, y, dr, dh = (torch.randn((tokens, width), device="cuda").bfloat16() for _ in range(4))
    w, q = (1 + 0.1 * torch.randn(width, device="cuda") for _ in range(2))
    r, h, dx, dy = (torch.empty_like(x) for _ in range(4))
    dw, dq = torch.empty_like(w), torch.empty_like(q)
    ws = torch.empty(gs.gs_residual_norm_workspace_bytes(tokens, width), dtype=torch.uint8, device="cuda")
    kw = dict(pre_weight=w, post_weight=q, post="rms")

    def forward():
        gs.gs_residual_norm(x, y, r, h, **kw)
        return r, h

    def gradient():
        gs.gs_residual_norm_bwd(x, y, dr, dh, dx, dy, ws, dpre_weight=dw, dpost_weight=dq, **kw)
        return dx, dy, dw, dq

    return forward, gradient


@pytest.mark.parametrize("of,widths", [(0, FORWARD), (1, GRADIENT)])
def test_norms_of_several_widths_from_several_threads(of, widths):
    import torch

    calls = [_calls(w)[of] for w in widths]
    want = [[t.clone() for t in call()] for call in calls]
    torch.cuda.synchronize()
    start, wrong = threading.Barrier(len(calls)), []

    def work(n):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                start.wait(60)
                for _ in range(3000):
                    got = calls[n]()
                if not all(torch.equal(a, b) for a, b in zip(got, want[n])):
                    wrong.append((widths[n], "other bits"))
        except Exception as e:  # noqa: BLE001
            wrong.append((widths[n], repr(e)))

    threads = [threading.Thread(target=work, args=(n,)) for n in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong


@pytest.mark.parametrize("of,widths", [(0, FORWARD), (1, GRADIENT)])
def test_norms_of_several_widths_in_one_graph(of, widths):
    # a wide call, then narrower ones: captured, called without the graph in between, replayed
    import torch

    calls = [_calls(w)[of] for w in sorted(widths, reverse=True)]
    want = [[t.clone() for t in call()] for call in calls]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [call() for call in calls]
    calls[-1]()
    for _ in range(2):
        for o in outs:
            for t in o:
                t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for o, w in zip(outs, want) for a, b in zip(o, w))
