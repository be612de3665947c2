"""The operators of a block run together, as a training step calls them: norms around the blocks with
gate and residual, packed projection, head norms with rotation, window attention, and back, then the
clipping of all gradients.  Against plain fp32 torch, replayed from a captured graph, and on two
streams at once."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

T_LENS = [300, 0, 77, 130]
C, HQ, HK, D = 192, 6, 2, 32
LEFT, SINKS = 50, 4


class Step:
    """Inputs, parameters and buffers of one step, and the step itself."""

    def __init__(self, seed=0):
        import torch

        import differentiable_gaussian_splatting_gb300 as gs

        self.gs, self.torch = gs, torch
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        n = lambda *s, std=1.0: torch.randn(s, generator=g, device="cuda") * std
        T = self.T = sum(T_LENS)
        bf = torch.bfloat16
        self.x, self.y = n(T, C).to(bf), n(T, C, std=0.7).to(bf)
        self.dr, self.dh = n(T, C, std=0.1).to(bf), n(T, C, std=0.1).to(bf)
        self.p = dict(post=1 + n(C, std=0.1), pre=1 + n(C, std=0.1), gate=n(len(T_LENS), C, std=0.5),
                      qkv=(n((HQ + 2 * HK) * D, C) * C ** -0.5).to(bf),
                      qw=1 + n(D, std=0.1), kw=1 + n(D, std=0.1),
                      proj=(n(C, HQ * D) * (HQ * D) ** -0.5).to(bf),
                      norm=1 + n(C, std=0.1), bias=n(C, std=0.1))
        cu = np.concatenate([[0], np.cumsum(T_LENS)])
        self.cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        # a token's place in its sequence; the first ones are registers without a place
        self.pos = torch.cat([torch.arange(k, device="cuda") - SINKS for k in T_LENS]).int()
        angle = torch.arange(400, device="cuda")[:, None] * 100.0 ** (
            -torch.arange(D // 2, device="cuda") / (D // 2))
        self.table = torch.cat([angle.cos(), angle.sin()], 1).contiguous()
        e = lambda *s, dtype=bf: torch.empty(s, dtype=dtype, device="cuda")
        f = torch.float32
        ws = lambda b: torch.empty(b, dtype=torch.uint8, device="cuda")
        self.r1, self.h1, self.r2, self.h2 = (e(T, C) for _ in range(4))
        self.qn, self.kn, self.o = e(T, HQ, D), e(T, HK, D), e(T, HQ, D)
        self.lse = e(HQ, T, dtype=f)
        self.ws_a = ws(gs.gs_attention_window_workspace_bytes(T, T, len(T_LENS), HQ, HK, D, LEFT, 0,
                                                              SINKS))
        self.ws_n = ws(gs.gs_residual_norm_workspace_bytes(T, C, len(T_LENS)))
        self.ws_h = ws(gs.gs_qk_norm_rope_workspace_bytes(T, HQ, HK, D))
        self.g = {k: e(*v.shape, dtype=f) for k, v in self.p.items() if v.dtype == f}
        self.dx, self.dy, self.dr1, self.dy2 = (e(T, C) for _ in range(4))
        self.dqn, self.dkn, self.dqkv = e(T, HQ, D), e(T, HK, D), e(T, HQ + 2 * HK, D)
        self.norm = e(1, dtype=f)
        self.ws_c = ws(gs.gs_clip_grad_norm_workspace_bytes(16))

    def run(self, max_norm=float("inf")):
        """(outputs and gradients by name)"""
        gs, torch, p, T = self.gs, self.torch, self.p, self.T
        first = dict(pre_weight=p["pre"], post_weight=p["post"], gate=p["gate"], cu=self.cu,
                     pre="rms", post="rms")
        second = dict(pre_weight=p["norm"], pre_bias=p["bias"], pre="layer", beta=0.5)
        gs.gs_residual_norm(self.x, self.y, self.r1, self.h1, **first)
        qkv = (self.h1 @ p["qkv"].t()).view(T, -1, D)
        q, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + HK], qkv[:, HQ + HK:]
        gs.gs_qk_norm_rope(q, k, p["qw"], p["kw"], self.table, self.pos, self.qn, self.kn)
        att = dict(cu_q=self.cu, cu_k=self.cu, causal=True)
        gs.gs_attention_window_fwd(self.qn, self.kn, v, self.o, self.lse, self.ws_a, LEFT, 0, SINKS,
                                   **att)
        y2 = self.o.view(T, -1) @ p["proj"].t()
        gs.gs_residual_norm(self.r1, y2, self.r2, self.h2, **second)
        # and back
        g = self.g
        gs.gs_residual_norm_bwd(self.r1, y2, self.dr, self.dh, self.dr1, self.dy2, self.ws_n, **second,
                                dpre_weight=g["norm"], dpre_bias=g["bias"])
        d_proj = self.dy2.t() @ self.o.view(T, -1)
        do = (self.dy2 @ p["proj"]).view(T, HQ, D)
        gs.gs_attention_window_bwd(self.qn, self.kn, v, self.o, self.lse, do, self.dqn, self.dkn,
                                   self.dqkv[:, HQ + HK:], self.ws_a, LEFT, 0, SINKS, **att)
        gs.gs_qk_norm_rope_bwd(q, k, p["qw"], p["kw"], self.table, self.pos, self.dqn, self.dkn,
                               self.dqkv[:, :HQ], self.dqkv[:, HQ:HQ + HK], g["qw"], g["kw"], self.ws_h)
        flat = self.dqkv.view(T, -1)
        d_qkv, dh1 = flat.t() @ self.h1, flat @ p["qkv"]
        gs.gs_residual_norm_bwd(self.x, self.y, self.dr1, dh1, self.dx, self.dy, self.ws_n, **first,
                                dpre_weight=g["pre"], dpost_weight=g["post"], dgate=g["gate"])
        grads = {**g, "proj": d_proj, "qkv": d_qkv}
        gs.gs_clip_grad_norm(list(grads.values()), max_norm, self.norm, self.ws_c)
        return {"r": self.r2, "h": self.h2, "dx": self.dx, "dy": self.dy, "total": self.norm,
                **{"d" + n: t for n, t in grads.items()}}

    def plain(self):
        """The same in fp32 torch, through autograd."""
        torch = self.torch
        p = {k: v.detach().float().requires_grad_() for k, v in self.p.items()}
        x, y = self.x.float().requires_grad_(), self.y.float().requires_grad_()
        rms = lambda v: v * torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-6)
        gate = torch.repeat_interleave(p["gate"], self.cu[1:] - self.cu[:-1], dim=0)
        r1 = x + gate * (rms(y) * p["post"])
        qkv = (rms(r1) * p["pre"] @ p["qkv"].t()).view(self.T, -1, D)
        placed = (self.pos >= 0)[:, None, None]
        row = self.table[self.pos.clamp_min(0).long()][:, None]
        c, s = row[..., :D // 2], row[..., D // 2:]

        def side(v, w):
            v = rms(v) * w
            a, b = v[..., :D // 2], v[..., D // 2:]
            return torch.where(placed, torch.cat([a * c - b * s, b * c + a * s], -1), v)

        q = side(qkv[:, :HQ], p["qw"])
        k = side(qkv[:, HQ:HQ + HK], p["kw"]).repeat_interleave(HQ // HK, 1)
        v = qkv[:, HQ + HK:].repeat_interleave(HQ // HK, 1)
        outs = []
        for a, b in zip(self.cu.tolist(), self.cu.tolist()[1:]):
            i, j = torch.arange(b - a, device="cuda")[:, None], torch.arange(b - a, device="cuda")
            seen = ((j >= i - LEFT) | (j < SINKS)) & (j <= i)
            w = torch.einsum("ihd,jhd->hij", q[a:b], k[a:b]) * D ** -0.5
            outs.append(torch.einsum("hij,jhd->ihd",
                                     torch.softmax(w.masked_fill(~seen, -torch.inf), -1), v[a:b]))
        y2 = torch.cat(outs).reshape(self.T, -1) @ p["proj"].t()
        r2 = r1 + 0.5 * y2
        h = torch.nn.functional.layer_norm(r2, (C,), p["norm"], p["bias"], 1e-6)
        torch.autograd.backward([r2, h], [self.dr.float(), self.dh.float()])
        grads = {n: t.grad for n, t in p.items()}
        total = torch.sqrt(sum(t.double().square().sum() for t in grads.values()))
        return {"r": r2, "h": h, "dx": x.grad, "dy": y.grad, "total": total.view(1),
                **{"d" + n: t for n, t in grads.items()}}


def test_step_against_plain_torch():
    step = Step()
    got, want = step.run(), step.plain()
    # bfloat16 holds h, the projections, their heads, P, the outputs and as much on the way back: a
    # dozen roundings of at most 2^-8, by norms
    for n, w in want.items():
        a, b = got[n].float(), w.detach().float()
        assert ((a - b).norm() / b.norm()).item() < 12 * 2.0 ** -8, n
    assert (got["dgate"][1] == 0).all()  # the empty sequence's
    # clipped to a tenth: every gradient by the same factor
    total, before = got["total"].item(), {n: got[n].clone() for n in got if n.startswith("d")}
    got = step.run(max_norm=total / 10)
    for n in before:
        if n in ("dx", "dy"):
            continue  # not among the parameters'
        a, b = got[n].float(), before[n].float() * 0.1
        assert ((a - b).norm() / b.norm()).item() < 2.0 ** -8 + 1e-6, n
    step.gs.gs_attention_status()


def test_step_replayed_from_a_graph():
    import torch

    step = Step(1)
    want = {n: t.clone() for n, t in step.run(0.5).items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step.run(0.5)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step.run(0.5)
    for t in got.values():
        t.fill_(float("nan"))
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        for n, t in got.items():
            assert torch.equal(t, want[n]), n
    # other inputs in the same places
    other = Step(2)
    want = {n: t.clone() for n, t in other.run(0.5).items()}
    for n in ("x", "y", "dr", "dh"):
        getattr(step, n).copy_(getattr(other, n))
    for n, t in step.p.items():
        t.copy_(other.p[n])
    graph.replay()
    torch.cuda.synchronize()
    for n, t in got.items():
        assert torch.equal(t, want[n]), n


def test_steps_on_two_streams_at_once():
    import torch

    steps = [Step(3), Step(4)]
    want = [{n: t.clone() for n, t in s.run(0.5).items()} for s in steps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(5):
        got = []
        for s, stream in zip(steps, streams):
            with torch.cuda.stream(stream):
                got.append(s.run(0.5))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            for n, t in g.items():
                assert torch.equal(t, w[n]), n


def _example():
    import importlib.util
    import os

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location(
        "predict_gaussians", os.path.join(root, "examples", "predict_gaussians.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("options", [dict(window=5), dict(clip=0.05), dict(norms=True),
                                     dict(window=9, clip=0.05, norms=True)])
def test_example_runs_with(options):
    losses = _example().train(steps=3, size=96, seed=1, **options)
    assert len(losses) == 3 and np.isfinite(losses).all()


def test_example_gradients_of_residual_norm():
    import torch

    ex = _example()
    torch.manual_seed(5)
    x, y = (torch.randn(77, 96, device="cuda").bfloat16() for _ in range(2))
    w, b = 1 + 0.1 * torch.randn(96, device="cuda"), 0.1 * torch.randn(96, device="cuda")
    dr, dh = (torch.randn(77, 96, device="cuda").bfloat16() for _ in range(2))
    for second in (y, None):
        ours = [t if t is None else t.clone().requires_grad_() for t in (x, second, w, b)]
        out = ex.ResidualNorm.apply(*ours, 1e-5)
        torch.autograd.backward(list(out), [dr, dh])
        plain = [t if t is None else t.clone().float().requires_grad_() for t in (x, second, w, b)]
        r = plain[0] if second is None else plain[0] + plain[1]
        h = torch.nn.functional.layer_norm(r, (96,), plain[2], plain[3], 1e-5)
        torch.autograd.backward([r, h], [dr.float(), dh.float()])
        # outputs and gradients are rounded to bfloat16 once: at most 2^-8, by norms (and without y
        # the stream's gradient is joined by autograd: twice)
        for a, c in ((out[0], r), (out[1], h),
                     *((p.grad, q.grad) for p, q in zip(ours, plain) if p is not None)):
            a, c = a.detach().float(), c.detach()
            assert ((a - c).norm() / c.norm()).item() < 2 * 2.0 ** -8
