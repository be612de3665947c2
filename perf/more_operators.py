"""More operators of a network that predicts Gaussians, as cases to time and to compare: what one
training step of a deep stack over large views calls beside the token operators.

A view is read as tokens, one for each 16 x 16 tile (64 tokens for the 128 x 128 view of the
synthetic configurations, 2,500 for 800 x 800, 4,346 for 1297 x 840, 8,160 for 1920 x 1080, 32,400
for 3840 x 2160), behind a few register tokens without a place.  The operators:

  window_attention  softmax attention over the tokens near a query and the first few (sinks), over
                    ragged batches with shared heads, for prompts, single tokens and training
  residual_norm     residual + gate x norm of a block's output, and the norm before the next
                    block, and their gradient
  clip_grad_norm    the norm over all gradients of a step, and their clipping

`run` computes them in plain 32-bit torch operations, or, where `own` is true, through this
repository's package.
"""

from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

PACKAGE = "differentiable_gaussian_splatting_gb300"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6

# the costliest cases that draw() may give: padded (query, key) cells over all heads, for the plain
# form's matrices, padded key tokens x heads of single queries, and values of what passes over memory
MOST_CELLS_FWD = 16320 * 16320 * 16
MOST_CELLS_BWD = 8160 * 8160 * 16
MOST_KEYS = 32 * 32400 * 4
MOST_VALUES = 32400 * 1024
MOST_GRADIENTS = 1500000 * 59


def _attn(name, direction, lens_q, lens_k, hq, hk, dim, left, right, sinks, causal):
    return {"name": name, "op": "window_attention", "dir": direction,
            "lens_q": " ".join(map(str, lens_q)), "lens_k": " ".join(map(str, lens_k)), "hq": hq,
            "hk": hk, "dim": dim, "left": left, "right": right, "sinks": sinks, "causal": causal,
            "dtype": "bf16"}


def _norm(name, direction, tokens, width, pre, post, gate, lens, bias, alpha, beta, dtype):
    return {"name": name, "op": "residual_norm", "dir": direction, "tokens": tokens, "width": width,
            "pre": pre, "post": post, "gate": gate, "lens": " ".join(map(str, lens)), "bias": bias,
            "alpha": alpha, "beta": beta, "dtype": dtype}


def _clip(name, sizes, ratio, dtype):
    """sizes: the tensors' elements, "KxN" for K tensors of N; ratio: their norm over the largest
    that is left as it is"""
    return {"name": name, "op": "clip_grad_norm", "dir": "", "sizes": sizes, "ratio": ratio,
            "dtype": dtype}


def _decode_lens():
    """32 views whose tiles are predicted one after the other, each at another tile"""
    return [32400 - 1013 * i for i in range(31)] + [1]


def _network(width, blocks):
    """The gradients of a network of the example's kind."""
    block = (f"{width * 2 * width} {width * width} 2x{4 * width * width} {4 * width} "
             f"{width} 2x64 4x{width}")
    return " ".join([f"{768 * width} {width}"] + [block] * blocks +
                    [f"2x{width} {112 * width} 112"])


def listed():
    return [
        # a 3840 x 2160 view is too long for all pairs: two 1920 x 1080 views, each tile sees the
        # 1,024 before it (8.5 rows of tiles) and four register tokens, grouped heads
        _attn("win-fwd-16320", "fwd", [16320], [16320], 16, 4, 128, 1023, 0, 4, True),
        # views of several sizes, an empty one and a lone token among them, both sides seen
        _attn("win-fwd-ragged", "fwd", [4346, 2500, 64, 1, 0, 1039], [4346, 2500, 64, 1, 0, 1039],
              8, 8, 64, 256, 256, 4, False),
        # the next tile of 32 views at once, the tiles before it as keys and values
        _attn("win-fwd-tokens", "fwd", [1] * 32, _decode_lens(), 16, 4, 128, 2047, 0, 4, True),
        # training on a 1920 x 1080 view, grouped heads
        _attn("win-bwd-8160", "bwd", [8160], [8160], 16, 4, 128, 1023, 0, 4, True),
        # a training batch of small and middling views, both sides seen
        _attn("win-bwd-ragged", "bwd", [2500, 64, 1, 0, 1039], [2500, 64, 1, 0, 1039], 8, 8, 64,
              256, 256, 16, False),
        # one 128 x 128 view at inference in the example's width: the call's latency
        _norm("norm-fwd-64", "fwd", 64, 256, "layer", "none", False, [], True, 1.0, 1.0, "bf16"),
        # views of several sizes, a gate for each, norms on both sides of the block
        _norm("norm-fwd-32400", "fwd", 32400, 1024, "rms", "rms", True,
              [16320, 8160, 4346, 2500, 0, 1039, 35], False, 1.0, 1.0, "bf16"),
        # training on the same
        _norm("norm-bwd-32400", "bwd", 32400, 1024, "rms", "rms", True,
              [16320, 8160, 4346, 2500, 0, 1039, 35], False, 1.0, 1.0, "bf16"),
        # training in fp32, an odd width, one scaled gate for all tokens
        _norm("norm-bwd-4346-f32", "bwd", 4346, 515, "layer", "layer", True, [], True, 1.25, 0.5,
              "f32"),
        # the example's network: few and small gradients, the calls' latency
        _clip("clip-network", _network(256, 3), 4.0, "f32"),
        # a wide and deep one of the kind in bfloat16
        _clip("clip-network-wide", _network(1024, 12), 2.0, "bf16"),
        # the parameters of 1.5M Gaussians with spherical harmonics of degree 3
        _clip("clip-scene-1.5M", "2x4500000 6000000 1500000 72000000", 3.0, "f32"),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _draw_attn(rng):
    direction = rng.choice(["fwd", "fwd", "bwd"])
    dim = rng.choice([16, 40, 64, 64, 72, 96, 128, 128])
    hk = rng.choice([1, 2, 3, 4, 8])
    hq = hk * rng.choice([1, 2, 3, 4])
    causal = rng.random() < 0.5
    left = _log_uniform(rng, 1, 4096) - 1
    right = 0 if causal else rng.choice([left, _log_uniform(rng, 1, 2048) - 1])
    sinks = rng.choice([0, 1, 4, 4, 16, 128])
    if direction == "fwd" and rng.random() < 0.4:  # single tokens
        batch = _log_uniform(rng, 1, 64)
        most = min(32400, MOST_KEYS // (batch * hk))
        lens_q, lens_k = [1] * batch, [_log_uniform(rng, 1, most) for _ in range(batch)]
        if batch > 2:
            i = rng.randrange(batch)
            lens_q[i], lens_k[i] = rng.choice([(0, 0), (1, 0), (0, 9)])
    else:
        batch = rng.choice([1, 1, 2, 3, 5])
        cells = (MOST_CELLS_FWD if direction == "fwd" else MOST_CELLS_BWD) / (hq * batch)
        most = min(8160, int(math.sqrt(cells)))
        lens_k = [_log_uniform(rng, 1, most) for _ in range(batch)]
        if rng.random() < 0.25:  # other numbers of queries than of keys, shorter or longer
            lens_q = [_log_uniform(rng, 1, most) for _ in range(batch)]
        else:
            lens_q = list(lens_k)
        if batch > 2:  # an empty view among them
            i = rng.randrange(1, batch)
            lens_q[i], lens_k[i] = rng.choice([(0, 0), (7, 0), (0, 9)])
    return _attn("", direction, lens_q, lens_k, hq, hk, dim, left, right, sinks, causal)


def _draw_norm(rng):
    width = _log_uniform(rng, 8, 2048)
    if rng.random() < 0.5:
        width = (width + 7) // 8 * 8
    dtype = rng.choice(["bf16", "f32"])
    tokens = _log_uniform(rng, 1, min(32400, MOST_VALUES // (width * (1 if dtype == "bf16" else 2))))
    lens = []
    gate = rng.random() < 0.7
    if gate and rng.random() < 0.6:
        cuts = sorted(rng.randint(0, tokens) for _ in range(rng.randint(0, 8)))
        lens = [b - a for a, b in zip([0] + cuts, cuts + [tokens])]
    return _norm("", rng.choice(["fwd", "bwd"]), tokens, width, rng.choice(["rms", "layer"]),
                 rng.choice(["none", "rms", "layer"]), gate, lens, rng.random() < 0.5,
                 rng.choice([1.0, 1.25, 2.0]), rng.choice([1.0, 0.5, 0.1]), dtype)


def _draw_clip(rng):
    left = _log_uniform(rng, 1000, MOST_GRADIENTS)
    sizes = []
    while left and len(sizes) < rng.choice([5, 40, 400]):
        n = min(left, _log_uniform(rng, 1, left))
        sizes.append(n)
        left -= n
    return _clip("", " ".join(map(str, sizes)), rng.choice([0.5, 1.5, 4.0, 100.0]),
                 rng.choice(["bf16", "f32"]))


def draw(rng):
    case = rng.choice([_draw_attn, _draw_attn, _draw_norm, _draw_clip])(rng)
    del case["name"]
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _lens(text):
    return [int(n) for n in text.split()]


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _offsets(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def _prepare_attn(case, seed):
    g = _generator(seed)
    lens_q, lens_k = _lens(case["lens_q"]), _lens(case["lens_k"])
    Tq, Tk, hq, hk, D = sum(lens_q), sum(lens_k), case["hq"], case["hk"], case["dim"]
    dtype = DTYPES[case["dtype"]]

    def heads(T, h):  # normed heads: every vector has root mean square 1
        x = torch.randn((T, h, D), generator=g, device="cuda")
        return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)).to(dtype)

    s = {"case": case, "q": heads(Tq, hq), "k": heads(Tk, hk), "v": _normal(g, (Tk, hk, D), dtype),
         "lens_q": lens_q, "lens_k": lens_k, "cu_q": _offsets(lens_q), "cu_k": _offsets(lens_k),
         "scale": D ** -0.5, "out": torch.empty((Tq, hq, D), dtype=dtype, device="cuda"),
         "lse": torch.empty((hq, Tq), device="cuda")}
    if case["dir"] == "bwd":
        # what the forward left, and the gradient that came back
        s["out"], s["lse"] = _plain_attention(s)
        s["dout"] = _normal(g, (Tq, hq, D), dtype)
        s["dq"], s["dk"], s["dv"] = (torch.empty_like(s[n]) for n in ("q", "k", "v"))
    return s


def _prepare_norm(case, seed):
    g = _generator(seed)
    T, C, dtype = case["tokens"], case["width"], DTYPES[case["dtype"]]
    lens = _lens(case["lens"]) or [T]
    f = torch.float32

    def vector(on, mean):
        return mean + 0.1 * _normal(g, (C,), f) if on else None

    post, bias = case["post"] != "none", case["bias"]
    s = {"case": case, "lens": lens, "cu": _offsets(lens) if case["lens"] else None,
         # a stream with a mean of its own in every channel, a block's output
         "x": (_normal(g, (T, C), f, 2.0) + _normal(g, (C,), f, 0.5)).to(dtype),
         "y": _normal(g, (T, C), dtype, 0.7),
         "pre_weight": vector(True, 1.0), "pre_bias": vector(bias, 0.0),
         "post_weight": vector(post, 1.0), "post_bias": vector(post and bias, 0.0),
         "gate": _normal(g, (len(lens), C), f, 0.5) if case["gate"] else None}
    if case["dir"] == "fwd":
        s["r"], s["h"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
        return s
    s["dr"], s["dh"] = _normal(g, (T, C), dtype, 0.1), _normal(g, (T, C), dtype, 0.1)
    s["dx"], s["dy"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
    for n in ("pre_weight", "pre_bias", "post_weight", "post_bias", "gate"):
        s["d" + n] = None if s[n] is None else torch.empty_like(s[n])
    return s


def _sizes(text):
    sizes = []
    for word in text.split():
        k, n = word.split("x") if "x" in word else (1, word)
        sizes += [int(n)] * int(k)
    return sizes


def _prepare_clip(case, seed):
    g, host = _generator(seed), random.Random(seed)
    dtype, sizes = DTYPES[case["dtype"]], _sizes(case["sizes"])
    # every parameter's gradient at its own scale; a part of a scene is out of sight: zeros
    scales = [10.0 ** host.uniform(-4.0, 0.0) for _ in sizes]
    grads = []
    for n, scale in zip(sizes, scales):
        x = torch.randn(n, generator=g, device="cuda")
        if n > 1000000:
            x[n // 3:n // 2] = 0.0
        grads.append(x.mul_(scale).to(dtype))
    expected = math.sqrt(sum(n * s * s for n, s in zip(sizes, scales)))
    # the clipped gradients lie side by side in one buffer, each at a 16-byte word
    at = np.concatenate([[0], np.cumsum([(n + 7) // 8 * 8 for n in sizes])]).tolist()
    flat = torch.zeros(at[-1], dtype=dtype, device="cuda")
    return {"case": case, "grads": grads, "flat": flat,
            "outs": [flat[a:a + n] for a, n in zip(at, sizes)],
            "max_norm": float(np.float32(expected / case["ratio"])),
            "norm": torch.empty(1, device="cuda")}


def prepare(case, seed):
    return {"window_attention": _prepare_attn, "residual_norm": _prepare_norm,
            "clip_grad_norm": _prepare_clip}[case["op"]](case, seed)


# ---------------------------------------------------------------------------
# plain forms, in 32 bits, rounded once at the end
# ---------------------------------------------------------------------------
def _padded(x, cu, lens):
    """[T, H, D] -> [B, H, longest, D] in 32 bits, zeros behind each sequence; and which are real."""
    longest = max(1, max(lens))
    j = torch.arange(longest, device="cuda")
    real = j < (cu[1:] - cu[:-1])[:, None]
    rows = (cu[:-1, None] + j).clamp_max(max(0, x.shape[0] - 1))
    if not x.shape[0]:
        return x.new_zeros((len(lens), x.shape[1], longest, x.shape[2]), dtype=torch.float32), real
    y = x[rows].float() * real[:, :, None, None]
    return y.transpose(1, 2), real


def _scores(s):
    c = s["case"]
    q, real_q = _padded(s["q"], s["cu_q"], s["lens_q"])
    k, real_k = _padded(s["k"], s["cu_k"], s["lens_k"])
    B, hq, n, D = q.shape
    q = q.reshape(B, c["hk"], -1, D)  # the queries of a group share their key head
    score = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"]).view(B, c["hk"], -1, n, k.shape[2])
    # the last query stands at the last key
    at = torch.arange(n, device="cuda") + ((s["cu_k"][1:] - s["cu_k"][:-1]) -
                                           (s["cu_q"][1:] - s["cu_q"][:-1]))[:, None]
    at, j = at[:, :, None], torch.arange(k.shape[2], device="cuda")
    keep = ((j >= at - c["left"]) & (j <= at + c["right"])) | (j < c["sinks"])
    if c["causal"]:
        keep &= j <= at
    keep = keep & real_q[:, :, None] & real_k[:, None, :]
    return q, k, score, keep[:, None, None], real_q


def _plain_attention(s):
    c = s["case"]
    q, k, score, keep, real_q = _scores(s)
    v, _ = _padded(s["v"], s["cu_k"], s["lens_k"])
    B, hk, G, n, m = score.shape
    score = score.masked_fill_(~keep, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, 0.0)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (top + total.log()).reshape(B, c["hq"], n)
    o = torch.matmul(p.view(B, hk, G * n, m), v).view(B, hk, G, n, -1)
    o = (o / torch.where(total > 0, total, 1.0)).reshape(B, c["hq"], n, -1)
    return (o.transpose(1, 2)[real_q].to(s["q"].dtype),
            lse.transpose(1, 2)[real_q].transpose(0, 1).contiguous())


def _plain_attention_bwd(s):
    c = s["case"]
    q, k, score, keep, real_q = _scores(s)
    B, hk, G, n, m = score.shape
    v, real_k = _padded(s["v"], s["cu_k"], s["lens_k"])
    do, _ = _padded(s["dout"], s["cu_q"], s["lens_q"])
    o, _ = _padded(s["out"], s["cu_q"], s["lens_q"])
    lse = _padded(s["lse"].t().unsqueeze(-1).nan_to_num(neginf=0.0), s["cu_q"], s["lens_q"])[0]
    delta = (do * o).sum(-1).view(B, hk, G, n, 1)
    do = do.reshape(B, hk, G * n, -1)
    p = score.sub_(lse.reshape(B, hk, G, n, 1)).masked_fill_(~keep, -math.inf).exp_()
    dv = torch.matmul(p.view(B, hk, G * n, m).transpose(-1, -2), do)
    ds = torch.matmul(do, v.transpose(-1, -2)).view(B, hk, G, n, m).sub_(delta).mul_(p)
    ds = ds.view(B, hk, G * n, m)
    dq = (torch.matmul(ds, k) * s["scale"]).view(B, c["hq"], n, -1)
    dk = torch.matmul(ds.transpose(-1, -2), q) * s["scale"]
    t = s["q"].dtype
    return {"dq": dq.transpose(1, 2)[real_q].to(t), "dk": dk.transpose(1, 2)[real_k].to(t),
            "dv": dv.transpose(1, 2)[real_k].to(t)}


def _centred(v, kind):
    """(values by their norm, reciprocal of the norm) of each row"""
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    r = torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
    return v * r, r


def _affine(v, w, b):
    v = v if w is None else v * w
    return v if b is None else v + b


def _by_token(s, gate):
    """the gate's row of every token"""
    if gate.shape[0] == 1:
        return gate
    return torch.repeat_interleave(gate, s["cu"][1:] - s["cu"][:-1], dim=0,
                                   output_size=s["case"]["tokens"])


def _by_sequence(s, x):
    return torch.stack([p.sum(0) for p in x.split(s["lens"])])


def _plain_norm(s):
    c, dtype = s["case"], s["x"].dtype
    u = s["y"].float()
    if c["post"] != "none":
        u = _affine(_centred(u, c["post"])[0], s["post_weight"], s["post_bias"])
    if s["gate"] is not None:
        u = u * _by_token(s, s["gate"])
    r = c["alpha"] * s["x"].float() + c["beta"] * u
    h = _affine(_centred(r, c["pre"])[0], s["pre_weight"], s["pre_bias"])
    return {"r": r.to(dtype), "h": h.to(dtype)}


def _norm_back(g, hat, rstd, kind):
    """gradient by a norm's input from that by its normed values"""
    d = g - hat * (g * hat).mean(-1, keepdim=True)
    if kind == "layer":
        d = d - g.mean(-1, keepdim=True)
    return d * rstd


def _plain_norm_bwd(s):
    c, dtype = s["case"], s["x"].dtype
    u = hat_y = s["y"].float()
    if c["post"] != "none":
        hat_y, rstd_y = _centred(u, c["post"])
        u = _affine(hat_y, s["post_weight"], s["post_bias"])
    gate = None if s["gate"] is None else _by_token(s, s["gate"])
    r = c["alpha"] * s["x"].float() + c["beta"] * (u if gate is None else u * gate)
    hat_r, rstd_r = _centred(r, c["pre"])
    dh = s["dh"].float()
    dr = s["dr"].float() + _norm_back(dh * s["pre_weight"], hat_r, rstd_r, c["pre"])
    out = {"dx": (c["alpha"] * dr).to(dtype)}
    du = c["beta"] * (dr if gate is None else dr * gate)
    out["dy"] = (du if c["post"] == "none" else
                 _norm_back(du * s["post_weight"], hat_y, rstd_y, c["post"])).to(dtype)
    out["dpre_weight"] = (dh * hat_r).sum(0)
    if s["pre_bias"] is not None:
        out["dpre_bias"] = dh.sum(0)
    if s["post_weight"] is not None:
        out["dpost_weight"] = (du * hat_y).sum(0)
    if s["post_bias"] is not None:
        out["dpost_bias"] = du.sum(0)
    if gate is not None:
        out["dgate"] = _by_sequence(s, c["beta"] * dr * u)
    return out


def _plain_clip(s):
    squares = torch.stack([torch.sum(x.float().square(), dtype=torch.float64) for x in s["grads"]])
    norm = squares.sum().sqrt()
    factor = torch.clamp_max(s["max_norm"] / norm, 1.0).float()
    for x, out in zip(s["grads"], s["outs"]):
        out.copy_(x.float() * factor)
    return {"norm": norm.float().view(1), "outs": s["flat"]}


# ---------------------------------------------------------------------------
# the package's calls
# ---------------------------------------------------------------------------
def _package():
    import importlib

    return importlib.import_module(PACKAGE)


def _workspace(s, size):
    s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return s["workspace"]


def _own_attention(s):
    gs, c = _package(), s["case"]
    ws = s.get("workspace")
    if ws is None:
        ws = _workspace(s, gs.gs_attention_window_workspace_bytes(
            s["q"].shape[0], s["k"].shape[0], len(s["lens_q"]), c["hq"], c["hk"], c["dim"],
            c["left"], c["right"], c["sinks"]))
    if c["dir"] == "fwd":
        gs.gs_attention_window_fwd(s["q"], s["k"], s["v"], s["out"], s["lse"], ws, c["left"],
                                   c["right"], c["sinks"], cu_q=s["cu_q"], cu_k=s["cu_k"],
                                   causal=c["causal"], scale=s["scale"])
        return {"out": s["out"], "lse": s["lse"]}
    gs.gs_attention_window_bwd(s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"], s["dq"],
                               s["dk"], s["dv"], ws, c["left"], c["right"], c["sinks"],
                               cu_q=s["cu_q"], cu_k=s["cu_k"], causal=c["causal"],
                               scale=s["scale"])
    return {"dq": s["dq"], "dk": s["dk"], "dv": s["dv"]}


_GRADIENTS = ("dpre_weight", "dpre_bias", "dpost_weight", "dpost_bias", "dgate")


def _own_norm(s):
    gs, c = _package(), s["case"]
    common = {n: s[n] for n in ("pre_weight", "pre_bias", "post_weight", "post_bias", "gate", "cu")}
    common.update(pre=c["pre"], post=c["post"], alpha=c["alpha"], beta=c["beta"], eps=EPS)
    if c["dir"] == "fwd":
        gs.gs_residual_norm(s["x"], s["y"], s["r"], s["h"], **common)
        return {"r": s["r"], "h": s["h"]}
    ws = s.get("workspace")
    if ws is None:
        ws = _workspace(s, gs.gs_residual_norm_workspace_bytes(c["tokens"], c["width"],
                                                               len(s["lens"])))
    gs.gs_residual_norm_bwd(s["x"], s["y"], s["dr"], s["dh"], s["dx"], s["dy"], ws, **common,
                            **{n: s[n] for n in _GRADIENTS})
    return {n: s[n] for n in ("dx", "dy") + _GRADIENTS if s[n] is not None}


def _own_clip(s):
    gs = _package()
    ws = s.get("workspace")
    if ws is None:
        ws = _workspace(s, gs.gs_clip_grad_norm_workspace_bytes(len(s["grads"])))
    gs.gs_clip_grad_norm(s["grads"], s["max_norm"], s["norm"], ws, outs=s["outs"])
    return {"norm": s["norm"], "outs": s["flat"]}


def run(state):
    case = state["case"]
    forward = case["dir"] == "fwd"
    if case["op"] == "window_attention":
        if own:
            return _own_attention(state)
        if not forward:
            return _plain_attention_bwd(state)
        out, lse = _plain_attention(state)
        return {"out": out, "lse": lse}
    if case["op"] == "residual_norm":
        if own:
            return _own_norm(state)
        return _plain_norm(state) if forward else _plain_norm_bwd(state)
    return _own_clip(state) if own else _plain_clip(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _bounds(case, n, m):
    """first and last-but-one key of every query's window, and the sinks it sees"""
    at = np.arange(n, dtype=np.int64) + m - n
    lo = np.clip(at - case["left"], 0, m)
    hi = np.clip(at + (0 if case["causal"] else case["right"]) + 1, lo, m)
    sinks = np.full_like(at, min(case["sinks"], m))
    if case["causal"]:
        sinks = np.clip(at + 1, 0, sinks)
    return lo, hi, sinks


def _seen(case):
    """(query, key) pairs that the mask leaves, for one head, and keys that some query sees"""
    pairs = keys = 0
    for n, m in zip(_lens(case["lens_q"]), _lens(case["lens_k"])):
        if not n or not m:
            continue
        lo, hi, sinks = _bounds(case, n, m)
        pairs += int((hi - lo + sinks - np.clip(np.minimum(sinks, hi) - lo, 0, None)).sum())
        some = hi > lo
        a, b = (int(lo[some].min()), int(hi[some].max())) if some.any() else (0, 0)
        last = int(sinks.max())
        keys += b - a + last - max(0, min(last, b) - a)
    return pairs, keys


def work(case):
    size = 2 if case.get("dtype") == "bf16" else 4
    if case["op"] == "window_attention":
        Tq, Tk = sum(_lens(case["lens_q"])), sum(_lens(case["lens_k"]))
        pairs, keys = _seen(case)
        q, row = Tq * case["hq"] * case["dim"], case["hk"] * case["dim"]
        rest = 4 * Tq * case["hq"]
        if case["dir"] == "fwd":
            return {"bytes": size * (2 * q + 2 * keys * row) + rest,
                    "flops": 4 * pairs * case["hq"] * case["dim"]}
        return {"bytes": size * (4 * q + 2 * keys * row + 2 * Tk * row) + rest,
                "flops": 10 * pairs * case["hq"] * case["dim"]}
    if case["op"] == "residual_norm":
        n, arrays = case["tokens"] * case["width"], 4 if case["dir"] == "fwd" else 6
        return {"bytes": n * size * arrays, "flops": n * (12 if case["dir"] == "fwd" else 40)}
    n = sum(_sizes(case["sizes"]))
    return {"bytes": 2 * n * size, "flops": 3 * n}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_attention(case, s):
    hq, hk, D = case["hq"], case["hk"], case["dim"]
    group, forward = hq // hk, case["dir"] == "fwd"
    d64 = {n: s[n].double() for n in ("q", "k", "v") + (() if forward else ("dout",))}
    Tq = s["q"].shape[0]
    out = torch.zeros((Tq, hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((hq, Tq), -math.inf, dtype=torch.float64, device="cuda")
    grads = {n: torch.zeros_like(d64[n]) for n in ("q", "k", "v")}
    a0 = b0 = 0
    for n, m in zip(s["lens_q"], s["lens_k"]):
        for r in range(0, n if m else 0, 1024):  # a block of query rows against the keys near it
            e = min(n, r + 1024)
            lo, hi, sinks = (torch.from_numpy(x[r:e]).cuda()[:, None] for x in _bounds(case, n, m))
            first = int(min(lo.min(), hi.min()))
            j = torch.cat([torch.arange(min(int(sinks.max()), first), device="cuda"),
                           torch.arange(first, int(hi.max()), device="cuda")])
            if int(sinks.max()) > first:  # sinks beyond the first key of the window
                j = torch.arange(max(int(hi.max()), int(sinks.max())), device="cuda")
            if not j.numel():
                continue
            seen = ((j >= lo) & (j < hi)) | (j < sinks)
            for g in range(hk):
                heads = slice(g * group, (g + 1) * group)
                kh, vh = d64["k"][b0 + j, g], d64["v"][b0 + j, g]
                qh = d64["q"][a0 + r:a0 + e, heads].transpose(0, 1)
                w = (qh @ kh.t() * s["scale"]).masked_fill(~seen, -math.inf)
                total = torch.logsumexp(w, -1)
                prob = torch.exp(w - torch.where(torch.isfinite(total), total, 0.0)[..., None])
                o = prob @ vh
                if forward:
                    out[a0 + r:a0 + e, heads] = o.transpose(0, 1)
                    lse[heads, a0 + r:a0 + e] = total
                    continue
                do = d64["dout"][a0 + r:a0 + e, heads].transpose(0, 1)
                back = prob * (do @ vh.t() - (do * o).sum(-1, keepdim=True)) * s["scale"]
                grads["q"][a0 + r:a0 + e, heads] = (back @ kh).transpose(0, 1)
                grads["k"][b0 + j, g] += torch.einsum("hij,hid->jd", back, qh)
                grads["v"][b0 + j, g] += torch.einsum("hij,hid->jd", prob, do)
        a0, b0 = a0 + n, b0 + m
    if forward:
        return {"out": out, "lse": lse}
    return {"d" + n: grads[n] for n in ("q", "k", "v")}


def _exact_norm(case, s):
    """Through autograd in 64 bits."""
    C = case["width"]
    leaves = {n: s[n].double().requires_grad_(case["dir"] == "bwd") if s[n] is not None else None
              for n in ("x", "y", "pre_weight", "pre_bias", "post_weight", "post_bias", "gate")}

    def norm(v, kind, w, b):
        mean = v.sum(-1, keepdim=True) / C if kind == "layer" else 0.0
        v = (v - mean) / ((v - mean).pow(2).sum(-1, keepdim=True) / C + EPS).sqrt()
        v = v if w is None else w * v
        return v if b is None else v + b

    rs, hs = [], []
    token = 0
    for i, n in enumerate(s["lens"]):
        y = leaves["y"][token:token + n]
        if case["post"] != "none":
            y = norm(y, case["post"], leaves["post_weight"], leaves["post_bias"])
        if leaves["gate"] is not None:
            y = y * leaves["gate"][i]
        rs.append(case["alpha"] * leaves["x"][token:token + n] + case["beta"] * y)
        hs.append(norm(rs[-1], case["pre"], leaves["pre_weight"], leaves["pre_bias"]))
        token += n
    r, h = torch.cat(rs), torch.cat(hs)
    if case["dir"] == "fwd":
        return {"r": r, "h": h}
    torch.autograd.backward([r, h], [s["dr"].double(), s["dh"].double()])
    return {"d" + n: v.grad for n, v in leaves.items() if v is not None}


def _exact_clip(s):
    norm = math.sqrt(math.fsum(float(x.double().pow(2).sum()) for x in s["grads"]))
    factor = min(1.0, s["max_norm"] / norm) if norm > 0 else 1.0
    flat = torch.zeros(s["flat"].numel(), dtype=torch.float64, device="cuda")
    for x, out in zip(s["grads"], s["outs"]):
        flat[out.storage_offset():out.storage_offset() + x.numel()] = x.double() * factor
    return {"norm": torch.tensor([norm], dtype=torch.float64, device="cuda"), "outs": flat}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "window_attention":
        return _exact_attention(case, s)
    return _exact_norm(case, s) if case["op"] == "residual_norm" else _exact_clip(s)
