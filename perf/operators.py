"""The token operators of a network that predicts Gaussians, as cases to time and to compare.

A network that is trained through the rasterizer reads a view as tokens, one for each 16 x 16
tile: 64 tokens for the 128 x 128 view of the synthetic configurations, 2,500 for 800 x 800,
4,346 for 1297 x 840, 8,160 for 1920 x 1080, 32,400 for 3840 x 2160.  The operators:

  qk_norm_rope   RMS norm of every query and key head and the position rotation, and its gradient
  attention      softmax attention over ragged batches with shared heads, and its gradient
  dropout_add    residual + dropout(x) from a counter-based generator, and its gradient

`run` computes them in plain 32-bit torch operations, or, where `own` is true, through this
repository's package.
"""

from __future__ import annotations

import math

import numpy as np
import torch

own = False

PACKAGE = "differentiable_gaussian_splatting_gb300"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6

# the costliest cases that draw() may give, per operator: padded (query, key) cells over all
# heads, for the plain form's matrices, and values of the operators that pass over memory once
MOST_CELLS_FWD = 16320 * 16320 * 16
MOST_CELLS_BWD = 8160 * 8160 * 16
MOST_VALUES = 32400 * 20 * 128


def _rope(name, direction, tokens, hq, hk, dim, rot, dtype, interleaved, registers):
    return {"name": name, "op": "qk_norm_rope", "dir": direction, "tokens": tokens, "hq": hq,
            "hk": hk, "dim": dim, "rot": rot, "dtype": dtype, "interleaved": interleaved,
            "registers": registers}


def _attn(name, direction, lens_q, lens_k, hq, hk, dim, causal):
    return {"name": name, "op": "attention", "dir": direction,
            "lens_q": " ".join(map(str, lens_q)), "lens_k": " ".join(map(str, lens_k)), "hq": hq,
            "hk": hk, "dim": dim, "causal": causal, "dtype": "bf16"}


def _drop(name, direction, rows, width, p, dtype, residual):
    return {"name": name, "op": "dropout_add", "dir": direction, "rows": rows, "width": width,
            "p": p, "dtype": dtype, "residual": residual}


def listed():
    return [
        # one 128 x 128 view at inference: the call's latency
        _rope("rope-fwd-64", "fwd", 64, 8, 8, 64, 64, "bf16", False, 0),
        # a 3840 x 2160 view, grouped heads, read out of the packed projection
        _rope("rope-fwd-32400", "fwd", 32400, 16, 4, 128, 128, "bf16", False, 0),
        # training in fp32 on a 1297 x 840 view, part of each head rotated, four register tokens
        _rope("rope-bwd-4350-f32", "bwd", 4350, 12, 12, 64, 48, "f32", True, 4),
        # training on a 3840 x 2160 view
        _rope("rope-bwd-32400", "bwd", 32400, 16, 4, 128, 128, "bf16", False, 0),
        # one 128 x 128 view at inference
        _attn("attn-fwd-64", "fwd", [64], [64], 8, 8, 64, False),
        # views of several sizes in one batch, an empty one and a lone token among them, tiles
        # predicted one after the other (causal), grouped heads
        _attn("attn-fwd-ragged", "fwd", [4346, 2500, 64, 1, 0, 1039], [4346, 2500, 64, 1, 0, 1039],
              16, 4, 128, True),
        # two 1920 x 1080 views attended jointly
        _attn("attn-fwd-16320", "fwd", [16320], [16320], 16, 16, 128, False),
        # a camera token per view reads all the view's tile tokens
        _attn("attn-fwd-pool", "fwd", [1, 1, 1, 1], [32400, 8160, 4346, 2500], 16, 16, 64, False),
        # a training batch of small and middling views
        _attn("attn-bwd-ragged", "bwd", [2500, 64, 1, 0, 1039], [2500, 64, 1, 0, 1039], 8, 8, 64,
              True),
        # training on a 1920 x 1080 view, grouped heads
        _attn("attn-bwd-8160", "bwd", [8160], [8160], 16, 4, 128, False),
        # the residual branch of a 3840 x 2160 view, 1,024 channels
        _drop("drop-fwd-32400", "fwd", 32400, 1024, 0.1, "bf16", True),
        # the gradient of a 128 x 128 view's branch in fp32, an odd width
        _drop("drop-bwd-64-f32", "bwd", 64, 515, 0.25, "f32", False),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    kind = rng.choice(["rope", "attn", "attn", "drop"])
    direction = rng.choice(["fwd", "bwd"])
    if kind == "rope":
        dim = 8 * rng.randint(2, 16)
        hk = rng.choice([1, 2, 3, 4, 8])
        hq = hk * rng.choice([1, 2, 3, 4])
        tokens = _log_uniform(rng, 1, min(32400, MOST_VALUES // ((hq + hk) * dim)))
        case = _rope("", direction, tokens, hq, hk, dim, rng.choice([dim, max(2, dim // 4 * 2)]),
                     rng.choice(["bf16", "f32"]), rng.random() < 0.5,
                     rng.randint(0, min(4, tokens - 1)))
        if case["dtype"] == "f32":
            case["tokens"] = max(1, case["tokens"] // 2)
            case["registers"] = min(case["registers"], case["tokens"] - 1)
    elif kind == "attn":
        dim = rng.choice([16, 40, 64, 64, 72, 96, 128, 128])
        hk = rng.choice([1, 2, 3, 4, 8])
        hq = hk * rng.choice([1, 2, 3, 4])
        causal = rng.random() < 0.4
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
        case = _attn("", direction, lens_q, lens_k, hq, hk, dim, causal)
    else:
        width = rng.randint(1, 1300)
        dtype = rng.choice(["bf16", "f32"])
        most = 32400 * 1024 // (width * (1 if dtype == "bf16" else 2))
        case = _drop("", direction, _log_uniform(rng, 1, min(32400, most)), width,
                     rng.choice([0.0, 0.1, 0.3, 0.5]), dtype,
                     direction == "fwd" and rng.random() < 0.7)
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


def _axial_table(n_pos, rot):
    """cos and sin [n_pos, rot] of tokens on a grid: half of the pairs turn with the row, half
    with the column of the token's tile."""
    wide = max(1, math.isqrt(n_pos))
    i = torch.arange(n_pos, device="cuda", dtype=torch.float64)
    row, col = torch.div(i, wide, rounding_mode="floor"), i % wide
    half = rot // 2
    rows = (half + 1) // 2
    f_row = 100.0 ** (-torch.arange(rows, device="cuda", dtype=torch.float64) / max(1, rows))
    f_col = 100.0 ** (-torch.arange(half - rows, device="cuda", dtype=torch.float64)
                      / max(1, half - rows))
    angle = torch.cat([row[:, None] * f_row, col[:, None] * f_col], 1)
    return torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()


def _prepare_rope(case, seed):
    g = _generator(seed)
    T, hq, hk, D = case["tokens"], case["hq"], case["hk"], case["dim"]
    dtype = DTYPES[case["dtype"]]
    # the projection of a token holds its queries, keys and values side by side
    packed = _normal(g, (T, hq + 2 * hk, D), torch.float32)
    packed *= 0.5 + torch.rand((T, hq + 2 * hk, 1), generator=g, device="cuda")
    packed = packed.to(dtype)
    n_pos = max(1, T - case["registers"])
    positions = torch.arange(T, device="cuda", dtype=torch.int32) - case["registers"]
    positions = torch.where(positions < 0, torch.full_like(positions, -1), positions)
    s = {"case": case, "packed": packed, "q": packed[:, :hq], "k": packed[:, hq:hq + hk],
         "qw": 1.0 + 0.1 * _normal(g, (D,), torch.float32),
         "kw": 1.0 + 0.1 * _normal(g, (D,), torch.float32),
         "table": _axial_table(n_pos, case["rot"]), "positions": positions,
         "q_out": torch.empty((T, hq, D), dtype=dtype, device="cuda"),
         "k_out": torch.empty((T, hk, D), dtype=dtype, device="cuda")}
    if case["dir"] == "bwd":
        s["dq_out"] = _normal(g, (T, hq, D), dtype, 0.1)
        s["dk_out"] = _normal(g, (T, hk, D), dtype, 0.1)
        s["dq"], s["dk"] = torch.empty_like(s["q_out"]), torch.empty_like(s["k_out"])
        s["dqw"], s["dkw"] = torch.empty_like(s["qw"]), torch.empty_like(s["kw"])
    return s


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


def _prepare_drop(case, seed):
    g = _generator(seed)
    shape, dtype = (case["rows"], case["width"]), DTYPES[case["dtype"]]
    s = {"case": case, "x": _normal(g, shape, dtype),
         "rng": torch.randint(0, 2 ** 62, (2,), generator=g, device="cuda", dtype=torch.int64),
         "out": torch.empty(shape, dtype=dtype, device="cuda")}
    s["residual"] = _normal(g, shape, dtype, 2.0) if case["residual"] else None
    return s


def prepare(case, seed):
    return {"qk_norm_rope": _prepare_rope, "attention": _prepare_attn,
            "dropout_add": _prepare_drop}[case["op"]](case, seed)


# ---------------------------------------------------------------------------
# plain forms, in 32 bits, rounded once at the end
# ---------------------------------------------------------------------------
def _pairs(x, interleaved):
    """The two values of each rotated pair, as (first, second)."""
    if interleaved:
        return x[..., 0::2], x[..., 1::2]
    h = x.shape[-1] // 2
    return x[..., :h], x[..., h:]


def _unpairs(a, b, interleaved):
    if interleaved:
        return torch.stack([a, b], -1).flatten(-2)
    return torch.cat([a, b], -1)


def _turn(x, table, positions, rot, interleaved, sign):
    """x [T, H, D] with the pairs of its first rot values turned by sign times the angle;
    tokens of a negative position stay as they are."""
    row = table[positions.clamp_min(0).long()]
    free = (positions < 0)[:, None]
    c = torch.where(free, 1.0, row[:, :rot // 2])[:, None]
    s = torch.where(free, 0.0, row[:, rot // 2:])[:, None] * sign
    a, b = _pairs(x[..., :rot], interleaved)
    return torch.cat([_unpairs(a * c - b * s, b * c + a * s, interleaved), x[..., rot:]], -1)


def _plain_rope(s):
    c = s["case"]

    def one(x, w):
        y = x.float()
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * w
        return _turn(y, s["table"], s["positions"], c["rot"], c["interleaved"], 1.0).to(x.dtype)

    return {"q": one(s["q"], s["qw"]), "k": one(s["k"], s["kw"])}


def _plain_rope_bwd(s):
    c = s["case"]

    def one(x, w, dy):
        x32 = x.float()
        r = torch.rsqrt(x32.square().mean(-1, keepdim=True) + EPS)
        g = _turn(dy.float(), s["table"], s["positions"], c["rot"], c["interleaved"], -1.0)
        xr = x32 * r
        wg = g * w
        dx = r * (wg - xr * (wg * xr).mean(-1, keepdim=True))
        return dx.to(x.dtype), (g * xr).sum((0, 1))

    (dq, dqw), (dk, dkw) = one(s["q"], s["qw"], s["dq_out"]), one(s["k"], s["kw"], s["dk_out"])
    return {"dq": dq, "dk": dk, "dqw": dqw, "dkw": dkw}


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
    keep = (real_q[:, :, None] & real_k[:, None, :])
    if c["causal"]:  # the last query sees the last key
        i, j = torch.arange(n, device="cuda"), torch.arange(k.shape[2], device="cuda")
        ahead = ((s["cu_k"][1:] - s["cu_k"][:-1]) - (s["cu_q"][1:] - s["cu_q"][:-1]))[:, None, None]
        keep = keep & (j[None, None, :] <= i[None, :, None] + ahead)
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
    p = score.sub_(lse.reshape(B, hk, G, n, 1)).exp_().masked_fill_(~keep, 0.0)
    dv = torch.matmul(p.view(B, hk, G * n, m).transpose(-1, -2), do)
    ds = torch.matmul(do, v.transpose(-1, -2)).view(B, hk, G, n, m).sub_(delta).mul_(p)
    ds = ds.view(B, hk, G * n, m)
    dq = (torch.matmul(ds, k) * s["scale"]).view(B, c["hq"], n, -1)
    dk = torch.matmul(ds.transpose(-1, -2), q) * s["scale"]
    t = s["q"].dtype
    return {"dq": dq.transpose(1, 2)[real_q].to(t), "dk": dk.transpose(1, 2)[real_k].to(t),
            "dv": dv.transpose(1, 2)[real_k].to(t)}


def _mulhilo(a, b):
    """High and low 32 bits of the product of a 32-bit constant and 32-bit values held in int64."""
    low, high = a * (b & 0xFFFF), a * (b >> 16)
    mid = high + (low >> 16)
    return mid >> 16, ((mid & 0xFFFF) << 16) | (low & 0xFFFF)


def _kept(n, rng, p):
    """Which of n elements stay: Philox4x32-10 (Salmon et al., 2011) keyed by the seed, counting
    groups of eight elements and the offset; 16 bits of its output for each element."""
    i = torch.arange((n + 7) // 8, device="cuda", dtype=torch.int64)
    seed, offset = rng[0], rng[1]
    mask = 0xFFFFFFFF
    k0, k1 = seed & mask, (seed >> 32) & mask
    c0, c1 = i & mask, (i >> 32) & mask
    c2, c3 = (offset & mask).expand_as(i), ((offset >> 32) & mask).expand_as(i)
    for _ in range(10):  # the generator's ten rounds, each on the last one's result
        h0, l0 = _mulhilo(0xD2511F53, c0)
        h1, l1 = _mulhilo(0xCD9E8D57, c2)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & mask, (k1 + 0xBB67AE85) & mask
    words = torch.stack([c0, c1, c2, c3], 1)
    bits = torch.stack([words & 0xFFFF, words >> 16], 2).reshape(-1)[:n]
    return bits >= _dropped(p)


def _dropped(p):
    """How many of the 65,536 values of an element's 16 bits drop it."""
    return int(math.floor(p * 65536.0 + 0.5))


def _plain_drop(s):
    c, x = s["case"], s["x"].float()
    keep = _kept(x.numel(), s["rng"], c["p"]).view(x.shape)
    y = torch.where(keep, x * (65536.0 / (65536 - _dropped(c["p"]))), 0.0)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(s["x"].dtype)


# ---------------------------------------------------------------------------
# the package's calls
# ---------------------------------------------------------------------------
def _package():
    import importlib

    return importlib.import_module(PACKAGE)


def _own_rope(s):
    gs, c = _package(), s["case"]
    gs.gs_qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], s["table"], s["positions"], s["q_out"],
                       s["k_out"], eps=EPS, interleaved=c["interleaved"])
    return {"q": s["q_out"], "k": s["k_out"]}


def _workspace(s, size):
    if "workspace" not in s:
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return s["workspace"]


def _own_rope_bwd(s):
    gs, c = _package(), s["case"]
    ws = s.get("workspace")
    if ws is None:
        ws = _workspace(s, gs.gs_qk_norm_rope_workspace_bytes(c["tokens"], c["hq"], c["hk"],
                                                              c["dim"]))
    gs.gs_qk_norm_rope_bwd(s["q"], s["k"], s["qw"], s["kw"], s["table"], s["positions"],
                           s["dq_out"], s["dk_out"], s["dq"], s["dk"], s["dqw"], s["dkw"], ws,
                           eps=EPS, interleaved=c["interleaved"])
    return {"dq": s["dq"], "dk": s["dk"], "dqw": s["dqw"], "dkw": s["dkw"]}


def _attention_workspace(s):
    ws = s.get("workspace")
    if ws is None:
        gs, c = _package(), s["case"]
        ws = _workspace(s, gs.gs_attention_workspace_bytes(
            s["q"].shape[0], s["k"].shape[0], len(s["lens_q"]), c["hq"], c["hk"], c["dim"]))
    return ws


def _own_attention(s):
    _package().gs_attention_fwd(s["q"], s["k"], s["v"], s["out"], s["lse"], _attention_workspace(s),
                                cu_q=s["cu_q"], cu_k=s["cu_k"], causal=s["case"]["causal"],
                                scale=s["scale"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_attention_bwd(s):
    _package().gs_attention_bwd(s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"], s["dq"],
                                s["dk"], s["dv"], _attention_workspace(s), cu_q=s["cu_q"],
                                cu_k=s["cu_k"], causal=s["case"]["causal"], scale=s["scale"])
    return {"dq": s["dq"], "dk": s["dk"], "dv": s["dv"]}


def _own_drop(s):
    gs, c = _package(), s["case"]
    if c["dir"] == "fwd":
        gs.gs_dropout_add(s["x"], s["residual"], s["out"], s["rng"], c["p"])
    else:
        gs.gs_dropout_add_bwd(s["x"], s["out"], s["rng"], c["p"])
    return {"out": s["out"]}


def run(state):
    case = state["case"]
    forward = case["dir"] == "fwd"
    if case["op"] == "qk_norm_rope":
        if own:
            return _own_rope(state) if forward else _own_rope_bwd(state)
        return _plain_rope(state) if forward else _plain_rope_bwd(state)
    if case["op"] == "attention":
        if own:
            return _own_attention(state) if forward else _own_attention_bwd(state)
        if not forward:
            return _plain_attention_bwd(state)
        out, lse = _plain_attention(state)
        return {"out": out, "lse": lse}
    # the gradient of the branch is the same mask and factor on the gradient that came back
    return _own_drop(state) if own else {"out": _plain_drop(state)}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _seen(case):
    """(query, key) pairs that the mask leaves, over all sequences, for one head."""
    total = 0
    for n, m in zip(_lens(case["lens_q"]), _lens(case["lens_k"])):
        if not case["causal"]:
            total += n * m
        else:  # query i sees min(m, max(0, i + 1 + m - n)) keys
            first = max(0, n - m)
            a, b = first + 1 + m - n, m
            total += (a + b) * (n - first) // 2 if n > first else 0
    return total


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "qk_norm_rope":
        T, D = case["tokens"], case["dim"]
        values = T * (case["hq"] + case["hk"]) * D
        rest = 4 * T + 4 * case["rot"] * max(1, T - case["registers"]) + 8 * D
        if case["dir"] == "fwd":
            return {"bytes": 2 * size * values + rest, "flops": 7 * values}
        return {"bytes": 3 * size * values + rest + 8 * D, "flops": 14 * values}
    if case["op"] == "attention":
        Tq, Tk = sum(_lens(case["lens_q"])), sum(_lens(case["lens_k"]))
        q, kv, seen = Tq * case["hq"] * case["dim"], Tk * case["hk"] * case["dim"], _seen(case)
        rest = 4 * Tq * case["hq"]
        if case["dir"] == "fwd":
            return {"bytes": size * (2 * q + 2 * kv) + rest,
                    "flops": 4 * seen * case["hq"] * case["dim"]}
        return {"bytes": size * (4 * q + 4 * kv) + rest,
                "flops": 10 * seen * case["hq"] * case["dim"]}
    n = case["rows"] * case["width"]
    return {"bytes": n * size * (3 if case["residual"] else 2), "flops": 2 * n}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_rope(case, s):
    T, D, R = case["tokens"], case["dim"], case["rot"]
    half = R // 2
    pos = s["positions"].long()
    angle_c = torch.ones((T, half), dtype=torch.float64, device="cuda")
    angle_s = torch.zeros_like(angle_c)
    placed = pos >= 0
    angle_c[placed] = s["table"].double()[pos[placed], :half]
    angle_s[placed] = s["table"].double()[pos[placed], half:]
    i = torch.arange(half, device="cuda")
    first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
    turn = torch.eye(D, dtype=torch.float64, device="cuda").repeat(T, 1, 1) if T * D * D < 1e8 else None

    def rotate(x, sign):
        if turn is not None:  # as one matrix for each token
            M = turn.clone()
            M[:, first, first], M[:, second, second] = angle_c, angle_c
            M[:, first, second], M[:, second, first] = -sign * angle_s, sign * angle_s
            return torch.einsum("tij,thj->thi", M, x)
        y = x.clone()
        z = torch.complex(x[..., first], x[..., second]) * torch.complex(angle_c, sign * angle_s)[:, None]
        y[..., first], y[..., second] = z.real, z.imag
        return y

    out = {}
    for n in ("q", "k"):
        x, w = s[n].double(), s[n + "w"].double()
        norm = (x.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt()
        if case["dir"] == "fwd":
            out[n] = rotate(x / norm * w, 1.0)
            continue
        g = rotate(s["d" + n + "_out"].double(), -1.0)
        # y_j = w_j x_j / norm:  dy_j/dx_i = w_j (delta_ij / norm - x_i x_j / (D norm^3))
        out["d" + n] = g * w / norm - x * (g * w * x).sum(-1, keepdim=True) / (D * norm.pow(3))
        out["d" + n + "w"] = (g * x / norm).sum((0, 1))
    return out if case["dir"] == "fwd" else {n: out[n] for n in ("dq", "dk", "dqw", "dkw")}


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
        for h in range(hq if n and m else 0):
            kh, vh = d64["k"][b0:b0 + m, h // group], d64["v"][b0:b0 + m, h // group]
            for r in range(0, n, 2048):  # a block of query rows against all keys
                e = min(n, r + 2048)
                qh = d64["q"][a0 + r:a0 + e, h]
                w = qh @ kh.t() * s["scale"]
                if case["causal"]:
                    hidden = torch.ones_like(w, dtype=torch.bool).triu(m - n + r + 1)
                    w = w.masked_fill(hidden, -math.inf)
                total = torch.logsumexp(w, -1)
                prob = torch.softmax(w, -1)
                prob = torch.where(torch.isfinite(total)[:, None], prob, 0.0)
                o = prob @ vh
                if forward:
                    out[a0 + r:a0 + e, h] = o
                    lse[h, a0 + r:a0 + e] = total
                    continue
                do = d64["dout"][a0 + r:a0 + e, h]
                back = prob * (do @ vh.t() - (do * o).sum(-1, keepdim=True)) * s["scale"]
                grads["q"][a0 + r:a0 + e, h] = back @ kh
                grads["k"][b0:b0 + m, h // group] += back.t() @ qh
                grads["v"][b0:b0 + m, h // group] += prob.t() @ do
        a0, b0 = a0 + n, b0 + m
    if forward:
        return {"out": out, "lse": lse}
    return {"d" + n: grads[n] for n in ("q", "k", "v")}


def _exact_drop(case, s):
    """The generator on the host, in whole numbers."""
    n = s["x"].numel()
    seed, offset = (int(v) for v in s["rng"].tolist())
    groups = np.arange((n + 7) // 8, dtype=np.uint64)
    low = np.uint64(0xFFFFFFFF)
    half = np.uint64(32)
    c = [groups & low, groups >> half, np.full_like(groups, offset & 0xFFFFFFFF),
         np.full_like(groups, offset >> 32)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> half) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> half) ^ c[3] ^ np.uint64(k[1]),
             a & low]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    bits = np.stack(c, 1).astype("<u4").view("<u2").reshape(-1)[:n]
    drop = math.floor(case["p"] * 65536 + 0.5)
    keep = torch.from_numpy(bits.astype(np.int32) >= drop).cuda().view(s["x"].shape)
    y = s["x"].double() * keep / (1.0 - drop / 65536.0)
    return {"out": y if s["residual"] is None else y + s["residual"].double()}


def exact(case, seed):
    s = prepare(case, seed)
    return {"qk_norm_rope": _exact_rope, "attention": _exact_attention,
            "dropout_add": _exact_drop}[case["op"]](case, s)
