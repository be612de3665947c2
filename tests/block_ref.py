"""Plain float64 definitions of the operators around the blocks (residual norms, gradient clipping,
window attention), with bounds on what fp32 arithmetic may add to them.  numpy only.

A bound counts roundings, each at most U = 2^-24 of the value rounded.  A sum over a row runs over
eight values of a thread, five steps across lanes and at most 32 warps: 45 roundings, each of at most
the sum of magnitudes.  SUM = 48 U covers it with the division by the width; a root halves a relative
error and adds two of its own."""

import numpy as np

U = 2.0 ** -24
SUM = 48 * U


# ---------------------------------------------------------------------------
# residual norms
# ---------------------------------------------------------------------------
def _mean(v):
    return v.mean(-1, keepdims=True)


def norm(v, e, kind, eps):
    """(normed values, bound on their error, factor, bound on its relative error) of rows v that are
    off by at most e"""
    if kind == "none":
        return v, e, np.ones((v.shape[0], 1)), np.zeros((v.shape[0], 1))
    if kind == "layer":
        m = _mean(v)
        e = e + _mean(e) + SUM * _mean(np.abs(v)) + U * (np.abs(v) + np.abs(m))
        v = v - m
    s = 1.0 / np.sqrt(_mean(v * v) + eps)
    # d s / s = -s^2 mean(v dv); the sum of squares, its root and reciprocal
    es = s * s * _mean(np.abs(v) * e + e * e) + SUM + 4 * U
    return v * s, (s * e) * (1 + es) + np.abs(v * s) * (es + U), s, es


def _norm_back(k, ek, vn, evn, s, es, kind):
    """(s (k - vn mean(k vn) [- mean k]), bound) for k off by ek, vn by evn, s by es of itself"""
    along, size = _mean(k * vn), _mean(np.abs(k * vn))
    ealong = _mean(np.abs(k) * evn + ek * np.abs(vn) + ek * evn) + (SUM + U) * size
    mean = _mean(k) if kind == "layer" else 0.0
    emean = _mean(ek) + SUM * _mean(np.abs(k)) if kind == "layer" else 0.0
    d = k - mean - vn * along
    ed = ek + emean + np.abs(vn) * ealong + evn * (np.abs(along) + ealong)
    ed = ed + 3 * U * (np.abs(k) + np.abs(mean) + np.abs(vn * along))
    return s * d, s * (ed + np.abs(d) * (es + 2 * U)) * (1 + es)


def residual_norm(x, y, pw=None, pb=None, qw=None, qb=None, gate=None, cu=None, pre="rms",
                  post="none", alpha=1.0, beta=1.0, eps=1e-6, dr=None, dh=None):
    """{name: (value, bound)}: r and h, and with dr or dh the gradients by x, y and the parameters.
    y may be None."""
    x = x.astype(np.float64)
    T, C = x.shape
    zero = np.zeros((T, C))
    one = lambda w, other: np.full(C, other) if w is None else w.astype(np.float64)
    pw_, pb_, qw_, qb_ = one(pw, 1.0), one(pb, 0.0), one(qw, 1.0), one(qb, 0.0)
    lens = [T] if cu is None else np.diff(cu)
    g = np.ones((T, C)) if gate is None else np.repeat(
        gate.astype(np.float64).reshape(len(lens), C), lens, 0)
    out = {}
    un, eun, su, esu = norm(zero if y is None else y.astype(np.float64), zero, post, eps)
    u = un * qw_ + qb_
    eu = np.abs(qw_) * eun + U * (np.abs(un * qw_) + np.abs(qb_))
    bg = beta * g
    r = alpha * x + bg * u
    er = np.abs(bg) * eu + 4 * U * (np.abs(bg * u) + np.abs(alpha * x))
    out["r"] = r, er
    vn, evn, sv, esv = norm(r, er, pre, eps)
    if pre != "none":
        h = vn * pw_ + pb_
        out["h"] = h, np.abs(pw_) * evn + 2 * U * (np.abs(vn * pw_) + np.abs(pb_))
    if dr is None and dh is None:
        return out
    d, ed = (zero, zero) if dr is None else (dr.astype(np.float64), zero)
    if pre != "none":
        gh = dh.astype(np.float64)
        k = gh * pw_
        b, eb = _norm_back(k, U * np.abs(k), vn, evn, sv, esv, pre)
        d, ed = d + b, ed + eb + U * (np.abs(d) + np.abs(b))
        out["pre_weight"] = (gh * vn).sum(0), (np.abs(gh) * evn).sum(0), (np.abs(gh * vn)).sum(0)
        out["pre_bias"] = gh.sum(0), np.zeros(C), np.abs(gh).sum(0)
    out["x"] = alpha * d, abs(alpha) * (ed + U * np.abs(d))
    if y is not None:
        du, edu = bg * d, np.abs(bg) * ed + 3 * U * np.abs(bg * d)
        out["post_weight"] = ((du * un).sum(0), (edu * np.abs(un) + np.abs(du) * eun).sum(0),
                              np.abs(du * un).sum(0))
        out["post_bias"] = du.sum(0), edu.sum(0), np.abs(du).sum(0)
        dg = beta * d * u
        # formed as weight x sum of d un + bias x sum of d: the terms' magnitudes apart
        mag = abs(beta) * np.abs(d) * (np.abs(un * qw_) + np.abs(qb_))
        edg = abs(beta) * (ed * (np.abs(un * qw_) + np.abs(qb_)) + np.abs(d * qw_) * eun)
        ends = np.concatenate([[0], np.cumsum(lens)])
        by = lambda a: np.stack([a[i:j].sum(0) for i, j in zip(ends[:-1], ends[1:])])
        out["gate"] = by(dg), by(edg), by(mag)
        if post != "none":
            k = du * qw_
            du, edu = _norm_back(k, np.abs(qw_) * edu + U * np.abs(k), un, eun, su, esu, post)
        out["y"] = du, edu
    # sums over tokens: a rounding a row and block on the way, at most
    for n in ("pre_weight", "pre_bias", "post_weight", "post_bias", "gate"):
        if n in out:
            v, e, mag = out[n]
            out[n] = v, e + (T + 40) * U * mag
    return out


# ---------------------------------------------------------------------------
# gradient norm and clipping
# ---------------------------------------------------------------------------
def clip_grad_norm(grads, max_norm):
    """(norm, clipped arrays)"""
    with np.errstate(over="ignore"):
        norm = np.sqrt(sum(float((g.astype(np.float64) ** 2).sum()) for g in grads))
    f = 0.0 if not np.isfinite(norm) else max_norm / norm if norm > max_norm else 1.0
    return norm, [g.astype(np.float64) * f if f else np.zeros(g.shape) for g in grads]


# ---------------------------------------------------------------------------
# window attention
# ---------------------------------------------------------------------------
def seen(n, m, left, right, sinks, causal):
    """[n, m]: which keys each query sees"""
    at, j = np.arange(n)[:, None] + m - n, np.arange(m)[None]
    s = ((j >= at - left) & (j <= at + right)) | (j < sinks)
    return s & (j <= at) if causal else s


def _sequences(Tq, Tk, cu_q, cu_k):
    if cu_q is None:
        return [(0, Tq, 0, Tk)]
    return [(int(cu_q[b]), int(cu_q[b + 1]), int(cu_k[b]), int(cu_k[b + 1]))
            for b in range(len(cu_q) - 1)]


def window_attention(q, k, v, scale, left, right, sinks, causal=False, cu_q=None, cu_k=None):
    """(out, lse, magnitude of out, largest magnitude of a score's terms per row)"""
    q, k, v = (t.astype(np.float64) for t in (q, k, v))
    Tq, hq, _ = q.shape
    group = hq // k.shape[1]
    out, mag = np.zeros_like(q), np.zeros_like(q)
    lse, smag = np.full((hq, Tq), -np.inf), np.zeros((hq, Tq))
    for q0, q1, k0, k1 in _sequences(Tq, k.shape[0], cu_q, cu_k):
        if q1 <= q0 or k1 <= k0:
            continue
        keep = seen(q1 - q0, k1 - k0, left, right, sinks, causal)
        some = keep.any(1)
        for h in range(hq):
            kk, vv = k[k0:k1, h // group], v[k0:k1, h // group]
            s = np.where(keep, scale * (q[q0:q1, h] @ kk.T), -np.inf)
            top = np.where(some, s.max(-1), 0.0)[:, None]
            e = np.exp(s - top)
            total = e.sum(-1, keepdims=True)
            with np.errstate(divide="ignore"):
                lse[h, q0:q1] = (top + np.log(total))[:, 0]
            p = e / np.where(total > 0, total, 1.0)
            out[q0:q1, h], mag[q0:q1, h] = p @ vv, p @ np.abs(vv)
            size = np.where(keep, np.abs(q[q0:q1, h]) @ np.abs(kk).T, 0.0)
            smag[h, q0:q1] = abs(scale) * size.max(-1)
    return out, lse, mag, smag


def window_attention_bwd(q, k, v, out, lse, dout, scale, left, right, sinks, causal=False, cu_q=None,
                         cu_k=None):
    """{name: (gradient, bound)}: P and dS are rounded to bfloat16 once each (2^-8 of a term), their
    fp32 terms stay below 2^-12 of the terms' magnitudes (a score of at most 128 products: 2^-17,
    which the exponential amplifies by at most the score's magnitude, below 32 here)."""
    q, k, v, out, dout = (t.astype(np.float64) for t in (q, k, v, out, dout))
    Tq, hq, _ = q.shape
    group, H, E = hq // k.shape[1], 2.0 ** -8, 2.0 ** -12
    g = {n: [np.zeros_like(t), np.zeros_like(t)] for n, t in (("q", q), ("k", k), ("v", v))}
    for q0, q1, k0, k1 in _sequences(Tq, k.shape[0], cu_q, cu_k):
        if q1 <= q0 or k1 <= k0:
            continue
        keep = seen(q1 - q0, k1 - k0, left, right, sinks, causal)
        for h in range(hq):
            kh = h // group
            qq, kk, vv, do = q[q0:q1, h], k[k0:k1, kh], v[k0:k1, kh], dout[q0:q1, h]
            ls = lse[h, q0:q1].astype(np.float64)[:, None]
            s = np.where(keep, scale * (qq @ kk.T), -np.inf)
            p = np.exp(s - np.where(np.isfinite(ls), ls, 0.0)) * np.isfinite(ls)
            delta = (do * out[q0:q1, h]).sum(-1, keepdims=True)
            delta_m = np.abs(do * out[q0:q1, h]).sum(-1, keepdims=True)
            ds = p * (do @ vv.T - delta)
            err = H * np.abs(ds) + E * p * (np.abs(do) @ np.abs(vv).T + delta_m)
            g["q"][0][q0:q1, h] = scale * ds @ kk
            g["q"][1][q0:q1, h] = abs(scale) * err @ np.abs(kk)
            g["k"][0][k0:k1, kh] += scale * ds.T @ qq
            g["k"][1][k0:k1, kh] += abs(scale) * err.T @ np.abs(qq)
            g["v"][0][k0:k1, kh] += p.T @ do
            g["v"][1][k0:k1, kh] += (H + E) * (p.T @ np.abs(do))
    return {n: tuple(t) for n, t in g.items()}
