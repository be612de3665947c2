"""Plain float64 definitions of the token operators, with the magnitudes of their terms (the
same sums over absolute values), from which the tests' tolerances are made.  numpy only."""

import numpy as np

U = 2.0 ** -24   # half a unit in the last place of fp32
H = 2.0 ** -8    # of bfloat16 (8 significant bits)


def bf16(x):
    """x rounded to bfloat16 (nearest, ties to even), as float32."""
    b = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000
    return b.astype(np.uint32).view(np.float32).reshape(np.shape(x))


# ---------------------------------------------------------------------------
# head norm + rotation
# ---------------------------------------------------------------------------
def _pairs(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def _angles(table, positions, T, rot):
    c, s = np.ones((T, rot // 2)), np.zeros((T, rot // 2))
    pos = np.arange(T) if positions is None else positions
    ok = pos >= 0
    if rot:
        c[ok], s[ok] = table[pos[ok], :rot // 2], table[pos[ok], rot // 2:]
    return c[:, None], s[:, None]


def turn(x, c, s, rot, interleaved):
    """(the turned rows, their magnitude)"""
    a, b = _pairs(rot, interleaved)
    y, m = x.copy(), np.abs(x)
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    m[..., a] = np.abs(x[..., a] * c) + np.abs(x[..., b] * s)
    m[..., b] = np.abs(x[..., b] * c) + np.abs(x[..., a] * s)
    return y, m


def head_norm(x, w, table, positions, eps, interleaved):
    """(y, magnitude) of one side; x [T, H, D], w [D] or None, table [P, rot] or None"""
    x = x.astype(np.float64)
    rot = 0 if table is None else table.shape[1]
    c, s = _angles(table, positions, x.shape[0], rot)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return turn(x * r * (1.0 if w is None else w.astype(np.float64)), c, s, rot, interleaved)


def head_norm_bwd(x, w, table, positions, eps, interleaved, dy):
    """(dx, its magnitude, dw, its magnitude)"""
    x, dy = x.astype(np.float64), dy.astype(np.float64)
    rot = 0 if table is None else table.shape[1]
    c, s = _angles(table, positions, x.shape[0], rot)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    g, gm = turn(dy, c, -s, rot, interleaved)
    w = np.ones(x.shape[-1]) if w is None else w.astype(np.float64)
    dx = r * (w * g - x * r * r * (w * g * x).mean(-1, keepdims=True))
    dxm = r * (np.abs(w) * gm + np.abs(x) * r * r * np.abs(w * gm * x).mean(-1, keepdims=True))
    return dx, dxm, (g * x * r).sum((0, 1)), (gm * np.abs(x) * r).sum((0, 1))


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def _sequences(Tq, Tk, cu_q, cu_k):
    if cu_q is None:
        yield 0, Tq, 0, Tk
        return
    for b in range(len(cu_q) - 1):
        yield int(cu_q[b]), int(cu_q[b + 1]), int(cu_k[b]), int(cu_k[b + 1])


def _scores(q, k, scale, causal):
    n, m = q.shape[0], k.shape[0]
    s = scale * (q @ k.T)
    if causal:
        s = np.where(np.arange(m)[None] <= np.arange(n)[:, None] + m - n, s, -np.inf)
    return s


def attention(q, k, v, scale, causal=False, cu_q=None, cu_k=None):
    """(out, lse, magnitude of out, largest magnitude of a score's terms per row)"""
    q, k, v = (t.astype(np.float64) for t in (q, k, v))
    Tq, hq, D = q.shape
    group = hq // k.shape[1]
    out, mag = np.zeros_like(q), np.zeros_like(q)
    lse, smag = np.full((hq, Tq), -np.inf), np.zeros((hq, Tq))
    for q0, q1, k0, k1 in _sequences(Tq, k.shape[0], cu_q, cu_k):
        if q1 == q0 or k1 == k0:
            continue
        for h in range(hq):
            kk, vv = k[k0:k1, h // group], v[k0:k1, h // group]
            s = _scores(q[q0:q1, h], kk, scale, causal)
            top = s.max(-1, keepdims=True)
            top = np.where(np.isfinite(top), top, 0.0)
            e = np.exp(s - top)
            l = e.sum(-1, keepdims=True)
            with np.errstate(divide="ignore"):
                lse[h, q0:q1] = (top + np.log(l))[:, 0]
            p = e / np.where(l > 0, l, 1.0)
            out[q0:q1, h], mag[q0:q1, h] = p @ vv, p @ np.abs(vv)
            smag[h, q0:q1] = abs(scale) * (np.abs(q[q0:q1, h]) @ np.abs(kk).T).max(-1)
    return out, lse, mag, smag


def attention_bwd(q, k, v, out, lse, dout, scale, causal=False, cu_q=None, cu_k=None):
    """{name: (gradient, bound on the rounding of P and dS to bfloat16 and of their fp32 terms)}
    of the formulas evaluated at the given out and lse.  Each of P and dS is rounded once (H);
    P's exponent and the differences dP - delta are fp32, whose errors stay below 2^-12 of the
    terms' magnitudes for the sizes tested (a score's sum of D <= 128 products: 2^-17; its
    exponential amplifies that by at most the score's magnitude, below 32 here)."""
    q, k, v, out, dout = (t.astype(np.float64) for t in (q, k, v, out, dout))
    Tq, hq, D = q.shape
    group = hq // k.shape[1]
    E = 2.0 ** -12
    g = {n: [np.zeros_like(t), np.zeros_like(t)] for n, t in (("q", q), ("k", k), ("v", v))}
    for q0, q1, k0, k1 in _sequences(Tq, k.shape[0], cu_q, cu_k):
        if q1 == q0 or k1 == k0:
            continue
        for h in range(hq):
            kh = h // group
            qq, kk, vv, do = q[q0:q1, h], k[k0:k1, kh], v[k0:k1, kh], dout[q0:q1, h]
            ls = lse[h, q0:q1].astype(np.float64)[:, None]
            s = _scores(qq, kk, scale, causal)
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


# ---------------------------------------------------------------------------
# dropout
# ---------------------------------------------------------------------------
def philox4x32_10(counter, key):
    """Philox4x32-10 in whole numbers: counter (4 words or arrays of them), key (2 words)."""
    c, k = [np.asarray(x, np.uint64) for x in counter], [int(x) for x in key]
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> half) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> half) ^ c[3] ^ np.uint64(k[1]),
             a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def kept(n, seed, offset, p):
    """(mask of the n elements, factor of the kept ones)"""
    seed, offset = int(seed) % 2 ** 64, int(offset) % 2 ** 64
    i = np.arange((n + 7) // 8, dtype=np.uint64)
    z = np.zeros_like(i)
    w = philox4x32_10([i & np.uint64(0xFFFFFFFF), i >> np.uint64(32), z + np.uint64(offset & 0xFFFFFFFF),
                       z + np.uint64(offset >> 32)], [seed & 0xFFFFFFFF, seed >> 32])
    bits = np.stack([x for v in w for x in (v & np.uint64(0xFFFF), v >> np.uint64(16))], 1)
    drop = int(np.floor(float(np.float32(p)) * 65536 + 0.5))
    return bits.reshape(-1)[:n] >= drop, 65536.0 / (65536 - drop)
