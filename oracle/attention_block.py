"""fp64 CPU oracle of the local attention block's operators: per-head norms with the position
rotation, attention in a sliding window with sinks, their gradients, and attention of one token over
a paged cache.

TEST INFRASTRUCTURE ONLY, as the other oracles here: it never imports the product and the product
never imports it. Plain numpy in fp64, whole softmax rows, loops over sequences and heads.

Visibility (0-based positions of one sequence of n tokens): key u is visible to query t if u <= t and
(u > t - window or u < sinks). Rows t >= n: o = 0, lse = -inf, zero gradients.
"""
from __future__ import annotations

import numpy as np

f64 = lambda a: np.asarray(a, np.float64)  # noqa: E731


def rotate(x, pos, inv_freq, sign=1.0):
    """x [..., H, dh] rotated by positions pos [...]: pairs (i, i + rot/2), rot = 2 len(inv_freq)."""
    x = f64(x)
    h = len(inv_freq)
    phi = sign * f64(pos)[..., None, None] * f64(inv_freq)
    c, s = np.cos(phi), np.sin(phi)
    a, b = x[..., :h], x[..., h:2 * h]
    return np.concatenate([a * c - b * s, b * c + a * s, x[..., 2 * h:]], -1)


def norm_rope(x, w, pos, inv_freq, eps):
    x = f64(x)
    if w is not None:
        x = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * f64(w)
    return rotate(x, pos, inv_freq)


def norm_rope_backward(x, w, pos, inv_freq, eps, dy):
    """(dx, dw) for the gradient dy of norm_rope; dw None without weights."""
    g = rotate(dy, pos, inv_freq, -1.0)
    if w is None:
        return g, None
    x, w = f64(x), f64(w)
    r = 1.0 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    xh, t = x * r, g * w
    dx = r * (t - xh * np.mean(t * xh, -1, keepdims=True))
    return dx, (g * xh).reshape(-1, x.shape[-1]).sum(0)


def visible(n, window, sinks):
    t, u = np.arange(n)[:, None], np.arange(n)[None]
    return (u <= t) & ((u > t - window) | (u < sinks))


def _probs(q, k, scale, see):
    s = np.where(see, scale * (q @ k.T), -np.inf)
    m = s.max(1, keepdims=True)
    e = np.exp(s - m)
    l = e.sum(1, keepdims=True)
    return e / l, (m + np.log(l))[:, 0]


def attention(q, k, v, window, sinks=0, lens=None, scale=None):
    """q [B,T,Hq,dh], k, v [B,T,Hkv,dh] -> o [B,T,Hq,dh], lse [B,Hq,T]."""
    q, k, v = f64(q), f64(k), f64(v)
    B, T, Hq, dh = q.shape
    G = Hq // k.shape[2]
    scale = scale or 1.0 / np.sqrt(dh)
    o, lse = np.zeros(q.shape), np.full((B, Hq, T), -np.inf)
    for b in range(B):
        n = T if lens is None else min(max(int(lens[b]), 0), T)
        if not n:
            continue
        see = visible(n, window, sinks)
        for h in range(Hq):
            p, lse[b, h, :n] = _probs(q[b, :n, h], k[b, :n, h // G], scale, see)
            o[b, :n, h] = p @ v[b, :n, h // G]
    return o, lse


def attention_backward(q, k, v, do, window, sinks=0, lens=None, scale=None):
    """(dq, dk, dv) for the gradient do of o."""
    q, k, v, do = f64(q), f64(k), f64(v), f64(do)
    B, T, Hq, dh = q.shape
    G = Hq // k.shape[2]
    scale = scale or 1.0 / np.sqrt(dh)
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    for b in range(B):
        n = T if lens is None else min(max(int(lens[b]), 0), T)
        if not n:
            continue
        see = visible(n, window, sinks)
        for h in range(Hq):
            g = h // G
            p, _ = _probs(q[b, :n, h], k[b, :n, g], scale, see)
            dp = do[b, :n, h] @ v[b, :n, g].T
            ds = p * (dp - (p * dp).sum(1, keepdims=True))
            dq[b, :n, h] = scale * ds @ k[b, :n, g]
            dk[b, :n, g] += scale * ds.T @ q[b, :n, h]
            dv[b, :n, g] += p.T @ do[b, :n, h]
    return dq, dk, dv


def attention_bounds(q, k, v, do, window, sinks=0, lens=None, scale=None):
    """Elementwise bounds of the errors of a computation of o, dq, dk, dv with bf16 inputs, fp32
    sums and exponentials, and P, dS, o and the results rounded to bf16, each rounding off by at most
    u = 2^-8 of the value (w = 2^-24 in fp32). With A = scale |q| |k|^T, the scores' error is at most
    (dh + 2) w A, so P's relative error is rp <= 2 (dh + 2) w max A + (n + 8) 2 w before its own
    rounding, and:
      lse: rp, then 4 w |lse|;
      o:  (rp + u) P |v|, then u |o|;
      dp: (dh + 2) w |do| |v|^T;  delta: |do| . (o's error), plus (dh + 2) w |do| . |o|;
      dS: rp |dS| + P (dp's error + delta's error), then u |dS|;
      dq: scale dS's error |k| (+ (n + 2) w of its terms), then u |dq|; dk alike over the heads' rows;
      dv: (rp + u) P^T |do| (+ (n + 2) w of its terms), then u |dv|.
    Returns the bounds of (lse, o, dq, dk, dv); do None: the last three None."""
    q, k, v = f64(q), f64(k), f64(v)
    B, T, Hq, dh = q.shape
    G = Hq // k.shape[2]
    scale = scale or 1.0 / np.sqrt(dh)
    u, w = 2.0 ** -8, 2.0 ** -24
    eo, eq, ek, ev = (np.zeros(x.shape) for x in (q, q, k, v))
    dq = dk = dv = None
    if do is not None:
        do = f64(do)
        dq, dk, dv = attention_backward(q, k, v, do, window, sinks, lens, scale)
    o, lse = attention(q, k, v, window, sinks, lens, scale)
    el = np.zeros(lse.shape)
    for b in range(B):
        n = T if lens is None else min(max(int(lens[b]), 0), T)
        if not n:
            continue
        see = visible(n, window, sinks)
        for h in range(Hq):
            g = h // G
            qq, kk, vv = q[b, :n, h], k[b, :n, g], v[b, :n, g]
            p, _ = _probs(qq, kk, scale, see)
            A = np.where(see, scale * np.abs(qq) @ np.abs(kk).T, 0.0).max(1, keepdims=True)
            rp = 2 * (dh + 2) * w * A + (n + 8) * 2 * w
            el[b, h, :n] = rp[:, 0] + 4 * w * np.abs(lse[b, h, :n])
            eo[b, :n, h] = (rp + u) * (p @ np.abs(vv)) * (1 + u) + u * np.abs(o[b, :n, h])
            if do is None:
                continue
            dd = do[b, :n, h]
            dp = dd @ vv.T
            delta = (p * dp).sum(1, keepdims=True)
            ds = p * (dp - delta)
            edp = (dh + 2) * w * (np.abs(dd) @ np.abs(vv).T)
            edl = (np.abs(dd) * (eo[b, :n, h] + (dh + 2) * w * np.abs(o[b, :n, h]))).sum(1, keepdims=True)
            eds = (rp * np.abs(ds) + p * (1 + rp) * (edp + edl)) * (1 + u) + u * np.abs(ds)
            sums = (n + 2) * w * np.abs(ds)
            eq[b, :n, h] = scale * (eds + sums) @ np.abs(kk)
            ek[b, :n, g] += scale * (eds + G * sums).T @ np.abs(qq)
            ev[b, :n, g] += ((rp + u + G * (n + 2) * w) * p * (1 + u)).T @ np.abs(dd)
    if do is not None:
        eq, ek, ev = (e * (1 + u) + u * np.abs(x) for e, x in ((eq, dq), (ek, dk), (ev, dv)))
        return el, eo, eq, ek, ev
    return el, eo, None, None, None


def paged_attention(q, k_pages, v_pages, table, lens, window, sinks=0, scale=None):
    """q [N,Hq,dh] over the pages' visible tokens -> o [N,Hq,dh]; beside it
    sum_u p_u |v_u| [N,Hq,dh] and max_u scale |q| |k_u| [N,Hq,1], which the error bounds need."""
    q, k_pages, v_pages = f64(q), f64(k_pages), f64(v_pages)
    N, Hq, dh = q.shape
    page, G = k_pages.shape[1], Hq // k_pages.shape[2]
    scale = scale or 1.0 / np.sqrt(dh)
    o, mag, most = np.zeros(q.shape), np.zeros(q.shape), np.zeros((N, Hq, 1))
    for n in range(N):
        u = np.arange(int(lens[n]))
        u = u[(u >= int(lens[n]) - window) | (u < sinks)]
        if not len(u):
            continue
        at = np.asarray(table)[n][u // page]
        kk, vv = k_pages[at, u % page], v_pages[at, u % page]
        for h in range(Hq):
            p, _ = _probs(q[n, h][None], kk[:, h // G], scale, np.ones((1, len(u)), bool))
            o[n, h] = p[0] @ vv[:, h // G]
            mag[n, h] = p[0] @ np.abs(vv[:, h // G])
            most[n, h] = scale * (np.abs(kk[:, h // G]) @ np.abs(q[n, h])).max()
    return o, mag, most
