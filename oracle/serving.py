"""fp64 CPU oracle of the serving operators: the e4m3 cache, attention of one token per sequence behind a shared prefix,
and linear attention with a decay for each head.

TEST INFRASTRUCTURE ONLY, as the other oracles here: it never imports the product and the product never imports it.
Plain numpy in fp64, loops over sequences, heads and tokens.
"""
from __future__ import annotations

import numpy as np

from .attention_block import f64, paged_attention


# ------------------------------------------------------------------------------------------- e4m3 cache
def scale_exponent(x):
    """The exponent of s for rows x [..., dh]: s = max(2^-117, the smallest 2^e with max |x| / 2^e <= 448)."""
    top = np.abs(f64(x)).max(-1)
    e = np.full(top.shape, -117)
    while (big := top > 448.0 * np.exp2(e.astype(np.float64))).any():
        e = e + big
    return e


E4M3 = np.array([(m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])  # codes 0 .. 126, ascending; 127 is NaN


def codes(y):
    """The e4m3 codes (0 .. 126, and 128 more for negative ones) nearest to y, ties to the even code."""
    a = np.abs(f64(y))
    hi = np.minimum(np.searchsorted(E4M3, a), 126)
    lo = np.maximum(hi - 1, 0)
    up, down = E4M3[hi] - a, a - E4M3[lo]
    c = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (c + 128 * np.signbit(f64(y))).astype(np.uint8)


def quantize(x):
    """(codes [..., dh] uint8, scale bytes [...] uint8) of rows x; NaN codes and scale where a row is not finite."""
    x = f64(x)
    ok = np.isfinite(x).all(-1)
    safe = np.where(ok[..., None], x, 0.0)
    e = scale_exponent(safe)
    c = codes(safe / np.exp2(e.astype(np.float64))[..., None])
    return np.where(ok[..., None], c, 127).astype(np.uint8), np.where(ok, e + 127, 255).astype(np.uint8)


def values(c, scales):
    """What codes and scale bytes stand for."""
    c, b = np.asarray(c), np.asarray(scales)
    table = np.concatenate([E4M3, [np.nan]])
    v = table[c & 127] * np.where(c & 128, -1.0, 1.0)
    return v * np.where(b == 255, np.nan, np.exp2(b.astype(np.float64) - 127))[..., None]


# --------------------------------------------------------------------------------------- shared prefix
def prefix_attention(q, k_pages, v_pages, prefix_table, prefix_len, table, lens, window, sinks=0, scale=None):
    """As attention_block.paged_attention (o, sum p |v|, max scale |q| |k|), sequence n's tokens being the prefix's
    and then its own: each is laid out afresh in pages of one token."""
    k_pages, v_pages = f64(k_pages), f64(v_pages)
    page, P = k_pages.shape[1], int(prefix_len)
    width = P + int(max(lens)) if len(lens) else P
    flat_k, flat_v = (x.reshape(-1, 1, *x.shape[2:]) for x in (k_pages, v_pages))
    rows = np.zeros((len(lens), max(width, 1)), np.int64)
    u = np.arange(P)
    for n, own in enumerate(lens):
        j = np.arange(int(own))
        rows[n, :P] = np.asarray(prefix_table)[u // page] * page + u % page
        rows[n, P:P + int(own)] = np.asarray(table)[n][j // page] * page + j % page
    return paged_attention(q, flat_k, flat_v, rows, P + np.asarray(lens), window, sinks, scale)


# ------------------------------------------------------------------------------------ linear attention
LEAST = -104.0  # smaller log decays count as this (exp of it is below 2^-149)


def linear_attention(q, k, v, log_decay, state=None, lens=None, scale=None):
    """q, k [B,T,Hk,dk], v [B,T,H,dv], log_decay [H] or [B,T,H] -> o [B,T,H,dv], state [B,H,dk,dv], and both again
    with absolute values for all inputs (what the error bounds need): the recurrence, token by token."""
    q, k, v = f64(q), f64(k), f64(v)
    B, T, Hk, dk = q.shape
    H, dv = v.shape[2:]
    scale = scale or 1.0 / np.sqrt(dk)
    g = np.maximum(np.broadcast_to(f64(log_decay), (B, T, H)), LEAST)
    s = np.zeros((B, H, dk, dv)) if state is None else f64(state).copy()
    a = np.abs(s)
    o, ao = np.zeros(v.shape), np.zeros(v.shape)
    group = np.arange(H) // (H // Hk)
    for b in range(B):
        n = T if lens is None else min(max(int(lens[b]), 0), T)
        for t in range(n):
            keep = np.exp(g[b, t])[:, None, None]
            kv = k[b, t, group][:, :, None] * v[b, t][:, None, :]
            s[b] = keep * s[b] + kv
            a[b] = keep * a[b] + np.abs(kv)
            o[b, t] = scale * (q[b, t, group][:, None, :] @ s[b])[:, 0]
            ao[b, t] = scale * (np.abs(q[b, t, group])[:, None, :] @ a[b])[:, 0]
    return o, s, ao, a
