"""CPU oracle for rotary positions, the paged cache's append and the attention
over it.

TEST INFRASTRUCTURE ONLY, like the rest of ``oracle``.  Plain definitions in
float64 numpy, one sequence and head at a time:

* rotation: pair (a, b) of a head at position t turns by t * inv_freq[i]:
  a' = m (a cos - b sin), b' = m (a sin + b cos); the backward negates the angle;
* append: new token i of a sequence with q_len new tokens and kv keys in all
  goes to key position kv - q_len + i: page table[pos // P], slot pos % P;
* attention: token at position t keeps keys j <= t (causal) and j > t - window
  (window > 0) of its sequence; s_j = scale q.k_j; out = softmax(s) v, taken
  over kept keys only (a key that is not kept never enters, whatever it
  holds); nothing kept: out = 0, lse = -inf.
"""
from __future__ import annotations

import math

import numpy as np


def angles(positions, inv_freq):
    """fp64 angles reduced modulo 2 pi from extended-precision products."""
    p = np.asarray(positions).astype(np.longdouble)[..., None]
    two_pi = 2 * np.pi + np.longdouble(2.4492935982947064e-16)  # 2 pi beyond fp64
    turns = p * (np.asarray(inv_freq, np.float64).astype(np.longdouble) / two_pi)
    return ((turns - np.rint(turns)) * two_pi).astype(np.float64)


def rotate(x, positions, inv_freq, layout="half", mscale=1.0, backward=False):
    """x [..., heads, dim], positions [...]."""
    x = np.asarray(x, np.float64)
    r = 2 * len(inv_freq)
    a = angles(positions, inv_freq)[..., None, :]
    c, s = mscale * np.cos(a), mscale * np.sin(a) * (-1.0 if backward else 1.0)
    y = x.copy()
    lo = slice(0, r // 2) if layout == "half" else slice(0, r, 2)
    hi = slice(r // 2, r) if layout == "half" else slice(1, r, 2)
    y[..., lo] = x[..., lo] * c - x[..., hi] * s
    y[..., hi] = x[..., lo] * s + x[..., hi] * c
    return y


def slots(cu, kv_lens, table, page):
    """(token row, position, page, slot) of every new token."""
    for b, kv in enumerate(kv_lens):
        n = cu[b + 1] - cu[b]
        for i in range(n):
            t = kv - n + i
            yield cu[b] + i, t, int(table[b][t // page]), t % page


def attend(q, k, v, kv_off, scale, causal=True, window=0):
    """One sequence and head: q [n, d], k, v [kv, d]; token i stands at kv_off + i.
    Returns (out [n, d], lse [n], weight [n, d] = softmax(s) |v|)."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    n, kv = q.shape[0], k.shape[0]
    out = np.zeros((n, v.shape[1]))
    mag = np.zeros((n, v.shape[1]))
    lse = np.full(n, -np.inf)
    for i in range(n):
        t = kv_off + i
        hi = min(kv, t + 1) if causal else kv
        lo = max(0, t - window + 1) if window > 0 else 0
        if hi <= lo:
            continue
        s = scale * (k[lo:hi] @ q[i])
        m = s.max()
        p = np.exp(s - m)
        lse[i] = m + math.log(p.sum())
        p /= p.sum()
        out[i] = p @ v[lo:hi]
        mag[i] = p @ np.abs(v[lo:hi])
    return out, lse, mag


def paged_attend(q, k_cache, v_cache, cu, kv_lens, table, scale, causal=True, window=0,
                 k_scale_inv=1.0, v_scale_inv=1.0):
    """q [tokens, heads, d], caches [pages, P, kv_heads, d] (values).  Returns
    (out, lse, mag); rows of no sequence stay 0 / -inf."""
    q = np.asarray(q, np.float64)
    page, hk = k_cache.shape[1], k_cache.shape[2]
    hq = q.shape[1]
    out, mag = np.zeros_like(q), np.zeros_like(q)
    lse = np.full(q.shape[:2], -np.inf)
    for b, kv in enumerate(kv_lens):
        n = cu[b + 1] - cu[b]
        if n == 0:
            continue
        first = max(0, kv - n - window + 1) // page * page if window > 0 else 0
        pos = np.arange(first, kv)
        pg = np.asarray([table[b][t // page] for t in pos], dtype=np.int64)
        rows = slice(cu[b], cu[b + 1])
        for h in range(hk):
            kk = np.asarray(k_cache[pg, pos % page, h], np.float64) * k_scale_inv
            vv = np.asarray(v_cache[pg, pos % page, h], np.float64) * v_scale_inv
            for g in range(hq // hk):
                hh = h * (hq // hk) + g
                o, l, m = attend(q[rows, hh], kk, vv, kv - n - first, scale, causal, window)
                out[rows, hh], lse[rows, hh], mag[rows, hh] = o, l, m
    return out, lse, mag
