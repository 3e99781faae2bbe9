"""fp64 oracle of attention with a window that keeps the first keys (sinks),
over keys that lie anywhere in a cache, and of its gradients -- TEST
INFRASTRUCTURE ONLY.

The logits are those of the page "SGLang and Miles Add Day-0 Support for
Inkling", section "Attention with Relative Positional Embedding":
    x(i, j) = s(i) (alpha q_i . k_j + [0 <= i-j < E] r_i . P[:, i-j]),
    s(i) = max(1, ln(i+1) / ln(base)),
seen where 0 <= i-j and (no window, i-j < window, or j < sink).  Sinks, and
chunks over pages, are not on the pages.

Plain numpy, one query head at a time, every pair of the matrix.  Beside each
result the functions give the sum of the magnitudes of its terms, by which the
tests bound roundings.
"""
from __future__ import annotations

import numpy as np


def f64(x):
    return None if x is None else x.detach().cpu().double().numpy()


def logits(q, k, r, P, first, *, alpha, window, sink, base):
    """(x, magnitude of its products, visible, distances, s) of rows q [n, 128]
    at positions first .. against keys k [m, 128] at 0 .. m - 1."""
    i = first + np.arange(len(q))
    d = i[:, None] - np.arange(len(k))[None, :]
    x, mag = alpha * (q @ k.T), abs(alpha) * (np.abs(q) @ np.abs(k).T)
    if P is not None and P.size:
        near = (d >= 0) & (d < P.shape[1])
        at = np.clip(d, 0, P.shape[1] - 1)
        x = x + np.where(near, np.take_along_axis(r @ P, at, 1), 0)
        mag = mag + np.where(near, np.take_along_axis(np.abs(r) @ np.abs(P), at, 1), 0)
    s = np.maximum(1.0, np.log(i + 1.0) / np.log(base)) if base > 1 else np.ones(len(q))
    seen = d >= 0
    if window > 0:
        seen &= (d < window) | (np.arange(len(k)) < sink)[None, :]
    return x * s[:, None], mag * s[:, None], seen, d, s


def sequences(where, q_lens):
    a = 0
    for w, n in zip(where, q_lens):
        yield w, slice(a, a + n), len(w) - n
        a += n


def forward(q, k, v, r, P, where, q_lens, **kw):
    """out [Tq, Hq, 128], lse [Hq, Tq], sum p |v| [Tq, Hq, 128] and the largest
    magnitude of a row's logit [Hq, Tq].  where[b]: cache rows of sequence b's keys."""
    q, k, v, r, P = (f64(t) for t in (q, k, v, r, P))
    Tq, Hq, D = q.shape
    g = Hq // k.shape[1]
    out, size = np.zeros((Tq, Hq, D)), np.zeros((Tq, Hq, D))
    lse, top = np.full((Hq, Tq), -np.inf), np.zeros((Hq, Tq))
    for w, at, first in sequences(where, q_lens):
        for h in range(Hq):
            x, mag, seen, _, _ = logits(q[at, h], k[w, h // g], None if r is None else r[at, h], P, first, **kw)
            x = np.where(seen, x, -np.inf)
            if x.size == 0:
                continue
            m = x.max(1, keepdims=True)
            p = np.exp(x - m)
            z = p.sum(1, keepdims=True)
            p /= z
            out[at, h], size[at, h] = p @ v[w, h // g], p @ np.abs(v[w, h // g])
            lse[h, at], top[h, at] = (m + np.log(z))[:, 0], np.where(seen, mag, 0).max(1)
    return out, lse, size, top


def backward(q, k, v, r, P, out, lse, dout, where, q_lens, **kw):
    """Gradients of sum(dout * out) from the saved out / lse, {name: (value,
    sum of the magnitudes of its terms)} for dq, dk, dv, dr."""
    alpha = kw["alpha"]
    q, k, v, r, P, out, lse, dout = (f64(t) for t in (q, k, v, r, P, out, lse, dout))
    Hq = q.shape[1]
    g = Hq // k.shape[1]
    res = {n: (np.zeros(t.shape), np.zeros(t.shape)) for n, t in (("dq", q), ("dk", k), ("dv", v))}
    if P is not None and P.size:
        res["dr"] = (np.zeros(r.shape), np.zeros(r.shape))
    for w, at, first in sequences(where, q_lens):
        for h in range(Hq):
            c = h // g
            x, _, seen, d, s = logits(q[at, h], k[w, c], None if r is None else r[at, h], P, first, **kw)
            p = np.where(seen, np.exp(np.where(seen, x - lse[h, at][:, None], 0)), 0)
            do = dout[at, h]
            dp, D = do @ v[w, c].T, (do * out[at, h]).sum(1, keepdims=True)
            # terms of dl and their magnitudes before the difference cancels
            dl = p * (dp - D) * s[:, None]
            big = np.abs(dl) + 2.0 ** -8 * p * (np.abs(do) @ np.abs(v[w, c]).T + (np.abs(do) * np.abs(out[at, h])).sum(1, keepdims=True)) * s[:, None]
            for n, val, mag in (("dq", alpha * dl @ k[w, c], abs(alpha) * big @ np.abs(k[w, c])),):
                res[n][0][at, h] += val
                res[n][1][at, h] += mag
            for n, val, mag in (("dk", alpha * dl.T @ q[at, h], abs(alpha) * big.T @ np.abs(q[at, h])),
                                ("dv", p.T @ do, p.T @ np.abs(do))):
                res[n][0][w, c] += val
                res[n][1][w, c] += mag
            if "dr" in res:
                near = (d >= 0) & (d < P.shape[1])
                by, byb = np.zeros((len(q[at]), P.shape[1])), np.zeros((len(q[at]), P.shape[1]))
                rows = np.broadcast_to(np.arange(d.shape[0])[:, None], d.shape)
                np.add.at(by, (rows[near], d[near]), dl[near])
                np.add.at(byb, (rows[near], d[near]), big[near])
                res["dr"][0][at, h] += by @ P.T
                res["dr"][1][at, h] += byb @ np.abs(P).T
    return res
