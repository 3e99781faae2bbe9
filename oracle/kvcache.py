"""fp64 oracle of the compressed K / V cache -- TEST INFRASTRUCTURE ONLY.

NVFP4 rows (E2M1 codes, an E4M3 scale per 16 dims, an fp32 factor per kv
head), relative attention over keys with explicit positions and the weight
each key receives, and the choice eviction makes.  Plain numpy, written from
the definitions; it shares nothing with the CUDA library.
"""
from __future__ import annotations

import math

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# every finite E4M3 magnitude by its code: 3 mantissa bits, bias 7, 0x7f is NaN
E4M3 = np.array([m / 512.0 for m in range(8)] +
                [(1 + m / 8.0) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8) if (e, m) != (15, 7)])


def _nearest(a: np.ndarray, grid: np.ndarray, unit) -> np.ndarray:
    """Index of the grid value nearest to a / unit (a >= 0), a tie to the even
    index.  a is compared with border * unit, which is exact in float64."""
    border = (grid[1:] + grid[:-1]) / 2
    out = np.zeros(a.shape, dtype=np.int64)
    for i, b in enumerate(border):
        edge = b * unit
        out += (a > edge) | ((a == edge) & (i % 2 == 1))
    return out


def quantize_nvfp4(x, factor=None):
    """x float [n, H, 128] (bf16 values), factor [H] -> (codes uint8 [n, H, 64],
    scales uint8 [n, H, 8])."""
    x = np.asarray(x, dtype=np.float32)
    n, H, D = x.shape
    with np.errstate(invalid="ignore", over="ignore"):
        t = x if factor is None else x / np.asarray(factor, np.float32)[None, :, None]
        t = t.astype(np.float64).reshape(n, H, D // 16, 16)
        top = np.abs(t).max(-1)                       # NaN if any is
        nan = np.isnan(top)
        scode = _nearest(np.where(nan, 0, top), E4M3, 6.0)
        s = E4M3[scode][..., None]
        code = np.where(s > 0, _nearest(np.abs(np.where(np.isnan(t), 0, t)), E2M1, s), 0)
    code = np.where(s > 0, code + 8 * np.signbit(t), 0).astype(np.uint8).reshape(n, H, D)
    scale = np.where(nan, 0x7F, scode).astype(np.uint8)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8), scale


def dequantize_nvfp4(codes, scales, factor=None):
    """float64 [n, H, 128]."""
    codes, scales = np.asarray(codes), np.asarray(scales)
    nib = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    v = np.where(nib & 8, -E2M1[nib & 7], E2M1[nib & 7])
    s = np.append(E4M3, np.nan)[scales & 0x7F] * np.where(scales & 0x80, -1.0, 1.0)
    v = v * np.repeat(s, 16, -1)
    return v if factor is None else v * np.asarray(factor, np.float64)[None, :, None]


def logits(q, k, r, P, q_pos, k_pos, *, alpha, window=0, base=0.0):
    """Masked logits of one query head: q [Lq, 128], k [Lk, 128], r [Lq, c] or
    None, positions [Lq], [Lk].  Returns (x [Lq, Lk], largest magnitude sum of
    a row's products: what rounding errors of its logits are relative to)."""
    q, k = np.asarray(q, np.float64), np.asarray(k, np.float64)
    d = np.asarray(q_pos)[:, None] - np.asarray(k_pos)[None, :]
    seen = (d >= 0) & (np.asarray(k_pos)[None, :] >= 0)
    if window > 0:
        seen &= d < window
    with np.errstate(invalid="ignore"):
        x = alpha * (q @ k.T)
        mag = abs(alpha) * (np.abs(q) @ np.abs(k).T)
    if r is not None:
        R = np.asarray(r, np.float64) @ np.asarray(P, np.float64)
        M = np.abs(np.asarray(r, np.float64)) @ np.abs(np.asarray(P, np.float64))
        E = R.shape[1]
        inside = (d >= 0) & (d < E)
        c = np.clip(d, 0, E - 1)
        x = x + np.where(inside, np.take_along_axis(R, c, 1), 0.0)
        mag = mag + np.where(inside, np.take_along_axis(M, c, 1), 0.0)
    if base > 0:
        s = np.maximum(1.0, np.log(np.asarray(q_pos, np.float64) + 1) / math.log(base))[:, None]
        x, mag = x * s, mag * s
    return np.where(seen, x, -np.inf), np.where(seen, mag, 0.0)


def softmax(x):
    """(weights [Lq, Lk], lse [Lq]); rows that see nothing: zeros and -inf."""
    m = x.max(1, initial=-np.inf)
    with np.errstate(invalid="ignore"):
        e = np.exp(x - np.where(np.isneginf(m), 0.0, m)[:, None])
        e = np.where(np.isneginf(x), 0.0, e)
        z = e.sum(1)
        lse = np.where(z == 0, -np.inf, np.where(np.isneginf(m), 0.0, m) + np.log(np.where(z == 0, 1.0, z)))
        return e / np.where(z == 0, 1.0, z)[:, None], lse


def kept_keys(weights, keep, recent, sink):
    """Ascending indices that eviction keeps of one (sequence, kv head)."""
    w = np.asarray(weights, np.float64)
    n = len(w)
    recent = min(recent, keep)
    sink = min(sink, keep - recent, n - recent)
    mid = np.arange(sink, n - recent)
    v = w[mid]
    nan = np.isnan(v)
    mid = mid[np.lexsort((mid, -np.where(nan, 0.0, v), nan))]      # numbers first, heaviest first, lower index first
    return np.sort(np.concatenate([np.arange(sink), mid[:keep - recent - sink], np.arange(n - recent, n)])).astype(np.int64)
