"""Inputs and checks shared by the tests of the compressed K / V cache."""
from __future__ import annotations

import dataclasses

import numpy as np
import torch

import relative_position_biased_gb300 as rpb
from oracle import kvcache as C
from relative_position_biased_gb300 import workloads as W


@dataclasses.dataclass
class Case:
    q_lens: tuple
    k_lens: tuple
    Hq: int
    Hkv: int
    r_dim: int = 16
    E: int = 64
    window: int = 0
    base: float = 0.0
    page: int = 0
    positions: bool = False
    factors: bool = True
    sign: float = 1.0        # of the logit scale
    seed: int = 0

    @property
    def alpha(self):
        return self.sign * (1 / np.sqrt(128))


def rows_of(lens, page, seed):
    """(cache rows, block table or None, [row of every key] per sequence);
    a paged pool has spare pages and a shuffled order."""
    if page == 0:
        starts = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
        return int(starts[-1]), None, [np.arange(starts[i], starts[i + 1]) for i in range(len(lens))]
    counts = [(n + page - 1) // page for n in lens]
    perm = np.random.default_rng(seed).permutation(sum(counts) + 2)
    table = np.full((len(lens), max(1, max(counts, default=1))), -1, np.int32)
    used, rows = 0, []
    for b, n in enumerate(lens):
        table[b, :counts[b]] = perm[used:used + counts[b]]
        used += counts[b]
        p = np.arange(n)
        rows.append(table[b][p // page].astype(np.int64) * page + p % page if n else np.zeros(0, np.int64))
    return (sum(counts) + 2) * page, torch.from_numpy(table), rows


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16)


def make(c: Case):
    """CPU inputs: q, r, P, bf16 K / V rows of the cache, positions, where every
    key lies."""
    rng = np.random.default_rng(c.seed)
    Tq = sum(c.q_lens)
    rows, table, where = rows_of(c.k_lens, c.page, c.seed + 1)
    d = dict(rows=rows, table=table, where=where, cu_q=W.cu_seqlens(c.q_lens), cu_k=W.cu_seqlens(c.k_lens))
    d["q"] = bf16(rng.standard_normal((Tq, c.Hq, 128)))
    d["r"] = bf16(rng.standard_normal((Tq, c.Hq, c.r_dim))) if c.E else None
    d["P"] = bf16(0.1 * rng.standard_normal((c.r_dim, c.E))) if c.E else None
    d["k"] = bf16(rng.standard_normal((rows, c.Hkv, 128)))
    d["v"] = bf16(0.5 * rng.standard_normal((rows, c.Hkv, 128)))
    d["kg"] = np.linspace(0.003, 0.01, c.Hkv).astype(np.float32) if c.factors else None
    d["vg"] = np.linspace(0.002, 0.001, c.Hkv).astype(np.float32) if c.factors else None
    if c.positions:
        kp = np.full((c.Hkv, rows), -1, np.int32)
        qp = []
        for b, (nq, nk) in enumerate(zip(c.q_lens, c.k_lens)):
            # the newest half in a run, gaps before; every seventh older key hidden
            new = min(nk, max(nq, nk // 2))
            for h in range(c.Hkv):
                old = np.cumsum(rng.integers(1, 9, nk - new))
                first = 8 * (nk - new) + 1
                p = np.concatenate([old, first + np.arange(new)])
                p[:nk - new][::7] = -1
                kp[h, where[b]] = p
            qp.append(8 * (nk - new) + 1 + new - nq)
        d["key_pos"], d["q_pos"] = torch.from_numpy(kp), torch.tensor(qp, dtype=torch.int32)
    return d


def quantized(c: Case, d):
    """Host cache (numpy codes and scales) of d's K / V rows, and the values."""
    out = {}
    for n, g in (("k", d["kg"]), ("v", d["vg"])):
        out[n], out[n + "_scale"] = C.quantize_nvfp4(d[n].float().numpy(), g)
        out[n + "_values"] = C.dequantize_nvfp4(out[n], out[n + "_scale"], g)
    return out


def device_cache(qc, d):
    t = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    return rpb.KvNvfp4(t(qc["k"]), t(qc["v"]), t(qc["k_scale"]), t(qc["v_scale"]), t(d["kg"]), t(d["vg"]))


def cuda(x):
    return None if x is None else x.cuda()


def call_kw(c: Case, d):
    kw = dict(max_seqlen_q=max(c.q_lens), max_seqlen_k=max(c.k_lens), alpha=c.alpha, window=c.window,
              log_scale_base=c.base, total_k=sum(c.k_lens))
    if c.page:
        kw.update(block_table=d["table"].cuda(), page_size=c.page)
    if c.positions:
        kw.update(key_pos=d["key_pos"].cuda(), q_pos=d["q_pos"].cuda())
    return kw


def each_head(c: Case, d, keys):
    """Yields (b, query head, kv head, first query row, logits, magnitudes) in fp64;
    keys [rows, Hkv, 128]."""
    q0 = 0
    for b, (nq, nk) in enumerate(zip(c.q_lens, c.k_lens)):
        for hq in range(c.Hq):
            h = hq // (c.Hq // c.Hkv)
            if c.positions:
                qp = int(d["q_pos"][b]) + np.arange(nq)
                kp = d["key_pos"][h].numpy()[d["where"][b]].astype(np.int64)
            else:
                qp, kp = np.arange(nk - nq, nk), np.arange(nk)
            f = lambda t: t[q0:q0 + nq, hq].double().numpy()  # noqa: E731
            x, mag = C.logits(f(d["q"]), keys[d["where"][b], h], f(d["r"]) if c.E else None,
                              d["P"].double().numpy() if c.E else None, qp, kp, alpha=c.alpha, window=c.window,
                              base=c.base)
            yield b, hq, h, q0, x, mag
        q0 += nq


# A logit is a sum of at most 128 + 64 products of exact operands, scaled and
# shifted a few times: in fp32, whatever the order and with truncating adds (a
# whole step of 2^-23 each), it is off by less than 200 * 2^-23 of the sum of
# its products' magnitudes.
LOGIT = 200 * 2.0 ** -23


def check_decode(c: Case, d, keys, values, out, lse):
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, hq, h, q0, x, mag in each_head(c, d, keys):
        nq = x.shape[0]
        p, z = C.softmax(x)
        v = values[d["where"][b], h]
        ref = p @ np.where((p > 0).any(0)[:, None], v, 0.0)
        spread = p @ np.abs(np.where((p > 0).any(0)[:, None], v, 0.0))
        dx = LOGIT * mag.max(1, initial=0.0)
        got, got_z = out[q0:q0 + nq, hq], lse[hq, q0:q0 + nq]
        empty = np.isneginf(z)
        assert (np.isneginf(got_z) == empty).all() and (got[empty] == 0).all()
        # softmax sums: exp2 to 2^-21, up to n adds of 2^-24 in the worst order,
        # of which a lane sees one in 128
        sums = 2.0 ** -21 + (x.shape[1] / 128 + 64) * 2.0 ** -24
        ok = ~empty
        assert (np.abs(got_z - z)[ok] <= (dx + sums + 2.0 ** -22 * np.abs(z))[ok]).all(), \
            (b, hq, np.abs(got_z - z)[ok].max())
        # weights are rounded to f16 (2^-11, below its range 2^-25 / 2^7 of the
        # largest), the result to bf16 (2^-8)
        tol = spread * (2.0 ** -11 + 2 * dx + 2 * sums)[:, None] + np.abs(v).max(initial=0) * x.shape[1] * 2.0 ** -32
        tol = tol * (1 + 2.0 ** -8) + np.abs(ref) * 2.0 ** -8 + 1e-30
        assert (np.abs(got - ref) <= tol)[ok].all(), (b, hq, (np.abs(got - ref) / tol)[ok].max())


def check_weights(c: Case, d, keys, lse, w_in, decay, got):
    """lse [Hq, Tq] as given to the call; got [Hkv, rows]."""
    got = got.double().cpu().numpy()
    want = np.zeros_like(got)
    tol = np.zeros_like(got)
    held = np.zeros(got.shape[1], bool)
    for b, (nq, nk) in enumerate(zip(c.q_lens, c.k_lens)):
        at = d["where"][b]
        held[at] = True
        if w_in is not None and decay != 0:
            old = at[:nk - nq]
            want[:, old] = decay * w_in[:, old].astype(np.float64)
            tol[:, old] = np.abs(want[:, old]) * 2.0 ** -23
    group = c.Hq // c.Hkv
    for b, hq, h, q0, x, mag in each_head(c, d, keys):
        nq = x.shape[0]
        z = lse[hq, q0:q0 + nq].astype(np.float64)[:, None]
        p = np.where(np.isneginf(x) | np.isneginf(z), 0.0, np.exp(np.where(np.isneginf(z), -np.inf, x - np.where(np.isneginf(z), 0, z))))
        want[h, d["where"][b]] += p.sum(0)
        # the logit's error, exp2 (its argument in base 2 carries 2^-23 of |x| + |lse|),
        # and nq * group adds
        rel = LOGIT * mag + 2.0 ** -21 + (np.abs(np.where(np.isneginf(x), 0, x)) + np.where(np.isneginf(z), 0, np.abs(z))) * 2.0 ** -22
        tol[h, d["where"][b]] += (p * (rel + (nq * group + 8) * 2.0 ** -24)).sum(0) * 1.01
    bad = np.abs(got - want) > tol + 1e-37
    assert not bad[:, held].any(), (np.abs(got - want) / (tol + 1e-37))[:, held].max()
    return held
