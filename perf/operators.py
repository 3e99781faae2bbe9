"""Cases for the compressed K / V cache: the 4-bit (NVFP4) cache with the
decode attention that reads it, the attention weight each cached key has
received, and eviction by that weight.

Formats and symbols
  cache    NVFP4: E2M1 codes [rows, Hkv, 64] (two per byte, low nibble first),
           E4M3 scales [rows, Hkv, 8] (one per 16 dims), an fp32 factor per kv
           head; a stored value is code * scale * factor.
  logits   x(i, j) = s(i) (alpha q_i . k_j + [0 <= d < E] r_i . P[:, d]),
           d = position of query i - position of key j, masked for d < 0 and
           (with a window) d >= window, s(i) = max(1, ln(i + 1) / ln(base)).
"""
import math

import numpy as np
import torch

own = False

D = 128
DEV = "cuda"

# ---------------------------------------------------------------- cases

# (operator, sizes).  Lengths are drawn from k_lo .. k_hi by len_seed.
_LISTED = [
    # one short conversation, one new token: the smallest call, latency counts
    dict(name="decode_one_short", op="decode", batch=1, q_len=1, k_lo=701, k_hi=701, Hq=4, Hkv=1, r_dim=32, E=64,
         window=0, base=0.0, page=0, evicted=False, len_seed=0),
    # a serving batch of full-attention layers, ragged lengths
    dict(name="decode_batch", op="decode", batch=64, q_len=1, k_lo=1024, k_hi=32768, Hq=16, Hkv=2, r_dim=64, E=1024,
         window=0, base=65536.0, page=0, evicted=False, len_seed=0),
    # the same batch in a sliding-window layer, paged cache
    dict(name="decode_paged_window", op="decode", batch=64, q_len=1, k_lo=1024, k_hi=32768, Hq=16, Hkv=2, r_dim=64,
         E=1024, window=4096, base=0.0, page=128, evicted=False, len_seed=0),
    # a 9-token verify step against a million keys
    dict(name="decode_verify_long", op="decode", batch=1, q_len=9, k_lo=1 << 20, k_hi=1 << 20, Hq=16, Hkv=2, r_dim=64,
         E=1024, window=0, base=65536.0, page=0, evicted=False, len_seed=0),
    # decode over a cache that eviction has thinned out: positions with gaps
    dict(name="decode_evicted", op="decode", batch=32, q_len=1, k_lo=2049, k_hi=8191, Hq=16, Hkv=2, r_dim=64, E=1024,
         window=0, base=65536.0, page=0, evicted=True, len_seed=1),
    # a prompt's rows go into the cache, and are read back for the next chunk
    dict(name="store_prompt", op="store", batch=4, q_len=8192, k_lo=8192, k_hi=8192, Hkv=2, page=0, len_seed=0),
    # one new token of every sequence of a batch, paged cache
    dict(name="store_tokens", op="store", batch=64, q_len=1, k_lo=1024, k_hi=8192, Hkv=2, page=128, len_seed=2),
    # the weights of a decode step over the 4-bit cache
    dict(name="weights_decode", op="weights", kind="nvfp4", batch=64, q_len=1, k_lo=1024, k_hi=32768, Hq=16, Hkv=2,
         r_dim=64, E=1024, window=0, base=65536.0, page=0, decay=0.96875, len_seed=0),
    # every row of a packed prompt votes, sliding-window layer
    dict(name="weights_prompt", op="weights", kind="bf16", batch=4, q_len=8192, k_lo=8192, k_hi=8192, Hq=16, Hkv=2,
         r_dim=64, E=1024, window=4096, base=0.0, page=0, decay=0.0, len_seed=0),
    # the last 32 rows of long prompts vote (full layer)
    dict(name="weights_observe", op="weights", kind="bf16", batch=4, q_len=32, k_lo=16384, k_hi=65536, Hq=16, Hkv=2,
         r_dim=64, E=1024, window=0, base=65536.0, page=0, decay=0.0, len_seed=0),
    # a serving batch's 4-bit paged cache is halved
    dict(name="evict_batch", op="evict", kind="nvfp4", batch=64, k_lo=1024, k_hi=32768, Hkv=2, keep=0.5, recent=1024,
         sink=4, page=128, len_seed=0),
    # a million-key bf16 cache shrinks to an eighth
    dict(name="evict_long", op="evict", kind="bf16", batch=1, k_lo=1 << 20, k_hi=1 << 20, Hkv=2, keep=0.125,
         recent=4096, sink=4, page=0, len_seed=0),
]


def listed():
    return [dict(c) for c in _LISTED]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "store", "weights", "weights", "evict"])
    Hq, Hkv = rng.choice([(16, 2), (8, 2), (4, 1), (8, 1), (16, 1), (12, 4), (4, 4)])
    page = rng.choice([0, 0, 64, 128, 256])
    seed = rng.randrange(1 << 20)
    batch = _log_int(rng, 1, 64)
    top = max(64, min(1 << 19, (1 << 20) // batch))        # keys of the batch stay below a million
    k_hi = _log_int(rng, 40, top)
    k_lo = max(33, k_hi // rng.randint(1, 16))
    k_hi = max(k_hi, k_lo)
    r_dim, E = rng.choice([(64, 1024), (32, 64), (16, 200), (0, 0), (64, 77), (24, 512)])
    window = rng.choice([0, 0, _log_int(rng, 16, 8192)])
    base = rng.choice([0.0, 65536.0, 64.0]) if window == 0 else 0.0
    if op == "decode":
        evicted = rng.random() < 0.3
        return dict(op=op, batch=batch, q_len=rng.choice([1, 1, 1, 2, 5, 9, 16]), k_lo=k_lo, k_hi=k_hi, Hq=Hq, Hkv=Hkv,
                    r_dim=r_dim, E=E, window=window, base=base, page=page, evicted=evicted, len_seed=seed)
    if op == "store":
        q_len = rng.choice([1, 1, 7, 33, k_lo])
        rows = min(q_len, max(1, 32768 // batch))
        return dict(op=op, batch=batch, q_len=min(rows, k_lo), k_lo=k_lo, k_hi=min(k_hi, max(k_lo, 16384)), Hkv=Hkv,
                    page=page, len_seed=seed)
    if op == "weights":
        kind = rng.choice(["bf16", "nvfp4"])
        q_len = rng.choice([1, 1, 4, 32, 64, 257, 2048])
        q_len = min(q_len, k_lo, max(1, (1 << 27) // (batch * k_hi)))
        return dict(op=op, kind=kind, batch=batch, q_len=q_len, k_lo=k_lo, k_hi=k_hi, Hq=Hq, Hkv=Hkv, r_dim=r_dim, E=E,
                    window=window, base=base, page=page, decay=rng.choice([0.0, 0.5, 0.96875, 1.0]), len_seed=seed)
    return dict(op=op, kind=rng.choice(["nvfp4", "bf16"]), batch=batch, k_lo=k_lo, k_hi=k_hi, Hkv=Hkv,
                keep=rng.choice([0.1, 0.25, 0.5, 0.9]), recent=rng.choice([0, 16, 64, 1024]), sink=rng.choice([0, 1, 4]),
                page=page, len_seed=seed)


# ---------------------------------------------------------------- lengths and layouts

def _lens(case):
    rng = np.random.default_rng(1000 + case["len_seed"])
    return [int(x) for x in rng.integers(case["k_lo"], case["k_hi"] + 1, case["batch"])]


def _keep_lens(case):
    return [max(1, min(n, int(n * case["keep"]))) for n in _lens(case)]


def _cu(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=DEV)


def _pages(case, lens, gen):
    """(cache rows, block table or None, row index of every key of every sequence)."""
    size = case["page"]
    starts = np.concatenate([[0], np.cumsum(lens)])
    if size == 0:
        return int(starts[-1]), None, [torch.arange(int(s), int(s) + n, device=DEV) for s, n in zip(starts, lens)]
    counts = [(n + size - 1) // size for n in lens]
    total = sum(counts) + 2
    perm = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((len(lens), max(counts)), -1, dtype=torch.int32, device=DEV)
    rows, used = [], 0
    for b, n in enumerate(lens):
        pg = perm[used:used + counts[b]]
        used += counts[b]
        table[b, :counts[b]] = pg
        p = torch.arange(n, device=DEV)
        rows.append(pg.long()[p // size] * size + p % size)
    return total * size, table, rows


def _normal(gen, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen, device=DEV) * std).to(torch.bfloat16)


def _kv(gen, rows, Hkv, std=1.0):
    """Rows with a few strong channels, as keys and values have."""
    ch = torch.exp(0.5 * torch.randn(Hkv, D, generator=gen, device=DEV)) * std
    return (torch.randn(rows, Hkv, D, generator=gen, device=DEV) * ch).to(torch.bfloat16)


# ---------------------------------------------------------------- NVFP4, elementwise

def _e4m3(x):
    """Nearest E4M3 value, ties to even, at most 448 (x >= 0, float64)."""
    e = torch.frexp(x)[1].to(x.dtype) - 1
    q = torch.exp2(torch.clamp(e, min=-6.0) - 3.0)
    return torch.clamp(torch.round(x / q) * q, max=448.0)


def _e2m1(x):
    """Nearest E2M1 value, ties to even, at most 6 (float64)."""
    a = x.abs()
    q = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0)).to(x.dtype)
    return torch.copysign(torch.clamp(torch.round(a / q) * q, max=6.0), x)


def _encode(x, factor):
    """bf16 [n, Hkv, 128] -> code bytes [n, Hkv, 64], scale bytes [n, Hkv, 8]."""
    n, H, _ = x.shape
    t = (x.float() / factor[None, :, None]).double().view(n, H, 8, 16)
    s = _e4m3(t.abs().amax(-1) / 6.0)
    y = torch.where(s[..., None] > 0, t / torch.where(s > 0, s, 1.0)[..., None], torch.zeros_like(t))
    v = _e2m1(y).view(n, H, D)
    a = v.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = code | (torch.signbit(v).to(torch.uint8) << 3)
    return code[..., 0::2] | (code[..., 1::2] << 4), s.float().to(torch.float8_e4m3fn).view(torch.uint8)


def _decode_values(codes, scales, factor):
    """Stored values, fp32 [n, Hkv, 128]."""
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    v = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1).flatten(-2)
    s = scales.view(torch.float8_e4m3fn).float().repeat_interleave(16, -1)
    return v * s * factor[None, :, None]


def _random_cache(gen, rows, Hkv):
    """A cache of `rows` rows as quantising such keys / values leaves it."""
    out = {}
    for n, std in (("k", 1.0), ("v", 0.25)):
        amax = 6.0 * std
        factor = torch.full((Hkv,), amax / 2688.0, device=DEV) * (1 + 0.1 * torch.rand(Hkv, generator=gen, device=DEV))
        codes = torch.empty(rows, Hkv, 64, dtype=torch.uint8, device=DEV)
        scales = torch.empty(rows, Hkv, 8, dtype=torch.uint8, device=DEV)
        for lo in range(0, rows, 1 << 17):
            hi = min(rows, lo + (1 << 17))
            codes[lo:hi], scales[lo:hi] = _encode(_kv(gen, hi - lo, Hkv, std), factor)
        out[n], out[n + "_scale"], out[n + "_global"] = codes, scales, factor
    return out


# ---------------------------------------------------------------- prepare

def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(seed * 7919 + case["len_seed"])
    lens = _lens(case)
    st = dict(case=case, lens=lens, cu_k=_cu(lens), max_k=max(lens), total_k=sum(lens))
    rows, table, where = _pages(case, lens, gen)
    st.update(rows=rows, table=table, where=where)
    Hkv = case["Hkv"]
    if case["op"] == "evict":
        keep = _keep_lens(case)
        if case["kind"] == "nvfp4":
            c = _random_cache(gen, rows, Hkv)
            planes = [c["k"], c["v"], c["k_scale"], c["v_scale"]]
        else:
            planes = [_normal(gen, rows, Hkv, D) for _ in range(2)]
        # heavy tailed, with ties among the keys that hardly anyone looked at
        w = torch.exp(3 * torch.randn(Hkv, rows, generator=gen, device=DEV))
        w = torch.where(w < 0.05, torch.zeros_like(w), w)
        st.update(planes=planes, weights=w, keep=keep, cu_keep=_cu(keep), total_keep=sum(keep))
        if own:
            st["dst"] = [torch.empty(sum(keep), *p.shape[1:], dtype=p.dtype, device=DEV) for p in planes]
        return st
    q_lens = [min(case["q_len"], n) for n in lens]
    st.update(q_lens=q_lens, cu_q=_cu(q_lens), max_q=max(q_lens))
    Tq = sum(q_lens)
    if case["op"] == "store":
        # the factors come from calibration: largest magnitude over 448 * 6
        st["k"], st["v"] = _kv(gen, Tq, Hkv), _kv(gen, Tq, Hkv, 0.25)
        kg = torch.full((Hkv,), 6.0 / 2688.0, device=DEV) * (1 + 0.1 * torch.rand(Hkv, generator=gen, device=DEV))
        st["cache"] = dict(
            k=torch.zeros(rows, Hkv, 64, dtype=torch.uint8, device=DEV),
            v=torch.zeros(rows, Hkv, 64, dtype=torch.uint8, device=DEV),
            k_scale=torch.zeros(rows, Hkv, 8, dtype=torch.uint8, device=DEV),
            v_scale=torch.zeros(rows, Hkv, 8, dtype=torch.uint8, device=DEV), k_global=kg, v_global=kg * 0.25)
        return _handles(st)
    Hq = case["Hq"]
    st["alpha"] = 1.0 / math.sqrt(D)
    # normalised queries meet keys of unit scale: logits of a few units
    st["q"] = _normal(gen, Tq, Hq, D)
    st["r"] = _normal(gen, Tq, Hq, case["r_dim"]) if case["E"] else None
    st["P"] = _normal(gen, case["r_dim"], case["E"], std=0.1) if case["E"] else None
    if case["op"] == "weights" and case["kind"] == "bf16":
        st["k"] = _normal(gen, rows, Hkv, D)
    else:
        st["cache"] = _random_cache(gen, rows, Hkv)
    if case["op"] == "decode":
        if case["evicted"]:
            # each head kept other keys: the newest half in a run, the rest thinned by gaps
            kp = torch.full((Hkv, rows), -1, dtype=torch.int32, device=DEV)
            qp = []
            for b, n in enumerate(lens):
                new = max(q_lens[b], n // 2)
                gaps = torch.randint(1, 16, (Hkv, n - new), generator=gen, device=DEV).cumsum(1)
                first = int(gaps.max()) + 1 if n > new else 0
                pos = torch.cat([gaps, first + torch.arange(new, device=DEV).expand(Hkv, new)], 1)
                kp[:, where[b]] = pos.to(torch.int32)
                qp.append(first + new - q_lens[b])
            st.update(key_pos=kp, q_pos=torch.tensor(qp, dtype=torch.int32, device=DEV))
        return _handles(st)
    st["weights_in"] = torch.rand(Hkv, rows, generator=gen, device=DEV) * 8
    # the forward pass left the logsumexp of every row
    lse = torch.empty(Hq, Tq, device=DEV)
    for b in range(len(lens)):
        K = _keys(st, b)
        a = sum(q_lens[:b])
        for h in range(Hkv):
            for lo in range(0, q_lens[b], 2048):
                hi = min(q_lens[b], lo + 2048)
                x = _logits(st, b, h, K, lo, hi)
                lse[h * (Hq // Hkv):(h + 1) * (Hq // Hkv), a + lo:a + hi] = torch.logsumexp(x, -1)
    st["lse"] = lse
    return _handles(st)


def _handles(st):
    """What a program holds between calls besides the tensors."""
    if own and "cache" in st:
        import relative_position_biased_gb300 as rpb
        st["handle"] = rpb.KvNvfp4(**st["cache"])
    return st


# ---------------------------------------------------------------- plain forms

def _keys(st, b, name="k"):
    """fp32 keys (or values) [Lk, Hkv, 128] of sequence b."""
    rows = st["where"][b]
    if "cache" not in st:
        return st[name][rows].float()
    c = st["cache"]
    return _decode_values(c[name][rows], c[name + "_scale"][rows], c[name + "_global"])


def _positions(st, b, h, lo, hi):
    n, nq = st["lens"][b], st["q_lens"][b]
    if "key_pos" in st:
        return st["q_pos"][b].long() + torch.arange(lo, hi, device=DEV), st["key_pos"][h, st["where"][b]].long()
    return n - nq + torch.arange(lo, hi, device=DEV), torch.arange(n, device=DEV)


def _logits(st, b, h, K, lo, hi):
    """Masked logits [group, hi - lo, Lk] of rows lo .. hi of sequence b and kv head h."""
    case = st["case"]
    g = case["Hq"] // case["Hkv"]
    a = sum(st["q_lens"][:b])
    q = st["q"][a + lo:a + hi, h * g:(h + 1) * g].float().transpose(0, 1)
    x = (q @ K[:, h].t()) * st["alpha"]
    qp, kp = _positions(st, b, h, lo, hi)
    d = qp[:, None] - kp[None, :]
    if case["E"]:
        R = st["r"][a + lo:a + hi, h * g:(h + 1) * g].float().transpose(0, 1) @ st["P"].float()
        bias = R.gather(2, d.clamp(0, case["E"] - 1).expand(g, -1, -1))
        x = x + torch.where((d >= 0) & (d < case["E"]), bias, torch.zeros_like(bias))
    if case["base"] > 0:
        s = torch.clamp(torch.log(qp.double() + 1) / math.log(case["base"]), min=1.0).float()
        x = x * s[None, :, None]
    seen = (d >= 0) & (kp >= 0)[None, :]
    if case["window"]:
        seen &= d < case["window"]
    return torch.where(seen, x, torch.full_like(x, -math.inf))


def _plain_decode(st):
    case = st["case"]
    Hq, Hkv = case["Hq"], case["Hkv"]
    g = Hq // Hkv
    out = torch.empty_like(st["q"])
    lse = torch.empty(Hq, st["q"].shape[0], device=DEV)
    a = 0
    for b, nq in enumerate(st["q_lens"]):
        K, V = _keys(st, b), _keys(st, b, "v")
        for h in range(Hkv):
            x = _logits(st, b, h, K, 0, nq)
            m = x.amax(-1, keepdim=True)
            m = torch.where(m == -math.inf, torch.zeros_like(m), m)
            p = torch.exp(x - m)
            z = p.sum(-1, keepdim=True)
            o = (p @ V[:, h]) / torch.where(z > 0, z, torch.ones_like(z))
            out[a:a + nq, h * g:(h + 1) * g] = o.transpose(0, 1).to(out.dtype)
            lse[h * g:(h + 1) * g, a:a + nq] = (m + torch.log(z))[..., 0]
        a += nq
    return out, lse


def _plain_store(st):
    c = st["cache"]
    rows = torch.cat([w[n - q:] for w, n, q in zip(st["where"], st["lens"], st["q_lens"])])
    outs = []
    for n in ("k", "v"):
        c[n][rows], c[n + "_scale"][rows] = _encode(st[n], c[n + "_global"])
        outs.append(_decode_values(c[n][rows], c[n + "_scale"][rows], c[n + "_global"]).to(torch.bfloat16))
    return tuple(outs)


def _plain_weights(st):
    case = st["case"]
    g = case["Hq"] // case["Hkv"]
    w = torch.zeros_like(st["weights_in"])
    a = 0
    for b, (n, nq) in enumerate(zip(st["lens"], st["q_lens"])):
        K = _keys(st, b)
        for h in range(case["Hkv"]):
            acc = torch.zeros(n, device=DEV)
            acc[:n - nq] = st["weights_in"][h, st["where"][b][:n - nq]] * case["decay"]
            for lo in range(0, nq, 4096):
                hi = min(nq, lo + 4096)
                x = _logits(st, b, h, K, lo, hi)
                acc += torch.exp(x - st["lse"][h * g:(h + 1) * g, a + lo:a + hi, None]).sum((0, 1))
            w[h, st["where"][b]] = acc
        a += nq
    return w


def _plain_evict(st):
    case = st["case"]
    total, Hkv = st["total_keep"], case["Hkv"]
    outs = [torch.empty(total, *p.shape[1:], dtype=p.dtype, device=DEV) for p in st["planes"]]
    pos = torch.empty(Hkv, total, dtype=torch.int32, device=DEV)
    w_out = torch.empty(Hkv, total, device=DEV)
    a = 0
    for b, (n, keep) in enumerate(zip(st["lens"], st["keep"])):
        recent = min(case["recent"], keep)
        sink = min(case["sink"], keep - recent, n - recent)
        rest = keep - recent - sink
        for h in range(Hkv):
            w = st["weights"][h, st["where"][b]]
            mid = torch.sort(w[sink:n - recent], descending=True, stable=True)[1][:rest] + sink
            idx = torch.cat([torch.arange(sink, device=DEV), torch.sort(mid)[0], torch.arange(n - recent, n, device=DEV)])
            rows = st["where"][b][idx]
            for o, p in zip(outs, st["planes"]):
                o[a:a + keep, h] = p[rows, h]
            pos[h, a:a + keep] = idx.to(torch.int32)
            w_out[h, a:a + keep] = w[idx]
        a += keep
    return (*outs, pos, w_out)


# ---------------------------------------------------------------- run

def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return {"decode": _plain_decode, "store": _plain_store, "weights": _plain_weights, "evict": _plain_evict}[op](st)
    import relative_position_biased_gb300 as rpb
    paged = dict(block_table=st["table"], page_size=case["page"]) if case["page"] else {}
    if op == "decode":
        return rpb.decode_nvfp4(st["q"], st["handle"], st["r"], st["P"], st["cu_q"], st["cu_k"], max_seqlen_q=st["max_q"],
                                max_seqlen_k=st["max_k"], alpha=st["alpha"], window=case["window"],
                                log_scale_base=case["base"], key_pos=st.get("key_pos"), q_pos=st.get("q_pos"),
                                total_k=st["total_k"], **paged)
    if op == "store":
        rpb.store_nvfp4(st["k"], st["v"], st["cu_q"], st["cu_k"], st["handle"], **paged)
        return rpb.load_nvfp4(st["handle"], st["cu_q"], st["cu_k"], total_q=st["k"].shape[0], **paged)
    if op == "weights":
        w = torch.zeros_like(st["weights_in"])     # rows that no sequence holds are left as they are
        return rpb.key_weights(st["q"], st["handle"] if case["kind"] == "nvfp4" else st["k"], st["r"], st["P"], st["lse"],
                               st["cu_q"], st["cu_k"], max_seqlen_q=st["max_q"], max_seqlen_k=st["max_k"],
                               alpha=st["alpha"], window=case["window"], log_scale_base=case["base"],
                               weights_in=st["weights_in"], decay=case["decay"], out=w, total_k=st["total_k"], **paged)
    pos, w = rpb.evict(st["planes"], st["dst"], st["weights"], st["cu_k"], st["cu_keep"], max_seqlen_k=st["max_k"],
                       total_k=st["total_k"], total_keep=st["total_keep"], recent=case["recent"], sink=case["sink"], **paged)
    return (*st["dst"], pos, w)


# ---------------------------------------------------------------- work

def _pairs(lens, q_lens, window):
    """Query-key pairs a head scores, and the keys that some query sees."""
    pairs = keys = 0
    for n, nq in zip(lens, q_lens):
        i = np.arange(n - nq, n, dtype=np.float64) + 1
        pairs += float(np.minimum(i, window).sum() if window else i.sum())
        keys += min(n, window + nq - 1) if window else n
    return pairs, keys


def work(case):
    lens = _lens(case)
    total, Hkv = sum(lens), case["Hkv"]
    if case["op"] == "evict":
        keep = sum(_keep_lens(case))
        row = 144 if case["kind"] == "nvfp4" else 512
        return {"bytes": 4 * total * Hkv + keep * Hkv * (2 * row + 8), "flops": total * Hkv}
    q_lens = [min(case["q_len"], n) for n in lens]
    Tq = sum(q_lens)
    if case["op"] == "store":
        return {"bytes": 2 * (2 * Tq * Hkv * (256 + 72)), "flops": 2 * 4 * Tq * Hkv * D}
    Hq = case["Hq"]
    window = 0 if case.get("evicted") else case["window"]
    pairs, keys = _pairs(lens, q_lens, window)
    flops = 2.0 * D * pairs * Hq
    small = Tq * Hq * 2 * (D + case["r_dim"]) + 2 * case["r_dim"] * case["E"] + 4 * Tq * Hq
    if case["op"] == "decode":
        row = 144 + (4 if case["evicted"] else 0)
        return {"bytes": keys * Hkv * row + small + Tq * Hq * 2 * D, "flops": 2 * flops}
    row = 72 if case["kind"] == "nvfp4" else 256
    return {"bytes": keys * Hkv * row + total * Hkv * (8 if case["decay"] else 4) + small, "flops": flops}


# ---------------------------------------------------------------- 64-bit definitions

def _values64(st, rows, name):
    """Stored values in float64, from the bits of the two formats."""
    if "cache" not in st:
        return st[name][rows].double()
    c = st["cache"]
    byte = c[name][rows].long()
    nib = torch.stack([byte % 16, byte // 16], -1).flatten(-2)
    e, m = (nib // 2) % 4, (nib % 2).double()
    mag = torch.where(e == 0, m / 2, (1 + m / 2) * torch.pow(2.0, e.double() - 1))
    val = torch.where(nib >= 8, -mag, mag)
    sb = c[name + "_scale"][rows].long()
    se, sm = sb // 8, (sb % 8).double()
    sc = torch.where(se == 0, sm / 512, (1 + sm / 8) * torch.pow(2.0, se.double() - 7))
    n, H = val.shape[:2]
    return (val.view(n, H, 8, 16) * sc[..., None]).view(n, H, D) * c[name + "_global"].double()[:, None]


def _x64(st, b, h, hh, lo, hi, K):
    """float64 logits of query head h * g + hh, rows lo .. hi."""
    case = st["case"]
    n, nq = st["lens"][b], st["q_lens"][b]
    head = h * (case["Hq"] // case["Hkv"]) + hh
    a = sum(st["q_lens"][:b])
    if case.get("evicted"):
        i = st["q_pos"][b].double() + torch.arange(lo, hi, device=DEV).double()
        j = st["key_pos"][h][st["where"][b]].double()
    else:
        i = torch.arange(n - nq + lo, n - nq + hi, device=DEV).double()
        j = torch.arange(n, device=DEV).double()
    x = st["alpha"] * torch.mm(st["q"][a + lo:a + hi, head].double(), K.t())
    dist = i[:, None] - j
    if case["E"]:
        table = torch.zeros(hi - lo, case["E"] + 1, dtype=torch.float64, device=DEV)
        table[:, :-1] = torch.mm(st["r"][a + lo:a + hi, head].double(), st["P"].double())
        slot = torch.where((dist >= 0) & (dist < case["E"]), dist, torch.full_like(dist, case["E"])).long()
        x += torch.take_along_dim(table, slot, 1)
    if case["base"] > 0:
        x *= torch.maximum(torch.ones_like(i), (i + 1).log() / math.log(case["base"]))[:, None]
    hide = (dist < 0) | (j < 0)
    if case["window"]:
        hide |= dist >= case["window"]
    return x.masked_fill_(hide, -math.inf)


def exact(case, seed):
    global own
    keep_own, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = keep_own
    lens = st["lens"]
    if case["op"] == "evict":
        w = st["weights"].cpu().numpy()
        where = [r.cpu().numpy() for r in st["where"]]
        total, Hkv = st["total_keep"], case["Hkv"]
        src = np.empty((Hkv, total), dtype=np.int64)
        pos = np.empty((Hkv, total), dtype=np.int32)
        a = 0
        for b, (n, keep) in enumerate(zip(lens, st["keep"])):
            p = np.arange(n)
            for h in range(Hkv):
                # newest first, then the first keys, then by weight (lower index first)
                rank = np.lexsort((p, -w[h, where[b]].astype(np.float64), (p >= case["sink"]).astype(int),
                                   (p < n - case["recent"]).astype(int)))
                if keep < case["recent"]:
                    chosen = np.arange(n - keep, n)
                elif keep < case["recent"] + case["sink"]:
                    chosen = np.sort(np.concatenate([np.arange(keep - min(case["recent"], n)),
                                                     np.arange(n - min(case["recent"], n), n)]))
                else:
                    chosen = np.sort(rank[:keep])
                pos[h, a:a + keep] = chosen
                src[h, a:a + keep] = where[b][chosen]
            a += keep
        rows = torch.from_numpy(src).to(DEV)
        heads = torch.arange(Hkv, device=DEV)[:, None]
        moved = [p[rows, heads].transpose(0, 1).contiguous() for p in st["planes"]]
        return (*moved, torch.from_numpy(pos).to(DEV), st["weights"].gather(1, rows).double())
    if case["op"] == "store":
        outs = []
        mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device=DEV)
        grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
        s_all = torch.tensor([m / 512 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)
                                                            if (e, m) != (15, 7)], dtype=torch.float64, device=DEV)
        for n in ("k", "v"):
            f = st["cache"][n + "_global"]
            t = (st[n].float() / f[:, None]).double()        # the one fp32 rounding of the definition
            rows, H = t.shape[:2]
            t = t.view(rows, H, 8, 16)
            need = t.abs().amax(-1) / 6
            up = torch.searchsorted(s_all, need).clamp(max=len(s_all) - 1)
            dn = (up - 1).clamp(min=0)
            du, dd = (s_all[up] - need).abs(), (need - s_all[dn]).abs()
            idx = torch.where((du < dd) | ((du == dd) & (up % 2 == 0)), up, dn)
            s = s_all[idx]
            a = t.abs()[..., None]
            edge = mids * s[..., None, None]
            odd = torch.arange(7, device=DEV) % 2 == 1        # a tie above an odd code moves up, to the even one
            k = ((a > edge) | ((a == edge) & odd)).sum(-1)
            k = torch.where(s[..., None] > 0, k, torch.zeros_like(k))
            val = torch.copysign(grid[k], t) * s[..., None]
            outs.append(val.view(rows, H, D) * f.double()[:, None])
        return tuple(outs)
    Hq, Hkv = case["Hq"], case["Hkv"]
    g = Hq // Hkv
    Tq = st["q"].shape[0]
    if case["op"] == "decode":
        out = torch.empty(Tq, Hq, D, dtype=torch.float64, device=DEV)
        lse = torch.empty(Hq, Tq, dtype=torch.float64, device=DEV)
        for b, nq in enumerate(st["q_lens"]):
            a = sum(st["q_lens"][:b])
            K, V = _values64(st, st["where"][b], "k"), _values64(st, st["where"][b], "v")
            for h in range(Hkv):
                for hh in range(g):
                    x = _x64(st, b, h, hh, 0, nq, K[:, h])
                    z = torch.logsumexp(x, 1)
                    p = torch.exp(x - torch.where(z.isinf(), torch.zeros_like(z), z)[:, None])
                    out[a:a + nq, h * g + hh] = p @ V[:, h]
                    lse[h * g + hh, a:a + nq] = z
        return out, lse
    w = torch.zeros(Hkv, st["rows"], dtype=torch.float64, device=DEV)
    for b, (n, nq) in enumerate(zip(lens, st["q_lens"])):
        a = sum(st["q_lens"][:b])
        K = _values64(st, st["where"][b], "k")
        for h in range(Hkv):
            col = torch.zeros(n, dtype=torch.float64, device=DEV)
            for hh in range(g):
                for lo in range(0, nq, 4096):
                    hi = min(nq, lo + 4096)
                    x = _x64(st, b, h, hh, lo, hi, K[:, h])
                    col += torch.exp(x - st["lse"][h * g + hh, a + lo:a + hi].double()[:, None]).sum(0)
            old = st["weights_in"][h][st["where"][b]].double() * case["decay"]
            old[n - nq:] = 0
            w[h][st["where"][b]] = col + old
    return w
