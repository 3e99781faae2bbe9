"""Cases for serving from a paged bf16 K / V cache and for sliding windows with
sinks: the attention prologue that writes its rows into pages, the attention of
new tokens (one, a chunk, a whole prompt) over the cache that holds them, and
the gradients of a window with sinks.

Symbols
  logits   x(i, j) = s(i) (alpha q_i . k_j + [0 <= d < E] r_i . P[:, d]), d = i - j,
           s(i) = max(1, ln(i + 1) / ln(base)).
  visible  d >= 0, and with a window: d < window or j < sink (the first keys stay).
  rows     the new tokens are the last Lq of a sequence's Lk keys.
  pages    key p of sequence b is pool row table[b, p // size] * size + p % size.
"""
import math

import numpy as np
import torch

own = False

D = 128
DEV = "cuda"

# ---------------------------------------------------------------- cases

# Lengths are drawn by len_seed: new tokens from q_lo .. q_hi, keys from k_lo .. k_hi (at least the new tokens).
_LISTED = [
    # one short conversation, one new token, small pages: the smallest call, latency counts
    dict(name="token_one_short", op="extend", batch=1, q_lo=1, q_hi=1, k_lo=301, k_hi=301, Hq=4, Hkv=1, r_dim=32, E=64,
         window=0, sink=0, base=0.0, page=16, len_seed=0),
    # a decode step of a serving batch in a sliding-window layer that keeps the first 4 keys
    dict(name="token_batch_sinks", op="extend", batch=64, q_lo=1, q_hi=1, k_lo=1024, k_hi=32768, Hq=16, Hkv=2, r_dim=64,
         E=1024, window=4096, sink=4, base=0.0, page=64, len_seed=0),
    # the same step in a full layer, 16-key pages
    dict(name="token_batch_full", op="extend", batch=64, q_lo=1, q_hi=1, k_lo=1024, k_hi=32768, Hq=16, Hkv=2, r_dim=64,
         E=1024, window=0, sink=0, base=65536.0, page=16, len_seed=0),
    # ragged short chunks (draft tokens, tails of prompts) on long prefixes, full layer
    dict(name="chunk_ragged_short", op="extend", batch=12, q_lo=3, q_hi=97, k_lo=2000, k_hi=50000, Hq=16, Hkv=2, r_dim=64,
         E=1024, window=0, sink=0, base=65536.0, page=32, len_seed=1),
    # a scheduler's prompt chunks over sliding-window pages with sinks
    dict(name="chunk_window_sinks", op="extend", batch=4, q_lo=2048, q_hi=2048, k_lo=8192, k_hi=32768, Hq=16, Hkv=2,
         r_dim=64, E=1024, window=4096, sink=4, base=0.0, page=128, len_seed=2),
    # one chunk at the end of a long document, full layer
    dict(name="chunk_long_prefix", op="extend", batch=1, q_lo=2048, q_hi=2048, k_lo=131072, k_hi=131072, Hq=16, Hkv=2,
         r_dim=64, E=1024, window=0, sink=0, base=65536.0, page=128, len_seed=0),
    # training: a packed batch through a sliding-window layer with sinks, contiguous keys
    dict(name="prompt_sinks", op="extend", batch=4, q_lo=8192, q_hi=8192, k_lo=0, k_hi=0, Hq=16, Hkv=2, r_dim=64, E=1024,
         window=4096, sink=4, base=0.0, page=0, len_seed=0),
    # its gradients
    dict(name="backward_sinks", op="backward", batch=4, q_lo=8192, q_hi=8192, k_lo=0, k_hi=0, Hq=16, Hkv=2, r_dim=64,
         E=1024, window=4096, sink=4, base=0.0, page=0, len_seed=0),
    # gradients of a few ragged sequences, a window below the bias's extent
    dict(name="backward_ragged", op="backward", batch=5, q_lo=90, q_hi=1500, k_lo=0, k_hi=0, Hq=8, Hkv=2, r_dim=16, E=200,
         window=96, sink=7, base=0.0, page=0, len_seed=3),
    # the prologue of four prompts of 8192 tokens, rows into 128-key pages
    dict(name="prologue_prompts", op="prologue", batch=4, q_lo=8192, q_hi=8192, k_lo=8192, k_hi=8192, Hq=16, Hkv=2,
         page=128, state=False, len_seed=0),
    # the prologue of one new token of every sequence of a batch
    dict(name="prologue_tokens", op="prologue", batch=64, q_lo=1, q_hi=1, k_lo=1024, k_hi=8192, Hq=16, Hkv=2, page=16,
         state=True, len_seed=2),
]


def listed():
    return [dict(c) for c in _LISTED]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["extend", "extend", "extend", "backward", "backward", "prologue"])
    Hq, Hkv = rng.choice([(16, 2), (8, 2), (4, 1), (8, 1), (16, 1), (12, 4), (4, 4)])
    page = rng.choice([0, 16, 32, 48, 64, 128, 256])
    seed = rng.randrange(1 << 20)
    batch = _log_int(rng, 1, 64)
    r_dim, E = rng.choice([(64, 1024), (32, 64), (16, 200), (0, 0), (64, 77), (24, 512)])
    window = rng.choice([0, _log_int(rng, 16, 8192), _log_int(rng, 16, 8192)])
    base = rng.choice([0.0, 65536.0, 64.0]) if window == 0 else 0.0
    sink = rng.choice([0, 1, 4, 16, 100])
    if op == "prologue":
        q_hi = _log_int(rng, 1, max(1, 32768 // batch))
        k_hi = min(32768, q_hi + _log_int(rng, 1, 8192))
        return dict(op=op, batch=batch, q_lo=max(1, q_hi // rng.randint(1, 4)), q_hi=q_hi, k_lo=min(q_hi, k_hi), k_hi=k_hi, Hq=Hq,
                    Hkv=Hkv, page=rng.choice([16, 32, 48, 64, 128, 256]), state=rng.random() < 0.5, len_seed=seed)
    if op == "backward":
        batch = rng.randint(1, 8)
        q_hi = _log_int(rng, 64, 24576 // batch)
        q_lo = max(1, q_hi // rng.randint(1, 8))
        return dict(op=op, batch=batch, q_lo=q_lo, q_hi=q_hi, k_lo=0, k_hi=0, Hq=Hq, Hkv=Hkv, r_dim=r_dim, E=E,
                    window=_log_int(rng, 16, 4096), sink=rng.choice([1, 2, 4, 7, 16, 40, 100]), base=rng.choice([0.0, 0.0, 64.0]),
                    page=0, len_seed=seed)
    prompt = page == 0 and rng.random() < 0.5
    if prompt:                                   # new tokens are all there is
        batch = min(batch, 8)
        q_hi = _log_int(rng, 128, 24576 // batch)
        return dict(op=op, batch=batch, q_lo=max(1, q_hi // rng.randint(1, 8)), q_hi=q_hi, k_lo=0, k_hi=0, Hq=Hq, Hkv=Hkv,
                    r_dim=r_dim, E=E, window=window, sink=sink, base=base, page=page, len_seed=seed)
    k_hi = _log_int(rng, 40, max(64, min(1 << 17, (1 << 20) // batch)))
    most = max(1, min(2048, (1 << 26) // (batch * k_hi)))
    q_hi = rng.choice([1, 1, 2, 9, 33, _log_int(rng, 1, 2048)])
    q_hi = min(q_hi, most, k_hi)
    return dict(op=op, batch=batch, q_lo=max(1, q_hi // rng.randint(1, 8)), q_hi=q_hi, k_lo=max(1, k_hi // rng.randint(1, 16)),
                k_hi=k_hi, Hq=Hq, Hkv=Hkv, r_dim=r_dim, E=E, window=window, sink=sink, base=base, page=page, len_seed=seed)


# ---------------------------------------------------------------- lengths and layouts

def _lens(case):
    """(new tokens, keys) of every sequence."""
    rng = np.random.default_rng(1000 + case["len_seed"])
    q = [int(x) for x in rng.integers(case["q_lo"], case["q_hi"] + 1, case["batch"])]
    k = [int(x) for x in rng.integers(case["k_lo"], case["k_hi"] + 1, case["batch"])]
    return q, [max(a, b) for a, b in zip(q, k)]


def _cu(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=DEV)


def _pages(case, lens, gen):
    """(cache rows, block table or None, row index of every key of every sequence)."""
    size = case["page"]
    starts = np.concatenate([[0], np.cumsum(lens)])
    if size == 0:
        return int(starts[-1]), None, [torch.arange(int(s), int(s) + n, device=DEV) for s, n in zip(starts, lens)]
    counts = [(n + size - 1) // size for n in lens]
    total = max(sum(counts) + 2, (128 + size - 1) // size)
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


# ---------------------------------------------------------------- prepare

def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(seed * 7919 + case["len_seed"])
    q_lens, lens = _lens(case)
    rows, table, where = _pages(case, lens, gen)
    Hq, Hkv, Tq = case["Hq"], case["Hkv"], sum(q_lens)
    st = dict(case=case, lens=lens, q_lens=q_lens, cu_q=_cu(q_lens), cu_k=_cu(lens), max_q=max(q_lens), max_k=max(lens),
              total_k=sum(lens), rows=rows, table=table, where=where)
    if case["op"] == "prologue":
        # pre-norm projections, the conv state the sequence's earlier rows left, a pool that holds other rows
        st["q"], st["k"], st["v"] = (_normal(gen, Tq, h, D, std=s) for h, s in ((Hq, 2.0), (Hkv, 2.0), (Hkv, 1.0)))
        st["conv"] = [0.3 * torch.randn(Hkv * D, 4, generator=gen, device=DEV) for _ in range(2)]
        st["norm"] = [1 + 0.2 * torch.randn(D, generator=gen, device=DEV) for _ in range(2)]
        st["state"] = [_normal(gen, len(lens), 3, Hkv * D) for _ in range(2)] if case["state"] else None
        st["state_out"] = [torch.zeros(len(lens), 3, Hkv * D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        st["pool"] = [_normal(gen, rows, Hkv, D) for _ in range(2)]
        return st
    st["alpha"] = 1.0 / math.sqrt(D)
    # normalised queries meet keys of unit scale: logits of a few units
    st["q"] = _normal(gen, Tq, Hq, D)
    st["r"] = _normal(gen, Tq, Hq, case["r_dim"]) if case["E"] else None
    st["P"] = _normal(gen, case["r_dim"], case["E"], std=0.1) if case["E"] else None
    st["k"], st["v"] = _normal(gen, rows, Hkv, D), _normal(gen, rows, Hkv, D)
    if case["op"] == "backward":
        # the forward pass left out and lse
        st["out"], st["lse"] = _plain_extend(st)
        st["dout"] = _normal(gen, Tq, Hq, D)
    return st


# ---------------------------------------------------------------- plain forms

def _blocks(st):
    """(b, kv head, first row in q, rows lo .. hi, keys that some of them sees) in blocks that fit."""
    case = st["case"]
    g = case["Hq"] // case["Hkv"]
    a = 0
    for b, (n, nq) in enumerate(zip(st["lens"], st["q_lens"])):
        step = max(1, min(nq, (1 << 28) // (g * n)))
        if case["window"]:
            step = max(step, min(nq, case["window"]))
        for lo in range(0, nq, step):
            hi = min(nq, lo + step)
            first = max(0, n - nq + lo - case["window"] + 1) if case["window"] else 0
            keys = torch.arange(first, n - nq + hi, device=DEV)
            if first > 0 and case["sink"] > 0:
                keys = torch.cat([torch.arange(min(case["sink"], first), device=DEV), keys])
            for h in range(case["Hkv"]):
                yield b, h, a, lo, hi, keys
        a += nq


def _logits(st, b, h, a, lo, hi, keys):
    """(masked logits [group, rows, keys], keys fp32, distances, row scales)."""
    case = st["case"]
    g = case["Hq"] // case["Hkv"]
    n, nq = st["lens"][b], st["q_lens"][b]
    K = st["k"][st["where"][b][keys], h].float()
    q = st["q"][a + lo:a + hi, h * g:(h + 1) * g].float().transpose(0, 1)
    x = (q @ K.t()) * st["alpha"]
    qp = n - nq + torch.arange(lo, hi, device=DEV)
    d = qp[:, None] - keys[None, :]
    if case["E"]:
        R = st["r"][a + lo:a + hi, h * g:(h + 1) * g].float().transpose(0, 1) @ st["P"].float()
        bias = R.gather(2, d.clamp(0, case["E"] - 1).expand(g, -1, -1))
        x = x + torch.where((d >= 0) & (d < case["E"]), bias, torch.zeros_like(bias))
    s = torch.ones(hi - lo, device=DEV)
    if case["base"] > 0:
        s = torch.clamp(torch.log(qp.double() + 1) / math.log(case["base"]), min=1.0).float()
        x = x * s[None, :, None]
    seen = d >= 0
    if case["window"]:
        seen &= (d < case["window"]) | (keys < case["sink"])[None, :]
    return torch.where(seen, x, torch.full_like(x, -math.inf)), K, d, s


def _plain_extend(st):
    case = st["case"]
    g = case["Hq"] // case["Hkv"]
    out = torch.empty_like(st["q"])
    lse = torch.empty(case["Hq"], st["q"].shape[0], device=DEV)
    for b, h, a, lo, hi, keys in _blocks(st):
        x = _logits(st, b, h, a, lo, hi, keys)[0]
        V = st["v"][st["where"][b][keys], h].float()
        m = x.amax(-1, keepdim=True)                       # (every row sees itself)
        p = torch.exp(x - m)
        z = p.sum(-1, keepdim=True)
        out[a + lo:a + hi, h * g:(h + 1) * g] = ((p @ V) / z).transpose(0, 1).to(out.dtype)
        lse[h * g:(h + 1) * g, a + lo:a + hi] = (m + torch.log(z))[..., 0]
    return out, lse


def _plain_backward(st):
    case = st["case"]
    g = case["Hq"] // case["Hkv"]
    dq, dk, dv = (torch.zeros(st[n].shape, device=DEV) for n in ("q", "k", "v"))
    dr = torch.zeros(st["r"].shape, device=DEV) if case["E"] else None
    for b, h, a, lo, hi, keys in _blocks(st):
        x, K, d, s = _logits(st, b, h, a, lo, hi, keys)
        rows, heads, at = slice(a + lo, a + hi), slice(h * g, (h + 1) * g), st["where"][b][keys]
        V = st["v"][at, h].float()
        do = st["dout"][rows, heads].float().transpose(0, 1)
        Dsum = (do * st["out"][rows, heads].float().transpose(0, 1)).sum(-1, keepdim=True)
        p = torch.exp(x - st["lse"][heads, rows, None])
        dv[at, h] += torch.einsum("gij,gid->jd", p, do)
        dl = p * (do @ V.t() - Dsum) * s[None, :, None]
        dq[rows, heads] = (dl @ K).transpose(0, 1) * st["alpha"]
        q = st["q"][rows, heads].float().transpose(0, 1)
        dk[at, h] += torch.einsum("gij,gid->jd", dl, q) * st["alpha"]
        if case["E"]:
            band = (d >= 0) & (d < case["E"])
            by_d = torch.zeros(g, hi - lo, case["E"], device=DEV)
            by_d.scatter_add_(2, d.clamp(0, case["E"] - 1).expand(g, -1, -1), torch.where(band, dl, torch.zeros_like(dl)))
            dr[rows, heads] = (by_d @ st["P"].float().t()).transpose(0, 1)
    grads = (dq, dk, dv) if dr is None else (dq, dk, dv, dr)
    return tuple(x.to(torch.bfloat16) for x in grads)


def _plain_prologue(st):
    case = st["case"]
    eps, H = 1e-6, case["Hkv"]

    def norm(x, gamma):
        return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * gamma

    q_out = norm(st["q"].float(), st["norm"][0]).to(torch.bfloat16)
    a = 0
    for b, (n, nq) in enumerate(zip(st["lens"], st["q_lens"])):
        rows = st["where"][b][n - nq:]
        for i, name in enumerate(("k", "v")):
            x = st[name][a:a + nq].reshape(nq, H * D)
            before = st["state"][i][b] if st["state"] else torch.zeros(3, H * D, dtype=x.dtype, device=DEV)
            x = torch.cat([before, x])
            st["state_out"][i][b] = x[nq:]
            x = x.float()
            y = x[3:]
            for lag in range(4):
                y = y + st["conv"][i][:, lag] * x[3 - lag:3 - lag + nq]
            y = y.view(nq, H, D)
            st["pool"][i][rows] = (norm(y, st["norm"][1]) if i == 0 else y).to(torch.bfloat16)
        a += nq
    return (q_out, *st["pool"], *st["state_out"])


# ---------------------------------------------------------------- run

def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return {"extend": _plain_extend, "backward": _plain_backward, "prologue": _plain_prologue}[op](st)
    import relative_position_biased_gb300 as rpb
    paged = dict(block_table=st["table"], page_size=case["page"]) if case["page"] else {}
    if op == "prologue":
        q_out = rpb.prologue(st["q"], st["k"], st["v"], *st["conv"], *st["norm"], st["cu_q"], st["cu_k"], *st["pool"], eps=1e-6,
                             conv_state_in=st["state"], conv_state_out=st["state_out"], **paged)
        return (q_out, *st["pool"], *st["state_out"])
    kw = dict(max_seqlen_q=st["max_q"], max_seqlen_k=st["max_k"], alpha=st["alpha"], window=case["window"],
              log_scale_base=case["base"], sink=case["sink"])
    if op == "extend":
        return rpb.extend(st["q"], st["k"], st["v"], st["r"], st["P"], st["cu_q"], st["cu_k"], total_k=st["total_k"], **paged, **kw)
    grads = rpb.backward(st["q"], st["k"], st["v"], st["r"], st["P"], st["out"], st["lse"], st["dout"], st["cu_q"], st["cu_k"], **kw)
    return grads if case["E"] else grads[:3]


# ---------------------------------------------------------------- work

def _pairs(case):
    """Query-key pairs a head scores, those inside the bias, and the keys that some row sees."""
    pairs = band = keys = 0
    for nq, n in zip(*_lens(case)):
        i = np.arange(n - nq, n, dtype=np.float64)
        W = case["window"] or n
        seen = np.minimum(i + 1, W)
        extra = np.minimum(case["sink"], i + 1 - seen)
        pairs += float((seen + extra).sum())
        # distances below E: in the window, or a sink
        far = np.clip(np.minimum(case["sink"] - 1, i - W) - np.maximum(i - case["E"] + 1, 0) + 1, 0, None)
        band += float((np.minimum(seen, case["E"]) + far).sum()) if case["E"] else 0.0
        first = max(0, n - nq - W + 1)
        keys += n - first + min(case["sink"], first)
    return pairs, band, keys


def work(case):
    q_lens, lens = _lens(case)
    Tq, Hq, Hkv = sum(q_lens), case["Hq"], case["Hkv"]
    if case["op"] == "prologue":
        state = 2 * len(lens) * 3 * Hkv * D * 2 * (2 if case["state"] else 1)
        return {"bytes": 2 * 2 * Tq * (Hq + 2 * Hkv) * D + state + 2 * Hkv * D * 16, "flops": Tq * D * (4 * Hq + 20 * Hkv)}
    pairs, band, keys = _pairs(case)
    rows, small = Tq * Hq, Tq * Hq * 2 * case["r_dim"] + 2 * case["r_dim"] * case["E"] + 4 * Tq * Hq
    if case["op"] == "extend":
        bias = 2.0 * case["r_dim"] * rows * min(case["E"], max(lens)) if case["E"] else 0.0
        return {"bytes": keys * Hkv * 4 * D + rows * 4 * D + small, "flops": 4.0 * D * pairs * Hq + bias}
    flops = 10.0 * D * pairs * Hq + 2.0 * case["r_dim"] * band * Hq
    return {"bytes": 2 * sum(lens) * Hkv * 4 * D + 4 * rows * 2 * D + small + rows * 2 * case["r_dim"], "flops": flops}


# ---------------------------------------------------------------- 64-bit definitions

def _spans(st, b, lo, hi):
    """Key ranges of rows lo .. hi: what windows reach, and the sinks before it."""
    case = st["case"]
    p_lo, p_hi = st["lens"][b] - st["q_lens"][b] + lo, st["lens"][b] - st["q_lens"][b] + hi
    start = max(0, p_lo + 1 - case["window"]) if case["window"] else 0
    spans = [(start, p_hi)]
    if start and case["sink"]:
        spans.append((0, min(start, case["sink"])))
    return spans


def _x64(st, b, head, tok, lo, hi, span):
    """float64 logits of one query head's rows lo .. hi against keys span, and their distances."""
    case = st["case"]
    kv = head // (case["Hq"] // case["Hkv"])
    i = torch.arange(lo, hi, device=DEV, dtype=torch.float64) + (st["lens"][b] - st["q_lens"][b])
    j = torch.arange(*span, device=DEV, dtype=torch.float64)
    dist = i[:, None] - j
    K = st["k"][st["where"][b][span[0]:span[1]], kv].double()
    x = torch.mm(st["q"][tok + lo:tok + hi, head].double(), K.t()).mul_(st["alpha"])
    if case["E"]:
        table = torch.zeros(hi - lo, case["E"] + 1, dtype=torch.float64, device=DEV)
        table[:, :-1] = torch.mm(st["r"][tok + lo:tok + hi, head].double(), st["P"].double())
        slot = torch.where((dist >= 0) & (dist < case["E"]), dist, torch.full_like(dist, case["E"])).long()
        x += torch.take_along_dim(table, slot, 1)
    s = torch.ones_like(i)
    if case["base"] > 0:
        s = torch.maximum(s, (i + 1).log() / math.log(case["base"]))
    x *= s[:, None]
    hide = dist < 0
    if case["window"]:
        hide |= (dist >= case["window"]) & (j >= case["sink"])
    return x.masked_fill_(hide, -math.inf), dist, s


def _exact_prologue(st):
    case = st["case"]
    H = case["Hkv"]
    q = st["q"].double()
    q_out = q / torch.sqrt(q.pow(2).sum(-1, keepdim=True) / D + 1e-6) * st["norm"][0].double()
    pools = [p.double() for p in st["pool"]]
    states = [torch.empty(len(st["lens"]), 3, H * D, dtype=torch.float64, device=DEV) for _ in range(2)]
    tok = 0
    for b, (n, nq) in enumerate(zip(st["lens"], st["q_lens"])):
        for i, name in enumerate(("k", "v")):
            hist = torch.zeros(nq + 3, H * D, dtype=torch.float64, device=DEV)
            if st["state"]:
                hist[:3] = st["state"][i][b].double()
            hist[3:] = st[name][tok:tok + nq].double().flatten(1)
            w = st["conv"][i].double()
            w = torch.cat([w[:, :1] + 1, w[:, 1:]], 1)                # the input added back
            y = sum(hist[3 - lag:nq + 3 - lag] * w[:, lag] for lag in range(4)).unflatten(1, (H, D))
            if name == "k":
                y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / D + 1e-6) * st["norm"][1].double()
            pools[i][st["where"][b][n - nq:]] = y
            states[i][b] = hist[nq:]
        tok += nq
    return (q_out, *pools, *states)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "prologue":
        return _exact_prologue(st)
    Hq, g = case["Hq"], case["Hq"] // case["Hkv"]
    Tq = st["q"].shape[0]
    if case["op"] == "extend":
        out = torch.empty(Tq, Hq, D, dtype=torch.float64, device=DEV)
        lse = torch.empty(Hq, Tq, dtype=torch.float64, device=DEV)
    else:
        dq, dk, dv = (torch.zeros(st[n].shape, dtype=torch.float64, device=DEV) for n in ("q", "k", "v"))
        dr = torch.zeros(st["r"].shape, dtype=torch.float64, device=DEV) if case["E"] else None
    tok = 0
    for b, nq in enumerate(st["q_lens"]):
        for lo in range(0, nq, 2048):
            hi = min(nq, lo + 2048)
            at = slice(tok + lo, tok + hi)
            for head in range(Hq):
                kv = head // g
                xs = [(sp, *_x64(st, b, head, tok, lo, hi, sp)) for sp in _spans(st, b, lo, hi)]
                if case["op"] == "extend":
                    z = torch.logsumexp(torch.stack([torch.logsumexp(x, 1) for _, x, _, _ in xs]), 0)
                    lse[head, at] = z
                    out[at, head] = sum((x - z[:, None]).exp_() @ st["v"][st["where"][b][sp[0]:sp[1]], kv].double()
                                        for sp, x, _, _ in xs)
                    continue
                do = st["dout"][at, head].double()
                mean = (do * st["out"][at, head].double()).sum(1, keepdim=True)
                for sp, x, dist, s in xs:
                    rows = st["where"][b][sp[0]:sp[1]]
                    p = (x - st["lse"][head, at].double()[:, None]).exp_()
                    dv[rows, kv] += p.t() @ do
                    dl = p * (do @ st["v"][rows, kv].double().t() - mean) * s[:, None]
                    dq[at, head] += st["alpha"] * (dl @ st["k"][rows, kv].double())
                    dk[rows, kv] += st["alpha"] * (dl.t() @ st["q"][at, head].double())
                    if case["E"]:
                        slot = torch.where((dist >= 0) & (dist < case["E"]), dist, torch.full_like(dist, case["E"])).long()
                        sums = torch.zeros(hi - lo, case["E"] + 1, dtype=torch.float64, device=DEV).scatter_add_(1, slot, dl)
                        dr[at, head] += sums[:, :-1] @ st["P"].double().t()
        tok += nq
    if case["op"] == "extend":
        return out, lse
    return (dq, dk, dv) if dr is None else (dq, dk, dv, dr)
