"""New tokens over a cache (contiguous or paged), windows with sinks and their
gradients, and the prologue into pages, on the GPU against the fp64 oracle.

Tolerances count roundings.  A logit is a sum of 128 + r_dim exact products in
fp32 (the tensor cores truncate): off by at most 256 * 2^-24 of its products'
magnitudes, which moves lse by as much and the weights by that factor.  out: the
weights round to bf16 (2^-8 of each), the part of some keys may be carried in
bf16 to the next kernel (2^-8 of it), and the result rounds once (2^-8).
Gradients: one factor of every product rounds to bf16, the result rounds once,
and dl is a difference whose sides are off by 2^-16 of their terms (the oracle's
magnitudes hold 2^-8 of them, which the factor 2^-8 brings to that)."""
import numpy as np
import pytest
import torch

import relative_position_biased_gb300 as rpb
from oracle import extend as X
from tests import kvcache_util as U
from tests.conftest import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    rpb.build()
    rpb.load_library()


@pytest.fixture(autouse=True)
def _clean_error_word():
    if gpu_available():
        rpb.relattn_get_device_error()
    yield


def ok():
    torch.cuda.synchronize()
    st = rpb.relattn_get_device_error()
    assert st == rpb.RELATTN_OK, (rpb.STATUS_NAMES.get(st, st), hex(rpb.relattn_last_device_error_word()))


def rules(c, sink):
    return dict(alpha=c.alpha, window=c.window, sink=sink, base=c.base)


def call(c, d, sink, **kw):
    """extend on the device; rows of the pool that hold no key are NaN."""
    held = np.zeros(d["rows"], bool)
    for w in d["where"]:
        held[w] = True
    k, v = d["k"].clone(), d["v"].clone()
    k[~torch.from_numpy(held)] = float("nan")
    v[~torch.from_numpy(held)] = float("nan")
    args = [U.cuda(t) for t in (d["q"], k, v, d["r"], d["P"], d["cu_q"], d["cu_k"])]
    opts = dict(U.call_kw(c, d), sink=sink)
    opts.update(kw)
    return rpb.extend(*args, **opts)


def bounds(c, d, sink):
    out, lse, size, top = X.forward(d["q"], d["k"], d["v"], d["r"], d["P"], d["where"], c.q_lens, **rules(c, sink))
    dx = 256 * 2.0 ** -24 * top + 2.0 ** -20
    e_out = 2.0 ** -8 * (2 * size + np.abs(out)) + 4 * dx.T[:, :, None] * size + 1e-30
    return out, lse, e_out, dx + 2.0 ** -20 * np.abs(lse)


def check(c, sink=0, **kw):
    d = U.make(c)
    out, lse = call(c, d, sink, **kw)
    ok()
    ref, z, e_out, e_lse = bounds(c, d, sink)
    got, got_z = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(got).all() and np.isfinite(got_z).all()
    bad = np.abs(got - ref) - e_out
    assert (bad <= 0).all(), ("out", np.unravel_index(bad.argmax(), bad.shape), np.abs(got - ref).max())
    bad = np.abs(got_z - z) - e_lse
    assert (bad <= 0).all(), ("lse", np.unravel_index(bad.argmax(), bad.shape), np.abs(got_z - z).max())
    return out, lse


# ------------------------------------------------------------------ lengths, layouts, masks

LAYOUTS = [(16, 2, 64, 1024), (4, 1, 32, 64), (12, 4, 16, 200), (4, 4, 16, 64), (8, 1, 0, 0), (6, 2, 24, 77), (5, 1, 7, 33),
           (8, 2, 8, 128)]


@pytest.mark.parametrize("Hq,Hkv,rd,E", LAYOUTS)
@pytest.mark.parametrize("page", [0, 16, 48, 128])
@pytest.mark.parametrize("q_lens,k_lens", [
    ((1,), (1,)), ((1, 1, 1), (301, 127, 700)), ((2, 0, 16, 1), (130, 64, 16, 515)), ((33, 7), (33, 400)), ((129, 70, 1), (385, 70, 256)),
])
def test_chunks(Hq, Hkv, rd, E, page, q_lens, k_lens):
    check(U.Case(q_lens, k_lens, Hq, Hkv, r_dim=rd, E=E, page=page, seed=len(q_lens) + page))


@pytest.mark.parametrize("Hq,Hkv,rd,E", LAYOUTS)
@pytest.mark.parametrize("window,sink", [(1, 0), (1, 1), (17, 4), (64, 200), (130, 3), (300, 130), (5000, 9)])
@pytest.mark.parametrize("page,q_lens,k_lens", [
    (32, (1, 1, 1), (40, 700, 333)), (0, (5, 1), (300, 700)), (64, (140, 3), (500, 260)), (0, (400, 90), (400, 90)),
])
def test_windows_with_sinks(Hq, Hkv, rd, E, window, sink, page, q_lens, k_lens):
    check(U.Case(q_lens, k_lens, Hq, Hkv, r_dim=rd, E=E, window=window, page=page, seed=window + sink), sink)


@pytest.mark.parametrize("num_splits", [1, 2])       # (0 takes the warp-MMA kernel for most of these)
@pytest.mark.parametrize("Hq,Hkv,rd,E", LAYOUTS)
@pytest.mark.parametrize("page,q_lens,k_lens,window,sink", [
    (0, (1,), (1,), 0, 0), (16, (1, 1), (17, 300), 0, 0), (16, (2, 0, 9), (64, 16, 129), 40, 3), (32, (33, 7), (33, 250), 0, 0),
    (0, (129, 1), (300, 256), 60, 2), (64, (40, 1), (41, 1), 9, 1),
])
def test_short_sequences_on_the_kernels_of_long_ones(Hq, Hkv, rd, E, page, q_lens, k_lens, window, sink, num_splits):
    check(U.Case(q_lens, k_lens, Hq, Hkv, r_dim=rd, E=E, window=window, page=page, seed=len(q_lens) + page), sink,
          num_splits=num_splits)


@pytest.mark.parametrize("k_len", [310, 320, 321, 330])
@pytest.mark.parametrize("q_len,window,sink", [(1, 0, 0), (1, 300, 19), (1, 300, 20), (20, 0, 0), (20, 290, 10), (20, 290, 11)])
def test_lengths_about_where_the_kernels_change(q_len, window, sink, k_len):
    check(U.Case((q_len,), (k_len,), 4, 1, r_dim=32, E=64, window=window, page=16, seed=k_len), sink)
    check(U.Case((q_len,), (k_len + 3000,), 4, 1, r_dim=32, E=64, window=window, page=16, seed=k_len), sink)


@pytest.fixture
def few_ctas():
    """(the test build runs the kernels that share their work on a few CTAs)"""
    with rpb.test_library():
        yield lambda n: rpb.relattn_test_band_ctas(n) == 0 or pytest.fail("no hook")
        rpb.relattn_test_band_ctas(0)


@pytest.mark.parametrize("ctas", [1, 2, 3, 7, 40])
@pytest.mark.parametrize("E,window,sink,num_splits", [(64, 0, 0, 0), (64, 700, 5, 0), (0, 0, 0, 0), (0, 300, 200, 3), (520, 0, 0, 2)])
@pytest.mark.parametrize("Hq,Hkv,page,q_lens,k_lens", [
    (8, 1, 16, (300, 5, 0, 70, 1), (1500, 2900, 40, 600, 333)),        # row tiles of one and of two, some cut
    (6, 2, 0, (90, 0, 0, 33), (2000, 0, 70, 2500)),                    # group 3: tiles that its heads do not fill
    (16, 2, 128, (17,), (6000,)),                                      # a tile in many shares
])
def test_shares_of_any_number_of_ctas(few_ctas, ctas, E, window, sink, num_splits, Hq, Hkv, page, q_lens, k_lens):
    few_ctas(ctas)
    check(U.Case(q_lens, k_lens, Hq, Hkv, r_dim=16 if E else 0, E=E, window=window, page=page, seed=ctas), sink,
          num_splits=num_splits)


def test_shares_of_many_sequences(few_ctas):
    """More sequences than a warp's 32 lanes and than the 12 warps that count their work, many of them empty or short."""
    rng = np.random.default_rng(8)
    q_lens = tuple(int(x) for x in rng.integers(0, 60, 90) * (rng.random(90) < 0.6))
    k_lens = tuple(n + int(x) for n, x in zip(q_lens, rng.integers(0, 600, 90) * (rng.random(90) < 0.5)))
    for ctas in (0, 5, 31):
        few_ctas(ctas)
        check(U.Case(q_lens, k_lens, 8, 1, r_dim=16, E=64, page=16, seed=2))


@pytest.mark.parametrize("q_len,num_splits", [(1, 0), (1, 1), (1, 3), (40, 0), (40, 1), (300, 0)])
@pytest.mark.parametrize("rd", [16, 7])                     # (7: the kernel of any shape)
def test_the_largest_window_and_number_of_sinks(q_len, num_splits, rd):
    top = 2 ** 31 - 1
    c = U.Case((q_len, 1), (900, 50), 8, 2, r_dim=rd, E=64, window=100, page=16, seed=1)
    d = U.make(c)
    a = call(c, d, top, num_splits=num_splits)
    b = call(c, d, 900, num_splits=num_splits)
    ok()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check(c, 900, num_splits=num_splits)
    check(U.Case((q_len, 1), (900, 50), 8, 2, r_dim=rd, E=64, window=top, page=16, seed=1), top, num_splits=num_splits)


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("base", [0.0, 16.0])
@pytest.mark.parametrize("q_lens,k_lens", [((1, 1), (90, 300)), ((40, 300), (90, 300))])
def test_log_scale_and_sign(sign, base, q_lens, k_lens):
    check(U.Case(q_lens, k_lens, 8, 2, r_dim=32, E=64, base=base, page=32, sign=sign, seed=5))


@pytest.mark.parametrize("q_lens,k_lens,window,sink", [
    ((1, 1), (9000, 4000), 0, 0), ((20,), (6000,), 0, 0), ((150,), (5000,), 1500, 5), ((600,), (2600,), 0, 0), ((9, 9), (5000, 1), 0, 0),
    ((64,), (5000,), 2000, 129),
])
@pytest.mark.parametrize("num_splits", [0, 1, 3])
def test_long_caches(q_lens, k_lens, window, sink, num_splits):
    k_lens = tuple(max(a, b) for a, b in zip(q_lens, k_lens))
    check(U.Case(q_lens, k_lens, 16, 2, r_dim=64, E=1024, window=window, page=16, seed=9), sink, num_splits=num_splits)


def test_many_sequences():
    rng = np.random.default_rng(4)
    k_lens = tuple(int(x) for x in rng.integers(1, 300, 150))
    check(U.Case((1,) * 150, k_lens, 8, 2, r_dim=16, E=64, page=16, seed=3))
    q_lens = tuple(min(n, int(x)) for n, x in zip(k_lens, rng.integers(0, 40, 150)))
    check(U.Case(q_lens, k_lens, 8, 2, r_dim=16, E=64, window=50, page=16, seed=3), 3)


@pytest.mark.parametrize("Hq,Hkv,rd,E", [(20, 1, 16, 64), (32, 1, 64, 128), (128, 1, 8, 64), (130, 1, 8, 64), (24, 8, 8, 136),
                                         (3, 1, 64, 64), (2, 1, 40, 600), (6, 6, 16, 2048)])
@pytest.mark.parametrize("q_lens,k_lens,window,sink", [((33, 1), (200, 150), 0, 0), ((5, 140), (700, 300), 90, 6)])
def test_groups_and_extents(Hq, Hkv, rd, E, q_lens, k_lens, window, sink):
    check(U.Case(q_lens, k_lens, Hq, Hkv, r_dim=rd, E=E, window=window, page=16, seed=Hq), sink)


def test_sequences_without_tokens_or_keys():
    for q_lens, k_lens in (((0, 1, 0), (0, 70, 300)), ((0, 40, 0, 20), (0, 70, 300, 20)), ((0,), (0,))):
        if sum(q_lens):
            check(U.Case(q_lens, k_lens, 8, 2, r_dim=16, E=64, page=32))
    # no rows at all: nothing is launched
    c = U.Case((0,), (60,), 8, 2, r_dim=16, E=64)
    out, lse = call(c, U.make(c), 0, max_seqlen_q=1)
    ok()
    assert out.shape == (0, 8, 128) and lse.shape == (8, 0)


@pytest.mark.parametrize("q_len", [1, 30])
def test_a_pool_of_more_than_32_bits_of_elements(q_len):
    """The pages used lie past 2^31 elements (and 2^32 bytes) of the pool."""
    page, pages = 64, 140000
    c = U.Case((q_len,), (500,), 8, 2, r_dim=16, E=64, window=200, page=page, seed=3)
    d = U.make(c)
    k, v = (torch.empty(pages * page, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert k.numel() > 1 << 31
    n = d["table"].shape[1]
    far = torch.arange(pages - n, pages, dtype=torch.int32).flip(0)
    for i in range(n):
        src, dst = int(d["table"][0, i]) * page, int(far[i]) * page
        k[dst:dst + page] = d["k"][src:src + page].cuda()
        v[dst:dst + page] = d["v"][src:src + page].cuda()
    kw = dict(U.call_kw(c, d), sink=4, block_table=far.view(1, -1).cuda())
    out, lse = rpb.extend(d["q"].cuda(), k, v, d["r"].cuda(), d["P"].cuda(), d["cu_q"].cuda(), d["cu_k"].cuda(), **kw)
    ok()
    ref, z, e_out, e_lse = bounds(c, d, 4)
    assert (np.abs(out.double().cpu().numpy() - ref) <= e_out).all()
    assert (np.abs(lse.double().cpu().numpy() - z) <= e_lse).all()
    # and the prologue writes there
    x, _ = prologue_inputs(c)
    cu = [U.W.cu_seqlens(m).cuda() for m in (c.q_lens, c.k_lens)]
    flat = [torch.zeros(500, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    rpb.prologue(*x.values(), *cu, *flat)
    rpb.prologue(*x.values(), *cu, k, v, block_table=far.view(1, -1).cuda(), page_size=page)
    ok()
    p = torch.arange(500 - q_len, 500)
    at = (far.long()[p // page] * page + p % page).cuda()
    assert torch.equal(flat[0][500 - q_len:], k[at]) and torch.equal(flat[1][500 - q_len:], v[at])


def test_python_refuses_other_layouts():
    c = U.Case((3,), (200,), 8, 2, r_dim=16, E=64, page=32)
    d = U.make(c)
    t = {n: U.cuda(d[n]) for n in ("q", "k", "v", "r", "P", "cu_q", "cu_k")}
    kw = dict(U.call_kw(c, d))
    run = lambda **over: rpb.extend(*dict(t, **over).values(), **kw)  # noqa: E731
    wide = torch.zeros(d["rows"], 2, 256, dtype=torch.bfloat16, device="cuda")
    for over in (dict(k=wide[..., :128]), dict(v=t["v"][:-32]), dict(q=t["q"].float()), dict(cu_k=t["cu_k"].long()),
                 dict(P=t["P"][:8]), dict(v=t["v"].cpu()), dict(k=wide[..., :128], v=wide[..., 128:])):
        with pytest.raises(ValueError):
            run(**over)
    with pytest.raises(ValueError, match="multiple of page_size"):
        rpb.extend(*t.values(), **dict(kw, page_size=80))
    with pytest.raises(ValueError, match="total_k rows"):
        rpb.extend(*t.values(), **dict(kw, block_table=None, total_k=100))
    with pytest.raises(rpb.RelattnError):                        # a workspace too small for the call
        rpb.extend(t["q"].repeat(20, 1, 1), t["k"], t["v"], t["r"].repeat(20, 1, 1), t["P"],
                   torch.tensor([0, 60], dtype=torch.int32, device="cuda"), t["cu_k"],
                   **dict(kw, max_seqlen_q=60, num_splits=2, workspace=torch.empty(16, device="cuda")))
    ok()


# ------------------------------------------------------------------ pages and rows that must not matter

@pytest.mark.parametrize("q_len,page", [(1, 16), (1, 64), (40, 16), (200, 128)])
def test_pages_behind_the_window_may_be_gone(q_len, page):
    c = U.Case((q_len,), (1500,), 8, 2, r_dim=32, E=64, window=100, page=page, seed=1)
    d = U.make(c)
    a = call(c, d, 5)
    ok()
    first = 1500 - q_len - 100 + 1
    gone = np.arange(d["table"].shape[1])
    gone = gone[((gone + 1) * page <= first) & (gone * page >= 5)]
    assert len(gone) > 3
    d["table"][0, gone] = torch.where(torch.arange(len(gone)) % 2 == 0, -7, 1 << 30).to(torch.int32)
    b = call(c, d, 5)
    ok()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("q_len", [1, 40, 200])
def test_a_needed_page_outside_the_pool_is_recorded(q_len):
    c = U.Case((q_len,), (600,), 8, 2, r_dim=32, E=64, page=64, seed=1)
    d = U.make(c)
    d["table"][0, 2] = 1 << 20
    out, _ = call(c, d, 0)
    torch.cuda.synchronize()
    assert rpb.relattn_get_device_error() == 6
    assert torch.isfinite(out).all()
    # its keys read as zero
    d["k"] = torch.cat([d["k"], torch.zeros(128, 2, 128, dtype=torch.bfloat16)])
    d["v"] = torch.cat([d["v"], torch.zeros(128, 2, 128, dtype=torch.bfloat16)])
    w = d["where"][0].copy()
    w[128:192] = d["rows"]
    ref, z, size, top = X.forward(d["q"], d["k"], d["v"], d["r"], d["P"], [w], c.q_lens, **rules(c, 0))
    assert (np.abs(out.double().cpu().numpy() - ref) <= 2.0 ** -7 * (size + np.abs(ref)) + 1e-3 * size).all()


@pytest.mark.parametrize("q_lens,k_lens", [((1, 1, 1), (50, 60, 70)), ((30, 20, 40), (50, 60, 70))])
def test_rows_of_no_sequence_and_bad_lengths_keep_their_outputs(q_lens, k_lens):
    c = U.Case(q_lens, k_lens, 8, 2, r_dim=16, E=64, page=32)
    d = U.make(c)
    Tq = sum(q_lens)
    pad = torch.cat([d["q"], d["q"][:1].expand(5, -1, -1)])
    d2 = dict(d, q=pad, r=torch.cat([d["r"], d["r"][:1].expand(5, -1, -1)]))
    out = torch.full((Tq + 5, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((8, Tq + 5), 7.0, device="cuda")
    call(c, d2, 0, out=out, lse=lse)
    ok()
    assert (out[Tq:] == 7).all() and (lse[:, Tq:] == 7).all()
    ref, z, e_out, e_lse = bounds(c, d, 0)
    assert (np.abs(out[:Tq].double().cpu().numpy() - ref) <= e_out).all()
    # a sequence longer than the bound is skipped and recorded, the others are not
    out.fill_(7.0)
    lse.fill_(7.0)
    call(c, d2, 0, out=out, lse=lse, max_seqlen_k=65)
    torch.cuda.synchronize()
    assert rpb.relattn_get_device_error() == 6
    n = q_lens[0] + q_lens[1]
    assert (np.abs(out[:n].double().cpu().numpy() - ref[:n]) <= e_out[:n]).all() and (out[n:] == 7).all()


# ------------------------------------------------------------------ streams, graphs, workspaces

@pytest.mark.parametrize("q_lens", [(1, 1), (70, 20), (200, 300)])
def test_captured_calls_follow_new_lengths_and_pages(q_lens):
    c = U.Case(q_lens, (900, 640), 8, 2, r_dim=32, E=64, window=200, page=32, seed=2)
    d = U.make(c)
    t = {n: U.cuda(d[n]) for n in ("q", "k", "v", "r", "P", "cu_q", "cu_k", "table")}
    kw = dict(U.call_kw(c, d), sink=4, block_table=t["table"], max_seqlen_q=max(q_lens), max_seqlen_k=900)
    run = lambda: rpb.extend(t["q"], t["k"], t["v"], t["r"], t["P"], t["cu_q"], t["cu_k"], **kw)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out, lse = run()
    for k_lens in ((900, 640), (300, 333), (q_lens[0], 510)):
        c2 = U.Case(q_lens, k_lens, 8, 2, r_dim=32, E=64, window=200, page=32, seed=7)
        d2 = U.make(c2)
        for n in ("q", "r", "P"):
            t[n].copy_(d2[n])
        t["k"][:d2["rows"]].copy_(d2["k"])
        t["v"][:d2["rows"]].copy_(d2["v"])
        t["cu_k"].copy_(d2["cu_k"])
        t["table"].fill_(-1)
        t["table"][:, :d2["table"].shape[1]].copy_(d2["table"])
        g.replay()
        ok()
        ref, z, e_out, e_lse = bounds(c2, d2, 4)
        assert (np.abs(out.double().cpu().numpy() - ref) <= e_out).all()
        assert (np.abs(lse.double().cpu().numpy() - z) <= e_lse).all()


@pytest.mark.parametrize("q_lens", [(1, 1, 1), (30, 70, 1), (260, 90, 1)])
def test_calls_repeat_bit_for_bit_on_any_stream(q_lens):
    c = U.Case(q_lens, (1900, 1640, 900), 16, 2, r_dim=64, E=512, page=16, seed=2)
    d = U.make(c)
    a = call(c, d, 0)
    s = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    both = [call(c, d, 0, stream=x.cuda_stream) for x in s]
    ok()
    for b in both:
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_random_batches_are_prefills():
    """Contiguous and paged, mixed lengths and kernels: relattn_prefill's out and
    lse.  Each is within 2^-8 (2 sum p |v| + |out|) <= 2^-8 3 max |v| of the exact
    out (P and out in bf16), and lse within 256 2^-24 of a logit's products."""
    rng = np.random.default_rng(12)
    for n in range(28):
        Hq, Hkv = [(16, 2), (8, 1), (4, 4), (12, 4), (20, 1), (6, 6)][n % 6]
        kind, E = n % 4, int(rng.choice([0, 64, 520, 1024]))
        b = (3, 200, 20, 1)[kind]
        q_lens = rng.integers(0, (900, 4, 2, 200)[kind], b) + (kind == 3)
        if kind == 2:
            q_lens[rng.integers(b)] = rng.integers(1, 1500)
        k_lens = q_lens + rng.integers(0, (3000, 300, 5000, 20000)[kind], b)
        if q_lens.sum() == 0:
            continue
        c = U.Case(tuple(q_lens.tolist()), tuple(k_lens.tolist()), Hq, Hkv, r_dim=16 if E else 0, E=E, page=int(rng.choice([16, 48, 128])),
                   window=int(rng.choice([0, 0, 90, 2000])), base=float(rng.choice([0, 16])), seed=n)
        d = U.make(c)
        at = torch.from_numpy(np.concatenate(d["where"]).astype(np.int64))
        t = {m: U.cuda(d[m]) for m in ("q", "r", "P", "cu_q", "cu_k")}
        k, v = d["k"][at].cuda(), d["v"][at].cuda()
        kw = dict(max_seqlen_q=int(q_lens.max()), max_seqlen_k=int(k_lens.max()), alpha=c.alpha, window=c.window, log_scale_base=c.base)
        want = rpb.prefill(t["q"], k, v, t["r"], t["P"], t["cu_q"], t["cu_k"], **kw)
        num_splits = int(rng.choice([0, 0, 1, 3]))
        for got in (rpb.extend(t["q"], k, v, t["r"], t["P"], t["cu_q"], t["cu_k"], num_splits=num_splits, **kw),
                    call(c, d, 0, num_splits=num_splits)):
            ok()
            assert (got[0].float() - want[0].float()).abs().max() <= 2 * 2.0 ** -8 * 3 * v.abs().max().float(), n
            assert (got[1] - want[1]).abs().max() <= 2 * 256 * 2.0 ** -24 * 200, n      # (products of a logit: below 200 here)


@pytest.mark.parametrize("q_lens,k_lens,window,num_splits", [
    ((1, 1), (5000, 40), 0, 0), ((300, 5, 70), (3000, 2900, 600), 0, 0), ((1300, 40), (4000, 40), 0, 0), ((1300, 40), (4000, 40), 500, 3),
    ((200, 100), (200, 100), 0, 1),
])
def test_a_workspace_may_hold_anything(q_lens, k_lens, window, num_splits):
    c = U.Case(q_lens, k_lens, 16, 2, r_dim=16, E=128, window=window, page=16, seed=4)
    d = U.make(c)
    a = call(c, d, 4, num_splits=num_splits)
    for fill in (0, 255, 1):
        b = call(c, d, 4, num_splits=num_splits, workspace=torch.full((1 << 27,), fill, dtype=torch.uint8, device="cuda"))
        ok()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("q_lens,k_lens,num_splits", [((1, 1), (5000, 40), 0), ((300, 5, 70), (3000, 2900, 600), 0),
                                                      ((1300, 40), (4000, 40), 0), ((300, 40), (4000, 600), 1), ((5,), (60,), 0)])
def test_out_and_workspace_of_sixteen_byte_alignment(q_lens, k_lens, num_splits):
    c = U.Case(q_lens, k_lens, 16, 2, r_dim=16, E=128, page=16, seed=4)
    d = U.make(c)
    a = call(c, d, 0, num_splits=num_splits)
    n = sum(q_lens) * 16 * 128
    out = torch.full((n + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty((1 << 27) + 16, dtype=torch.uint8, device="cuda")[16:]
    mine = out[8:8 + n].view(sum(q_lens), 16, 128)
    assert mine.data_ptr() % 32 == 16 and ws.data_ptr() % 32 == 16
    b = call(c, d, 0, num_splits=num_splits, out=mine, workspace=ws)
    ok()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and (out[:8] == 7).all() and (out[8 + n:] == 7).all()


# ------------------------------------------------------------------ gradients

def grads(c, sink):
    d = U.make(c)
    t = {n: U.cuda(d[n]) for n in ("q", "k", "v", "r", "P", "cu_q", "cu_k")}
    kw = dict(max_seqlen_q=max(c.q_lens), max_seqlen_k=max(c.k_lens), alpha=c.alpha, window=c.window, log_scale_base=c.base)
    out, lse = rpb.extend(*t.values(), sink=sink, **kw)
    dout = U.bf16(np.random.default_rng(8).standard_normal(out.shape)).cuda()
    args = (t["q"], t["k"], t["v"], t["r"], t["P"], out, lse, dout, t["cu_q"], t["cu_k"])
    return d, out, lse, dout, args, kw


def check_grads(c, sink):
    d, out, lse, dout, args, kw = grads(c, sink)
    got = rpb.backward(*args, sink=sink, **kw)
    ok()
    ref = X.backward(d["q"], d["k"], d["v"], d["r"], d["P"], out, lse, dout, d["where"], c.q_lens, **rules(c, sink))
    _, _, _, top = X.forward(d["q"], d["k"], d["v"], d["r"], d["P"], d["where"], c.q_lens, **rules(c, sink))
    slack = 1 + 2 * 256 * 2.0 ** -24 * top.max() * 2 ** 8
    for n, g in zip(("dq", "dk", "dv", "dr"), got):
        if n not in ref:
            assert g is None or not g.any()
            continue
        val, mag = ref[n]
        diff = np.abs(g.double().cpu().numpy() - val)
        # dq / dr: 2^-8 of the part of some keys carried by another product chain is within the terms'
        lim = 2.0 ** -8 * (slack * mag + np.abs(val)) + 1e-30
        bad = diff - lim
        assert (bad <= 0).all(), (n, np.unravel_index(bad.argmax(), bad.shape), diff.max(), lim.ravel()[bad.argmax()])


GRAD_LAYOUTS = [(16, 2, 64, 1024), (4, 1, 32, 64), (12, 4, 16, 200), (4, 4, 16, 64), (8, 1, 0, 0), (6, 2, 24, 77)]


@pytest.mark.parametrize("Hq,Hkv,rd,E", GRAD_LAYOUTS)
@pytest.mark.parametrize("window,sink", [(1, 1), (20, 4), (64, 16), (90, 17), (200, 70)])
@pytest.mark.parametrize("q_lens,k_lens", [((1,), (1,)), ((40, 21), (40, 21)), ((300, 1, 150), (300, 90, 200)), ((130,), (430,))])
def test_gradients(Hq, Hkv, rd, E, window, sink, q_lens, k_lens):
    check_grads(U.Case(q_lens, k_lens, Hq, Hkv, r_dim=rd, E=E, window=window, seed=sink), sink)


@pytest.mark.parametrize("Hq,Hkv,rd,E", [(16, 2, 64, 1024), (4, 4, 0, 0), (20, 1, 16, 128)])
@pytest.mark.parametrize("window", [1, 70, 600])
@pytest.mark.parametrize("q_lens,k_lens", [((1000, 3, 0, 250), (1000, 900, 20, 251)), ((7,) * 150, (7, 30, 300) * 50)])
def test_gradients_of_sinks_that_are_all_keys_need_no_window(Hq, Hkv, rd, E, window, q_lens, k_lens):
    """Both sums are over the same pairs, in another order; each gradient is within
    2^-7 of the exact one's norm (the library's bound for relattn_backward)."""
    d, out, lse, dout, args, kw = grads(U.Case(q_lens, k_lens, Hq, Hkv, r_dim=rd, E=E, seed=window), 0)
    a = rpb.backward(*args, **kw)
    b = rpb.backward(*args, **dict(kw, window=window), sink=1024)
    ok()
    for x, y in zip(a, b):
        if x is not None:
            assert (x.float() - y.float()).norm() <= 2 * 2.0 ** -7 * x.float().norm()


def test_gradients_of_inconsistent_lengths_leave_the_sequence_out():
    c = U.Case((60, 90, 50), (60, 90, 50), 8, 2, r_dim=16, E=64, window=20)
    d, out, lse, dout, args, kw = grads(c, 3)
    good = rpb.backward(*args, sink=3, **kw)
    ok()
    got = [torch.full_like(t, 7.0) for t in good]
    rpb.backward(*args, sink=3, **dict(kw, max_seqlen_q=60, max_seqlen_k=60), **dict(zip(("dq", "dk", "dv", "dr"), got)))
    torch.cuda.synchronize()
    assert rpb.relattn_get_device_error() == 6
    for a, b in zip(good, got):
        assert torch.equal(a[:60], b[:60]) and torch.equal(a[150:], b[150:]) and (b[60:150] == 7).all()


def test_gradients_captured_and_replayed():
    c = U.Case((200, 120), (200, 120), 8, 2, r_dim=16, E=64, window=40)
    d, out, lse, dout, args, kw = grads(c, 3)
    want = rpb.backward(*args, sink=3, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        rpb.backward(*args, sink=3, **kw)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            got = rpb.backward(*args, sink=3, **kw)
    for t in got:
        t.zero_()
    torch.cuda.synchronize()
    g.replay()
    ok()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_a_workspace_of_gradients_may_hold_anything():
    d, out, lse, dout, args, kw = grads(U.Case((300, 120), (300, 200), 8, 2, r_dim=16, E=128, window=40), 30)
    a = rpb.backward(*args, sink=30, **kw)
    for fill in (0, 255):
        b = rpb.backward(*args, sink=30, workspace=torch.full((1 << 26,), fill, dtype=torch.uint8, device="cuda"), **kw)
        ok()
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_gradients_log_scale_and_longer():
    check_grads(U.Case((700, 500), (700, 650), 8, 2, r_dim=32, E=64, window=128, base=16.0, seed=1), 5)
    check_grads(U.Case((1500,), (1500,), 8, 1, r_dim=16, E=200, window=300, seed=1), 4)


def test_no_sink_is_the_plain_backward_bit_for_bit():
    c = U.Case((300, 150), (300, 200), 8, 2, r_dim=32, E=64, window=70)
    d, out, lse, dout, args, kw = grads(c, 0)
    a = rpb.backward(*args, **kw)
    prm = rpb.RelattnBwdParams(
        fwd=rpb.make_params(*args[:5], *args[8:], out=out, lse=lse, **kw), dout=dout.data_ptr(),
        **{n: torch.empty_like(t).data_ptr() for n, t in ()})
    got = [torch.empty_like(t) for t in a]
    prm.dq, prm.dk, prm.dv, prm.dr = (t.data_ptr() for t in got)
    st, n = rpb.relattn_backward_sinks_workspace_size(prm, 0)
    assert st == 0 and n == rpb.relattn_backward_workspace_size(prm)[1]
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    prm.workspace, prm.workspace_bytes = ws.data_ptr(), n
    assert rpb.relattn_backward_sinks(prm, 0, torch.cuda.current_stream().cuda_stream) == 0
    ok()
    assert all(torch.equal(x, y) for x, y in zip(a, got))


def test_gradients_repeat_bit_for_bit():
    c = U.Case((900, 450), (900, 450), 16, 2, r_dim=64, E=256, window=200)
    _, _, _, _, args, kw = grads(c, 4)
    a, b = rpb.backward(*args, sink=4, **kw), rpb.backward(*args, sink=4, **kw)
    ok()
    assert all(torch.equal(x, y) for x, y in zip(a, b))


# ------------------------------------------------------------------ the prologue into pages, and all together

def prologue_inputs(c, seed=0, state=True):
    rng = np.random.default_rng(seed)
    Tq, C = sum(c.q_lens), c.Hkv * 128
    f = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda()  # noqa: E731
    x = dict(q=f(Tq, c.Hq, 128).bfloat16(), k=f(Tq, c.Hkv, 128).bfloat16(), v=f(Tq, c.Hkv, 128).bfloat16(),
             conv_k=0.3 * f(C, 4), conv_v=0.3 * f(C, 4), norm_q=1 + 0.1 * f(128), norm_k=1 + 0.1 * f(128))
    st = [f(len(c.q_lens), 3, C).bfloat16() for _ in range(2)] if state else None
    return x, st


@pytest.mark.parametrize("Hq,Hkv", [(16, 2), (4, 1), (64, 64)])       # (the last takes the kernel without staging)
@pytest.mark.parametrize("page,q_lens,k_lens", [(16, (1, 1), (17, 300)), (48, (100, 3, 0, 70), (100, 60, 9, 500)), (128, (40,), (256,))])
def test_prologue_into_pages_writes_the_contiguous_prologues_rows(Hq, Hkv, page, q_lens, k_lens):
    c = U.Case(q_lens, k_lens, Hq, Hkv, r_dim=0, E=0, page=page)
    rows, table, where = U.rows_of(k_lens, page, 3)
    x, st = prologue_inputs(c)
    cu = [U.W.cu_seqlens(n).cuda() for n in (q_lens, k_lens)]
    flat = [torch.full((sum(k_lens), Hkv, 128), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pool = [torch.full((rows, Hkv, 128), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    outs = [[torch.zeros_like(t) for t in st] for _ in range(2)]
    q1 = rpb.prologue(*x.values(), *cu, *flat, conv_state_in=st, conv_state_out=outs[0])
    q2 = rpb.prologue(*x.values(), *cu, *pool, conv_state_in=st, conv_state_out=outs[1], block_table=table.cuda(), page_size=page)
    ok()
    assert torch.equal(q1, q2) and all(torch.equal(a, b) for a, b in zip(*outs))
    at = torch.from_numpy(np.concatenate(where)).cuda()
    rest = torch.ones(rows, dtype=torch.bool, device="cuda")
    rest[at] = False
    for f, p in zip(flat, pool):
        assert torch.equal(f, p[at]) and (p[rest] == 9).all()


def test_prologue_skips_pages_outside_the_pool():
    c = U.Case((20, 20), (40, 40), 4, 2, r_dim=0, E=0, page=16)
    rows, table, where = U.rows_of(c.k_lens, 16, 3)
    x, _ = prologue_inputs(c)
    cu = [U.W.cu_seqlens(n).cuda() for n in (c.q_lens, c.k_lens)]
    table[0, 2] = 1 << 20
    pool = [torch.full((rows, 2, 128), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    rpb.prologue(*x.values(), *cu, *pool, block_table=table.cuda(), page_size=16)
    torch.cuda.synchronize()
    assert rpb.relattn_get_device_error() == 6
    for p in pool:
        assert (p[torch.from_numpy(where[0][32:]).cuda()] == 9).all()
        assert (p[torch.from_numpy(np.concatenate([where[0][20:32], where[1][20:]])).cuda()] != 9).any(-1).all()


def test_a_conversation_through_pages():
    """Two prompts in chunks, then single tokens: every step's prologue writes
    pages and its attention reads them; each step against the oracle over the
    rows that the contiguous prologue gives."""
    c = U.Case((0, 0), (0, 0), 8, 2, r_dim=16, E=64, window=150, page=16)
    steps = [(200, 35), (70, 1), (1, 90), (1, 1), (1, 1), (5, 1)]
    total = [sum(s[i] for s in steps) for i in range(2)]
    rows, table, where = U.rows_of(total, 16, 5)
    pool = [torch.full((rows, 2, 128), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    state = [torch.zeros(2, 3, 256, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    x0, _ = prologue_inputs(U.Case((1,), (1,), 8, 2), seed=7)
    rng = np.random.default_rng(6)
    P = U.bf16(0.1 * rng.standard_normal((16, 64)))
    have = [0, 0]
    for n, s in enumerate(steps):
        have = [a + b for a, b in zip(have, s)]
        cs = U.Case(s, tuple(have), 8, 2, r_dim=16, E=64, window=150, page=16)
        x, _ = prologue_inputs(cs, seed=20 + n, state=False)
        x.update({k: x0[k] for k in ("conv_k", "conv_v", "norm_q", "norm_k")})
        cu = [U.W.cu_seqlens(v).cuda() for v in (s, have)]
        new = [torch.empty_like(t) for t in state]
        q = rpb.prologue(*x.values(), *cu, *pool, conv_state_in=state, conv_state_out=new, block_table=table.cuda(), page_size=16)
        state = new
        r = U.bf16(rng.standard_normal((sum(s), 8, 16)))
        out, lse = rpb.extend(q, *pool, r.cuda(), P.cuda(), *cu, max_seqlen_q=max(s), max_seqlen_k=max(have), alpha=cs.alpha,
                              window=150, sink=4, block_table=table.cuda(), page_size=16, total_k=sum(have))
        ok()
        d = dict(q=q, k=pool[0], v=pool[1], r=r, P=P, where=[w[:m] for w, m in zip(where, have)])
        ref, z, e_out, e_lse = bounds(cs, d, 4)
        assert (np.abs(out.double().cpu().numpy() - ref) <= e_out).all(), n
        assert (np.abs(lse.double().cpu().numpy() - z) <= e_lse).all(), n
