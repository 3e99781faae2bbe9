"""The compressed K / V cache on the GPU against the fp64 oracle: NVFP4 rows in
and out, decode over them, the weight each key receives, eviction, and a run
of them together.  Tolerances count roundings (tests/kvcache_util.py)."""
import numpy as np
import pytest
import torch

import relative_position_biased_gb300 as rpb
from oracle import kvcache as C
from relative_position_biased_gb300 import workloads as W
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
    assert st == rpb.RELATTN_OK, rpb.STATUS_NAMES.get(st, st)


def host(t):
    return t.cpu().numpy()


# ------------------------------------------------------------------ store and load

@pytest.mark.parametrize("q_lens,k_lens,Hkv,page,factors", [
    ((1,), (1,), 1, 0, False),
    ((37, 0, 5), (37, 3, 260), 2, 0, True),
    ((1,) * 9, (33, 1, 64, 65, 100, 7, 31, 32, 96), 2, 32, True),
    ((130, 64), (130, 200), 3, 64, False),
])
def test_store_writes_the_chunk_rows_and_no_others(q_lens, k_lens, Hkv, page, factors):
    c = U.Case(q_lens, k_lens, Hkv, Hkv, page=page, factors=factors)
    d = U.make(c)
    rows = np.concatenate([w[len(w) - n:] for w, n in zip(d["where"], q_lens)])
    k, v = d["k"][rows], d["v"][rows]
    cache = rpb.empty_nvfp4(d["rows"], Hkv, "cuda", *(U.cuda(None if g is None else torch.from_numpy(g))
                                                     for g in (d["kg"], d["vg"])))
    for t in cache[:4]:
        t.fill_(0xA5)
    kw = dict(block_table=d["table"].cuda(), page_size=page) if page else {}
    cu = (d["cu_q"].cuda(), d["cu_k"].cuda())
    rpb.store_nvfp4(k.cuda(), v.cuda(), *cu, cache, **kw)
    ok()
    other = np.setdiff1d(np.arange(d["rows"]), rows)
    for x, codes, scales, g in ((k, cache.k, cache.k_scale, d["kg"]), (v, cache.v, cache.v_scale, d["vg"])):
        want_c, want_s = C.quantize_nvfp4(x.float().numpy(), g)
        np.testing.assert_array_equal(host(scales)[rows], want_s)
        np.testing.assert_array_equal(host(codes)[rows], want_c)
        assert (host(codes)[other] == 0xA5).all() and (host(scales)[other] == 0xA5).all()
    lk, lv = rpb.load_nvfp4(cache, *cu, total_q=len(rows), **kw)
    ok()
    for x, got, g in ((k, lk, d["kg"]), (v, lv, d["vg"])):
        ref = C.dequantize_nvfp4(*C.quantize_nvfp4(x.float().numpy(), g), g)
        # code * scale is exact; the factor's product rounds to fp32, then to bf16
        assert (np.abs(host(got.double()) - ref) <= np.abs(ref) * (2.0 ** -8 * (1 + 2.0 ** -20) + 2.0 ** -24)).all()


def test_calls_follow_a_cache_to_other_memory():
    x = U.bf16(np.ones((40, 1, 128))).cuda()
    cu = W.cu_seqlens([40]).cuda()
    cache = rpb.empty_nvfp4(40, 1, "cuda")
    left = [cache.k.view(cache.k.shape), cache.k_scale.view(cache.k_scale.shape)]      # (kept alive)
    rpb.store_nvfp4(x, x, cu, cu, cache)
    cache.k.data = torch.zeros_like(cache.k)
    cache.k_scale.set_(torch.zeros_like(cache.k_scale))
    rpb.store_nvfp4(2 * x, 2 * x, cu, cu, cache)
    ok()
    assert torch.equal(cache.k, left[0]) and not torch.equal(cache.k_scale, left[1]) and (cache.k_scale != 0).all()
    k, v = rpb.load_nvfp4(cache, cu, cu, total_q=40)
    ok()
    assert torch.equal(k, v) and (k > 1.5).all()


def _store_one(x, factor=None):
    n = x.shape[0]
    cu = W.cu_seqlens([n]).cuda()
    g = None if factor is None else torch.from_numpy(factor).cuda()
    cache = rpb.empty_nvfp4(n, x.shape[1], "cuda", g, g)
    rpb.store_nvfp4(x.cuda(), x.cuda(), cu, cu, cache)
    ok()
    return host(cache.k), host(cache.k_scale), host(cache.v), host(cache.v_scale)


@pytest.mark.parametrize("factor", [None, np.float32(0.0123), np.float32(2.0 ** -20), np.float32(3e4)])
def test_store_rounds_exactly(factor):
    """Every bf16 magnitude as a block's largest element, and elements next to
    and on the borders of the codes."""
    mags = torch.arange(0, 0x7f80, dtype=torch.int16).view(torch.bfloat16).float().numpy()
    n = (len(mags) + 7) // 8
    rng = np.random.default_rng(3)
    x = np.zeros((n, 8, 16), np.float32)
    x[:, :, 0] = np.resize(mags, n * 8).reshape(n, 8)
    x[:, :, 1:8] = x[:, :, :1] * np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], np.float32) / 6
    x[:, :, 8:] = x[:, :, :1] * rng.uniform(-1, 1, (n, 8, 8))
    xb = U.bf16(x.reshape(n, 1, 128))
    f = None if factor is None else np.array([factor], np.float32)
    ck, sk, cv, sv = _store_one(xb, f)
    want_c, want_s = C.quantize_nvfp4(xb.float().numpy(), f)
    np.testing.assert_array_equal(sk, want_s)
    np.testing.assert_array_equal(ck, want_c)
    np.testing.assert_array_equal(cv, want_c)
    np.testing.assert_array_equal(sv, want_s)


@pytest.mark.parametrize("factor", [None, 0.0123, 2.0 ** -20, 3e4, 1e-25])
def test_store_keeps_the_sign_of_zero(factor):
    """-0 (and magnitudes that round to it) beside nonzero elements, whichever way
    the quotient is made."""
    rng = np.random.default_rng(8)
    x = rng.standard_normal((40, 2, 128)).astype(np.float32)
    x *= (2.0 ** rng.integers(-60, 60, (40, 2, 8, 1))).repeat(16, 3).reshape(x.shape)
    x[rng.random(x.shape) < 0.3] = -0.0
    x[rng.random(x.shape) < 0.2] = 0.0
    x[rng.random(x.shape) < 0.1] = -1e-38
    xb = U.bf16(x)
    f = None if factor is None else np.full(2, factor, np.float32)
    ck, sk, cv, sv = _store_one(xb, f)
    want_c, want_s = C.quantize_nvfp4(xb.float().numpy(), f)
    assert ((want_c & 15) == 8).any() and (want_s > 0).any()
    for c, s in ((ck, sk), (cv, sv)):
        np.testing.assert_array_equal(s, want_s)
        np.testing.assert_array_equal(c, want_c)


def test_store_of_infinities_and_nan():
    x = np.ones((3, 1, 128), np.float32)
    x[0, 0, 3] = np.inf
    x[1, 0, 20] = -np.inf
    x[2, 0, 127] = np.nan
    ck, sk, _, _ = _store_one(U.bf16(x))
    want_c, want_s = C.quantize_nvfp4(x)
    np.testing.assert_array_equal(sk, want_s)
    np.testing.assert_array_equal(ck[:2], want_c[:2])
    assert sk[2, 0, 7] == 0x7F and (sk[2, 0, :7] == want_s[2, 0, :7]).all()


def test_store_records_bad_pages_and_lengths():
    x = U.bf16(np.ones((40, 1, 128)))
    cache = rpb.empty_nvfp4(64, 1, "cuda")
    table = torch.tensor([[1, 7]], dtype=torch.int32, device="cuda")      # page 7 is not in the pool
    cu = W.cu_seqlens([40]).cuda()
    rpb.store_nvfp4(x.cuda(), x.cuda(), cu, cu, cache, block_table=table, page_size=32)
    torch.cuda.synchronize()
    assert rpb.relattn_get_device_error() == 6
    assert (host(cache.k)[32:] != 0).all() and (host(cache.k)[:32] == 0).all()
    k, _ = rpb.load_nvfp4(cache, cu, cu, total_q=40, block_table=table, page_size=32)
    assert rpb.relattn_get_device_error() == 6
    # a block of ones: 1 / 6 is nearest to the scale 11 / 64, 64 / 11 to the code 6
    assert (host(k.float())[:32] == 6 * 11 / 64).all() and (host(k.float())[32:] == 0).all()
    # more chunk rows than keys, and keys past the cache: skipped, recorded
    for ck in ([8], [100]):
        cache = rpb.empty_nvfp4(64, 1, "cuda")
        rpb.store_nvfp4(x.cuda(), x.cuda(), cu, W.cu_seqlens(ck).cuda(), cache)
        assert rpb.relattn_get_device_error() == 6
        assert (host(cache.k) == 0).all()


# ------------------------------------------------------------------ decode

def run_decode(c, d, qc, cache=None, **kw):
    out, lse = rpb.decode_nvfp4(d["q"].cuda(), cache or U.device_cache(qc, d), U.cuda(d["r"]), U.cuda(d["P"]),
                                d["cu_q"].cuda(), d["cu_k"].cuda(), **{**U.call_kw(c, d), **kw})
    ok()
    return out, lse


DECODE = [
    U.Case((1,), (1,), 1, 1, E=0, r_dim=0, factors=False),
    U.Case((1,), (31,), 4, 1),
    U.Case((1, 1, 1, 1, 1), (32, 33, 127, 128, 129), 8, 1),
    U.Case((1,), (2900,), 16, 2, r_dim=64, E=1024, base=64.0),
    U.Case((9, 3, 1), (700, 130, 5), 16, 2, r_dim=64, E=256, base=64.0),       # 72 rows per kv head
    U.Case((16, 2), (300, 65), 2, 2, E=77, r_dim=24),                          # 16 rows, one head each
    U.Case((1, 0, 1), (257, 9, 640), 24, 1, E=100, r_dim=5),                   # 24 rows of one token
    U.Case((1, 1), (1500, 20), 16, 2, window=1),
    U.Case((4, 1, 2), (1500, 513, 90), 8, 2, window=100, E=64),
    U.Case((1, 1), (3000, 700), 12, 4, window=512, E=1024, r_dim=64),
    U.Case((1,) * 7, (33, 1, 64, 65, 1000, 7, 96), 16, 2, page=32),
    U.Case((5, 2), (1000, 321), 4, 1, page=64, window=200),
    U.Case((1, 1, 1), (600, 65, 2050), 16, 2, positions=True, base=64.0),
    U.Case((3, 9), (600, 65), 4, 2, positions=True, E=40, page=32),
    U.Case((1, 2), (900, 300), 8, 1, positions=True, window=150),
    # more than 32 rows of a kv head
    U.Case((16, 9), (1700, 300), 32, 2, E=300, r_dim=64, base=64.0),           # 256: two blocks of rows
    U.Case((7, 16, 0, 1), (900, 16, 5, 2050), 24, 2, page=32, window=130, E=64),
    U.Case((3,), (20000,), 16, 1, E=1024, r_dim=16),
    U.Case((5, 16), (129, 400), 8, 1, E=0, r_dim=0, window=1, factors=False),
    U.Case((9, 11, 12), (640, 96, 4097), 16, 2, E=1500, r_dim=8, page=96, sign=-1.0),
]


@pytest.mark.parametrize("i", range(len(DECODE)))
@pytest.mark.parametrize("splits", [0, 1, 3])
def test_decode(i, splits):
    c = DECODE[i]
    d = U.make(c)
    qc = U.quantized(c, d)
    out, lse = run_decode(c, d, qc, num_splits=splits)
    U.check_decode(c, d, qc["k_values"], qc["v_values"], out, lse)


@pytest.mark.parametrize("splits", [0, 1, 5, 100000])
@pytest.mark.parametrize("c", [
    U.Case((1, 1), (700, 2050), 16, 2, base=64.0),                             # 8 rows
    U.Case((3, 1), (2900, 40), 12, 2, E=100, window=300),                      # 18
    U.Case((9, 2), (700, 4100), 8, 1, E=256, r_dim=64),                        # 72
    U.Case((1, 2), (600, 2065), 8, 2, positions=True),
], ids=["8", "18", "72", "positions"])
def test_decode_under_a_bound_far_above_the_lengths(c, splits):
    """max_seqlen_k is a bound only: the workspace stays that of as many partials as
    the GPU runs CTAs, at most 4 an SM."""
    d = U.make(c)
    qc = U.quantized(c, d)
    bound = (1 << 31) - (1 << 16)
    out, lse = run_decode(c, d, qc, num_splits=splits, max_seqlen_k=bound)
    U.check_decode(c, d, qc["k_values"], qc["v_values"], out, lse)
    prm = rpb.RelattnParams(q=1 << 20, k=None, v=None, r=1 << 20, P=1 << 20, cu_seqlens_q=1 << 20, cu_seqlens_k=1 << 20,
                            batch=2, total_q=sum(c.q_lens), total_k=sum(c.k_lens), max_seqlen_q=max(c.q_lens),
                            max_seqlen_k=bound, num_heads_q=c.Hq, num_heads_kv=c.Hkv, head_dim=128, r_dim=c.r_dim,
                            rel_extent=c.E, window=c.window, alpha=0.1, log_scale_base=c.base, out=1 << 20, lse=1 << 20,
                            workspace=None, workspace_bytes=0, num_splits=splits)
    st, n = rpb.relattn_decode_nvfp4_workspace_size(prm, rpb.RelattnPositions(1 << 20, 1 << 20) if c.positions else None)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    row = sum(c.q_lens) * c.Hq
    assert st == 0 and n <= row * (4 * sms * (128 + 1) * 4 + c.E * 4) + 512


@pytest.mark.parametrize("nq,length,splits,batch", [
    (9, 1 << 27, 0, 1), (9, 1 << 22, 1, 1), (9, 1 << 22, 3, 1), (9, 1 << 21, 0, 390),
    (1, (1 << 31) - (1 << 16), 0, 1), (1, 1 << 24, 1, 1), (1, 1 << 23, 0, 390), (4, 1 << 24, 2, 1)])
def test_long_sums_keep_their_magnitude(nq, length, splits, batch):
    """The first sequence has one page of 65536 keys again and again, with values
    whose mean is 1.  The matrix instructions add to fp32 by truncation; a piece
    takes at most 4096 such additions, each short of less than a step (2^-23) of
    what has been summed, so outputs are short of at most 4096 * 2^-23 of their
    size.  The roundings of bf16 and of the f16 weights average out over the rows
    and dims (2^-12 is left for them); a weight's sum of 2^15 fp32 additions is
    off by half a step (2^-24) each at most."""
    page, Hq = 1 << 16, 8
    c = U.Case((nq,), (page,), Hq, 1, E=0, r_dim=0, factors=False, page=page)
    d = U.make(c)
    d["v"] = (d["v"].float() + 1.0).to(torch.bfloat16)
    qc = U.quantized(c, d)
    n = length // page
    table = torch.full((batch, n), int(d["table"][0, 0]), dtype=torch.int32, device="cuda")
    q = torch.cat([d["q"], d["q"][:1].expand(batch - 1, -1, -1)]).cuda().contiguous()
    cu_q = W.cu_seqlens([nq] + [1] * (batch - 1)).cuda()
    cu_k = W.cu_seqlens([length] + [70] * (batch - 1)).cuda()
    out, lse = rpb.decode_nvfp4(q, U.device_cache(qc, d), None, None, cu_q, cu_k, max_seqlen_q=nq, max_seqlen_k=length,
                                alpha=c.alpha, total_k=length + 70 * (batch - 1), block_table=table, page_size=page,
                                num_splits=splits)
    ok()
    K, V = qc["k_values"][d["where"][0], 0], qc["v_values"][d["where"][0], 0]
    short = []
    for hq in range(Hq):
        f = d["q"][:, hq].double().numpy()
        x0, _ = C.logits(f, K, None, None, np.full(nq, page), np.arange(page), alpha=c.alpha)
        x1, _ = C.logits(f, K, None, None, np.arange(page - nq, page), np.arange(page), alpha=c.alpha)      # the last copy
        m = x0.max(1)[:, None]
        s = (n - 1) * np.exp(x0 - m) + np.exp(x1 - m)
        ref = s @ V / s.sum(1)[:, None]
        short.append((host(out[:nq, hq].double()) - ref) / ref)
        z = np.log(s.sum(1)) + m[:, 0]
        assert np.abs(host(lse[hq, :nq].double()) - z).max() <= 2.0 ** 15 * 2.0 ** -24 + 2.0 ** -22 * np.abs(z).max()
        if batch > 1:                                    # and a short one beside it
            p, z = C.softmax(C.logits(f[:1], K[:70], None, None, [69], np.arange(70), alpha=c.alpha)[0])
            assert np.abs(host(out[-1, hq].double()) - (p @ V[:70])[0]).max() <= 2.0 ** -7 * np.abs(V).max()
            assert abs(float(lse[hq, -1]) - z[0]) <= 1e-5
    assert abs(np.mean(short)) <= 4096 * 2.0 ** -23 + 2.0 ** -12, np.mean(short)


@pytest.mark.parametrize("batch", [65, 513])
def test_decode_of_many_sequences(batch):
    """Past 384 sequences every unit has a CTA of its own."""
    rng = np.random.default_rng(batch)
    c = U.Case((1,) * batch, tuple(int(x) for x in rng.integers(1, 90, batch)), 4, 2, E=64)
    d = U.make(c)
    qc = U.quantized(c, d)
    out, lse = run_decode(c, d, qc)
    U.check_decode(c, d, qc["k_values"], qc["v_values"], out, lse)


@pytest.mark.parametrize("q_len", [1, 5])
def test_decode_with_large_and_tiny_queries(q_len):
    """Rows of far apart magnitudes in one unit, and a logit range that moves the
    running maximum by hundreds."""
    c = U.Case((q_len,), (900,), 8, 1, E=64)
    d = U.make(c)
    q = d["q"].float()
    q *= torch.tensor([1e-30, 1e-4, 0.0, 1.0, 30.0, 300.0, 3.0, 1e-38])[None, :, None]
    d["q"] = q.to(torch.bfloat16)
    qc = U.quantized(c, d)
    out, lse = run_decode(c, d, qc)
    U.check_decode(c, d, qc["k_values"], qc["v_values"], out, lse)


def test_rows_that_see_no_key_and_rows_of_no_sequence():
    c = U.Case((1, 2), (64, 200), 4, 1, positions=True)
    d = U.make(c)
    d["key_pos"][:, d["where"][0]] = -1                  # sequence 0: every key hidden
    d["key_pos"][:, d["where"][1]] = 10                  # sequence 1: every key after its queries
    d["q_pos"] = torch.tensor([5, 9], dtype=torch.int32)  # ... of row 0, at the second's position
    qc = U.quantized(c, d)
    for splits in (0, 1, 2):
        q = torch.cat([d["q"], d["q"][:2]]).cuda()       # two rows behind the last sequence
        r = torch.cat([d["r"], d["r"][:2]]).cuda()
        out = torch.full_like(q, 7.0)
        lse = torch.full((4, 5), 7.0, device="cuda")
        rpb.decode_nvfp4(q, U.device_cache(qc, d), r, d["P"].cuda(), d["cu_q"].cuda(), d["cu_k"].cuda(), out=out,
                         lse=lse, num_splits=splits, **U.call_kw(c, d))
        ok()
        assert (out[3:] == 7).all() and (lse[:, 3:] == 7).all()
        U.check_decode(c, d, qc["k_values"], qc["v_values"], out[:3], lse[:, :3])
        assert torch.isneginf(lse[:, :2]).all() and torch.isfinite(lse[:, 2]).all()


@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("Hq", [1, 3, 4])                # up to 9, 27 and 36 rows
def test_nan_in_masked_places_stays_there(window, Hq):
    """NaN scales in rows that only some query rows see: the others are clean."""
    c = U.Case((9, 2), (300, 150), Hq, 1, window=window, E=64)
    d = U.make(c)
    qc = U.quantized(c, d)
    bad = [int(d["where"][0][295]), int(d["where"][1][149])]    # seen by the last rows only
    if window:
        bad.append(int(d["where"][0][253]))                     # seen by row 0 and 1 (positions 291, 292)
        bad.append(int(d["where"][0][100]))                     # seen by none
    for n in ("k_scale", "v_scale"):
        qc[n][bad] = 0x7F
    out, lse = run_decode(c, d, qc)
    out, lse = host(out.float()), host(lse)
    sees = {0: [r for r in range(9) if 291 + r >= 295 or (window and r < 2)], 1: [1]}
    keys = np.where(np.isnan(C.dequantize_nvfp4(qc["k"], qc["k_scale"], d["kg"])), 0, qc["k_values"])
    values = np.where(np.isnan(C.dequantize_nvfp4(qc["v"], qc["v_scale"], d["vg"])), 0, qc["v_values"])
    clean = np.ones(11, bool)
    for b, q0 in ((0, 0), (1, 9)):
        for r in sees[b]:
            clean[q0 + r] = False
    assert np.isnan(out[~clean]).all() and np.isnan(lse[:, ~clean]).all()
    assert np.isfinite(out[clean]).all() and np.isfinite(lse[:, clean]).all()
    for b, hq, h, q0, x, mag in U.each_head(c, d, keys):
        p, z = C.softmax(x)
        for r in range(x.shape[0]):
            if clean[q0 + r]:
                # a rounding of bf16 and one of f16 on sums of magnitude below 1
                assert np.abs(out[q0 + r, hq] - p[r] @ values[d["where"][b], h]).max() < 2.0 ** -8
                assert abs(lse[hq, q0 + r] - z[r]) < 1e-3


@pytest.mark.parametrize("Hq", [1, 3, 4])
def test_one_nan_value_reaches_its_own_dims_only(Hq):
    c = U.Case((9,), (300,), Hq, 1, E=0, r_dim=0)
    d = U.make(c)
    qc = U.quantized(c, d)
    qc["v_scale"][295, 0, 3] = 0x7F                     # dims 48 .. 63 of a key that rows 4 .. 8 see
    out, lse = run_decode(c, d, qc)
    nan = np.isnan(host(out.float()))
    want = np.zeros((9, Hq, 128), bool)
    want[4:, :, 48:64] = True
    np.testing.assert_array_equal(nan, want)
    assert torch.isfinite(lse).all()


def test_decode_reports_bad_pages_positions_and_lengths():
    c = U.Case((1, 1), (300, 40), 4, 1, page=32)
    d = U.make(c)
    qc = U.quantized(c, d)
    good, _ = run_decode(c, d, qc)
    bad = d["table"].clone()
    bad[0, 3] = 10 ** 6
    args = (d["q"].cuda(), U.device_cache(qc, d), d["r"].cuda(), d["P"].cuda(), d["cu_q"].cuda(), d["cu_k"].cuda())
    kw = U.call_kw(c, d)
    out, lse = rpb.decode_nvfp4(*args, **{**kw, "block_table": bad.cuda()})
    torch.cuda.synchronize()
    assert rpb.relattn_get_device_error() == 6
    assert torch.isfinite(out.float()).all() and torch.equal(out[1], good[1])
    # a sequence longer than max_seqlen_k is skipped; the other one is computed
    out = torch.full_like(out, 7.0)
    rpb.decode_nvfp4(*args, **{**kw, "max_seqlen_k": 100}, out=out)
    assert rpb.relattn_get_device_error() == 6
    assert (out[0] == 7).all()
    # (its own plan may split it differently: one bf16 rounding apart)
    assert (out[1].float() - good[1].float()).abs().max() <= 2.0 ** -8 * good[1].float().abs().max()
    pos = torch.zeros(1, d["rows"], dtype=torch.int32, device="cuda")
    rpb.decode_nvfp4(*args, **kw, key_pos=pos, q_pos=torch.tensor([-3, 5], dtype=torch.int32, device="cuda"), out=out)
    assert rpb.relattn_get_device_error() == 6
    assert (out[0] == 7).all()


def test_cache_offsets_past_32_bits():
    """Pages at the end of a pool whose codes take more than 4 GB."""
    page, pages, Hkv = 128, (1 << 33) // (128 * 4 * 64) + 4, 4
    c = U.Case((1, 2), (300, 129), 8, Hkv, E=64)
    d = U.make(c)
    qc = U.quantized(c, d)
    small = U.device_cache(qc, d)
    rows = page * pages
    big = rpb.KvNvfp4(*(torch.empty(rows, Hkv, t.shape[2], dtype=torch.uint8, device="cuda") for t in small[:4]),
                      small.k_global, small.v_global)
    assert big.k.numel() > 1 << 32
    table = torch.tensor([[pages - 1, 0, pages - 3], [pages - 2, 1, -1]], dtype=torch.int32)
    where = []
    for b, n in enumerate(c.k_lens):
        p = np.arange(n)
        where.append(table[b].numpy()[p // page].astype(np.int64) * page + p % page)
        for s, t in zip(small[:4], big[:4]):
            t[torch.from_numpy(where[b]).cuda()] = s[torch.from_numpy(d["where"][b]).cuda()]
    kw = {**U.call_kw(c, d), "block_table": table.cuda(), "page_size": page}
    args = (U.cuda(d["r"]), U.cuda(d["P"]))
    cu = (d["cu_q"].cuda(), d["cu_k"].cuda())
    out, lse = rpb.decode_nvfp4(d["q"].cuda(), big, *args, *cu, **kw)
    ok()
    U.check_decode(c, d, qc["k_values"], qc["v_values"], out, lse)
    w = rpb.key_weights(d["q"].cuda(), big, *args, lse, *cu, **kw, decay=0.0,
                        out=torch.empty(Hkv, rows, device="cuda"))
    ok()
    got = torch.zeros(Hkv, d["rows"], device="cuda")
    for b in range(2):
        got[:, torch.from_numpy(d["where"][b]).cuda()] = w[:, torch.from_numpy(where[b]).cuda()]
    U.check_weights(c, d, qc["k_values"], host(lse), None, 0.0, got)
    # and the rows of its tail come back out of it
    keep = [100, 60]
    dst = [torch.empty(160, Hkv, t.shape[2], dtype=torch.uint8, device="cuda") for t in big[:4]]
    pos, _ = rpb.evict(big[:4], dst, w, cu[1], W.cu_seqlens(keep).cuda(), max_seqlen_k=300, recent=50, sink=2,
                       total_k=429, total_keep=160, block_table=table.cuda(), page_size=page)
    ok()
    for b, o in ((0, 0), (1, 100)):
        for h in range(Hkv):
            p = host(pos[h, o:o + keep[b]])
            np.testing.assert_array_equal(p, C.kept_keys(host(w)[h, where[b]], keep[b], 50, 2))
            for s, t in zip(small[:4], dst):
                np.testing.assert_array_equal(host(t)[o:o + keep[b], h], host(s)[d["where"][b][p], h])


# ------------------------------------------------------------------ key weights

WEIGHTS = [
    U.Case((1,), (1,), 1, 1, E=0, r_dim=0),
    U.Case((1, 1, 1), (33, 1000, 127), 8, 1),
    U.Case((2, 0, 1), (257, 40, 700), 16, 2, r_dim=64, E=256, base=64.0),      # 16 rows
    U.Case((9,), (700,), 16, 2, E=64),                                         # 72 rows
    U.Case((32, 5), (300, 1025), 4, 2, E=77, r_dim=24, base=64.0),             # an observation window
    U.Case((200, 1, 130), (200, 1, 130), 4, 1, E=64),                          # whole prompts
    U.Case((300, 40), (300, 90), 8, 2, E=64, window=50),
    U.Case((1, 1), (1500, 700), 16, 2, window=100, E=1024, r_dim=64),          # keys out of sight decay
    U.Case((1,) * 4, (33, 64, 500, 7), 8, 2, page=32),
    U.Case((20, 3), (150, 90), 8, 2, page=64, window=33),
    U.Case((1, 1), (600, 65), 16, 2, positions=True),
    U.Case((30, 3), (150, 90), 8, 2, positions=True, page=32, window=60),
    # rows past the bias band, several steps of 256 rows, ragged ends
    U.Case((700, 33, 1), (700, 33, 1), 6, 2, E=64, window=300, base=64.0),
    U.Case((500, 90), (777, 90), 4, 2, E=0, r_dim=0),
    U.Case((300,), (900,), 8, 1, E=0, r_dim=0, window=200, page=32),
    U.Case((520, 17), (520, 300), 2, 2, E=64, r_dim=16, page=64, base=64.0),   # 32 tokens in 32 rows
    U.Case((400,), (400,), 16, 1, E=100, r_dim=5),                             # unaligned r and P
    U.Case((31,), (2000,), 8, 1, E=64),
    U.Case((5,), (2000,), 16, 1, E=64),                                        # too few tokens for the tcgen05 kernel
    U.Case((330, 130), (330, 200), 1, 1, E=100, r_dim=16),                     # 128 tokens a step
    U.Case((300,), (400,), 4, 2, E=300, r_dim=64, window=250),                 # 64
    U.Case((150, 70), (190, 70), 8, 2, E=64, r_dim=8, base=64.0),              # 32
    U.Case((270,), (270,), 24, 2, E=128, r_dim=32),                            # group 12: unused row slots
    U.Case((140,), (300,), 40, 1, E=64, r_dim=16, page=32),                    # group 40: 3 tokens
    U.Case((40, 3), (90, 33), 64, 1, E=32, r_dim=16),
]


@pytest.mark.parametrize("i", range(len(WEIGHTS)))
@pytest.mark.parametrize("kind", ["bf16", "nvfp4"])
@pytest.mark.parametrize("decay", [0.0, 0.75])
def test_key_weights(i, kind, decay):
    c = WEIGHTS[i]
    d = U.make(c)
    qc = U.quantized(c, d)
    keys = qc["k_values"] if kind == "nvfp4" else d["k"].double().numpy()
    k = U.device_cache(qc, d) if kind == "nvfp4" else d["k"].cuda()
    lse = np.zeros((c.Hq, sum(c.q_lens)), np.float32)
    for b, hq, h, q0, x, mag in U.each_head(c, d, keys):
        lse[hq, q0:q0 + x.shape[0]] = C.softmax(x)[1]
    rng = np.random.default_rng(5)
    w_in = rng.uniform(0, 9, (c.Hkv, d["rows"])).astype(np.float32)
    given = w_in.copy()
    if decay == 0:
        given[:] = np.nan                                # not read
    for b, (nq, nk) in enumerate(zip(c.q_lens, c.k_lens)):
        given[:, d["where"][b][nk - nq:]] = np.nan       # the newest rows' are not read either
    kw = U.call_kw(c, d)
    args = (d["q"].cuda(), k, U.cuda(d["r"]), U.cuda(d["P"]), torch.from_numpy(lse).cuda(), d["cu_q"].cuda(),
            d["cu_k"].cuda())
    out = torch.full((c.Hkv, d["rows"]), 7.0, device="cuda")
    rpb.key_weights(*args, weights_in=torch.from_numpy(given).cuda(), decay=decay, out=out, **kw)
    ok()
    held = U.check_weights(c, d, keys, lse, w_in, decay, out)
    assert (host(out)[:, ~held] == 7).all()
    place = torch.from_numpy(given).cuda()               # in place: the same bits
    rpb.key_weights(*args, weights_in=place, decay=decay, out=place, **kw)
    ok()
    assert torch.equal(place[:, torch.from_numpy(held).cuda()], out[:, torch.from_numpy(held).cuda()])


@pytest.mark.parametrize("kind", ["bf16", "nvfp4"])
@pytest.mark.parametrize("kw", [dict(q=1), dict(q=1, positions=True), dict(q=1, window=20, page=32), dict(q=5, page=64),
                                dict(q=5, positions=True, E=9), dict(q=18), dict(q=18, window=40)],
                         ids=["1", "1-pos", "1-win", "5", "5-pos", "18", "18-win"])
def test_key_weights_of_many_sequences(kind, kw):
    """Past 384 sequences few rows leave the walk too; some sequences have no row,
    some no key."""
    rng = np.random.default_rng(kw["q"])
    k_lens = rng.integers(0, 90, 400)
    q_lens = np.minimum(rng.integers(0, kw["q"] + 1, 400), k_lens)
    q_lens[0] = kw["q"]
    k_lens[0] = 300
    c = U.Case(tuple(map(int, q_lens)), tuple(map(int, k_lens)), 8, 2, **{"E": 64, **{n: v for n, v in kw.items() if n != "q"}})
    d = U.make(c)
    qc = U.quantized(c, d)
    keys = qc["k_values"] if kind == "nvfp4" else d["k"].double().numpy()
    k = U.device_cache(qc, d) if kind == "nvfp4" else d["k"].cuda()
    lse = np.full((c.Hq, sum(c.q_lens)), 5.0, np.float32)
    w_in = np.random.default_rng(6).uniform(0, 9, (c.Hkv, d["rows"])).astype(np.float32)
    out = torch.full((c.Hkv, d["rows"]), 7.0, device="cuda")
    rpb.key_weights(d["q"].cuda(), k, d["r"].cuda(), d["P"].cuda(), torch.from_numpy(lse).cuda(), d["cu_q"].cuda(),
                    d["cu_k"].cuda(), weights_in=torch.from_numpy(w_in).cuda(), decay=0.5, out=out, **U.call_kw(c, d))
    ok()
    held = U.check_weights(c, d, keys, lse, w_in, 0.5, out)
    assert (host(out)[:, ~held] == 7).all()


@pytest.mark.parametrize("kw", [dict(q=1, positions=True), dict(q=3, page=32, window=30), dict(q=9), dict(q=9, positions=True)],
                         ids=["1-pos", "3-win", "9", "9-pos"])
def test_decode_of_many_sequences_of_every_kind(kw):
    rng = np.random.default_rng(kw["q"] + 1)
    k_lens = rng.integers(0, 90, 390)
    q_lens = np.minimum(rng.integers(0, kw["q"] + 1, 390), k_lens)
    q_lens[0], k_lens[0] = kw["q"], 300
    c = U.Case(tuple(map(int, q_lens)), tuple(map(int, k_lens)), 8, 2, **{"E": 64, **{n: v for n, v in kw.items() if n != "q"}})
    d = U.make(c)
    qc = U.quantized(c, d)
    out, lse = run_decode(c, d, qc)
    U.check_decode(c, d, qc["k_values"], qc["v_values"], out, lse)


@pytest.mark.parametrize("kind", ["bf16", "nvfp4"])
@pytest.mark.parametrize("E,page,window", [(64, 0, 0), (0, 32, 0), (200, 96, 3000)])
def test_key_weights_of_more_tiles_than_sms(kind, E, page, window):
    """Every SM takes several tiles of 128 keys, of sequences of all lengths, some
    without a tile or without a row that sees it."""
    c = U.Case((20, 0, 17, 40, 1, 33), (5000, 700, 17, 9000, 1, 2049), 6, 6, E=E, r_dim=16 if E else 0, page=page,
               window=window, base=64.0)
    assert sum(-(-n // 128) for n in c.k_lens) * c.Hkv > 5 * 152
    d = U.make(c)
    qc = U.quantized(c, d)
    keys = qc["k_values"] if kind == "nvfp4" else d["k"].double().numpy()
    k = U.device_cache(qc, d) if kind == "nvfp4" else d["k"].cuda()
    lse = np.zeros((c.Hq, sum(c.q_lens)), np.float32)
    for b, hq, h, q0, x, mag in U.each_head(c, d, keys):
        lse[hq, q0:q0 + x.shape[0]] = C.softmax(x)[1]
    w_in = np.random.default_rng(6).uniform(0, 9, (c.Hkv, d["rows"])).astype(np.float32)
    out = torch.full((c.Hkv, d["rows"]), 7.0, device="cuda")
    rpb.key_weights(d["q"].cuda(), k, U.cuda(d["r"]), U.cuda(d["P"]), torch.from_numpy(lse).cuda(), d["cu_q"].cuda(),
                    d["cu_k"].cuda(), weights_in=torch.from_numpy(w_in).cuda(), decay=0.5, out=out, **U.call_kw(c, d))
    ok()
    held = U.check_weights(c, d, keys, lse, w_in, 0.5, out)
    assert (host(out)[:, ~held] == 7).all()


@pytest.mark.parametrize("q_len,bias", [(1, False), (5, True), (20, True)])
def test_key_weights_of_a_cache_without_rows(q_len, bias):
    """Query rows of no sequence and no key at all: nothing to do, no error."""
    q = torch.ones(q_len, 8, 128, dtype=torch.bfloat16, device="cuda")
    r = torch.ones(q_len, 8, 8, dtype=torch.bfloat16, device="cuda") if bias else None
    P = torch.ones(8, 16, dtype=torch.bfloat16, device="cuda") if bias else None
    lse, zero = torch.zeros(8, q_len, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    some = torch.full((64, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    w = torch.full((2, 64), 7.0, device="cuda")
    work = torch.zeros(1 << 20, device="cuda")
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    fwd = rpb.RelattnParams(q=ptr(q), k=ptr(some), v=None, r=ptr(r), P=ptr(P), cu_seqlens_q=ptr(zero), cu_seqlens_k=ptr(zero),
                            batch=1, total_q=q_len, total_k=0, max_seqlen_q=q_len, max_seqlen_k=4096, num_heads_q=8,
                            num_heads_kv=2, head_dim=128, r_dim=8 if bias else 0, rel_extent=16 if bias else 0, window=50,
                            alpha=0.1, log_scale_base=0.0, out=None, lse=ptr(lse))
    prm = rpb.RelattnKeyWeightsParams(fwd=fwd, weights_out=ptr(w), decay=1.0, workspace=ptr(work), workspace_bytes=4 << 20)
    assert rpb.relattn_key_weights(prm, torch.cuda.current_stream().cuda_stream) == rpb.RELATTN_OK
    ok()
    assert (w == 7).all()


@pytest.mark.parametrize("page", [0, 1024])
@pytest.mark.parametrize("kind", ["bf16", "nvfp4"])
def test_key_weights_under_a_bound_far_above_the_lengths(kind, page):
    """max_seqlen_k is a bound only.  Paged, it makes 400 million units, nearly all
    without a tile: passing over them takes seconds, and no wait gives up."""
    c = U.Case((20, 17, 40, 33, 18, 64), (500, 700, 40, 90, 1025, 64), 8, 4, E=64, page=page)
    d = U.make(c)
    qc = U.quantized(c, d)
    keys = qc["k_values"] if kind == "nvfp4" else d["k"].double().numpy()
    k = U.device_cache(qc, d) if kind == "nvfp4" else d["k"].cuda()
    lse = np.full((c.Hq, sum(c.q_lens)), 6.0, np.float32)
    kw = U.call_kw(c, d)
    kw["max_seqlen_k"] = (1 << 31) - (1 << 16)
    if page:
        wide = torch.full((6, 1 << 21), -1, dtype=torch.int32, device="cuda")
        wide[:, :d["table"].shape[1]] = d["table"].cuda()
        kw["block_table"] = wide
    out = torch.full((c.Hkv, d["rows"]), 7.0, device="cuda")
    rpb.key_weights(d["q"].cuda(), k, d["r"].cuda(), d["P"].cuda(), torch.from_numpy(lse).cuda(), d["cu_q"].cuda(),
                    d["cu_k"].cuda(), decay=0.0, out=out, **kw)
    ok()
    held = U.check_weights(c, d, keys, lse, None, 0.0, out)
    assert (host(out)[:, ~held] == 7).all()


@pytest.mark.parametrize("kind", ["bf16", "nvfp4"])
def test_rows_without_a_logsumexp_and_nan_keys(kind):
    """A row with lse = -inf gives nothing, and a NaN key spoils its own weight
    only where a row sees it."""
    for q_lens in ((3,), (40,)):
        c = U.Case(q_lens, (200,), 4, 1, E=0, r_dim=0, window=60)
        d = U.make(c)
        qc = U.quantized(c, d)
        nq = q_lens[0]
        bad = [20, 199]                                  # out of every window; seen by the last row
        if kind == "bf16":
            d["k"][bad] = float("nan")
            k, keys = d["k"].cuda(), d["k"].double().numpy()
        else:
            qc["k_scale"][bad] = 0x7F
            k, keys = U.device_cache(qc, d), C.dequantize_nvfp4(qc["k"], qc["k_scale"], d["kg"])
        lse = np.full((4, nq), 5.0, np.float32)
        lse[:, 0] = -np.inf
        w = rpb.key_weights(d["q"].cuda(), k, None, None, torch.from_numpy(lse).cuda(), d["cu_q"].cuda(),
                            d["cu_k"].cuda(), **U.call_kw(c, d))
        ok()
        nan = np.isnan(host(w))[0]
        assert nan.nonzero()[0].tolist() == [199]
        want = np.zeros(200)
        for b, hq, h, q0, x, mag in U.each_head(c, d, np.where(np.isnan(keys), 0, keys)):
            want += np.exp(x - 5.0)[1:].sum(0)
        # logits of a few units, off by less than 1e-4 (the bound of check_weights)
        assert np.allclose(host(w)[0, :199], want[:199], rtol=1e-4, atol=1e-30)


@pytest.mark.parametrize("kind", ["bf16", "nvfp4"])
@pytest.mark.parametrize("q_len,Hq,positions", [(0, 4, False), (1, 1, False), (1, 4, False), (2, 8, False), (3, 4, False),
                                                (9, 4, False), (40, 4, False), (1, 4, True), (40, 4, True)])
def test_nan_keys_that_only_silent_rows_see(kind, q_len, Hq, positions):
    """NaN keys in the sight of nobody but rows with lse = -inf, slots without a row
    and a sequence without rows: their weights decay like all others."""
    c = U.Case((q_len, 1), (700, 300), Hq, 1, E=0, r_dim=0, positions=positions)
    d = U.make(c)
    qc = U.quantized(c, d)
    bad = [3, 150, 699 - q_len]                          # of the first sequence
    if kind == "bf16":
        d["k"][bad] = float("nan")
        d["k"][200] = float("inf")
        bad.append(200)
        k = d["k"].cuda()
    else:
        qc["k_scale"][bad] = 0x7F
        k = U.device_cache(qc, d)
    lse = np.full((Hq, q_len + 1), -np.inf, np.float32)
    lse[:, q_len:] = 5.0                                 # the second sequence's row votes
    w_in = np.random.default_rng(9).uniform(1, 9, (1, 1000)).astype(np.float32)
    w = rpb.key_weights(d["q"].cuda(), k, None, None, torch.from_numpy(lse).cuda(), d["cu_q"].cuda(), d["cu_k"].cuda(),
                        weights_in=torch.from_numpy(w_in).cuda(), decay=0.5, **U.call_kw(c, d))
    ok()
    want = 0.5 * w_in[0, :700]
    want[700 - q_len:] = 0
    np.testing.assert_array_equal(host(w)[0, :700], want)
    assert np.isfinite(host(w)[0, 700:]).all() and (host(w)[0, 700:] > 0).any()


@pytest.mark.parametrize("Hq", [1, 3, 8])
def test_a_key_of_logit_minus_infinity_has_no_weight(Hq):
    """An infinite element that every row answers with -inf: weight 0, in slots
    without a row too."""
    c = U.Case((1,), (300,), Hq, 1, E=0, r_dim=0)
    d = U.make(c)
    d["k"][40, 0, 7] = float("inf")
    d["q"][:, :, 7] = -1.0
    w = rpb.key_weights(d["q"].cuda(), d["k"].cuda(), None, None, torch.full((Hq, 1), 5.0, device="cuda"),
                        d["cu_q"].cuda(), d["cu_k"].cuda(), **U.call_kw(c, d))
    ok()
    assert host(w)[0, 40] == 0 and np.isfinite(host(w)).all() and (np.delete(host(w)[0], 40) > 0).all()


@pytest.mark.parametrize("kind", ["bf16", "nvfp4"])
def test_key_weights_of_lengths_that_cannot_be_side_by_side(kind):
    """cu_seqlens_k out of order: every second sequence passes the checks by itself,
    together they have more keys than 32 bits count.  Nothing is done."""
    batch, page = 300, 1 << 20
    cu_k = torch.tensor([0, (1 << 31) - (1 << 16)] * (batch // 2) + [0], dtype=torch.int32, device="cuda")
    table = torch.full((batch, 1 << 11), -1, dtype=torch.int32, device="cuda")
    q = torch.ones(batch, 8, 128, dtype=torch.bfloat16, device="cuda")
    k = torch.ones(page, 1, 128, dtype=torch.bfloat16, device="cuda")
    if kind == "nvfp4":
        k = rpb.empty_nvfp4(page, 1, "cuda")
    out = torch.full((1, page), 7.0, device="cuda")
    rpb.key_weights(q, k, None, None, torch.zeros(8, batch, device="cuda"),
                    torch.arange(batch + 1, dtype=torch.int32, device="cuda"), cu_k, max_seqlen_q=1,
                    max_seqlen_k=(1 << 31) - (1 << 16), alpha=0.1, out=out, total_k=page, block_table=table, page_size=page)
    torch.cuda.synchronize()
    assert rpb.relattn_get_device_error() == 6
    assert (out == 7).all()


# ------------------------------------------------------------------ eviction

def _planes(rows, Hkv, kinds, seed=0):
    g = torch.Generator().manual_seed(seed)
    out = []
    for n in kinds:
        if n == "bf16":
            out.append(torch.randn(rows, Hkv, 128, generator=g).to(torch.bfloat16))
        else:
            out.append(torch.randint(0, 256, (rows, Hkv, n), generator=g, dtype=torch.uint8))
    return out


@pytest.mark.parametrize("k_lens,keep,recent,sink,kinds,page,page_to,ties", [
    ((1,), (1,), 0, 0, ("bf16",), 0, 0, False),
    ((50, 7, 0, 33), (20, 7, 0, 1), 4, 2, (64, 64, 8, 8), 0, 0, False),
    ((50, 64), (3, 10), 16, 4, ("bf16", "bf16"), 0, 0, True),               # fewer kept than recent
    ((4097, 511), (1000, 510), 0, 0, (128, 128, 4, 4), 0, 0, True),
    ((4096, 5000), (4096, 4999), 100, 100, (3,), 0, 0, False),              # odd bytes, all kept
    ((1000, 300), (400, 128), 64, 4, (64, 64, 8, 8), 32, 64, False),        # pages to pages
    ((17000, 9000), (2000, 8000), 128, 4, (8,), 0, 0, True),
    ((40000,), (5000,), 0, 0, (8,), 128, 0, False),                         # two CTAs a cluster
    ((150001,), (75000,), 1024, 4, (8,), 0, 0, True),                       # eight
    ((300001, 40), (290000, 7), 5, 1, (16, 1), 0, 0, True),                 # sixteen
    ((800000,), (1234,), 100, 3, (8,), 0, 0, False),                        # more keys than shared memory holds
    ((790000, 100), (400000, 99), 0, 0, (4,), 64, 32, True),
    # and of more (sequence, head) pairs than the selection by all SMs takes
    ((150001, 20, 0, 9, 1), (75000, 3, 0, 9, 1), 1024, 4, (8,), 0, 0, True),
    ((300001, 40, 33, 8, 7), (290000, 7, 33, 1, 2), 5, 1, (16, 1), 32, 0, True),
    ((800000, 5, 6, 0, 2), (1234, 5, 1, 0, 2), 100, 3, (8,), 0, 0, False),
    ((1900000, 70000), (3000, 69999), 10, 4, (4,), 0, 0, True),             # more than all SMs' shared memory holds
])
def test_evict(k_lens, keep, recent, sink, kinds, page, page_to, ties):
    Hkv = 2
    rows, table, where = U.rows_of(k_lens, page, 3)
    rows_to, table_to, where_to = U.rows_of(keep, page_to, 4)
    rng = np.random.default_rng(6)
    w = rng.exponential(1.0, (Hkv, rows)).astype(np.float32)
    if ties:
        w = np.round(w, 1)
        w[:, ::13] = -w[:, ::13]
        w[:, 5::101] = np.nan
        w[:, 6::103] = np.inf
        w[:, 7::107] = -0.0
    planes = _planes(rows, Hkv, kinds)
    dst = [torch.full((rows_to, *p.shape[1:]), 3, dtype=p.dtype, device="cuda") for p in planes]
    kw = {}
    if page:
        kw.update(block_table=table.cuda(), page_size=page)
    if page_to:
        kw.update(block_table_keep=table_to.cuda(), page_size_keep=page_to)
    key_pos = torch.from_numpy(rng.integers(0, 1 << 30, (Hkv, rows)).astype(np.int32))
    for pos_in in (None, key_pos):
        pos, wk = rpb.evict([p.cuda() for p in planes], dst, torch.from_numpy(w).cuda(), W.cu_seqlens(k_lens).cuda(),
                            W.cu_seqlens(keep).cuda(), max_seqlen_k=max(k_lens), recent=recent, sink=sink,
                            total_k=sum(k_lens), total_keep=sum(keep), key_pos=U.cuda(pos_in), **kw)
        ok()
        used = np.zeros(rows_to, bool)
        for b, (n, kk) in enumerate(zip(k_lens, keep)):
            used[where_to[b]] = True
            for h in range(Hkv):
                idx = C.kept_keys(w[h, where[b]], kk, recent, sink)
                assert len(idx) == kk
                src = where[b][idx]
                want = idx if pos_in is None else key_pos[h].numpy()[src]
                np.testing.assert_array_equal(host(pos)[h, where_to[b]], want)
                np.testing.assert_array_equal(host(wk)[h, where_to[b]], w[h, src])
                for p, q in zip(planes, dst):
                    assert torch.equal(q[torch.from_numpy(where_to[b]).cuda(), h].cpu(), p[torch.from_numpy(src), h])
        assert (host(pos)[:, ~used] == -1).all() and (host(wk)[:, ~used] == 0).all()
        for q in dst:
            assert (q.cpu().float()[torch.from_numpy(~used)] == 3).all()


def test_sizes_past_32_bits_are_refused_or_mean_all():
    n, big = 300, 1 << 32
    w = torch.rand(1, n, device="cuda")
    cu, cu_keep = W.cu_seqlens([n]).cuda(), W.cu_seqlens([40]).cuda()
    for recent, sink, want in ((big, 0, np.arange(260, 300)), (0, big, np.arange(40)), (big, big, np.arange(260, 300))):
        pos, _ = rpb.evict([], [], w, cu, cu_keep, max_seqlen_k=n, recent=recent, sink=sink, total_keep=40)
        ok()
        np.testing.assert_array_equal(host(pos)[0], want)
    q = torch.zeros(1, 1, 128, dtype=torch.bfloat16, device="cuda")
    cache, lse, cu1 = rpb.empty_nvfp4(n, 1, "cuda"), torch.zeros(1, 1, device="cuda"), W.cu_seqlens([1]).cuda()
    good = dict(max_seqlen_q=1, max_seqlen_k=n, window=0, total_k=n)
    for name, value in (("max_seqlen_q", big + 1), ("max_seqlen_k", big + n), ("window", big + 4), ("window", -big + 4),
                        ("total_k", big + n)):
        kw = {**good, name: value}
        with pytest.raises(ValueError, match="32 bits"):
            rpb.decode_nvfp4(q, cache, None, None, cu1, cu, alpha=0.1, **kw)
        with pytest.raises(ValueError, match="32 bits"):
            rpb.key_weights(q, cache, None, None, lse, cu1, cu, alpha=0.1, **kw)
    with pytest.raises(ValueError, match="32 bits"):
        rpb.decode_nvfp4(q, cache, None, None, cu1, cu, alpha=0.1, num_splits=big + 1, **good)
    for kw in (dict(max_seqlen_k=big + n), dict(total_keep=big + 40), dict(total_k=big + n), dict(recent=-big + 4)):
        with pytest.raises(ValueError, match="32 bits"):
            rpb.evict([torch.zeros(n, 1, 4, device="cuda")], [torch.zeros(40, 1, 4, device="cuda")], w, cu, cu_keep,
                      **{**dict(max_seqlen_k=n, recent=0, total_keep=40), **kw})


def test_evict_of_equal_weights_keeps_the_first():
    n = 20000
    w = torch.zeros(1, n, device="cuda")
    pos, _ = rpb.evict([], [], w, W.cu_seqlens([n]).cuda(), W.cu_seqlens([777]).cuda(), max_seqlen_k=n, recent=0,
                       total_keep=777)
    ok()
    assert torch.equal(pos[0].cpu(), torch.arange(777, dtype=torch.int32))


def test_evict_without_planes_into_pages():
    """Positions and weights alone, at the rows of a paged cache: rows_keep says how
    many it has."""
    lens, keep, Hkv = (300, 170), (40, 33), 2
    rows_to, table, where = U.rows_of(keep, 32, 4)
    w = torch.rand(Hkv, sum(lens), device="cuda")
    args = (w, W.cu_seqlens(lens).cuda(), W.cu_seqlens(keep).cuda())
    kw = dict(max_seqlen_k=300, recent=8, sink=2, total_keep=sum(keep), block_table_keep=table.cuda(), page_size_keep=32)
    pos, wk = rpb.evict([], [], *args, rows_keep=rows_to, **kw)
    ok()
    assert pos.shape == wk.shape == (Hkv, rows_to)
    used = np.zeros(rows_to, bool)
    for b in range(2):
        used[where[b]] = True
        for h in range(Hkv):
            v = host(w)[h, sum(lens[:b]):sum(lens[:b]) + lens[b]]
            idx = C.kept_keys(v, keep[b], 8, 2)
            np.testing.assert_array_equal(host(pos)[h, where[b]], idx)
            np.testing.assert_array_equal(host(wk)[h, where[b]], v[idx])
    assert (host(pos)[:, ~used] == -1).all() and (host(wk)[:, ~used] == 0).all()
    with pytest.raises(ValueError, match="rows must be a multiple of page_size"):
        rpb.evict([], [], *args, **kw)
    p = torch.zeros(sum(lens), Hkv, 4, device="cuda")
    with pytest.raises(ValueError, match="rows_keep"):
        rpb.evict([p], [p.new_zeros(rows_to, Hkv, 4)], *args, rows_keep=rows_to - 32, **kw)


@pytest.mark.parametrize("given", [(True, True), (True, False), (False, True)])
def test_evict_keeps_what_given_outputs_hold_elsewhere(given):
    w = torch.rand(2, 300, device="cuda")
    p = torch.rand(300, 2, 4, device="cuda")
    to = torch.zeros(100, 2, 4, device="cuda")
    pos = torch.full((2, 100), 7, dtype=torch.int32, device="cuda") if given[0] else None
    wk = torch.full((2, 100), 7.0, device="cuda") if given[1] else None
    pos, wk = rpb.evict([p], [to], w, W.cu_seqlens([300]).cuda(), W.cu_seqlens([60]).cuda(), max_seqlen_k=300, recent=5,
                        total_keep=60, key_pos_out=pos, weights_out=wk)
    ok()
    assert (pos[:, 60:] == (7 if given[0] else -1)).all() and (wk[:, 60:] == (7 if given[1] else 0)).all()
    assert (pos[:, :60] >= 0).all() and torch.equal(wk[0, :60], w[0][pos[0, :60].long()])


def test_evict_of_nothing_clears_new_outputs():
    p = torch.rand(30, 1, 4, device="cuda")
    to = torch.zeros(10, 1, 4, device="cuda")
    pos, wk = rpb.evict([p], [to], torch.rand(1, 30, device="cuda"), W.cu_seqlens([30]).cuda(), W.cu_seqlens([0]).cuda(),
                        max_seqlen_k=30, recent=0, total_keep=0)
    ok()
    assert (pos == -1).all() and (wk == 0).all() and pos.shape == (1, 10)


def test_evict_skips_and_records_bad_lengths():
    w = torch.rand(1, 100, device="cuda")
    p = torch.rand(100, 1, 4, device="cuda")
    out = torch.full((50, 1, 4), 3.0, device="cuda")
    cu_k = torch.tensor([0, 20, 100], dtype=torch.int32, device="cuda")
    cu_keep = torch.tensor([0, 30, 50], dtype=torch.int32, device="cuda")      # 30 of 20
    pos, _ = rpb.evict([p], [out], w, cu_k, cu_keep, max_seqlen_k=100, recent=5, total_keep=50)
    torch.cuda.synchronize()
    assert rpb.relattn_get_device_error() == 6
    assert (out[:30] == 3).all() and (pos[:, :30] == -1).all()
    idx = C.kept_keys(host(w)[0, 20:], 20, 5, 0)
    np.testing.assert_array_equal(host(pos)[0, 30:], idx)
    assert torch.equal(out[30:, 0], p[20 + torch.from_numpy(idx).cuda(), 0])


@pytest.mark.parametrize("max_k", [100, 40000])           # selected by clusters, and by all SMs
@pytest.mark.parametrize("cu_keep,bad", [([0, 10, 40], 1), ([-5, 10, 30], 0)])
def test_evict_moves_nothing_of_a_sequence_partly_outside(max_k, cu_keep, bad):
    """A sequence whose kept rows start before the first or end behind the last
    place moves no row, whatever the workspace held (here, numbers of rows)."""
    w = torch.rand(2, 100, device="cuda")
    p = torch.rand(100, 2, 4, device="cuda")
    out = torch.full((30, 2, 4), 3.0, device="cuda")
    cu_k = torch.tensor([0, 20, 100], dtype=torch.int32, device="cuda")
    work = torch.full((1 << 20,), 3, dtype=torch.int32, device="cuda")
    pos, wk = rpb.evict([p], [out], w, cu_k, torch.tensor(cu_keep, dtype=torch.int32, device="cuda"), max_seqlen_k=max_k,
                        recent=30, total_keep=30, workspace=work)
    torch.cuda.synchronize()
    assert rpb.relattn_get_device_error() == 6
    good, skipped = (slice(0, 10), slice(10, 30)) if bad == 1 else (slice(10, 30), slice(0, 10))
    end = 20 if bad == 1 else 100
    assert torch.equal(out[good], p[end - (good.stop - good.start):end])      # the newest
    assert (out[skipped] == 3).all() and (pos[:, skipped] == -1).all() and (wk[:, skipped] == 0).all()


# ------------------------------------------------------------------ streams, graphs, runs

def test_captured_calls_replay_and_streams_do_not_share():
    """Two captured decodes with workspaces of their own, replayed together with
    new inputs; and a call on a side stream."""
    c = U.Case((1, 2), (700, 300), 8, 2, E=64)
    d = U.make(c)
    qc = U.quantized(c, d)
    cache = U.device_cache(qc, d)
    cu = (d["cu_q"].cuda(), d["cu_k"].cuda())
    r, P, kw = d["r"].cuda(), d["P"].cuda(), U.call_kw(c, d)
    qs = [d["q"].cuda(), (d["q"] * 0.5).cuda()]
    want = [rpb.decode_nvfp4(q, cache, r, P, *cu, **kw) for q in qs]
    weights = [rpb.key_weights(q, cache, r, P, o[1], *cu, **kw) for q, o in zip(qs, want)]
    graphs, bufs = [], []
    for i in range(2):
        q = torch.zeros_like(qs[i])
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            rpb.decode_nvfp4(q, cache, r, P, *cu, **kw)              # warm up
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o, z = rpb.decode_nvfp4(q, cache, r, P, *cu, **kw)
            w = rpb.key_weights(q, cache, r, P, z, *cu, **kw)
        graphs.append(g)
        bufs.append((q, o, z, w))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for i in range(2):
            bufs[i][0].copy_(qs[i])
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(bufs[i][1], want[i][0]) and torch.equal(bufs[i][2], want[i][1])
            assert torch.equal(bufs[i][3], weights[i])
    side = torch.cuda.Stream()
    out, lse = rpb.decode_nvfp4(qs[0], cache, r, P, *cu, **kw, stream=side.cuda_stream)
    w = rpb.key_weights(qs[0], cache, r, P, lse, *cu, **kw, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(out, want[0][0]) and torch.equal(lse, want[0][1]) and torch.equal(w, weights[0])
    ok()


@pytest.mark.parametrize("nq,Hq,positions", [(1, 8, False), (2, 8, True), (9, 8, False), (9, 8, True)])
def test_captured_calls_follow_new_lengths(nq, Hq, positions):
    """A graph captured under bounds, for a batch with room to spare, replayed with
    other lengths, pages and positions: decode, key weights and eviction."""
    batch, Hkv, page, top, E = 5, 2, 32, 4000, 64
    slots = -(-top // page)
    rows = batch * slots // 2 * page
    cap = dict(cu_q=torch.zeros(batch + 1, dtype=torch.int32, device="cuda"), cu_k=torch.zeros(batch + 1, dtype=torch.int32, device="cuda"),
               cu_keep=torch.zeros(batch + 1, dtype=torch.int32, device="cuda"),
               table=torch.full((batch, slots), -1, dtype=torch.int32, device="cuda"),
               q=torch.zeros(batch * nq, Hq, 128, dtype=torch.bfloat16, device="cuda"),
               r=torch.zeros(batch * nq, Hq, 16, dtype=torch.bfloat16, device="cuda"),
               P=torch.zeros(16, E, dtype=torch.bfloat16, device="cuda"),
               key_pos=torch.zeros(Hkv, rows, dtype=torch.int32, device="cuda"), q_pos=torch.zeros(batch, dtype=torch.int32, device="cuda"))
    cache = rpb.empty_nvfp4(rows, Hkv, "cuda", torch.ones(Hkv, device="cuda"), torch.ones(Hkv, device="cuda"))
    to = torch.zeros(500, Hkv, 8, dtype=torch.uint8, device="cuda")
    pos = dict(key_pos=cap["key_pos"], q_pos=cap["q_pos"]) if positions else {}
    kw = dict(max_seqlen_q=nq, max_seqlen_k=top, alpha=1 / np.sqrt(128), total_k=600, block_table=cap["table"], page_size=page, **pos)

    def step():
        out, lse = rpb.decode_nvfp4(cap["q"], cache, cap["r"], cap["P"], cap["cu_q"], cap["cu_k"], **kw)
        w = rpb.key_weights(cap["q"], cache, cap["r"], cap["P"], lse, cap["cu_q"], cap["cu_k"], decay=0.0, **kw)
        kept, wk = rpb.evict([cache.k_scale], [to], w, cap["cu_k"], cap["cu_keep"], max_seqlen_k=top, recent=4, sink=1, total_k=600,
                             total_keep=500, block_table=cap["table"], page_size=page)
        return out, lse, w, kept

    step()                                               # warm up (on no sequence)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for q_lens, k_lens in (((1, nq, 0, 1, nq), (7, 500, 33, 1, 40)), ((nq,) * 5, (nq, 3500, 90, 64, 700)),
                           ((1, 0, 0, 0, 0), (2000, 0, 0, 0, 0)), ((nq, 1), (3000, 4000))):
        q_lens, k_lens = q_lens + (0,) * (5 - len(q_lens)), k_lens + (0,) * (5 - len(k_lens))
        c = U.Case(q_lens, k_lens, Hq, Hkv, E=E, page=page, positions=positions, seed=sum(k_lens))
        d = U.make(c)
        qc = U.quantized(c, d)
        n = d["rows"]
        assert n <= rows
        for t, x in zip(cache, U.device_cache(qc, d)):
            t[:len(x)].copy_(x)
        for name in ("q", "r"):
            cap[name][:len(d[name])].copy_(d[name])
        cap["P"].copy_(d["P"])
        cap["cu_q"].copy_(d["cu_q"])
        cap["cu_k"].copy_(d["cu_k"])
        keep = [k // 20 for k in k_lens]
        cap["cu_keep"].copy_(W.cu_seqlens(keep))
        cap["table"][:, :d["table"].shape[1]].copy_(d["table"])
        if positions:
            cap["key_pos"][:, :n].copy_(d["key_pos"])
            cap["q_pos"].copy_(d["q_pos"])
        graph.replay()
        ok()
        out, lse, w, kept = got
        Tq = sum(q_lens)
        U.check_decode(c, d, qc["k_values"], qc["v_values"], out[:Tq], lse[:, :Tq])
        U.check_weights(c, d, qc["k_values"], host(lse[:, :Tq]), None, 0.0, w[:, :n])
        o = 0
        for b, k in enumerate(keep):
            for h in range(Hkv):
                idx = C.kept_keys(host(w)[h, d["where"][b]], k, 4, 1)
                np.testing.assert_array_equal(host(kept)[h, o:o + k], idx)
                assert torch.equal(to[o:o + k, h], cache.k_scale[torch.from_numpy(d["where"][b][idx]).cuda(), h])
            o += k


def test_calls_of_many_rows_and_long_sequences_replay_side_by_side():
    """Decodes of 40 rows, key weights of 160 rows and selections by all SMs, in
    two graphs that replay on two streams at once."""
    c = U.Case((5, 4), (40000, 300), 16, 2, E=64)
    d = U.make(c)
    qc = U.quantized(c, d)
    cache = U.device_cache(qc, d)
    cu = (d["cu_q"].cuda(), d["cu_k"].cuda())
    r, P, kw = d["r"].cuda(), d["P"].cuda(), U.call_kw(c, d)
    c2 = U.Case((20, 3), c.k_lens, 16, 2, E=64, seed=3)
    d2 = U.make(c2)
    q2, r2, P2, cu2, kw2 = d2["q"].cuda(), d2["r"].cuda(), d2["P"].cuda(), d2["cu_q"].cuda(), U.call_kw(c2, d2)
    lse2 = torch.full((16, 23), 8.0, device="cuda")
    cu_keep = W.cu_seqlens([9000, 200]).cuda()

    def step(q, w):
        o, z = rpb.decode_nvfp4(q, cache, r, P, *cu, **kw)
        w = rpb.key_weights(q2, cache, r2, P2, lse2, cu2, cu[1], weights_in=w, decay=0.5, **kw2)
        to = torch.zeros(9200, 2, 8, dtype=torch.uint8, device="cuda")
        pos, wk = rpb.evict([cache.k_scale], [to], w, cu[1], cu_keep, max_seqlen_k=40000, recent=64, sink=4,
                            total_k=40300, total_keep=9200)
        return o, z, w, to, pos, wk

    rng = torch.Generator(device="cuda").manual_seed(1)
    ins = [(d["q"].cuda() * f, torch.rand(2, 40300, device="cuda", generator=rng)) for f in (1.0, 0.5)]
    want = [step(q, w) for q, w in ins]
    ok()
    graphs, held = [], []
    for q, w in ins:
        g, q0, w0 = torch.cuda.CUDAGraph(), torch.zeros_like(q), torch.zeros_like(w)
        with torch.cuda.graph(g):
            got = step(q0, w0)
        graphs.append(g)
        held.append((q0, w0, got))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for (q, w), (q0, w0, _) in zip(ins, held):
            q0.copy_(q)
            w0.copy_(w)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
                g.replay()
        torch.cuda.synchronize()
        ok()
        for x, (_, _, got) in zip(want, held):
            for a, b in zip(x, got):
                assert torch.equal(a, b)


def test_a_prompt_is_cached_weighed_evicted_and_decoded():
    """The operators in the order a server calls them: a prompt's rows go into a
    4-bit paged cache, its last rows vote, half of the keys leave, and a
    token is decoded over the rest at its own position."""
    page, lens, Hq, Hkv, E = 64, (300, 700), 8, 2, 64
    c = U.Case(lens, lens, Hq, Hkv, E=E, r_dim=16, base=64.0)
    d = U.make(c)
    rows, table, where = U.rows_of([n + 1 for n in lens], page, 9)
    table = table.cuda()
    cache = rpb.empty_nvfp4(rows, Hkv, "cuda")
    cu = W.cu_seqlens(lens).cuda()
    q, k, v, r, P = (d[n].cuda() for n in ("q", "k", "v", "r", "P"))
    kw = dict(alpha=c.alpha, log_scale_base=64.0, max_seqlen_k=max(lens))
    out, lse = rpb.prefill(q, k, v, r, P, cu, cu, max_seqlen_q=max(lens), **kw)
    rpb.store_nvfp4(k, v, cu, cu, cache, block_table=table, page_size=page)
    k4, v4 = rpb.load_nvfp4(cache, cu, cu, total_q=sum(lens), block_table=table, page_size=page)
    # the last 16 rows of each prompt vote, on the cached keys
    last = torch.cat([torch.arange(sum(lens[:b + 1]) - 16, sum(lens[:b + 1])) for b in range(2)]).cuda()
    cu_obs = W.cu_seqlens([16, 16]).cuda()
    w = rpb.key_weights(q[last], cache, r[last], P, lse[:, last].contiguous(), cu_obs, cu, max_seqlen_q=16, decay=0.0,
                        total_k=sum(lens), block_table=table, page_size=page, **kw)
    ok()
    host_k = np.zeros((rows, Hkv, 128))
    host_v = np.zeros((rows, Hkv, 128))
    for b in range(2):
        o = sum(lens[:b])
        host_k[where[b][:lens[b]]] = k4[o:o + lens[b]].double().cpu().numpy()
        host_v[where[b][:lens[b]]] = v4[o:o + lens[b]].double().cpu().numpy()
    c_obs = U.Case((16, 16), lens, Hq, Hkv, E=E, base=64.0)
    d_obs = dict(d, q=d["q"][last.cpu()], r=d["r"][last.cpu()], where=[where[b][:lens[b]] for b in range(2)])
    U.check_weights(c_obs, d_obs, host_k, host(lse[:, last]), None, 0.0, w)
    # half of the keys stay, in contiguous rows with room for one more
    keep = [n // 2 for n in lens]
    dst = rpb.empty_nvfp4(sum(keep), Hkv, "cuda")
    cu_keep = W.cu_seqlens(keep).cuda()
    pos, wk = rpb.evict(cache[:4], dst[:4], w, cu, cu_keep, max_seqlen_k=max(lens), recent=20, sink=4,
                        total_k=sum(lens), total_keep=sum(keep), block_table=table, page_size=page)
    ok()
    kept = [[C.kept_keys(host(w)[h, where[b][:lens[b]]], keep[b], 20, 4) for h in range(Hkv)] for b in range(2)]
    # the next token: its row joins each sequence, in pages of its own
    rows2, table2, where2 = U.rows_of([n + 1 for n in keep], 32, 11)
    cache2 = rpb.empty_nvfp4(rows2, Hkv, "cuda")
    pos2 = torch.full((Hkv, rows2), -1, dtype=torch.int32, device="cuda")
    rng = np.random.default_rng(12)
    new_k, new_v, new_q = (U.bf16(rng.standard_normal((2, H, 128))) for H in (Hkv, Hkv, Hq))
    new_r = U.bf16(rng.standard_normal((2, Hq, 16)))
    for b in range(2):
        a = sum(keep[:b])
        at = torch.from_numpy(where2[b]).cuda()
        for s, t in zip(dst[:4], cache2[:4]):
            t[at[:-1]] = s[a:a + keep[b]]
        pos2[:, at[:-1]] = pos[:, a:a + keep[b]]
        pos2[:, at[-1]] = lens[b]
    cu1, cu2 = W.cu_seqlens([1, 1]).cuda(), W.cu_seqlens([n + 1 for n in keep]).cuda()
    t2 = table2.cuda()
    rpb.store_nvfp4(new_k.cuda(), new_v.cuda(), cu1, cu2, cache2, block_table=t2, page_size=32)
    out, lse2 = rpb.decode_nvfp4(new_q.cuda(), cache2, new_r.cuda(), P, cu1, cu2, max_seqlen_q=1,
                                 max_seqlen_k=max(keep) + 1, alpha=c.alpha, log_scale_base=64.0, key_pos=pos2,
                                 q_pos=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                 block_table=t2, page_size=32, total_k=sum(keep) + 2)
    ok()
    keys = np.zeros((rows2, Hkv, 128))
    vals = np.zeros((rows2, Hkv, 128))
    kp = np.full((Hkv, rows2), -1, np.int32)
    for b in range(2):
        for h in range(Hkv):
            keys[where2[b][:-1], h] = host_k[where[b][kept[b][h]], h]
            vals[where2[b][:-1], h] = host_v[where[b][kept[b][h]], h]
            kp[h, where2[b][:-1]] = kept[b][h]
            kp[h, where2[b][-1]] = lens[b]
        keys[where2[b][-1]] = C.dequantize_nvfp4(*C.quantize_nvfp4(new_k[b:b + 1].float().numpy()))[0]
        vals[where2[b][-1]] = C.dequantize_nvfp4(*C.quantize_nvfp4(new_v[b:b + 1].float().numpy()))[0]
    np.testing.assert_array_equal(host(pos2), kp)
    c2 = U.Case((1, 1), tuple(n + 1 for n in keep), Hq, Hkv, E=E, base=64.0, positions=True)
    d2 = dict(q=new_q, r=new_r, P=d["P"], where=where2, key_pos=torch.from_numpy(kp),
              q_pos=torch.tensor(lens, dtype=torch.int32))
    U.check_decode(c2, d2, keys, vals, out, lse2)


def test_a_thinned_bf16_cache_under_the_plain_decode():
    """Without a log-scale and with the bias inside the newest keys, the bf16
    decode reads an evicted cache as it is."""
    lens, keep, Hq, Hkv, E = (400, 900), (150, 300), 8, 2, 64
    c = U.Case((1, 1), lens, Hq, Hkv, E=E)
    d = U.make(c)
    cu1, cu = W.cu_seqlens([1, 1]).cuda(), W.cu_seqlens(lens).cuda()
    q, k, v, r, P = (d[n].cuda() for n in ("q", "k", "v", "r", "P"))
    kw = dict(max_seqlen_q=1, alpha=c.alpha)
    out, lse = rpb.decode(q, k, v, r, P, cu1, cu, max_seqlen_k=900, **kw)
    w = rpb.key_weights(q, k, r, P, lse, cu1, cu, max_seqlen_k=900, **kw)
    ok()
    dst = [torch.empty(sum(keep), Hkv, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    cu_keep = W.cu_seqlens(keep).cuda()
    pos, _ = rpb.evict([k, v], dst, w, cu, cu_keep, max_seqlen_k=900, recent=E, total_keep=sum(keep))
    out2, lse2 = rpb.decode(q, *dst, r, P, cu1, cu_keep, max_seqlen_k=300, **kw)
    ok()
    for b, hq, h, q0, x, mag in U.each_head(c, d, d["k"].double().numpy()):
        idx = C.kept_keys(host(w)[h, d["where"][b]], keep[b], E, 0)
        np.testing.assert_array_equal(host(pos)[h, sum(keep[:b]):sum(keep[:b]) + keep[b]], idx)
        p, z = C.softmax(x[:, idx])
        ref = p @ d["v"].double().numpy()[d["where"][b][idx], h]
        # the framework's own bounds for this decode
        assert np.abs(out2[q0, hq].double().cpu().numpy() - ref[0]).max() <= 2e-2
        assert abs(float(lse2[hq, q0]) - z[0]) <= 1e-3
