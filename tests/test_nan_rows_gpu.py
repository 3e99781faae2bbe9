"""A NaN logit in the forward and decode calls: the rows that see it give NaN in out
and lse whatever the kernel and however the keys are split, other rows are as
without it.  (A split whose sum is NaN must not pass for one without keys.)"""
import numpy as np
import pytest
import torch

import relative_position_biased_gb300 as rpb
from tests import kvcache_util as U
from tests import test_extend_gpu as X
from tests.conftest import gpu_available
from tests.test_extend_gpu import _clean_error_word, _lib  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]


def check(c, call, back):
    d = U.make(c)
    want, z, e_out, e_lse = X.bounds(c, d, 0)
    hit = np.zeros((sum(c.q_lens), c.Hq), bool)
    at = 0
    for b, (nq, nk) in enumerate(zip(c.q_lens, c.k_lens)):
        j, g = max(nk - 1 - back, 0), b % c.Hkv
        d["k"][d["where"][b][j], g] = float("nan")
        pos = nk - nq + np.arange(nq)
        sees = (pos >= j) & ((c.window <= 0) | (pos - j < c.window))
        hit[at:at + nq, g * (c.Hq // c.Hkv):(g + 1) * (c.Hq // c.Hkv)] = sees[:, None]
        at += nq
    t = [U.cuda(d[n]) for n in ("q", "k", "v", "r", "P", "cu_q", "cu_k")]
    out, lse = call(d, t, dict(max_seqlen_q=max(c.q_lens), max_seqlen_k=max(c.k_lens), alpha=c.alpha, window=c.window))
    X.ok()
    got, got_z = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isnan(got[hit]).all() and np.isnan(got_z[hit.T]).all()
    assert (np.abs(got - want)[~hit] <= e_out[~hit]).all()
    assert (np.abs(got_z - z)[~hit.T] <= e_lse[~hit.T]).all()


@pytest.mark.parametrize("back", [0, 90, 700])
@pytest.mark.parametrize("Hq,Hkv,rd,E,window", [(16, 2, 64, 128, 0), (4, 4, 16, 64, 300), (8, 2, 0, 0, 0), (6, 2, 7, 33, 0)])
def test_prefill(Hq, Hkv, rd, E, window, back):
    check(U.Case((900, 300), (900, 300), Hq, Hkv, r_dim=rd, E=E, window=window), lambda d, t, kw: rpb.prefill(*t, **kw), back)


@pytest.mark.parametrize("back", [0, 90, 700, 3000])
@pytest.mark.parametrize("num_splits", [0, 1, 3])
@pytest.mark.parametrize("Hq,Hkv,rd,E,window,q_lens", [
    (16, 2, 64, 128, 0, (1, 1)),           # few rows, keys along the products' rows
    (16, 2, 64, 128, 0, (9, 16)),          # 128-row blocks
    (4, 4, 16, 64, 1000, (5, 1)),
    (6, 2, 7, 33, 0, (1, 3)),              # the kernel of any shape
])
def test_decode(Hq, Hkv, rd, E, window, q_lens, num_splits, back):
    c = U.Case(q_lens, (5000, 900), Hq, Hkv, r_dim=rd, E=E, window=window)
    check(c, lambda d, t, kw: rpb.decode(*t, num_splits=num_splits, **kw), back)


@pytest.mark.parametrize("back", [0, 700])
@pytest.mark.parametrize("q_lens", [(1, 1), (9, 3)])
def test_decode_paged(q_lens, back):
    c = U.Case(q_lens, (5000, 900), 16, 2, r_dim=64, E=128, page=128)
    check(c, lambda d, t, kw: rpb.decode_paged(*t, d["table"].cuda(), page_size=128, **kw), back)


@pytest.mark.parametrize("nan", [[], [0], [2], [0, 1, 2]])
@pytest.mark.parametrize("empty", [[], [1]])
def test_combine(nan, empty):
    """Rows of partials: NaN stays, -inf is a split without keys whatever it holds."""
    n, T, H = 3, 70, 4
    rng = np.random.default_rng(1)
    o = torch.from_numpy(rng.standard_normal((n, T, H, 128)).astype(np.float32)).cuda()
    z = torch.from_numpy(rng.standard_normal((n, T, H)).astype(np.float32)).cuda()
    for s in empty:
        z[s, 10:], o[s, 10:] = -float("inf"), float("nan")
    for s in nan:
        z[s, 5:60], o[s, 5:60] = float("nan"), float("nan")
    out = torch.empty(T, H, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(H, T, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    assert rpb.relattn_combine(o.data_ptr(), z.data_ptr(), n, T, H, out.data_ptr(), lse.data_ptr(), st) == 0
    torch.cuda.synchronize()
    bad = z.isnan().any(0)
    w = torch.exp(z.double() - z.double().nan_to_num(-1e30).amax(0))
    ref = (w[..., None] * torch.where(z[..., None] == -float("inf"), torch.zeros_like(o), o).double()).sum(0) / w.sum(0)[..., None]
    assert out[bad].isnan().all() and lse.T[bad].isnan().all()
    # weights, products and sums in fp32 (2^-16 of |o| < 6 at most), one rounding of out
    assert (out.double() - ref)[~bad].abs().max() <= 2.0 ** -8 * ref[~bad].abs().max() + 6 * 2.0 ** -16
    assert (lse.T.double() - torch.logsumexp(z.double(), 0))[~bad].abs().max() <= 2.0 ** -16


@pytest.mark.parametrize("num_splits", [0, 1, 3])
@pytest.mark.parametrize("q_lens", [(1, 2), (9, 3)])
@pytest.mark.parametrize("which", ["decode", "decode_mxfp8", "decode_nvfp4", "extend"])
def test_a_nan_in_q_is_its_rows_alone(which, q_lens, num_splits):
    if which == "decode_mxfp8" and q_lens[0] > 2:
        pytest.skip("16 rows per kv head at most")
    c = U.Case(q_lens, (5000, 900), 16, 2, r_dim=64, E=128)
    d = U.make(c)
    kw = dict(max_seqlen_q=max(q_lens), max_seqlen_k=5000, alpha=c.alpha, num_splits=num_splits)
    t = {n: U.cuda(d[n]) for n in ("q", "k", "v", "r", "P", "cu_q", "cu_k")}
    rest = (t["r"], t["P"], t["cu_q"], t["cu_k"])
    if which == "decode_mxfp8":
        (k8, ks), (v8, vs) = rpb.quantize_mxfp8(t["k"]), rpb.quantize_mxfp8(t["v"])
        run = lambda q: rpb.decode_mxfp8(q, k8, v8, ks, vs, *rest, **kw)  # noqa: E731
    elif which == "decode_nvfp4":
        cache = U.device_cache(U.quantized(c, d), d)
        run = lambda q: rpb.decode_nvfp4(q, cache, *rest, **kw)[:2]  # noqa: E731
    else:
        run = lambda q: getattr(rpb, which)(q, t["k"], t["v"], *rest, **kw)  # noqa: E731
    want = run(t["q"])
    q = t["q"].clone()
    q[0, 3, 100], q[-1, 9, 0] = float("nan"), float("nan")
    hit = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    hit[0, 3] = hit[-1, 9] = True
    out, lse = run(q)
    X.ok()
    assert out[hit].isnan().all() and lse.T[hit].isnan().all()
    assert torch.equal(out[~hit], want[0][~hit]) and torch.equal(lse.T[~hit], want[1].T[~hit])
