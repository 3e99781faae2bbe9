"""Refusals of the compressed-cache entry points (no GPU needed: every one is
decided on the host before a device is touched)."""
import copy
import ctypes
import pickle

import pytest
import torch

import relative_position_biased_gb300 as rpb

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 5
A = 1 << 20                                    # aligned stand-ins for device pointers, never read here


@pytest.fixture(scope="module", autouse=True)
def _lib():
    rpb.build()
    rpb.load_library()


def fwd(**kw):
    d = dict(q=A, k=2 * A, r=3 * A, P=4 * A, cu_seqlens_q=5 * A, cu_seqlens_k=6 * A, batch=2, total_q=2, total_k=600,
             max_seqlen_q=1, max_seqlen_k=400, num_heads_q=8, num_heads_kv=2, head_dim=128, r_dim=16, rel_extent=64,
             window=0, alpha=0.1, log_scale_base=0.0, out=7 * A, lse=8 * A, workspace=None, workspace_bytes=0)
    d.update(kw)
    return rpb.RelattnParams(**d)


def cache(**kw):
    d = dict(k=20 * A, v=22 * A, k_scale=24 * A, v_scale=26 * A, k_global=None, v_global=None, rows=600)
    d.update(kw)
    return rpb.RelattnKvNvfp4(**d)


def pages(**kw):
    d = dict(block_table=30 * A, max_pages_per_seq=7, page_size=64, num_pages=10)
    d.update(kw)
    return rpb.RelattnPagedKV(**d)


@pytest.mark.parametrize("kw,want", [
    (dict(head_dim=64), UNSUPPORTED), (dict(num_heads_kv=3), INVALID), (dict(max_seqlen_q=17, max_seqlen_k=17), UNSUPPORTED),
    (dict(r_dim=65), UNSUPPORTED), (dict(alpha=float("nan")), INVALID), (dict(log_scale_base=1.0), INVALID),
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(lse=None), INVALID), (dict(q=A + 2), INVALID),
    (dict(r=None), INVALID), (dict(total_k=601), INVALID), (dict(batch=-1), INVALID),
    (dict(batch=40000), UNSUPPORTED), (dict(max_seqlen_k=0), INVALID),
    (dict(max_seqlen_k=(1 << 31) - (1 << 16) + 1, total_k=(1 << 31) - 1), UNSUPPORTED),
])
def test_decode_refuses_parameters(kw, want):
    assert rpb.relattn_decode_nvfp4(fwd(**kw), cache()) == want


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), INVALID), (dict(v=20 * A + 8), INVALID), (dict(k_scale=None), INVALID),
    (dict(v_scale=A + 4), INVALID), (dict(k_global=A + 1), INVALID), (dict(rows=599), INVALID), (dict(rows=-1), INVALID),
    (dict(rows=1 << 31), UNSUPPORTED),
])
def test_decode_refuses_caches(kw, want):
    assert rpb.relattn_decode_nvfp4(fwd(), cache(**kw)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(page_size=0), INVALID), (dict(page_size=48), UNSUPPORTED), (dict(num_pages=0), INVALID),
    (dict(block_table=None), INVALID), (dict(block_table=A + 2), INVALID), (dict(max_pages_per_seq=6), INVALID),
    (dict(num_pages=11), INVALID), (dict(num_pages=1 << 26), UNSUPPORTED),
])
def test_decode_refuses_pages(kw, want):
    assert rpb.relattn_decode_nvfp4(fwd(), cache(rows=640), None, pages(**kw)) == want


def test_decode_refuses_half_given_positions():
    for kw in (dict(key_pos=A, q_pos=None), dict(key_pos=None, q_pos=A), dict(key_pos=A + 2, q_pos=A)):
        assert rpb.relattn_decode_nvfp4(fwd(), cache(), rpb.RelattnPositions(**kw)) == INVALID


def rows(**kw):
    d = dict(k=A, v=2 * A, cu_seqlens_q=3 * A, cu_seqlens_k=4 * A, batch=2, total_q=40, num_heads_kv=2, head_dim=128,
             cache=ctypes.pointer(cache()), pages=None)
    d.update(kw)
    return rpb.RelattnCacheRowsParams(**d)


@pytest.mark.parametrize("kw,want", [
    (dict(head_dim=64), UNSUPPORTED), (dict(cache=None), INVALID), (dict(k=None), INVALID), (dict(v=A + 8), INVALID),
    (dict(cu_seqlens_k=None), INVALID), (dict(total_q=-1), INVALID), (dict(num_heads_kv=0), INVALID),
    (dict(k=20 * A), INVALID), (dict(v=24 * A + 600 * 16 - 16), INVALID),          # inside the codes / the scales
    (dict(pages=ctypes.pointer(pages(page_size=33))), UNSUPPORTED),
])
def test_store_and_load_refuse(kw, want):
    assert rpb.relattn_store_nvfp4(rows(**kw)) == want
    assert rpb.relattn_load_nvfp4(rows(**kw)) == want


def weights(f=None, **kw):
    d = dict(fwd=f or fwd(out=None, v=None), cache=None, positions=None, pages=None, weights_in=40 * A, weights_out=42 * A,
             decay=0.5, workspace=50 * A, workspace_bytes=1 << 20)
    d.update(kw)
    return rpb.RelattnKeyWeightsParams(**d)


@pytest.mark.parametrize("p,want", [
    (lambda: weights(decay=-0.5), INVALID), (lambda: weights(decay=float("inf")), INVALID),
    (lambda: weights(weights_out=None), INVALID), (lambda: weights(weights_out=A + 2), INVALID),
    (lambda: weights(weights_out=40 * A + 400), INVALID),                          # overlaps, not in place
    (lambda: weights(f=fwd(k=None)), INVALID), (lambda: weights(f=fwd(lse=None)), INVALID),
    (lambda: weights(workspace=None), WORKSPACE), (lambda: weights(workspace_bytes=2 * 8 * 64 * 4 - 1), WORKSPACE),
    (lambda: weights(workspace=A + 4), WORKSPACE),
    (lambda: weights(f=fwd(batch=40000)), UNSUPPORTED),
    (lambda: weights(cache=ctypes.pointer(cache(rows=599))), INVALID),
    (lambda: weights(cache=ctypes.pointer(cache(v_scale=None))), INVALID),
])
def test_key_weights_refuse(p, want):
    assert rpb.relattn_key_weights(p()) == want


def test_key_weights_refuse_more_units_than_a_grid_holds():
    """2^24 tiles of 128 keys for each of 130 heads; of a contiguous cache its rows
    count, and few rows are walked whatever the bound."""
    many = dict(out=None, v=None, batch=65, total_q=65 * 20, max_seqlen_q=20, max_seqlen_k=(1 << 31) - (1 << 16))
    wide = ctypes.pointer(pages(page_size=1 << 20, num_pages=1, max_pages_per_seq=1 << 11))
    big = ctypes.pointer(cache(rows=1 << 20))
    for c in (None, big):
        p = weights(f=fwd(**many), cache=c, pages=wide, weights_in=None, workspace_bytes=1 << 40)
        assert rpb.relattn_key_weights(p) == UNSUPPORTED
    # (these pass the check and stop at the next one)
    assert rpb.relattn_key_weights(weights(f=fwd(**many), workspace=None)) == WORKSPACE
    few = dict(many, max_seqlen_q=1, total_q=65)
    assert rpb.relattn_key_weights(weights(f=fwd(**few), cache=big, pages=wide, weights_in=None, workspace=None)) == WORKSPACE


def evict(**kw):
    d = dict(weights=A, cu_seqlens_k=2 * A, cu_seqlens_keep=3 * A, key_pos=None, batch=2, total_k=600, total_keep=100,
             max_seqlen_k=400, num_heads_kv=2, sink=4, recent=16, rows=600, rows_keep=100, pages=None, pages_keep=None,
             num_planes=0, weights_out=4 * A, key_pos_out=5 * A, workspace=50 * A, workspace_bytes=1 << 20)
    planes = kw.pop("planes", [])
    d.update(kw)
    p = rpb.RelattnEvictParams(**d)
    for i, x in enumerate(planes):
        p.planes[i] = rpb.RelattnPlane(*x)
        p.num_planes = i + 1
    return p


@pytest.mark.parametrize("kw,want", [
    (dict(weights=None), INVALID), (dict(cu_seqlens_keep=None), INVALID), (dict(total_keep=601), INVALID),
    (dict(rows=599), INVALID), (dict(rows_keep=99), INVALID), (dict(sink=-1), INVALID), (dict(recent=-1), INVALID),
    (dict(num_planes=9), INVALID), (dict(num_planes=1), INVALID), (dict(planes=[(6 * A, 8 * A, 0)]), INVALID),
    (dict(planes=[(6 * A, 6 * A + 64, 64)]), INVALID), (dict(planes=[(6 * A, 8 * A, 64), (10 * A, 8 * A, 64)]), INVALID),
    (dict(weights_out=A), INVALID), (dict(weights_out=5 * A), INVALID), (dict(key_pos=5 * A), INVALID),
    (dict(workspace=None), WORKSPACE), (dict(workspace_bytes=100 * 3 * 4 - 1), WORKSPACE), (dict(workspace=A + 8), WORKSPACE),
    (dict(pages=ctypes.pointer(pages(page_size=16, num_pages=40)), rows=640), UNSUPPORTED),
    (dict(rows=1 << 31), UNSUPPORTED), (dict(max_seqlen_k=(1 << 31) - (1 << 16) + 1), UNSUPPORTED),
    # few long sequences need more than the kept rows' numbers
    (dict(max_seqlen_k=40000, rows=40000, total_k=40000, workspace_bytes=100 * 3 * 4), WORKSPACE),
])
def test_evict_refuses(kw, want):
    assert rpb.relattn_evict(evict(**kw)) == want


def test_evict_refuses_more_units_than_a_grid_holds():
    """16 CTAs each of 2^27 (sequence, kv head) pairs: before anything is launched."""
    for batch, want in ((1 << 26, UNSUPPORTED), ((1 << 26) - 1, WORKSPACE)):
        assert rpb.relattn_evict(evict(batch=batch, max_seqlen_k=400, clear_out=1, workspace=None)) == want


def test_evict_workspace_size_refuses_negative_sizes():
    for kw in (dict(batch=-1), dict(max_seqlen_k=-1), dict(total_keep=-1), dict(num_heads_kv=0)):
        assert rpb.relattn_evict_workspace_size(evict(**kw))[0] == INVALID
    assert rpb.relattn_evict_workspace_size(evict(batch=-1, max_seqlen_k=40000))[0] == INVALID


def test_empty_calls_are_accepted():
    assert rpb.relattn_decode_nvfp4(fwd(batch=0, total_q=0), cache()) == 0
    assert rpb.relattn_store_nvfp4(rows(batch=0)) == 0
    assert rpb.relattn_load_nvfp4(rows(total_q=0)) == 0
    assert rpb.relattn_key_weights(weights(f=fwd(batch=0))) == 0
    assert rpb.relattn_evict(evict(batch=0)) == 0
    assert rpb.relattn_evict(evict(total_keep=0)) == 0


def test_null_parameters():
    lib = rpb.load_library()
    assert lib.relattn_store_nvfp4(None, None) == INVALID
    assert lib.relattn_load_nvfp4(None, None) == INVALID
    assert lib.relattn_decode_nvfp4(None, None, None, None, None) == INVALID
    assert lib.relattn_decode_nvfp4(ctypes.byref(fwd()), None, None, None, None) == INVALID
    assert lib.relattn_key_weights(None, None) == INVALID
    assert lib.relattn_evict(None, None) == INVALID
    n = ctypes.c_size_t(0)
    assert lib.relattn_decode_nvfp4_workspace_size(None, None, ctypes.byref(n)) == INVALID
    assert lib.relattn_key_weights_workspace_size(None, ctypes.byref(n)) == INVALID
    assert lib.relattn_evict_workspace_size(None, ctypes.byref(n)) == INVALID


def test_workspace_sizes():
    st, n = rpb.relattn_key_weights_workspace_size(weights())
    assert (st, n) == (0, 2 * 8 * 64 * 4)
    assert rpb.relattn_key_weights_workspace_size(weights(f=fwd(r_dim=0, rel_extent=0))) == (0, 0)
    assert rpb.relattn_evict_workspace_size(evict()) == (0, 100 * 3 * 4)
    st, n = rpb.relattn_evict_workspace_size(evict(max_seqlen_k=40000))
    assert st == 0 and n > 4 * 3 * 2048 * 4                # three histograms of every (sequence, head)
    assert rpb.relattn_evict_workspace_size(evict(max_seqlen_k=40000, batch=5)) == (0, 100 * 3 * 4)


def test_python_checks_name_the_argument():
    """The conveniences refuse wrong tensors before the library sees them."""
    c = rpb.empty_nvfp4(64, 2, "cpu")
    k = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        rpb.store_nvfp4(k, k, cu, cu, c)
    q = torch.zeros(1, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        rpb.decode_nvfp4(q, c, None, None, cu, cu, max_seqlen_q=1, max_seqlen_k=4, alpha=1.0)
    with pytest.raises(ValueError, match="k must be torch.bfloat16"):
        rpb.store_nvfp4(k.float(), k, cu, cu, c)
    with pytest.raises(ValueError, match="v must have shape"):
        rpb.store_nvfp4(k, k[:2], cu, cu, c)
    with pytest.raises(ValueError, match="cu_seqlens_k must have shape"):
        rpb.store_nvfp4(k, k, cu, cu[:1], c)
    with pytest.raises(ValueError, match="contiguous"):
        rpb.store_nvfp4(torch.zeros(4, 2, 256, dtype=torch.bfloat16)[..., ::2], k, cu, cu, c)
    with pytest.raises(ValueError, match="cache.v must be torch.uint8"):
        rpb.KvNvfp4(c.k, c.v.float(), c.k_scale, c.v_scale)
    with pytest.raises(ValueError, match="cache.k_scale must have shape"):
        rpb.KvNvfp4(c.k, c.v, c.k_scale[:, :1], c.v_scale)
    with pytest.raises(ValueError, match="cache.v_global must have shape"):
        rpb.KvNvfp4(*c[:4], None, torch.ones(3))
    with pytest.raises(ValueError, match="KvNvfp4"):
        rpb.store_nvfp4(k, k, cu, cu, tuple(c))
    with pytest.raises(ValueError, match="page_size"):
        rpb.store_nvfp4(k, k, cu, cu, c, block_table=torch.zeros(1, 2, dtype=torch.int32), page_size=48)


def test_a_workspace_is_one_block_of_memory():
    """A strided tensor's elements are not the bytes the library would write."""
    cpu = torch.device("cpu")
    for w in (torch.zeros(64, 4)[:, :2], torch.zeros(256)[::2], torch.zeros(1).expand(256)):
        with pytest.raises(ValueError, match="workspace must be contiguous"):
            rpb._workspace(512, w, cpu)
    w = torch.zeros(256)[128:]
    assert rpb._workspace(512, w, cpu) == (w, w.data_ptr(), 512)


def test_caches_made_from_a_cache_are_checked_too():
    c = rpb.empty_nvfp4(64, 2, "cpu")
    g = torch.ones(2)
    other = rpb.empty_nvfp4(64, 2, "cpu")
    d = c._replace(k=other.k, k_global=g)
    assert isinstance(d, rpb.KvNvfp4) and (d.rows, d.num_heads_kv, d.device) == (64, 2, c.device)
    assert (d.c_struct.k, d.c_struct.k_global, d.c_struct.v) == (other.k.data_ptr(), g.data_ptr(), c.v.data_ptr())
    with pytest.raises(ValueError, match="cache.v must have shape"):
        c._replace(v=c.v[:32])
    with pytest.raises(ValueError, match="cache.k_global must be torch.float32"):
        c._replace(k_global=g.double())
    assert rpb.KvNvfp4._make(tuple(c)).c_struct.k == c.k.data_ptr()
    assert copy.copy(c).c_struct.k == c.k.data_ptr()
    for e in (copy.deepcopy(c), pickle.loads(pickle.dumps(c))):
        assert e.c_struct.k == e.k.data_ptr() != c.k.data_ptr() and e.rows == 64


def test_a_cache_follows_its_tensors_to_other_memory():
    """Memory that a tensor has left is never passed to the library."""
    g = torch.ones(2)
    c = rpb.empty_nvfp4(64, 2, "cpu", k_global=g)
    other = rpb.empty_nvfp4(64, 2, "cpu")
    c.k.data = other.k
    c.v_scale.set_(other.v_scale)
    g.data = torch.full((2,), 2.0)
    rpb._cache(c, c.device)
    s = c.c_struct
    assert (s.k, s.v, s.k_scale, s.v_scale, s.k_global, s.v_global, s.rows) == (
        other.k.data_ptr(), c.v.data_ptr(), c.k_scale.data_ptr(), other.v_scale.data_ptr(), g.data_ptr(), None, 64)
    c.v.data = torch.zeros(32, 2, 64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="cache.v must have shape"):
        rpb._cache(c, c.device)


def test_every_call_names_a_wrong_cache():
    c = rpb.empty_nvfp4(64, 2, "cpu")
    cu = torch.tensor([0, 4], dtype=torch.int32)
    k = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    for wrong in (tuple(c), None, c.k):
        with pytest.raises(ValueError, match="cache must be a KvNvfp4"):
            rpb.load_nvfp4(wrong, cu, cu, total_q=4)
        with pytest.raises(ValueError, match="cache must be a KvNvfp4"):
            rpb.store_nvfp4(k, k, cu, cu, wrong)
    with pytest.raises(ValueError, match="CUDA"):
        rpb.load_nvfp4(c, cu, cu, total_q=4)
