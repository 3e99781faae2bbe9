"""relattn_extend on what the tests of its lengths and layouts leave out: blocks of
the band that straddle 64 keys, unusual values.  Tolerances as in test_extend_gpu.py."""
import numpy as np
import pytest
import torch

from tests import kvcache_util as U
from tests import test_extend_gpu as X
from tests.conftest import gpu_available
from tests.test_extend_gpu import _clean_error_word, _lib  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]


@pytest.mark.parametrize("more", range(0, 64, 7))
@pytest.mark.parametrize("Hq,Hkv", [(16, 2), (4, 1), (12, 4)])       # (the last has 192 distances at hand)
def test_pieces_of_the_band_whose_blocks_straddle_64_keys(Hq, Hkv, more):
    """The band in pieces: the first step of all but the nearest reads three chunks of
    distances where a block's rows straddle a multiple of 64."""
    X.check(U.Case((40,), (3000 + more,), Hq, Hkv, r_dim=16, E=1024, page=16, seed=more))


# Shapes that take every kernel: (Hq, Hkv, r_dim, E, page, tokens, keys, window, sink, num_splits)
PATHS = [
    (4, 1, 32, 64, 16, (1, 3), (200, 310), 0, 0, 0),             # short: one launch of the warp-MMA kernel
    (6, 2, 7, 33, 48, (40,), (500,), 90, 5, 0),                  # a shape that TMA does not describe
    (16, 2, 64, 256, 16, (1, 1), (5000, 900), 0, 0, 0),          # few rows, in splits
    (8, 2, 16, 64, 0, (2, 1), (900, 700), 0, 0, 1),              # in one
    (16, 2, 16, 128, 16, (40,), (2000,), 0, 0, 1),               # many rows, nothing cut: the band hands its rows on
    (4, 4, 16, 64, 0, (300, 70), (900, 600), 0, 0, 1),
    (16, 2, 64, 128, 64, (300, 70), (3000, 2600), 1000, 70, 1),
    (8, 1, 16, 128, 128, (600, 5, 200), (5000, 2000, 3500), 0, 0, 0),    # row tiles cut
    (16, 2, 16, 1024, 16, (40,), (6000,), 0, 0, 0),              # the band cut
    (16, 2, 0, 0, 16, (40,), (6000,), 0, 0, 0),                  # no band
    (16, 2, 16, 1024, 0, (300,), (300,), 0, 0, 1),               # nothing but the band
]


def place(p):
    Hq, Hkv, rd, E, page, q_lens, k_lens, window, sink, splits = p
    c = U.Case(q_lens, k_lens, Hq, Hkv, r_dim=rd, E=E, window=window, page=page, seed=Hq + len(q_lens))
    return c, U.make(c), sink, splits


def rows_of(c, b):
    first = sum(c.q_lens[:b])
    return slice(first, first + c.q_lens[b])


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("value", [float("inf"), -float("inf")])
def test_an_infinite_value_of_v_gives_infinities(path, value):
    """A key that every row of its sequence sees holds an infinity in one channel:
    every row's weight of it is above zero, so that channel is that infinity."""
    c, d, sink, splits = place(path)
    at = []
    for b, (nq, nk) in enumerate(zip(c.q_lens, c.k_lens)):
        g, ch = b % c.Hkv, 7 + 64 * (b % 2)
        d["v"][d["where"][b][max(nk - nq - 5, 0)], g, ch] = value
        at.append((rows_of(c, b), slice(g * (c.Hq // c.Hkv), (g + 1) * (c.Hq // c.Hkv)), ch))
    out, _ = X.call(c, d, sink, num_splits=splits)
    X.ok()
    for rows, heads, ch in at:
        assert (out[rows, heads, ch] == value).all()


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan"), 1e30, -3e38])
def test_one_large_value_of_v_stays_in_its_channel(path, value):
    """A key that every row of its sequence sees holds an infinity, a NaN or a value
    far above the others in one channel: that channel follows, the others do not change."""
    c, d, sink, splits = place(path)
    at = []
    for b, (nq, nk) in enumerate(zip(c.q_lens, c.k_lens)):
        g, ch = b % c.Hkv, 7 + 64 * (b % 2)
        d["v"][d["where"][b][max(nk - nq - 5, 0)], g, ch] = value
        at.append((rows_of(c, b), slice(g * (c.Hq // c.Hkv), (g + 1) * (c.Hq // c.Hkv)), ch))
    out, lse = X.call(c, d, sink, num_splits=splits)
    X.ok()
    got, got_z = out.double().cpu().numpy(), lse.double().cpu().numpy()
    finite = dict(d, v=torch.where(d["v"].isfinite(), d["v"], torch.zeros_like(d["v"])))
    ref, z, e_out, e_lse = X.bounds(c, finite, sink)
    # the sums of a row are fp32 and divided at the end; their weights are up to 2^8, so
    # a value of more than 2^120 (3e38 is 2^128) may pass the largest fp32 on the way
    if not abs(value) < 2.0 ** 120:
        for rows, heads, ch in at:
            hit = got[rows, heads, ch]
            right = np.isnan(hit) if np.isnan(value) else hit == np.sign(value) * np.inf
            if np.isfinite(value):
                right |= np.abs(hit - ref[rows, heads, ch]) <= e_out[rows, heads, ch]
            assert right.all(), hit
            got[rows, heads, ch] = ref[rows, heads, ch] = 0
    assert (np.abs(got - ref) <= e_out).all(), np.abs(got - ref).max()
    assert (np.abs(got_z - z) <= e_lse).all()


@pytest.mark.parametrize("path", PATHS)
def test_channels_of_any_size(path):
    """Channels of v from 2^-60 to 2^60 of the others: each is right to its own size."""
    c, d, sink, splits = place(path)
    scale = torch.exp2(torch.arange(128.0) * 37 % 121 - 60)
    d["v"] = (d["v"].float() * scale).bfloat16()
    out, lse = X.call(c, d, sink, num_splits=splits)
    X.ok()
    ref, z, e_out, e_lse = X.bounds(c, d, sink)
    assert (np.abs(out.double().cpu().numpy() - ref) <= e_out).all()


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("back", [0, 7, 150, 260, 800])
def test_a_nan_key_reaches_the_rows_that_see_it_whatever_is_cut(path, back):
    """out and lse of the rows that see a key of NaN are NaN; other rows are as without it."""
    c, d, sink, splits = place(path)
    want, z, e_out, e_lse = X.bounds(c, d, sink)
    hit = np.zeros((sum(c.q_lens), c.Hq), bool)
    for b, (nq, nk) in enumerate(zip(c.q_lens, c.k_lens)):
        j, g = max(nk - 1 - back, 0), b % c.Hkv
        d["k"][d["where"][b][j], g] = float("nan")
        pos = nk - nq + np.arange(nq)
        sees = (pos >= j) & ((c.window <= 0) | (pos - j < c.window) | (j < sink))
        hit[rows_of(c, b), g * (c.Hq // c.Hkv):(g + 1) * (c.Hq // c.Hkv)] |= sees[:, None]
    out, lse = X.call(c, d, sink, num_splits=splits)
    X.ok()
    got, got_z = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isnan(got[hit]).all() and np.isnan(got_z[hit.T]).all()
    assert (np.abs(got - want)[~hit] <= e_out[~hit]).all()
    assert (np.abs(got_z - z)[~hit.T] <= e_lse[~hit.T]).all()


def test_a_batch_of_many_empty_sequences_and_heads():
    """Sequences times heads above 2^25, with 17 tokens in all: the call runs, and asks for the workspace that it takes."""
    batch, H, q_len, k_len = 65535, 520, 17, 400
    c = U.Case((q_len,), (k_len,), H, H, r_dim=16, E=64, seed=4)
    d = U.make(c)
    for n, m in (("cu_q", q_len), ("cu_k", k_len)):
        d[n] = torch.zeros(batch + 1, dtype=torch.int32)
        d[n][40000:] = m
    out, lse = X.call(c, d, 0)
    X.ok()
    ref, z, e_out, e_lse = X.bounds(c, d, 0)
    assert (np.abs(out.double().cpu().numpy() - ref) <= e_out).all()
    assert (np.abs(lse.double().cpu().numpy() - z) <= e_lse).all()
