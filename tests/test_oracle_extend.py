"""The oracle of windows with sinks: without sinks it is the forward and backward
oracle's, sinks are what a brute-force softmax says, gradients match differences."""
import numpy as np
import pytest
import torch

import oracle
from oracle import extend as X
from relative_position_biased_gb300 import workloads as W


def make(q_lens, k_lens, Hq, Hkv, rd, E, seed=0):
    rng = np.random.default_rng(seed)
    t = lambda *s, f=1.0: torch.from_numpy(f * rng.standard_normal(s))  # noqa: E731
    Tq, Tk = sum(q_lens), sum(k_lens)
    starts = np.concatenate([[0], np.cumsum(k_lens)])
    return dict(q=t(Tq, Hq, 128), k=t(Tk, Hkv, 128), v=t(Tk, Hkv, 128), r=t(Tq, Hq, rd), P=t(rd, E, f=0.1)), \
        [np.arange(a, b) for a, b in zip(starts[:-1], starts[1:])]


@pytest.mark.parametrize("window,base", [(0, 0.0), (0, 8.0), (9, 0.0), (50, 8.0)])
def test_without_sinks_it_is_the_forward_and_backward_oracle(window, base):
    q_lens, k_lens = (12, 5, 1), (12, 40, 33)
    d, where = make(q_lens, k_lens, 4, 2, 6, 16)
    cu = W.cu_seqlens(q_lens), W.cu_seqlens(k_lens)
    kw = dict(alpha=0.09, window=window)
    out, lse, _, _ = X.forward(*d.values(), where, q_lens, sink=0, base=base, **kw)
    o, z = oracle.forward(*d.values(), *cu, log_scale_base=base, **kw)
    assert np.allclose(out, o, rtol=1e-12, atol=1e-13) and np.allclose(lse.T, z, rtol=1e-12)
    dout = torch.from_numpy(np.random.default_rng(1).standard_normal(out.shape))
    got = X.backward(*d.values(), torch.from_numpy(out), torch.from_numpy(lse), dout, where, q_lens, sink=0, base=base, **kw)
    for n, ref in zip(("dq", "dk", "dv", "dr"), oracle.backward(*d.values(), dout, *cu, log_scale_base=base, **kw)):
        assert np.allclose(got[n][0], ref, rtol=1e-10, atol=1e-12), n
        assert (np.abs(got[n][0]) <= got[n][1] * (1 + 1e-12)).all()


def test_a_sink_past_every_key_is_full_attention():
    d, where = make((20,), (20,), 2, 1, 4, 8)
    a = X.forward(*d.values(), where, (20,), alpha=0.1, window=3, sink=20, base=0.0)
    b = X.forward(*d.values(), where, (20,), alpha=0.1, window=0, sink=0, base=0.0)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_sinks_by_brute_force():
    d, where = make((7,), (15,), 2, 1, 4, 12)
    out, lse, _, _ = X.forward(*d.values(), where, (7,), alpha=0.1, window=3, sink=2, base=4.0)
    q, k, v, r, P = (t.numpy() for t in d.values())
    for t in range(7):
        i = 8 + t
        for h in range(2):
            keys = sorted(set(range(2)) | set(range(max(0, i - 2), i + 1)))
            s = max(1.0, np.log(i + 1) / np.log(4.0))
            x = np.array([s * (0.1 * q[t, h] @ k[j, 0] + (r[t, h] @ P[:, i - j] if i - j < 12 else 0)) for j in keys])
            e = np.exp(x)
            assert np.isclose(lse[h, t], np.log(e.sum()), rtol=1e-12)
            assert np.allclose(out[t, h], (e[:, None] * v[keys, 0]).sum(0) / e.sum(), rtol=1e-10)


@pytest.mark.parametrize("window,sink,E", [(3, 2, 12), (6, 4, 4), (2, 9, 30)])
def test_gradients_by_differences(window, sink, E):
    d, where = make((9, 4), (9, 13), 2, 1, 3, E, seed=2)
    kw = dict(alpha=0.08, window=window, sink=sink, base=5.0)
    q_lens = (9, 4)
    out, lse, _, _ = X.forward(*d.values(), where, q_lens, **kw)
    rng = np.random.default_rng(3)
    dout = rng.standard_normal(out.shape)
    got = X.backward(*d.values(), torch.from_numpy(out), torch.from_numpy(lse), torch.from_numpy(dout), where, q_lens, **kw)
    for n in ("q", "k", "v", "r"):
        step = rng.standard_normal(d[n].shape)
        ends = []
        for e in (1e-5, -1e-5):
            moved = dict(d, **{n: d[n] + e * torch.from_numpy(step)})
            ends.append((X.forward(*moved.values(), where, q_lens, **kw)[0] * dout).sum())
        want = (ends[0] - ends[1]) / 2e-5
        assert np.isclose((got["d" + n][0] * step).sum(), want, rtol=1e-6, atol=1e-8), n
