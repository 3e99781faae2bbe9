"""Pins of the compressed-cache oracle (CPU): format values, borders and
rounding, the attention against the forward oracle, and eviction's choice."""
import math

import numpy as np
import pytest
import torch

from oracle import kvcache as C
from relative_position_biased_gb300 import workloads as W


def _block(vals):
    x = np.zeros((1, 1, 128), np.float32)
    x[0, 0, :len(vals)] = vals
    return x


def test_e4m3_values_match_torch():
    codes = torch.arange(127, dtype=torch.uint8)
    np.testing.assert_array_equal(C.E4M3, codes.view(torch.float8_e4m3fn).double().numpy())


def test_representable_values_round_trip():
    vals = np.concatenate([C.E2M1, -C.E2M1[1:]]).astype(np.float32)     # amax 6: scale 1
    codes, scales = C.quantize_nvfp4(_block(vals))
    assert scales[0, 0, 0] == 0x38 and (scales[0, 0, 1:] == 0).all()
    np.testing.assert_array_equal(C.dequantize_nvfp4(codes, scales)[0, 0, :15], vals)


def test_ties_go_to_the_even_code():
    ties = np.array([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -2.5], np.float32)
    got = C.dequantize_nvfp4(*C.quantize_nvfp4(_block(ties)))[0, 0, :10]
    np.testing.assert_array_equal(got, [6, 0, 1, 1, 2, 2, 4, 4, 0, -2])


def test_scale_ties_saturation_zero_and_nan():
    # 6 * (1 + 1/16) is between the scales 1 and 1.125: the tie goes to the even code 0x38
    assert C.quantize_nvfp4(_block([6 * 1.0625]))[1][0, 0, 0] == 0x38
    assert C.quantize_nvfp4(_block([6 * 1.1875]))[1][0, 0, 0] == 0x3A
    codes, scales = C.quantize_nvfp4(_block([1e6, 1.0]))
    assert scales[0, 0, 0] == 0x7E
    assert C.dequantize_nvfp4(codes, scales)[0, 0, 0] == 448 * 6
    codes, scales = C.quantize_nvfp4(_block([1e-5]))           # scale rounds to zero
    assert scales[0, 0, 0] == 0 and (codes == 0).all()
    codes, scales = C.quantize_nvfp4(_block([np.nan, 1.0]))
    assert scales[0, 0, 0] == 0x7F and np.isnan(C.dequantize_nvfp4(codes, scales)[0, 0, 1])


def test_factor_scales_the_rows():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 2, 128)).astype(np.float32)
    a = C.dequantize_nvfp4(*C.quantize_nvfp4(x))
    f = np.array([0.25, 4.0], np.float32)
    b = C.dequantize_nvfp4(*C.quantize_nvfp4(x * f[:, None], f), f)
    np.testing.assert_allclose(b, a * f[:, None], rtol=0, atol=0)


def test_relative_error_of_normal_values_is_bounded():
    # the scale's rounding moves the largest element by at most 2^-4, and the
    # widest code step is a third of the element below it
    rng = np.random.default_rng(1)
    x = rng.standard_normal((64, 2, 128)).astype(np.float32)
    y = C.dequantize_nvfp4(*C.quantize_nvfp4(x))
    amax = np.repeat(np.abs(x).reshape(64, 2, 8, 16).max(-1), 16, -1)
    assert (np.abs(y - x) <= amax * (1 / 6 + 1 / 16)).all()


@pytest.mark.parametrize("window,base", [(0, 0.0), (40, 0.0), (0, 64.0)])
def test_attention_matches_the_forward_oracle(window, base, oracle_mod):
    w = W.custom("kvc", [9, 3], [100, 60], 4, 2, 16, 32, window=window, log_scale_base=base)
    inp = W.make_inputs(w)
    f = {k: v.double().numpy() for k, v in inp.items()}
    out, lse = oracle_mod.forward(inp["q"], inp["k"], inp["v"], inp["r"], inp["P"], inp["cu_seqlens_q"],
                                  inp["cu_seqlens_k"], alpha=w.alpha, window=window, log_scale_base=base)
    q0 = k0 = 0
    for nq, nk in zip(w.q_lens, w.k_lens):
        for h in range(4):
            x, _ = C.logits(f["q"][q0:q0 + nq, h], f["k"][k0:k0 + nk, h // 2], f["r"][q0:q0 + nq, h], f["P"],
                            np.arange(nk - nq, nk), np.arange(nk), alpha=w.alpha, window=window, base=base)
            p, z = C.softmax(x)
            np.testing.assert_allclose(p @ f["v"][k0:k0 + nk, h // 2], out[q0:q0 + nq, h], atol=1e-12)
            np.testing.assert_allclose(z, lse[q0:q0 + nq, h], atol=1e-12)
        q0, k0 = q0 + nq, k0 + nk


def test_rows_that_see_nothing():
    x = np.full((2, 3), -np.inf)
    x[1, 0] = 0.5
    p, z = C.softmax(x)
    assert (p[0] == 0).all() and z[0] == -np.inf and p[1, 0] == 1 and z[1] == 0.5


def test_gaps_in_the_positions_keep_distances():
    rng = np.random.default_rng(2)
    q, k, r, P = (rng.standard_normal(s) for s in ((1, 128), (50, 128), (1, 8), (8, 20)))
    full, mag = C.logits(q, k, r, P, [49], np.arange(50), alpha=0.1, window=30)
    keep = np.array([0, 3, 21, 22, 40, 48, 49])
    part, _ = C.logits(q, k[keep], r, P, [49], keep, alpha=0.1, window=30)
    # the two products may add their 128 terms in different orders: each sum is
    # within 128 * 2^-53 of its terms' magnitudes of the exact one, twice that apart
    np.testing.assert_array_equal(np.isneginf(part), np.isneginf(full[:, keep]))
    seen = ~np.isneginf(part)
    assert (np.abs(part - full[:, keep])[seen] <= (256 * 2.0 ** -53 * mag[:, keep])[seen]).all()


def test_eviction_choice():
    w = [5.0, 1.0, 3.0, 3.0, 3.0, np.nan, 0.0, 2.0]
    assert C.kept_keys(w, 4, 1, 1).tolist() == [0, 2, 3, 7]
    assert C.kept_keys(w, 3, 0, 0).tolist() == [0, 2, 3]
    assert C.kept_keys(w, 2, 5, 5).tolist() == [6, 7]
    assert C.kept_keys(w, 8, 0, 0).tolist() == list(range(8))
    assert C.kept_keys(w, 7, 0, 0).tolist() == [0, 1, 2, 3, 4, 6, 7]
    assert C.kept_keys([0.0, -0.0, 0.0], 2, 0, 0).tolist() == [0, 1]
    assert not math.isnan(C.kept_keys([np.nan], 1, 0, 0)[0])
