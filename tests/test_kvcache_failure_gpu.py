"""Failure paths of the compressed cache's kernels that wait, without faulting
the GPU: a hook of the test build leaves one key tile out of the tensor-core
kernels, the bounded waits behind it run out after about a second, every role
stops, tensor memory is freed, the host reads RELATTN_ERR_TIMEOUT, and the next
call is right.  In the same way a CTA stays away from an eviction's grid-wide
selection."""
import numpy as np
import pytest
import torch

import relative_position_biased_gb300 as rpb
from oracle import kvcache as C
from relative_position_biased_gb300 import workloads as W
from tests import kvcache_util as U

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _test_build():
    rpb.build()
    with rpb.test_library():
        yield


def times_out(call, tile):
    assert rpb.relattn_get_device_error() == rpb.RELATTN_OK      # start clean
    assert rpb.relattn_test_skip_k_tile(tile) == rpb.RELATTN_OK
    try:
        call()                                                   # the launch itself succeeds
        torch.cuda.synchronize()                                 # and every CTA ends
        st, word = rpb.relattn_get_device_error(), rpb.relattn_last_device_error_word()
    finally:
        rpb.relattn_test_skip_k_tile(-1)
    assert st == rpb.RELATTN_ERR_TIMEOUT, (st, hex(word))
    assert word & 2 and (word >> 8) > 0


@pytest.mark.parametrize("tile", [0, 2])
def test_decode_of_many_rows_gives_up_and_recovers(tile):
    c = U.Case((9,), (700,), 8, 1, E=64)                         # 72 rows
    d = U.make(c)
    qc = U.quantized(c, d)
    cache = U.device_cache(qc, d)
    call = lambda: rpb.decode_nvfp4(d["q"].cuda(), cache, d["r"].cuda(), d["P"].cuda(), d["cu_q"].cuda(),  # noqa: E731
                                    d["cu_k"].cuda(), num_splits=1, **U.call_kw(c, d))
    times_out(call, tile)
    out, lse = call()
    assert rpb.relattn_get_device_error() == rpb.RELATTN_OK
    U.check_decode(c, d, qc["k_values"], qc["v_values"], out, lse)


def test_key_weights_of_many_rows_give_up_and_recover():
    c = U.Case((40,), (300,), 8, 1, E=64)
    d = U.make(c)
    keys = d["k"].double().numpy()
    lse = np.full((c.Hq, 40), 6.0, np.float32)
    w_in = np.zeros((c.Hkv, d["rows"]), np.float32)

    def call():
        return rpb.key_weights(d["q"].cuda(), d["k"].cuda(), d["r"].cuda(), d["P"].cuda(), torch.from_numpy(lse).cuda(),
                               d["cu_q"].cuda(), d["cu_k"].cuda(), decay=0.0, **U.call_kw(c, d))

    times_out(call, 0)
    out = call()
    assert rpb.relattn_get_device_error() == rpb.RELATTN_OK
    U.check_weights(c, d, keys, lse, w_in, 0.0, out)


@pytest.mark.parametrize("cta", [0, 5])
def test_eviction_by_all_sms_gives_up_moves_nothing_and_recovers(cta):
    """The workspace holds numbers of rows, which nobody takes for a selection's."""
    lens, keep = [40000, 70], [9000, 40]
    w = torch.rand(2, sum(lens), device="cuda")
    p = torch.rand(sum(lens), 2, 4, device="cuda")
    out = torch.full((sum(keep), 2, 4), 3.0, device="cuda")
    work = torch.full((1 << 20,), 7, dtype=torch.int32, device="cuda")

    def call():
        return rpb.evict([p], [out], w, W.cu_seqlens(lens).cuda(), W.cu_seqlens(keep).cuda(), max_seqlen_k=40000,
                         recent=16, sink=2, total_keep=sum(keep), workspace=work)

    times_out(call, cta)
    assert (out == 3).all()
    pos, wk = call()
    assert rpb.relattn_get_device_error() == rpb.RELATTN_OK
    for b in range(2):
        a, o = sum(lens[:b]), sum(keep[:b])
        for h in range(2):
            idx = C.kept_keys(w[h, a:a + lens[b]].cpu().numpy(), keep[b], 16, 2)
            np.testing.assert_array_equal(pos[h, o:o + keep[b]].cpu().numpy(), idx)
            assert torch.equal(out[o:o + keep[b], h], p[a + torch.from_numpy(idx).cuda(), h])
