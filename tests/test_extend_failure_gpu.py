"""Failure paths of relattn_extend's kernels that wait, without faulting the GPU:
a hook of the test build leaves one key tile out, the bounded waits behind it run
out after about a second, every role stops, tensor memory is freed, the host
reads RELATTN_ERR_TIMEOUT, and the next call is right."""
import pytest
import torch

import relative_position_biased_gb300 as rpb
from tests import kvcache_util as U
from tests import test_extend_gpu as X

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _test_build():
    rpb.build()
    with rpb.test_library():
        yield


@pytest.mark.parametrize("q_len,E,num_splits,tile", [
    (1, 64, 1, 1),              # few rows
    (40, 64, 1, 0),             # the band's first block of keys; the other keys' first tile
    (40, 64, 1, 2),             # a later one
    (40, 0, 1, 3),              # no band
    (40, 64, 3, 1),             # partials
])
@pytest.mark.parametrize("page", [0, 16])
def test_extend_gives_up_and_recovers(q_len, E, num_splits, tile, page):
    c = U.Case((q_len,), (900,), 8, 1, r_dim=16 if E else 0, E=E, page=page)
    d = U.make(c)
    call = lambda: X.call(c, d, 0, num_splits=num_splits)  # noqa: E731
    assert rpb.relattn_get_device_error() == rpb.RELATTN_OK      # start clean
    assert rpb.relattn_test_skip_k_tile(tile) == rpb.RELATTN_OK
    try:
        call()                                                   # the launches themselves succeed
        torch.cuda.synchronize()                                 # and every CTA ends
        st, word = rpb.relattn_get_device_error(), rpb.relattn_last_device_error_word()
    finally:
        rpb.relattn_test_skip_k_tile(-1)
    assert st == rpb.RELATTN_ERR_TIMEOUT, (st, hex(word))
    assert word & 2 and (word >> 8) > 0
    X.check(c, num_splits=num_splits)
