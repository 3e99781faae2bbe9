"""relattn_extend on what the tests of its lengths and layouts leave out: blocks of
the band that straddle 64 keys, unusual values.  Tolerances as in test_extend_gpu.py."""
import pytest

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
