"""A call with a stream of its own: what it allocates for itself belongs to that
stream, so that memory which the caller's stream takes and writes meanwhile is
other memory."""
import pytest
import torch

import relative_position_biased_gb300 as rpb
from tests import kvcache_util as U
from tests import test_extend_gpu as X
from tests.conftest import gpu_available
from tests.test_extend_gpu import _clean_error_word, _lib  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]


def late(call, sizes):
    """call(stream) on a stream that is kept busy, then the caller's stream takes
    blocks of the given sizes (bytes) and fills them with NaN."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)                       # about 0.1 s
    got = call(s.cuda_stream)
    held = [torch.full((max(n // 4, 1),), float("nan"), device="cuda") for n in sizes for _ in range(3)]
    torch.cuda.synchronize()
    X.ok()
    del held
    return got


@pytest.mark.parametrize("sink", [0, 4])
def test_backward(sink):
    c = U.Case((300, 150), (300, 200), 16, 2, r_dim=32, E=64, window=70)
    d, out, lse, dout, args, kw = X.grads(c, sink)
    want = rpb.backward(*args, sink=sink, **kw)
    X.ok()
    prm = rpb.RelattnBwdParams(fwd=rpb.make_params(*args[:5], *args[8:], out=out, lse=lse, **kw), dout=dout.data_ptr())
    n = rpb.relattn_backward_sinks_workspace_size(prm, sink)[1]
    got = late(lambda s: rpb.backward(*args, sink=sink, stream=s, **kw), [n])
    assert all(torch.equal(a, b) for a, b in zip(want, got))
