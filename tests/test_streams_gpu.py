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


@pytest.mark.parametrize("which,q_lens", [("decode", (1, 1)), ("decode", (9, 16)), ("decode_paged", (1, 1)), ("decode_paged", (9, 16)),
                                          ("decode_mxfp8", (1, 2))])     # (16 rows per kv head at most)
def test_decode(which, q_lens):
    c = U.Case(q_lens, (5000, 900), 16, 2, r_dim=64, E=128, page=128 if which == "decode_paged" else 0)
    d = U.make(c)
    t = {n: U.cuda(d[n]) for n in ("q", "k", "v", "r", "P", "cu_q", "cu_k")}
    kw = dict(max_seqlen_q=max(q_lens), max_seqlen_k=5000, alpha=c.alpha)
    if which == "decode_paged":
        kw.update(page_size=128, total_k=5900)
        args = (*t.values(), d["table"].cuda())
    elif which == "decode_mxfp8":
        (k8, ks), (v8, vs) = rpb.quantize_mxfp8(t["k"]), rpb.quantize_mxfp8(t["v"])
        args = (t["q"], k8, v8, ks, vs, t["r"], t["P"], t["cu_q"], t["cu_k"])
    else:
        args = tuple(t.values())
    want = getattr(rpb, which)(*args, **kw)
    X.ok()
    splits = 152                                             # (a workspace of any number of them)
    sizes = [n * sum(q_lens) * 16 * 129 * 4 for n in range(2, splits, 5)]
    got = late(lambda s: getattr(rpb, which)(*args, stream=s, **kw), sizes)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_calls_by_name_and_on_the_default_stream():
    c = U.Case((40,), (40,), 4, 1, r_dim=16, E=64)
    d = U.make(c)
    names = dict(q="q", k="k", v="v", r="r", P="P", cu_seqlens_q="cu_q", cu_seqlens_k="cu_k")
    t = {n: U.cuda(d[m]) for n, m in names.items()}
    kw = dict(max_seqlen_q=40, max_seqlen_k=40, alpha=c.alpha)
    a = rpb.prefill(**t, **kw)
    b = rpb.prefill(**t, **kw, stream=0)
    X.ok()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
