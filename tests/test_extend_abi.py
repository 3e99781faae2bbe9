"""Refusals of relattn_extend, relattn_backward_sinks and relattn_prologue_paged
(no GPU needed: every one is decided on the host before a device is touched)."""
import pytest
import torch

import relative_position_biased_gb300 as rpb

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 5
A = 1 << 24                                    # aligned stand-ins for device pointers, never read here


@pytest.fixture(scope="module", autouse=True)
def _lib():
    rpb.build()
    rpb.load_library()


def fwd(**kw):
    d = dict(q=A, k=2 * A, v=3 * A, r=4 * A, P=5 * A, cu_seqlens_q=6 * A, cu_seqlens_k=7 * A, batch=2, total_q=40, total_k=600,
             max_seqlen_q=30, max_seqlen_k=400, num_heads_q=8, num_heads_kv=2, head_dim=128, r_dim=16, rel_extent=64,
             window=100, alpha=0.1, log_scale_base=0.0, out=8 * A, lse=9 * A, workspace=None, workspace_bytes=0)
    d.update(kw)
    return rpb.RelattnParams(**d)


def pages(**kw):
    d = dict(block_table=30 * A, max_pages_per_seq=9, page_size=48, num_pages=20)
    d.update(kw)
    return rpb.RelattnPagedKV(**d)


@pytest.mark.parametrize("kw,want", [
    (dict(head_dim=64), UNSUPPORTED), (dict(num_heads_kv=3), INVALID), (dict(r_dim=65), UNSUPPORTED),
    (dict(alpha=float("inf")), INVALID), (dict(log_scale_base=1.0), INVALID), (dict(q=None), INVALID), (dict(v=None), INVALID),
    (dict(out=None), INVALID), (dict(lse=None), INVALID), (dict(k=A + 8), INVALID), (dict(P=None), INVALID),
    (dict(batch=-1), INVALID), (dict(batch=65536), UNSUPPORTED), (dict(max_seqlen_k=29), INVALID),
    (dict(num_heads_q=65536, num_heads_kv=65536), UNSUPPORTED),
    (dict(max_seqlen_k=(1 << 31) - (1 << 16) + 1), UNSUPPORTED),
    # out over q (the call reads it on), or over a part of k, v or r
    (dict(out=A), INVALID), (dict(out=A + 40 * 8 * 256 - 16), INVALID), (dict(k=8 * A - 600 * 2 * 256 + 256), INVALID),
    (dict(v=8 * A + 512), INVALID), (dict(r=8 * A - 16), INVALID),
])
def test_extend_refuses_parameters(kw, want):
    assert rpb.relattn_extend(fwd(**kw)) == want
    assert rpb.relattn_extend_workspace_size(fwd(**kw))[0] == want


@pytest.mark.parametrize("kw,want", [
    (dict(page_size=0), INVALID), (dict(page_size=-16), INVALID), (dict(page_size=24), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED),
    (dict(num_pages=0), INVALID), (dict(block_table=None), INVALID), (dict(block_table=A + 2), INVALID),
    (dict(max_pages_per_seq=8), INVALID), (dict(max_pages_per_seq=0), INVALID), (dict(num_pages=1 << 26), UNSUPPORTED),
])
def test_extend_refuses_pages(kw, want):
    assert rpb.relattn_extend(fwd(), pages(**kw), 4) == want
    assert rpb.relattn_extend_workspace_size(fwd(), pages(**kw), 4)[0] == want


def test_extend_refuses_a_negative_sink():
    assert rpb.relattn_extend(fwd(), None, -1) == INVALID


def test_empty_calls_do_nothing():
    assert rpb.relattn_extend(fwd(batch=0, total_q=0), None, 4) == 0
    assert rpb.relattn_extend(fwd(total_q=0), pages(), 4) == 0
    assert rpb.relattn_extend_workspace_size(fwd(total_q=0), pages(), 4) == (0, 0)


def bwd(f=None, **kw):
    d = dict(dout=40 * A, dq=41 * A, dk=42 * A, dv=43 * A, dr=44 * A, workspace=50 * A, workspace_bytes=1 << 40)
    d.update(kw)
    return rpb.RelattnBwdParams(fwd=f or fwd(), **d)


def test_backward_refuses():
    assert rpb.relattn_backward_sinks(bwd(), -1) == INVALID
    assert rpb.relattn_backward_sinks(bwd(), 1025) == UNSUPPORTED
    assert rpb.relattn_backward_sinks(bwd(dq=None), 4) == INVALID
    assert rpb.relattn_backward_sinks(bwd(fwd(r_dim=12)), 4) == UNSUPPORTED
    assert rpb.relattn_backward_sinks(bwd(workspace=None), 4) == WORKSPACE
    need = rpb.relattn_backward_sinks_workspace_size(bwd(), 4)
    assert need[0] == 0
    assert rpb.relattn_backward_sinks(bwd(workspace_bytes=need[1] - 1), 4) == WORKSPACE
    assert rpb.relattn_backward_sinks_workspace_size(bwd(), 1025)[0] == UNSUPPORTED


def test_backward_workspace():
    plain = rpb.relattn_backward_workspace_size(bwd())[1]
    assert rpb.relattn_backward_sinks_workspace_size(bwd(), 0) == (0, plain)
    assert rpb.relattn_backward_sinks_workspace_size(bwd(fwd(window=0)), 4)[1] == rpb.relattn_backward_workspace_size(bwd(fwd(window=0)))[1]
    # dq 40 x 8 x 128 fp32; dk, dv 2 x 2 x 4 x 2 x 128; partials: 2 heads x (40 x 4 / 128 + 2) slots (128 rows each) of 2 x 16 x 128
    plain = (plain + 255) // 256 * 256
    want = plain + 40 * 8 * 512 + 2 * 2 * 4 * 1024 + 2 * 3 * 2 * 16 * 512
    assert rpb.relattn_backward_sinks_workspace_size(bwd(), 4) == (0, want)
    # the bias reaches past the window: dr 40 x 8 x 16 fp32 as well
    assert rpb.relattn_backward_sinks_workspace_size(bwd(fwd(window=63)), 4) == (0, want + 40 * 8 * 64)


def prologue(**kw):
    names = ("q", "k", "v", "conv_k", "conv_v", "norm_q", "norm_k", "cu_seqlens_q", "cu_seqlens_k", "q_out", "k_cache", "v_cache")
    d = {n: (i + 1) * A for i, n in enumerate(names)}
    d.update(eps=1e-6, batch=1, total_q=8, total_k=0, num_heads_q=4, num_heads_kv=2, head_dim=128)
    d.update(kw)
    return rpb.RelattnPrologueParams(**d)


@pytest.mark.parametrize("kw,pkw,want", [
    (dict(head_dim=64), {}, UNSUPPORTED), (dict(q=None), {}, INVALID), (dict(k_cache=None), {}, INVALID),
    (dict(v_cache=12 * A + 8), {}, INVALID), (dict(eps=0.0), {}, INVALID),
    (dict(k_cache=2 * A - 20 * 48 * 512 + 512), {}, INVALID),      # the pool's last row overlaps k
    ({}, dict(page_size=20), UNSUPPORTED), ({}, dict(page_size=0), INVALID), ({}, dict(num_pages=0), INVALID),
    ({}, dict(block_table=None), INVALID), ({}, dict(max_pages_per_seq=0), INVALID),
])
def test_prologue_refuses(kw, pkw, want):
    assert rpb.relattn_prologue_paged(prologue(**kw), pages(**pkw)) == want


def test_prologue_of_no_sequence_does_nothing():
    assert rpb.relattn_prologue_paged(prologue(batch=0, q=None), pages()) == 0


def test_python_refuses_before_the_library():
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    cu = torch.tensor([0, 2], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA device"):
        rpb.extend(q, q[:, :2].contiguous(), q[:, :2].contiguous(), None, None, cu, cu, max_seqlen_q=2, max_seqlen_k=2, alpha=0.1)
    with pytest.raises(ValueError, match="32 bits"):
        rpb.backward(q, q, q, None, None, q, q, q, cu, cu, max_seqlen_q=2, max_seqlen_k=2, alpha=0.1, sink=1 << 33)
