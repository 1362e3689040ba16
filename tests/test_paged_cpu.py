"""Paged caches on the CPU: every argument error of the C entry points is
decided before anything is launched, and the binding refuses wrong tensors."""
import ctypes

import pytest
import torch

from sparse_compressed_kv_gb300 import build as B
from sparse_compressed_kv_gb300 import csa
from tests import paged_helpers as H

INVALID, UNSUPPORTED, CAPACITY, WORKSPACE = 1, 2, 3, 7
PTR = 4096


@pytest.fixture(scope="module")
def lib():
    B.build()
    return csa.load()


def plan(**changes):
    ptrs = {n: PTR + 256 * i for i, (n, t) in enumerate(csa.csa_page_plan_t._fields_)
            if t is ctypes.c_void_p}
    return csa.csa_page_plan_t(**{**dict(num_seqs=4, ratio=4, page_rows=16, max_pages=8,
                                         num_pages=32, tok_cap=8, row_cap=4, swa_cap=128), **ptrs,
                                  **changes})


@pytest.mark.parametrize("changes,code", [
    (dict(num_seqs=0), INVALID), (dict(ratio=0), INVALID), (dict(page_rows=0), INVALID),
    (dict(max_pages=0), INVALID), (dict(num_pages=0), INVALID), (dict(swa_cap=0), INVALID),
    (dict(tok_cap=-1), INVALID), (dict(row_cap=-1), INVALID),
    (dict(num_seqs=8193), UNSUPPORTED), (dict(num_pages=1 << 31), UNSUPPORTED),
    (dict(num_pages=1 << 28), UNSUPPORTED), (dict(tok_cap=1 << 31), UNSUPPORTED),
    (dict(row_cap=1 << 31), UNSUPPORTED),
    (dict(seq_len=None), INVALID), (dict(new_len=None), INVALID), (dict(table=None), INVALID),
    (dict(free_ring=None), INVALID), (dict(free_pos=None), INVALID), (dict(row_off=None), INVALID),
    (dict(tok_seq=None), INVALID), (dict(swa_slot=None), INVALID), (dict(row_slot=None), INVALID),
    (dict(tok_pos=PTR + 4), INVALID), (dict(tok_seq=PTR + 2), INVALID),
    (dict(seq_len=PTR, seq_len_out=PTR), INVALID), (dict(free_pos=PTR, free_pos_out=PTR), INVALID),
])
def test_plan_refusals(lib, changes, code):
    p = plan(**changes)
    assert lib.csa_page_plan(ctypes.byref(p), PTR, None) == code


def test_plan_null_arguments(lib):
    p = plan()
    assert lib.csa_page_plan(None, PTR, None) == INVALID
    assert lib.csa_page_plan(ctypes.byref(p), None, None) == INVALID


def job(**changes):
    return csa.csa_append_job_t(**{**dict(rows=PTR, slots=PTR, num_rows=3, row_pitch=1024,
                                          row_bytes=1024, page_rows=16, num_pages=4, page_stride=16,
                                          cache=PTR), **changes})


@pytest.mark.parametrize("changes,code", [
    (dict(num_rows=-1), INVALID), (dict(row_bytes=0), INVALID), (dict(row_bytes=24), INVALID),
    (dict(page_rows=0), INVALID), (dict(num_pages=0), INVALID), (dict(page_stride=15), INVALID),
    (dict(row_pitch=1008), INVALID), (dict(row_pitch=1032), INVALID), (dict(rows=None), INVALID),
    (dict(slots=None), INVALID), (dict(cache=None), INVALID), (dict(rows=PTR + 8), INVALID),
    (dict(cache=PTR + 8), INVALID), (dict(slots=PTR + 4), INVALID),
    (dict(num_pages=1 << 31), UNSUPPORTED), (dict(num_pages=1 << 28), UNSUPPORTED),
    (dict(row_bytes=65552, row_pitch=65552), UNSUPPORTED), (dict(num_rows=1 << 31), UNSUPPORTED),
    (dict(page_stride=1 << 31), UNSUPPORTED),
])
def test_append_refusals(lib, changes, code):
    jobs = (csa.csa_append_job_t * 2)(job(), job(**changes))
    assert lib.csa_paged_append(jobs, 2, PTR, None) == code


def test_append_counts(lib):
    jobs = (csa.csa_append_job_t * 5)(*[job() for _ in range(5)])
    assert lib.csa_paged_append(jobs, 0, PTR, None) == INVALID
    assert lib.csa_paged_append(jobs, 5, PTR, None) == UNSUPPORTED
    assert lib.csa_paged_append(None, 1, PTR, None) == INVALID
    assert lib.csa_paged_append(jobs, 1, None, None) == INVALID
    # nothing to copy: nothing launched, whatever the pointers
    empty = (csa.csa_append_job_t * 1)(job(num_rows=0, rows=None, slots=None, cache=None))
    assert lib.csa_paged_append(empty, 1, PTR, None) == 0


def layout(**changes):
    return csa.csa_paged_layout_t(**{**dict(num_seqs=2, num_tokens=3, page_rows=16, max_pages=8,
                                            tok_seq=PTR, tok_pos=PTR, row_len=PTR, table=PTR,
                                            swa_kv=PTR, swa_cap=128, swa_first_pos=PTR), **changes})


def attend(lib, L, P, *, cache=PTR, num_pages=16, page_stride=16, q=PTR, sinks=None, out_type=0,
           out=PTR, status=PTR, ws=PTR, ws_bytes=1 << 40):
    return lib.csa_paged_attention(ctypes.byref(L), ctypes.byref(P), cache, num_pages, page_stride, q,
                                   sinks, out_type, out, status, ws, ws_bytes, None)


@pytest.mark.parametrize("changes,code", [
    (dict(num_seqs=0), INVALID), (dict(num_tokens=-1), INVALID), (dict(page_rows=0), INVALID),
    (dict(max_pages=0), INVALID), (dict(num_tokens=8193), UNSUPPORTED),
    (dict(max_pages=1 << 27), UNSUPPORTED), (dict(tok_seq=None), INVALID),
    (dict(tok_pos=None), INVALID), (dict(row_len=None), INVALID), (dict(table=None), INVALID),
    (dict(swa_kv=None), INVALID), (dict(swa_first_pos=None), INVALID), (dict(swa_cap=127), CAPACITY),
    (dict(num_seqs=1 << 24), UNSUPPORTED), (dict(swa_kv=PTR + 8), INVALID),
    (dict(tok_pos=PTR + 4), INVALID),
])
def test_attention_layout_refusals(lib, changes, code):
    assert attend(lib, layout(**changes), csa.params(16, 1)) == code


@pytest.mark.parametrize("changes,code", [
    (dict(hd=256), UNSUPPORTED), (dict(n_heads=0), INVALID), (dict(n_heads=129), UNSUPPORTED),
    (dict(window=-1), INVALID), (dict(ratio=0), INVALID), (dict(scale=float("nan")), INVALID),
])
def test_attention_param_refusals(lib, changes, code):
    P = csa.params(16, 1)
    for k, v in changes.items():
        setattr(P, k, v)
    assert attend(lib, layout(), P) == code
    n = ctypes.c_size_t(0)
    assert lib.csa_paged_workspace_size(ctypes.byref(layout()), ctypes.byref(P), ctypes.byref(n)) == code


@pytest.mark.parametrize("changes,code", [
    (dict(cache=None), INVALID), (dict(q=None), INVALID), (dict(out=None), INVALID),
    (dict(status=None), INVALID), (dict(cache=PTR + 8), INVALID), (dict(q=PTR + 8), INVALID),
    (dict(out=PTR + 4), INVALID), (dict(num_pages=0), INVALID), (dict(page_stride=15), INVALID),
    (dict(num_pages=1 << 31), UNSUPPORTED), (dict(num_pages=1 << 27), UNSUPPORTED),
    (dict(out_type=2), INVALID), (dict(ws=None), WORKSPACE), (dict(ws_bytes=16), WORKSPACE),
    (dict(ws=PTR + 16), INVALID), (dict(sinks=PTR + 2), INVALID),
])
def test_attention_buffer_refusals(lib, changes, code):
    assert attend(lib, layout(), csa.params(16, 1), **changes) == code


def test_attention_without_tokens_or_window(lib):
    # no tokens: nothing launched; no window: the ring may be missing
    assert attend(lib, layout(num_tokens=0, tok_seq=None), csa.params(16, 1), q=None) == 0
    P = csa.params(16, 1, window=0)
    n = ctypes.c_size_t(0)
    L = layout(swa_kv=None, swa_first_pos=None, swa_cap=0)
    assert lib.csa_paged_workspace_size(ctypes.byref(L), ctypes.byref(P), ctypes.byref(n)) == 0
    assert attend(lib, L, P, q=None) == INVALID     # decided after the ring, by q


def test_binding_refuses_host_tensors_and_wrong_types():
    i64 = torch.zeros(1, dtype=torch.int64)
    with pytest.raises(ValueError, match="tok_seq"):
        csa.PagedLayout(i64, i64, i64, torch.zeros(1, 1, dtype=torch.int32), 16)
    with pytest.raises(ValueError, match="shape"):
        csa.PagedLayout(i64.int(), i64, i64, torch.zeros(2, 1, dtype=torch.int32), 16)
    with pytest.raises(ValueError, match="cache"):
        csa.AppendJob(torch.zeros(2, 8), i64, torch.zeros(1, 4, 9), 4)
    with pytest.raises(ValueError, match="GPU"):
        csa.AppendJob(torch.zeros(1, 8), i64, torch.zeros(1, 4, 8), 4)
    t = H.plan_tensors("cpu", seq_len=[0], new_len=[1], table=[[0]], free_ring=[0], free_pos=[0, 1],
                       tok_cap=1, row_cap=1)
    with pytest.raises(ValueError, match="GPU"):
        csa.PagePlan(ratio=4, page_rows=16, swa_cap=128, **t)
    with pytest.raises(ValueError, match="table"):
        csa.PagePlan(ratio=4, page_rows=16, swa_cap=128, **dict(t, table=t["table"][0]))


def test_plan_reference_by_hand():
    # ratio 4, pages of 2 blocks.  Request 0 holds 7 tokens (1 block, page 5)
    # and brings 10: blocks 1..3, one more page (from the ring: 9).  Request 1
    # is over and gives back pages 3 and 8 (9 tokens' worth: 2 blocks = 1
    # page, so only page 3).  Request 2 brings its first 3 tokens: no block.
    got, bad = H.plan_reference(
        ratio=4, page_rows=2, swa_cap=4, seq_len=[7, 9, 0], new_len=[10, -1, 3],
        table=[[5, -5], [3, 8], [-5, -5]], free_ring=[9, 4] + [-7] * 8, free_pos=[0, 2],
        tok_cap=14, row_cap=3)
    assert bad == 0
    assert got["table"] == [[5, 9], [3, 8], [-5, -5]]
    assert got["free_ring"][:3] == [9, 4, 3] and got["free_pos_out"] == [1, 3]
    assert got["row_slot"] == [11, 18, 19] and got["row_off"] == [0, 3, 3, 3]
    assert got["tok_seq"] == [0] * 10 + [2] * 3 + [-1] and got["tok_off"] == [0, 10, 10, 13]
    assert got["tok_pos"] == list(range(7, 17)) + [0, 1, 2, -1]
    assert got["swa_slot"] == [-1] * 6 + [1, 2, 3, 0] + [8, 9, 10, -1]
    assert got["seq_len_out"] == [17, 0, 3] and got["row_len"] == [4, 0, 0]
    assert got["swa_first_pos"] == [13, 0, 0]


def test_attention_reference_by_hand():
    # one row and no window: its softmax weight is 1
    p = H.Paged(1, row_len=[1], tokens=[(0, 4)], window=0, heads=2)
    assert torch.equal(p.reference()[0, 0], p.rows_of(0)[0])
    # a sink as large as the one logit halves the output
    p.sinks = (p.scale * p.q[0].double() @ p.rows_of(0)[0]).float()
    assert torch.allclose(p.reference()[0], 0.5 * p.rows_of(0).expand(2, -1), rtol=1e-6)
