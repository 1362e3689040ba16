"""The paged caches on the CPU: which tensors the binding takes, what it makes of
their strides, and which arrays the C entry points refuse to share memory."""
import ctypes

import pytest
import torch

from sparse_compressed_kv_gb300 import build as B
from sparse_compressed_kv_gb300 import csa

INVALID = 1
PTR = 4096


@pytest.fixture(scope="module")
def lib():
    B.build()
    return csa.load()


def test_page_stride_of_a_pool_and_its_parts():
    pool = torch.zeros(5, 12, 4, 2)
    assert csa._page_stride(pool, 12) == 12 and csa._page_stride(pool, 3) == 12
    for first in (0, 4, 8):         # a layer's part of interleaved pages
        assert csa._page_stride(pool[:, first:first + 4], 4) == 12
    assert csa._page_stride(pool[:, 3:4], 1) == 12
    assert csa._page_stride(pool[2:3, 3:7], 4) == 4         # one page: no next one
    assert csa._page_stride(pool[::2, :6], 6) == 24         # every other page
    # a page of one row, whose own stride says nothing
    assert csa._page_stride(pool.view(5, 12, 8)[:, ::12], 1) == 12


@pytest.mark.parametrize("make,page_rows", [
    (lambda p: p[:, :4], 5),                                 # fewer rows than a page
    (lambda p: p[:, ::2], 6),                                # rows of a page apart
    (lambda p: p[..., :4], 12),                              # rows that are parts of rows
    (lambda p: p.transpose(0, 1), 5),
    (lambda p: p[:1, :4].expand(5, 4, 8), 4),                # every page the same
    (lambda p: p.as_strided((5, 4, 8), (30, 8, 1)), 4),      # pages that overlap
    (lambda p: p.as_strided((5, 4, 8), (36, 8, 1)), 4),      # no whole number of rows apart
])
def test_page_stride_refusals(make, page_rows):
    with pytest.raises(ValueError, match="page"):
        csa._page_stride(make(torch.zeros(5, 12, 8)), page_rows)


def test_append_job_takes_a_part_of_a_pool():
    pool = torch.zeros(5, 12, 8)
    i64 = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError, match="GPU"):             # (all that a CPU tensor lacks)
        csa.AppendJob(torch.zeros(2, 8), i64, pool[:, 4:8], 4)
    with pytest.raises(ValueError, match="page"):
        csa.AppendJob(torch.zeros(2, 8), i64, pool[:, 4:8], 5)
    with pytest.raises(ValueError, match="page"):
        csa.AppendJob(torch.zeros(2, 8), i64, pool[:, ::2], 4)


def _plan_at(lib, **at):
    """A small plan whose arrays lie apart, but for those named in `at`."""
    sizes = dict(seq_len=32, new_len=16, table=128, free_ring=128, free_pos=16, seq_len_out=32, row_len=32,
                 swa_first_pos=32, free_pos_out=16, tok_off=40, row_off=40, tok_seq=32, tok_pos=64, swa_slot=64,
                 row_slot=32, status=4)
    ptr = {n: PTR + 256 * i for i, n in enumerate(sizes)}
    ptr.update({n: ptr[o] + d for n, (o, d) in at.items()})
    status = ptr.pop("status")
    p = csa.csa_page_plan_t(num_seqs=4, ratio=4, page_rows=16, max_pages=8, num_pages=32, tok_cap=8, row_cap=4,
                            swa_cap=128, **ptr)
    return lib.csa_page_plan(ctypes.byref(p), status, None)


WRITTEN = ("table", "free_ring", "seq_len_out", "row_len", "swa_first_pos", "free_pos_out", "tok_off", "row_off",
           "tok_seq", "tok_pos", "swa_slot", "row_slot", "status")


@pytest.mark.parametrize("name", WRITTEN)
def test_plan_refuses_outputs_over_other_arrays(lib, name):
    # every CTA reads the inputs while others write the outputs: the same array, or
    # one that begins inside another
    for other in ("seq_len", "new_len", "free_pos") + tuple(n for n in WRITTEN if n != name):
        assert _plan_at(lib, **{name: (other, 0)}) == INVALID, other
        assert _plan_at(lib, **{name: (other, 8 if other != "status" else 0)}) == INVALID, other


def test_plan_takes_arrays_that_only_touch(lib):
    # (CSA_ERR_CUDA or _UNSUPPORTED: the checks are through, and this machine has no GPU)
    if torch.cuda.is_available():
        pytest.skip("the pointers are not real")
    assert _plan_at(lib) not in (0, INVALID)
    assert _plan_at(lib, row_len=("seq_len_out", 32), tok_pos=("tok_seq", 32)) not in (0, INVALID)
    # the inputs may share memory with each other
    assert _plan_at(lib, new_len=("seq_len", 0)) not in (0, INVALID)


ATTENTION = dict(out=2 * 3 * 16 * 512, ws=0, status=4, q=2 * 3 * 16 * 512, sinks=64, tok_seq=12, tok_pos=24,
                 row_len=16, table=64, swa_kv=2 * 128 * 1024, swa_first_pos=16)


def _attend_at(lib, window=128, **at):
    """A small bf16 attention whose arrays lie apart, but for those named in `at`."""
    P = csa.params(16, 1, window)
    size = ctypes.c_size_t(0)
    L = csa.csa_paged_layout_t(num_seqs=2, num_tokens=3, page_rows=16, max_pages=8, swa_cap=128)
    assert lib.csa_paged_workspace_size(ctypes.byref(L), ctypes.byref(P), ctypes.byref(size)) == 0
    ptr, end = {}, 4096
    for n, bytes_ in dict(ATTENTION, ws=size.value).items():
        ptr[n] = end
        end += -(-bytes_ // 256) * 256 + 256
    ptr.update({n: ptr[o] + d for n, (o, d) in at.items()})
    for n in ("tok_seq", "tok_pos", "row_len", "table", "swa_kv", "swa_first_pos"):
        setattr(L, n, ptr[n])
    return lib.csa_paged_attention(ctypes.byref(L), ctypes.byref(P), end, 16, 16, ptr["q"], ptr["sinks"], 1,
                                   ptr["out"], ptr["status"], ptr["ws"], size.value, None)


@pytest.mark.parametrize("name", ["out", "ws", "status"])
def test_attention_refuses_outputs_over_other_arrays(lib, name):
    for other in ATTENTION:
        if other == name:
            continue
        assert _attend_at(lib, **{name: (other, 0)}) == INVALID, other
        if ATTENTION[other] > 256:      # one that begins inside another
            assert _attend_at(lib, **{name: (other, 256)}) == INVALID, other


def test_attention_takes_arrays_that_only_touch(lib):
    if torch.cuda.is_available():
        pytest.skip("the pointers are not real")
    assert _attend_at(lib) not in (0, INVALID)
    assert _attend_at(lib, sinks=("out", ATTENTION["out"])) not in (0, INVALID)
    # without a window the ring is not used, wherever it is said to be
    assert _attend_at(lib, window=0, swa_kv=("out", 0)) not in (0, INVALID)


def test_binding_refuses_a_ring_without_its_first_positions():
    i32, i64 = torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int64)
    with pytest.raises(ValueError, match="swa_first_pos"):
        csa.PagedLayout(i32, i64, i64, torch.zeros(1, 1, dtype=torch.int32), 16,
                        swa_kv=torch.zeros(1, 128, 512, dtype=torch.bfloat16))


class _Job:
    def __init__(self, device):
        self.device, self.c = device, csa.csa_append_job_t()


def test_binding_refuses_jobs_that_are_not_one_call():
    assert csa.AppendJobs(iter([_Job(0), _Job(0)])).device == 0
    for jobs in ([], [_Job(0)] * 5, [_Job(0), _Job(1)]):
        with pytest.raises(ValueError, match="job"):
            csa.AppendJobs(jobs)


def test_binding_refuses_a_stream_of_another_device(monkeypatch):
    class Stream:
        def __init__(self, index):
            self.device_index, self.cuda_stream = index, 77
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    assert csa._device_stream("f", 0, Stream(0)) == 77
    with pytest.raises(ValueError, match="stream"):
        csa._device_stream("f", 0, Stream(1))
    with pytest.raises(ValueError, match="current device"):
        csa._device_stream("f", 1, Stream(1))


def test_binding_takes_any_object_with_a_stream(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    assert csa._device_stream("f", 0, type("Wrapped", (), dict(cuda_stream=99))()) == 99
