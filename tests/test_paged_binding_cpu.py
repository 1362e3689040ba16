"""The paged caches' binding on the CPU: which tensors it takes, and what it
makes of their strides."""
import pytest
import torch

from sparse_compressed_kv_gb300 import csa


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
