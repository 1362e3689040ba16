"""Paged caches on the GPU: calls that the documentation allows and that lie
off the usual path, against float64 or Python integers."""
import pytest
import torch

from sparse_compressed_kv_gb300 import csa
from tests import paged_helpers as H

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("heads", [1, 7, 9, 31, 33, 63, 65, 97, 127])
def test_attention_head_counts_inside_a_group(cuda_device, heads, dtype):
    # the last group of eight heads is partly stored, and several tokens follow one
    # another in a CTA: lanes that store and lanes that do not go on to the next
    # token's loads together
    T = 330
    p = H.Paged(heads, row_len=[150, 97, 40], tokens=[(t % 3, 160 + 370 * (t % 3 == 0) + t % 7) for t in range(T)],
                heads=heads, page_rows=24, window=20, swa_cap=40)
    got, status = p.run(cuda_device, dtype)
    assert status == 0
    tokens = list(range(0, T, 29)) + [T - 1]
    H.check(got, p.reference(tokens=tokens), dtype, tokens)
    again, _ = p.run(cuda_device, dtype)
    assert torch.equal(got, again)
