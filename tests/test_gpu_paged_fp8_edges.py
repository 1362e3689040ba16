"""8-bit paged caches on the GPU, at the ends of what the calls allow."""
import pytest
import torch

from sparse_compressed_kv_gb300 import csa
from tests import fp8_helpers as F
from tests import paged_helpers as H

pytestmark = pytest.mark.gpu

F32, BF16, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
BOTH = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])


def status_word(device):
    return torch.zeros(1, dtype=torch.int32, device=device)


# ---------------------------------------------------------------- the longest token

@BOTH
def test_attention_of_as_many_rows_as_a_call_allows(cuda_device, dtype):
    # table and window hold 2^31 - 65 rows, the limit, and the slots' padding takes them
    # past 2^31 - 64: one page over and over, every weight the same, so that the sums of
    # the ones in the pages and the zeros in the window are exact
    dev, P, M = cuda_device, 65535, 32767
    n = M * P
    window = (1 << 31) - 65 - n
    assert n % 8 == 1 and 0 < window < 1 << 17
    codes = torch.full((1, P, H.HD), 0x38, dtype=torch.uint8, device=dev)          # 1.0
    ring = torch.zeros(1, window, H.HD, dtype=torch.uint8, device=dev)
    pos = n + 5
    layout = csa.PagedLayoutFp8(torch.zeros(1, dtype=torch.int32, device=dev), torch.tensor([pos], device=dev),
                                torch.tensor([n], device=dev), torch.zeros(1, M, dtype=torch.int32, device=dev), P,
                                ring.view(F8), torch.ones(1, window, device=dev),
                                torch.tensor([pos - window + 1], device=dev))
    prm = csa.params(16, 1, window, 1)
    q = torch.zeros(1, 16, H.HD, dtype=BF16, device=dev)
    out, status = torch.full((1, 16, H.HD), 7.0, dtype=dtype, device=dev), status_word(dev)
    csa.csa_paged_attention_fp8(layout, prm, codes.view(F8), torch.ones(1, P, device=dev), q, out, status,
                                csa.paged_workspace(layout, prm))
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    # a join of up to 152 parts and two divisions, half of 2^-23 each; a bf16 output 2^-9 besides
    want = n / (n + window)
    assert float((out.double() - want).abs().max()) <= 155 * 2 ** -24 + (2 ** -8 if dtype == BF16 else 0)
