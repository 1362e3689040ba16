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


# ---------------------------------------------------------------- small weights

@BOTH
@pytest.mark.parametrize("T,n", [(1, 60000), (4, 20000), (160, 3500), (160, 20000), (160, 60000), (153, 262144)], ids=str)
def test_attention_sums_of_small_weights(cuda_device, T, n, dtype):
    # one row whose weight is 2^12 to 2^22 times that of each of the others, which are all
    # equal, so that whatever rounds their weights rounds them alike
    dev, heads = cuda_device, 64
    g = torch.Generator(device=dev).manual_seed(n + T)
    randn = lambda *shape: torch.randn(*shape, device=dev, generator=g)
    common, peak = randn(H.HD), randn(H.HD)
    # the peak's logit over the others': 12 to 22 powers of two, from head to head
    over = (12 + 10 * torch.rand(T, heads, 1, device=dev, generator=g)) * 0.6931 * H.HD ** 0.5
    unit = torch.stack([peak, common])
    along = torch.linalg.solve(unit @ unit.T, unit)          # [2, 512]: . peak, . common = (1, 0), (0, 1)
    q = 0.3 * randn(T, heads, H.HD)
    q = q - q @ unit.T @ along + over * along[0]             # over to the peak, 0 to the others
    rows = common.repeat(n, 1)
    rows[n // 3] = peak
    cache, scales = torch.zeros(n // 4, 4, H.HD, device=dev).to(F8), torch.zeros(n // 4, 4, device=dev)
    status = status_word(dev)
    csa.csa_paged_append_fp8(csa.AppendJobsFp8([csa.AppendJobFp8(rows, torch.arange(n, device=dev), cache, scales, 4)]),
                             status)
    layout = csa.PagedLayoutFp8(torch.zeros(T, dtype=torch.int32, device=dev),
                                torch.full((T,), 4 * n, dtype=torch.int64, device=dev), torch.tensor([n], device=dev),
                                torch.arange(n // 4, device=dev).int()[None], 4)
    prm = csa.params(heads, 1, 0, 4)
    q = q.to(BF16)
    out = torch.empty(T, heads, H.HD, device=dev, dtype=dtype)
    csa.csa_paged_attention_fp8(layout, prm, cache, scales, q, out, status, csa.paged_workspace(layout, prm))
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    two = F.values(*F.quantise(torch.stack([peak, common]).double().cpu().numpy())).to(dev)
    for t in range(0, T, max(1, T // 4)):
        l = prm.scale * q[t].double() @ two.T
        w = torch.exp(l - l.amax(1, keepdim=True)) * torch.tensor([1.0, n - 1.0], device=dev)
        w = w / w.sum(1, keepdim=True)
        assert float((l[:, 0] - l[:, 1]).min()) > 6
        ref = w @ two
        # A weight's rounding is handed on within its sequence of rows, 16 a head and part
        # of the token, each of which loses half of 2^-16 at the end where the largest is 2^7; and
        # a weight is a multiple of 2^-24, rounded.  (Handing nothing on: n 2^-24.)
        parts = 3 if T > 152 else 152 // T + 2
        floor = (16 * parts * 2 ** -24 + n * 2 ** -32) * float(w[:, 0].max())
        # equal weights round alike above that, too: by 2^-9 and 2^-11 for a bf16 output
        tol = F.REL[dtype] + floor + (2 ** -9 + 2 ** -11 if dtype == BF16 else 2 ** -18)
        err = (out[t].double() - ref).norm(dim=1) / ref.norm(dim=1)
        assert float(err.max()) <= tol, f"token {t}: off by {float(err.max()):.3e}, not {tol:.3e}"
