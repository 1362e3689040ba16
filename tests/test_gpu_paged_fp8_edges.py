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
@pytest.mark.parametrize("T,n", [(1, 60000), (4, 20000), (160, 3500), (160, 20000), (160, 60000),
                                 (153, 262144)], ids=str)
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


# ---------------------------------------------------------------- as exact as an f32 output is said to be

# Relative 2-norm errors of a token's output of 64 heads, for the random rows of PagedFp8
# (emulated: weights in six terms 1.0e-6 at most, the query in two 1.5e-6):
#   logits: 16 instructions into a truncating accumulator, half a last place (0.36 2^-23 on
#     average over a binade) of a running sum of two thirds of the final one: 4.6e-7 of
#     a logit of 2 (root mean square, in powers of two): 1.0e-6;
#   output: 12 instructions a chunk of 64 rows, likewise: 3.5e-7 a chunk.
# With the sixth term left out it would be 1.4e-5, with five rounded ones 7e-6 (64 heads).
def f32_bound(chunks):
    return 1.0e-6 + 1.5e-6 + 1.0e-6 + 3.5e-7 * chunks


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("rows,window,chunks", [(64, 0, 1), (150, 40, 3), (256, 128, 6)], ids=str)
def test_attention_f32_keeps_all_terms(cuda_device, rows, window, chunks, seed):
    p = F.PagedFp8(100 + seed, row_len=[rows] * 5, tokens=[(b, 4 * rows) for b in range(5)], heads=64, window=window,
                   page_rows=[16, 64, 3, 8][seed], sinks=seed % 2 == 1)
    got, status = p.run(cuda_device, F32)
    assert status == 0
    F.check(got, p.reference(), F32, rel=f32_bound(chunks))


def test_attention_f32_of_peaked_logits(cuda_device):
    # logits of several hundred: a weight's relative error is its logit's absolute one.
    # The accumulators': 4.6e-7 of the logit alike for rows whose logits are alike, and
    # 4 x 0.14 2^-23 x 700 at random, 5e-5; the query's small values: two of 512 off by 0.6
    # of 2^-17 of 14 at random, times rows of 17 and the scale: 7e-5; together 9e-5 (root mean
    # square), times weight and what it is taken from, at most half the output: six times that.
    # (A bf16 output's weights alone are off by up to 2^-9 + 2^-11, 2.4e-3.)
    p = F.PagedFp8(5, row_len=[640], tokens=[(0, 2560)], heads=64, page_rows=64, window=0, spread=0)
    j = torch.arange(640)
    at = (p.table[0, j // 64].long(), j % 64)
    codes, k = F.quantise((p.cache[at] * (1 + j[:, None] / 40)).numpy())
    p.codes[at], p.scales[at] = torch.from_numpy(codes), torch.from_numpy(k).float()
    p.requantised()
    p.q *= 4
    ref = p.reference()
    got, status = p.run(cuda_device, F32)
    assert status == 0
    err = (got.double().cpu() - ref).norm(dim=2) / ref.norm(dim=2)
    assert float(err.max()) <= 6 * 9e-5


# ---------------------------------------------------------------- long sums of a bf16 output

def test_attention_bf16_sums_in_several_stretches(cuda_device):
    # 45,000 rows in one CTA are three stretches between which the sums go to the
    # partial and back; the second stretch's rows raise the maximum by more than 2^8, and the
    # first one's still weigh a tenth
    dev, n, T = cuda_device, 45056, 320
    g = torch.Generator(device=dev).manual_seed(31)
    rows = torch.randn(n, H.HD, device=dev, generator=g)
    rows *= torch.tensor([1.0, 2.4, 1.5], device=dev)[torch.arange(n, device=dev) * 3 // n][:, None]
    cache, scales = torch.zeros(n // 32, 32, H.HD, device=dev).to(F8), torch.zeros(n // 32, 32, device=dev)
    table = torch.randperm(n // 32, device=dev, generator=g).int()[None]
    j = torch.arange(n, device=dev)
    status = status_word(dev)
    csa.csa_paged_append_fp8(csa.AppendJobsFp8([csa.AppendJobFp8(rows, table[0, j // 32].long() * 32 + j % 32, cache,
                                                                 scales, 32)]), status)
    q = torch.randn(T, 64, H.HD, device=dev, generator=g).to(BF16)
    pos = 4 * (n - torch.arange(T, device=dev) * 7)
    layout = csa.PagedLayoutFp8(torch.zeros(T, dtype=torch.int32, device=dev), pos, torch.tensor([n], device=dev),
                                table, 32)
    prm = csa.params(64, 1, 0, 4)
    out = torch.empty(T, 64, H.HD, device=dev, dtype=BF16)
    csa.csa_paged_attention_fp8(layout, prm, cache, scales, q, out, status, csa.paged_workspace(layout, prm))
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    vals = F.values(*F.quantise(rows.double().cpu().numpy())).to(dev)
    for t in range(0, T, 53):
        v = vals[:int(pos[t]) // 4]
        w = torch.softmax(prm.scale * q[t].double() @ v.T, 1)
        assert 0.01 < float(w[:, :n // 3].sum(1).mean()) < 0.5
        ref = w @ v
        assert (out[t].double() - ref).norm() <= F.REL[BF16] * ref.norm()


# ---------------------------------------------------------------- sizes and orders

def test_append_and_read_rows_past_32_bit_offsets(cuda_device):
    # 4.3 GiB of rows in, and of rows out; the cache's codes pass 2^31 bytes
    dev, n, P = cuda_device, (1 << 22) + 77, 64
    g = torch.Generator(device=dev).manual_seed(41)
    rows = torch.empty(n, 512, dtype=BF16, device=dev)
    for a in range(0, n, 1 << 20):
        rows[a:a + (1 << 20)] = torch.randn(min(1 << 20, n - a), 512, device=dev, generator=g)
    pages = -(-n // P)
    slots = torch.arange(n, device=dev).flip(0)
    cache, scales = torch.zeros(pages, P, 512, dtype=torch.uint8, device=dev), torch.zeros(pages, P, device=dev)
    out, status = torch.zeros(n, 512, dtype=BF16, device=dev), status_word(dev)
    csa.csa_paged_append_fp8(csa.AppendJobsFp8([csa.AppendJobFp8(rows, slots, cache.view(F8), scales, P)]), status)
    csa.csa_paged_read_fp8(cache.view(F8), scales, slots, out, status, P)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for a in range(0, n, 1 << 18):
        x, y = rows[a:a + (1 << 18)].float(), out[a:a + (1 << 18)].float()
        assert bool(((x - y).abs() <= torch.maximum(x.abs() * 2 ** -4, x.abs().amax(1, keepdim=True) * 2 ** -17)).all())
    at = torch.tensor([0, 1, n // 2, n - 2, n - 1], device=dev)
    assert torch.equal(out[at].double().cpu(), F.values(*F.quantise(rows[at].double().cpu().numpy())))


@BOTH
def test_attention_of_tokens_in_any_order(cuda_device, dtype):
    # sequences and positions out of order, padding between, a position twice (with two queries)
    tokens = [(2, 900), (0, 40), (-1, -1), (1, 1300), (2, 901), (0, 400), (1, 1300), (2, 10), (-1, -1), (0, 399)]
    p = F.PagedFp8(71, row_len=[100, 325, 225], tokens=tokens, heads=24, sinks=True, swa_cap=1500)
    got, status = p.run(cuda_device, dtype)
    assert status == 0
    F.check(got, p.reference(), dtype, [t for t, (b, _) in enumerate(tokens) if b >= 0])
    assert bool((got[[2, 8]] == 7).all())


@BOTH
@pytest.mark.parametrize("row_len,pos,window", [([0], 9000, 7000), ([37], 5151, 5000), ([2500], 10003, 3001)],
                         ids=str)
def test_attention_of_wide_windows(cuda_device, row_len, pos, window, dtype):
    p = F.PagedFp8(72, row_len=row_len, tokens=[(0, pos), (0, pos - 2)], heads=40, window=window, swa_cap=window + 9,
                   page_rows=5)
    got, status = p.run(cuda_device, dtype)
    assert status == 0
    F.check(got, p.reference(), dtype)


def test_attention_of_the_most_tokens_and_heads(cuda_device):
    tokens = [(t % 3, 200 + t % 57) for t in range(8192)]
    p = F.PagedFp8(73, row_len=[64, 50, 3], tokens=tokens, heads=128, window=30, swa_cap=100)
    some = list(range(0, 8192, 431)) + [8191]
    got, status = p.run(cuda_device, F32)
    assert status == 0
    F.check(got, p.reference(tokens=some), F32, some)


@BOTH
def test_attention_of_one_page_of_many_rows(cuda_device, dtype):
    p = F.PagedFp8(74, row_len=[70001, 3], tokens=[(0, 4 * 69000 + 2), (1, 14)], heads=16, page_rows=1 << 17, window=0,
                   spare_pages=0)
    got, status = p.run(cuda_device, dtype)
    assert status == 0
    F.check(got, p.reference(), dtype)


def test_attention_rows_without_weight_add_nothing(cuda_device):
    # 64 rows that hold all the weight, then 131,008 whose weights are below 2^-50 of theirs:
    # what the last of the first rounds away must not go on through the others.  A weight
    # of the 64 is off at random by 2.9e-6 (logits of 63 powers of two in 16 truncated steps,
    # 4 x 0.14 2^-23 of them), 1.0e-6 (six terms) and 4e-6 (the query's small values, two of
    # 512 off by 0.6 of 2^-17 of 14); times a row's part that is not in all of them, 22.6, and
    # the weights' 2-norm, at most 0.25, over an output of 11.3: half of each
    dev, T, n, live, heads = cuda_device, 153, 1 << 17, 64, 64
    g = torch.Generator(device=dev).manual_seed(51)
    randn = lambda *shape: torch.randn(*shape, device=dev, generator=g)
    u = randn(H.HD)
    rows = randn(n, H.HD)
    rows -= (rows @ u)[:, None] * u / (u @ u)                # nothing along u
    rows[:live] += 0.5 * u
    q = randn(T, heads, H.HD) + 40 * H.HD ** 0.5 / (0.5 * float(u @ u)) * u
    cache, scales = torch.zeros(n // 16, 16, H.HD, device=dev).to(F8), torch.zeros(n // 16, 16, device=dev)
    status = status_word(dev)
    csa.csa_paged_append_fp8(csa.AppendJobsFp8([csa.AppendJobFp8(rows, torch.arange(n, device=dev), cache, scales,
                                                                 16)]), status)
    layout = csa.PagedLayoutFp8(torch.zeros(T, dtype=torch.int32, device=dev),
                                torch.full((T,), 4 * n, dtype=torch.int64, device=dev), torch.tensor([n], device=dev),
                                torch.arange(n // 16, device=dev).int()[None], 16)
    prm = csa.params(heads, 1, 0, 4)
    q, out = q.to(BF16), torch.empty(T, heads, H.HD, device=dev)
    csa.csa_paged_attention_fp8(layout, prm, cache, scales, q, out, status, csa.paged_workspace(layout, prm))
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    vals = F.values(*F.quantise(rows.double().cpu().numpy())).to(dev)
    for t in range(0, T, 38):
        l = prm.scale * q[t].double() @ vals.T
        assert 25 < float(l[:, :live].amax(1).min()) and float(l.max()) < 55
        assert float((l[:, live:].amax(1) - l[:, :live].amax(1)).max()) < -34.7
        ref = torch.softmax(l, 1) @ vals
        err = (out[t].double() - ref).norm() / ref.norm()
        assert err <= (2.9e-6 + 1.0e-6 + 4e-6) / 2
