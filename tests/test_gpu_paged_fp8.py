"""8-bit paged caches on the GPU: the quantising append and the read bit for bit,
the attention against float64 over the values the codes stand for, and the calls
together as a serving step makes them."""
import numpy as np
import pytest
import torch

from sparse_compressed_kv_gb300 import csa
from tests import fp8_helpers as F
from tests import paged_helpers as H
from tests.gpu_helpers import Guarded

pytestmark = pytest.mark.gpu

F32, BF16, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
BOTH = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])


def status_word(device):
    return torch.zeros(1, dtype=torch.int32, device=device)


# ---------------------------------------------------------------- append and read

def awkward(n, width, dtype, seed):
    """Rows of every magnitude, some with zeros, ties, infinities or NaN."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, width, generator=g) * torch.exp2(torch.randint(-20, 20, (n, 1), generator=g).float())
    for i in range(n):
        kind = i % 11
        if kind == 1:
            x[i] = 0
        elif kind == 2:                     # ties between codes, and the largest value itself
            x[i] = (torch.randint(0, 16, (width,), generator=g) + 0.5 + 16) * 2.0 ** (i % 7)
            x[i, 0] = 448 * 2.0 ** (i % 7 - 4)
        elif kind == 3:
            x[i, i % width], x[i, (i + 7) % width], x[i, (i + 9) % width] = np.inf, -np.inf, np.nan
        elif kind == 4:
            x[i] *= 2.0 ** -100             # below the smallest scale
        elif kind == 5:
            x[i] *= 2.0 ** 80               # above the largest
        elif kind == 6:
            x[i] = np.nan
        elif kind == 7:                     # one large value: the rest in the subnormal range
            x[i, i % width] = 2.0 ** 30
        elif kind == 8:
            x[i, :] = -0.0
            x[i, 0] = 1e-39                 # a subnormal
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("n,width,extra,page_rows,gap,scale_gap,pages", [
    (1, 512, 0, 64, 0, 0, 2), (5, 16, 0, 1, 0, 0, 40), (37, 80, 16, 3, 2, 1, 21), (300, 128, 8, 16, 8, 0, 30),
    (2500, 512, 0, 64, 128, 128, 45), (64, 1024, 32, 7, 0, 5, 12), (90, 272, 0, 5, 3, 3, 30),
    (0, 512, 0, 64, 0, 0, 2),
])
def test_append(cuda_device, n, width, extra, page_rows, gap, scale_gap, pages, dtype):
    dev = cuda_device
    rows = awkward(n, width, dtype, n + width)
    g = torch.Generator().manual_seed(n)
    slots = torch.randperm(pages * page_rows, generator=g)[:n].long()
    slots[torch.rand(n, generator=g) < 0.2] = -1
    src = torch.zeros(max(n, 1), width + extra, dtype=dtype, device=dev)[:n, :width]
    src.copy_(rows)
    cache = Guarded((pages, page_rows + gap, width), torch.uint8, dev, 0x55)
    scales = Guarded((pages, page_rows + scale_gap), F32, dev, 9.0)
    want, want_s = cache.t.cpu(), scales.t.cpu()
    codes, k = F.quantise(rows.double().numpy())
    for i, s in enumerate(slots.tolist()):
        if s >= 0:
            want[s // page_rows, s % page_rows] = torch.from_numpy(codes[i])
            want_s[s // page_rows, s % page_rows] = float(k[i])
    status = status_word(dev)
    jobs = csa.AppendJobsFp8([csa.AppendJobFp8(src, slots.to(dev), cache.t.view(F8), scales.t, page_rows)])
    csa.csa_paged_append_fp8(jobs, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and cache.intact() and scales.intact()
    got = cache.t.cpu()
    nan = (want & 127) == 127                 # (a NaN's sign is not defined)
    assert torch.equal(got | (nan * 128), want | (nan * 128))
    assert torch.equal(scales.t.cpu(), want_s)


def test_append_several_caches_and_bad_slots(cuda_device):
    dev, status = cuda_device, status_word(cuda_device)
    g = torch.Generator().manual_seed(3)
    jobs, checks = [], []
    for k, (n, width, dt) in enumerate([(33, 512, BF16), (33, 128, F32), (50, 512, BF16), (9, 1024, F32)]):
        rows = torch.randn(n, width, generator=g).to(dt)
        slots = torch.randperm(96, generator=g)[:n]
        cache = torch.full((12, 11, width), 3, dtype=torch.uint8)
        scales = torch.full((12, 8), 5.0)
        want, want_s = cache.clone(), scales.clone()
        codes, scale = F.quantise(rows.double().numpy())
        if k == 2:      # past the pool: skipped, and said so
            slots[4], slots[7] = 96, 1 << 40
        for i, s in enumerate(slots.tolist()):
            if s < 96:
                want[s // 8, s % 8], want_s[s // 8, s % 8] = torch.from_numpy(codes[i]), float(scale[i])
        cache, scales = cache.to(dev), scales.to(dev)
        jobs.append(csa.AppendJobFp8(rows.to(dev), slots.to(dev), cache.view(F8), scales, 8))
        checks.append((cache, want, scales, want_s))
    csa.csa_paged_append_fp8(csa.AppendJobsFp8(jobs), status)
    torch.cuda.synchronize()
    assert int(status.item()) == csa.DEV_BAD_INDEX
    for cache, want, scales, want_s in checks:
        assert torch.equal(cache.cpu(), want) and torch.equal(scales.cpu(), want_s)


def test_append_of_more_rows_than_a_pass_of_the_grid(cuda_device):
    dev, n = cuda_device, 40000
    g = torch.Generator(device=dev).manual_seed(4)
    rows = torch.randn(n, 512, device=dev, generator=g).to(BF16)
    slots = torch.randperm(n, device=dev, generator=g)
    cache, scales = torch.zeros(n // 32, 32, 512, device=dev).to(F8), torch.zeros(n // 32, 32, device=dev)
    status = status_word(dev)
    csa.csa_paged_append_fp8(csa.AppendJobsFp8([csa.AppendJobFp8(rows, slots, cache, scales, 32)]), status)
    out = torch.zeros(n, 512, device=dev)
    csa.csa_paged_read_fp8(cache, scales, slots, out, status, 32)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    codes, k = F.quantise(rows.cpu().double().numpy())
    assert torch.equal(out.cpu().double(), F.values(codes, k))
    # what the format promises: half a step of the value, or of the subnormal range
    x, s = rows.double().cpu(), torch.from_numpy(k)[:, None]
    assert ((out.double().cpu() - x).abs() <= torch.maximum(x.abs() * 2 ** -4, s * 2.0 ** -10)).all()


@BOTH
@pytest.mark.parametrize("n,width,extra,page_rows,gap,scale_gap,pages", [
    (1, 512, 0, 64, 0, 0, 2), (5, 16, 0, 1, 0, 0, 40), (37, 80, 16, 3, 2, 1, 21), (300, 128, 8, 16, 8, 0, 30),
    (2500, 512, 0, 64, 128, 128, 45), (64, 1024, 32, 7, 0, 5, 12), (90, 272, 0, 5, 3, 3, 30),
    (0, 512, 0, 64, 0, 0, 2),
])
def test_read(cuda_device, n, width, extra, page_rows, gap, scale_gap, pages, dtype):
    dev = cuda_device
    g = torch.Generator().manual_seed(n + width)
    codes = torch.randint(0, 256, (pages, page_rows + gap, width), dtype=torch.uint8, generator=g)
    # scales as the append writes them, and others; the largest and smallest
    scales = torch.exp2(torch.randint(-60, 61, (pages, page_rows + scale_gap), generator=g).float())
    scales[::3] *= torch.rand(scales[::3].shape, generator=g) + 0.5
    slots = torch.randint(0, pages * page_rows, (n,), generator=g)       # the same one several times
    slots[torch.rand(n, generator=g) < 0.2] = -1
    bad = n > 30
    if bad:
        slots[3], slots[4] = pages * page_rows, 1 << 50
    out = Guarded((max(n, 1), width + extra), dtype, dev, 7.0)
    status = status_word(dev)
    csa.csa_paged_read_fp8(codes.to(dev).view(F8), scales.to(dev), slots.to(dev), out.t[:n, :width], status,
                           page_rows)
    torch.cuda.synchronize()
    assert int(status.item()) == (csa.DEV_BAD_INDEX if bad else 0) and out.intact()
    want = torch.full((n, width), 7.0, dtype=torch.float64)
    keep = (slots >= 0) & (slots < pages * page_rows)
    s = slots[keep]
    want[keep] = F.values(codes[s // page_rows, s % page_rows], scales[s // page_rows, s % page_rows])
    assert torch.equal(out.t[:n, :width].cpu().nan_to_num(99), want.to(F32).to(dtype).nan_to_num(99))
    assert (out.t[:, width:] == 7).all()


def test_far_ends_of_large_pools(cuda_device):
    # offsets past 2^32 bytes of codes
    dev = cuda_device
    pages, stride = 70000, 128
    pool = torch.zeros(pages, stride, 512, dtype=torch.uint8, device=dev)
    part, scales = pool.view(F8)[:, 64:], torch.zeros(pages, 64, device=dev)
    rows = torch.randn(3, 512, device=dev).to(BF16)
    slots = torch.tensor([pages * 64 - 1, 0, (pages // 2 + 1) * 64], device=dev)
    status, out = status_word(dev), torch.zeros(3, 512, dtype=BF16, device=dev)
    csa.csa_paged_append_fp8(csa.AppendJobsFp8([csa.AppendJobFp8(rows, slots, part, scales, 64)]), status)
    csa.csa_paged_read_fp8(part, scales, slots, out, status, 64)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert torch.equal(out.double().cpu(), F.values(*F.quantise(rows.double().cpu().numpy())))
    assert pool.view(torch.int64).ne(0).sum(2).ne(0).sum() == 3      # three rows, nothing else


# ---------------------------------------------------------------- attention

CASES = {
    "one-row": dict(row_len=[1], tokens=[(0, 4)], heads=1, window=0, page_rows=1),
    "tiny": dict(row_len=[256], tokens=[(0, 1024)], heads=16),
    "window-only": dict(row_len=[0, 1], tokens=[(0, 2), (1, 3)], heads=64, window=128),
    "nothing": dict(row_len=[0, 5], tokens=[(0, 3), (1, 20)], heads=8, window=0),
    "window-1": dict(row_len=[70], tokens=[(0, 280)], heads=24, window=1, page_rows=7),
    "ragged": dict(row_len=[63, 64, 65, 0, 130, 1, 400], tokens=[(b, p) for b, p in enumerate(
        [252, 256, 260, 0, 521, 5, 1600])], heads=64, page_rows=24, gap=8, sinks=True),
    "drafts": dict(row_len=[500, 90], tokens=[(0, 1996 + i) for i in range(4)] + [(1, 360 + i) for i in range(4)],
                   heads=128, page_rows=24, gap=8, sinks=True),
    "padding": dict(row_len=[200, 300], tokens=[(-1, -1), (1, 1200), (-1, -1), (0, 800), (-1, -1)], heads=40),
    "ratio-1": dict(row_len=[1000], tokens=[(0, 999), (0, 500)], ratio=1, heads=64, page_rows=100),
    "ratio-128": dict(row_len=[300, 20], tokens=[(0, 38500), (1, 2600)], ratio=128, heads=64, page_rows=2),
    "long": dict(row_len=[20000], tokens=[(0, 80000)], heads=64, page_rows=64),
    "two-long": dict(row_len=[9000, 5000], tokens=[(0, 36000), (1, 20000)], heads=128, page_rows=8, sinks=True),
    "many": dict(row_len=[150 + i for i in range(170)], tokens=[(i, 700 + i) for i in range(170)], heads=16),
}


@BOTH
@pytest.mark.parametrize("name", CASES)
def test_attention(cuda_device, name, dtype):
    p = F.PagedFp8(len(name), **CASES[name])
    got, status = p.run(cuda_device, dtype)
    seen = [t for t, b in enumerate(p.tok_seq.tolist()) if b >= 0]

    def lost(t):                        # window positions that the ring no longer holds
        b, x = int(p.tok_seq[t]), int(p.tok_pos[t])
        first = max(0, x - p.window + 1)
        return {min(int(p.row_len[b]), x // p.ratio) + i for i in range(int(p.swa_first_pos[b]) - first)
                if p.window and first + i <= x}

    assert status == (csa.DEV_MISSING_SWA if any(lost(t) for t in seen) else 0)
    assert any(lost(t) for t in seen) == (name == "ratio-1")     # (two tokens far apart)
    F.check(got, p.reference(lost), dtype, seen)
    for t, b in enumerate(p.tok_seq.tolist()):
        if b < 0:       # padding: the output is left as it was
            assert (got[t] == 7).all()
    again, _ = p.run(cuda_device, dtype)
    assert torch.equal(got, again)      # bit for bit


@pytest.mark.parametrize("seed", range(24))
def test_attention_random_shapes(cuda_device, seed):
    # token counts around the number of CTAs, any page size, heads and window
    rng = np.random.default_rng(300 + seed)
    B = int(rng.choice([1, 2, 5, 40, 151, 152, 153, 170]))
    new = int(rng.choice([1, 1, 2, 3]))
    ratio = int(rng.choice([1, 4, 128]))
    most = int(rng.choice([3, 70, 400, 1500])) if B < 100 else int(rng.choice([3, 70, 400]))
    ctx = [int(rng.integers(0, most + 1)) * ratio + int(rng.integers(0, ratio)) for _ in range(B)]
    p = F.PagedFp8(seed, row_len=[(c + new) // ratio for c in ctx],
                   tokens=[(b, ctx[b] + i) for b in range(B) for i in range(new)], ratio=ratio,
                   page_rows=int(rng.choice([1, 2, 3, 8, 12, 16, 50, 64, 128])), gap=int(rng.choice([0, 8, 3])),
                   heads=int(rng.choice([1, 3, 8, 16, 33, 64, 100])) if B < 100 else 8,
                   window=int(rng.choice([0, 1, 20, 128])), sinks=bool(rng.integers(2)))
    dtype = [F32, BF16][seed % 2]
    got, status = p.run(cuda_device, dtype)
    assert status == 0
    tokens = sorted(set(rng.integers(0, B * new, 40).tolist()) | {0, B * new - 1})
    F.check(got, p.reference(tokens=tokens), dtype, tokens)


@BOTH
@pytest.mark.parametrize("heads", [1, 7, 15, 17, 33, 63, 65, 97, 127])
def test_attention_head_counts_inside_a_group(cuda_device, heads, dtype):
    p = F.PagedFp8(heads, row_len=[90, 400], tokens=[(0, 360), (1, 1600)], heads=heads, sinks=True)
    got, status = p.run(cuda_device, dtype)
    assert status == 0
    F.check(got, p.reference(), dtype)


@BOTH
def test_attention_peaked_and_large_logits(cuda_device, dtype):
    # logits up to several hundred, rising along the rows: the running maximum
    # moves many times, and far rows weigh nothing
    p = F.PagedFp8(5, row_len=[640], tokens=[(0, 2560)], heads=64, page_rows=64, window=0, spread=0)
    j = torch.arange(640)
    at = (p.table[0, j // 64].long(), j % 64)
    codes, k = F.quantise((p.cache[at] * (1 + j[:, None] / 40)).numpy())
    p.codes[at], p.scales[at] = torch.from_numpy(codes), torch.from_numpy(k).float()
    p.requantised()
    p.q *= 4
    ref = p.reference()
    got, status = p.run(cuda_device, dtype)
    assert status == 0
    l = p.scale * p.q[0].double() @ p.rows_of(0).T
    assert 100 < float(l.max()) < 1000
    # a weight's relative error is its logit's absolute error: 19 steps of 2^-23 of at
    # most 1000, and the query's small values (2^-17 times rows 17 and queries 4 times as large)
    tol = F.REL[dtype] + 2 * (1000 * 19 * 2 ** -23 + 17 * 4 * 2 ** -17)
    err = (got.double().cpu() - ref).norm(dim=2)
    assert (err <= tol * ref.norm(dim=2)).all()


@BOTH
@pytest.mark.parametrize("T,n", [(100, 640), (60, 400), (30, 300), (1, 20000), (160, 3000)], ids=str)
def test_attention_rising_maximum(cuda_device, T, n, dtype):
    # rows in steps of 64 whose logits rise by more than the rescaling's threshold
    dev = cuda_device
    g = torch.Generator().manual_seed(T)
    rows = torch.randn(n, H.HD, generator=g) * (2 + 2.2 * (torch.arange(n) % 192 // 64))[:, None]
    codes, k = F.quantise(rows.double().numpy())
    vals = F.values(codes, k).to(dev)
    pages = -(-n // 16)
    table = torch.randperm(pages, generator=g)
    cache, scales = torch.full((pages, 16, H.HD), 127, dtype=torch.uint8), torch.full((pages, 16), float("nan"))
    j = torch.arange(n)
    cache[table[j // 16], j % 16], scales[table[j // 16], j % 16] = torch.from_numpy(codes), torch.from_numpy(k).float()
    q = torch.randn(T, 64, H.HD, generator=g).to(BF16).to(dev)
    layout = csa.PagedLayoutFp8(torch.zeros(T, dtype=torch.int32, device=dev),
                                torch.full((T,), 4 * n, dtype=torch.int64, device=dev),
                                torch.tensor([n], device=dev), table.int()[None].to(dev), 16)
    prm = csa.params(64, 1, 0, 4)
    status, out = status_word(dev), torch.empty(T, 64, H.HD, device=dev, dtype=dtype)
    csa.csa_paged_attention_fp8(layout, prm, cache.to(dev).view(F8), scales.to(dev), q, out, status,
                                csa.paged_workspace(layout, prm))
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for t in range(0, T, max(1, T // 12)):
        l = prm.scale * q[t].double() @ vals.T
        assert 15 < float(l.max()) < 40           # (the threshold: 8 ln 2 = 5.5)
        ref = torch.softmax(l, 1) @ vals
        # weights: 19 steps of 2^-23 of a logit of at most 40, and the query's small
        # values (rows up to 6.4 instead of 2), in weights and their sum
        tol = F.REL[dtype] + 2 * (40 * 19 * 2 ** -23 + 3.2 * 2 ** -17)
        err = (out[t].double() - ref).norm(dim=1) / ref.norm(dim=1)
        assert float(err.max()) <= tol, f"token {t}: off by {float(err.max()):.3e}"


@BOTH
def test_attention_scales_far_apart(cuda_device, dtype):
    # rows of one token from 2^-12 to 2^3, in no order; other tokens at the ends of the range,
    # where every weight is the same or the largest row takes all
    p = F.PagedFp8(15, row_len=[700, 100, 90, 80], tokens=[(0, 2800), (1, 400), (2, 360), (3, 320)], heads=64,
                   window=0)
    g = torch.Generator().manual_seed(16)
    for b, (n, lo, hi) in enumerate([(700, -18, -3), (100, -60, -59), (90, -60, -20), (80, -60, -60)]):
        j = torch.arange(n)
        at = (p.table[b, j // 16].long(), j % 16)
        p.scales[at] = torch.exp2(torch.randint(lo, hi + 1, (n,), generator=g).float())
    p.requantised()
    got, status = p.run(cuda_device, dtype)
    assert status == 0
    # (rows up to 448 / 8 instead of 3.5 * 2: the query's small values weigh 8 times as much, and logits 8 times)
    F.check(got, p.reference(), dtype, rel=F.REL[dtype] + 2 * 8 * (12 * 19 * 2 ** -23 + 2 ** -17))


def test_attention_scales_that_are_no_powers_of_two(cuda_device):
    p = F.PagedFp8(17, row_len=[300], tokens=[(0, 1200)], heads=64, sinks=True)
    g = torch.Generator().manual_seed(18)
    for s in (p.scales, p.swa_scales):
        s *= 1 + torch.rand(s.shape, generator=g)
    p.scales[p.table[0, 3].long(), 5] = 0        # a row of weight, without a value
    p.scales[p.table[0, 4].long(), 1] *= -1
    p.requantised()
    got, status = p.run(cuda_device, F32)
    assert status == 0
    F.check(got, p.reference(), F32, rel=2 * F.REL[F32])     # (logits and rows twice as large)


def test_attention_zero_rows_and_queries(cuda_device):
    p = F.PagedFp8(19, row_len=[100, 40], tokens=[(0, 400), (1, 160)], heads=16, window=4)
    p.codes[p.table[0, :7].long()] = 0
    p.scales[p.table[0, :7].long()] = 2.0 ** -60
    p.swa_codes[0], p.swa_scales[0] = 0, 2.0 ** -60
    p.q[1] = 0                                    # every weight the same
    p.requantised()
    got, status = p.run(cuda_device, F32)
    assert status == 0 and (got[0] == 0).all()
    F.check(got, p.reference(), F32, [1])


@pytest.mark.parametrize("magnitude", [2.0 ** -100, 2.0 ** -130, 2.0 ** 30])
def test_attention_queries_of_any_magnitude(cuda_device, magnitude):
    p = F.PagedFp8(20, row_len=[100], tokens=[(0, 400)], heads=16, window=4)
    p.q = (p.q.double() * magnitude).to(BF16)
    p.scale = 512 ** -0.5 / magnitude if magnitude > 1 else p.scale
    got, status = p.run(cuda_device, F32)
    assert status == 0
    F.check(got, p.reference(), F32)


@BOTH
def test_attention_not_a_number_stays_where_it_is(cuda_device, dtype):
    p = F.PagedFp8(21, row_len=[100, 100, 100], tokens=[(0, 400), (1, 400), (2, 400)], heads=64)
    clean, _ = p.run(cuda_device, dtype)
    p.codes[p.table[0, 2].long(), 3, 77] = 127     # one value of one row: every head's weights hold it
    p.q[2, 5, 100] = float("inf")
    p.q[2, 9, 3] = float("nan")
    got, status = p.run(cuda_device, dtype)
    assert status == 0
    assert got[0].isnan().all()
    assert torch.equal(got[1], clean[1])
    rest = [h for h in range(64) if h not in (5, 9)]
    assert got[2, [5, 9]].isnan().all() and torch.equal(got[2, rest], clean[2, rest])


@BOTH
@pytest.mark.parametrize("row_len,tokens", [([100], [(0, 400)]), ([20000], [(0, 80000)]),
                                            ([900, 30], [(0, 3600), (1, 130)])], ids=["whole", "cut", "two"])
def test_attention_sinks_of_any_value(cuda_device, row_len, tokens, dtype):
    p = F.PagedFp8(22, row_len=row_len, tokens=tokens, heads=8, sinks=True)
    p.sinks = torch.tensor([0.0, -float("inf"), float("inf"), float("nan"), 60.0, -200.0, 300.0, 3.0])
    got, status = p.run(cuda_device, dtype)
    assert status == 0
    p.sinks = p.sinks.clone()
    ref = p.reference()
    for t in range(len(tokens)):
        assert (got[t, 2] == 0).all() and got[t, 3].isnan().all()
        for h in (0, 1, 5, 7):
            norm = ref[t, h].norm()
            assert (got[t, h].double().cpu() - ref[t, h]).norm() <= 2 * F.REL[dtype] * norm
        for h in (4, 6):                          # the sink takes all
            assert got[t, h].abs().max() <= 1e-20


@pytest.mark.parametrize("scale", [0.0, -0.05])
def test_attention_other_scales(cuda_device, scale):
    p = F.PagedFp8(6, row_len=[150], tokens=[(0, 600)], heads=64, page_rows=16)
    p.scale = scale
    got, status = p.run(cuda_device, F32)
    assert status == 0
    F.check(got, p.reference(), F32)


@BOTH
@pytest.mark.parametrize("page_rows", [16, 6])
def test_attention_bad_pages_lengths_and_window(cuda_device, page_rows, dtype):
    P = page_rows
    p = F.PagedFp8(7, row_len=[100, 40, 30, 25], tokens=[(0, 400), (1, 160), (2, 120), (3, 100)], heads=16,
                   page_rows=P, window=32)
    pages = p.cache.shape[0]
    p.table[0, 1] = pages          # past the pool
    p.table[0, 3] = -1
    p.swa_first_pos[1] = 150       # the ring lost positions 129 .. 149
    p.row_len[3] = -3              # read as 0
    lost = set(range(P, 2 * P)) | set(range(3 * P, 4 * P))
    gone = {0: lost, 1: {40 + i for i in range(150 - (160 - 32 + 1))}, 2: None, 3: None}
    got, status = p.run(cuda_device, dtype)
    assert status == csa.DEV_BAD_INDEX | csa.DEV_MISSING_SWA | csa.DEV_BAD_LENGTH
    p.table.clamp_(0, pages - 1)
    p.row_len.clamp_(min=0)
    p.cache.nan_to_num_(0.0)       # the reference reads lost rows before it drops them
    F.check(got, p.reference(lambda t: gone[t]), dtype)


def test_attention_layout_errors(cuda_device):
    p = F.PagedFp8(8, row_len=[20, 20], tokens=[(0, 80), (1, 80), (0, 60)], heads=16, max_pages=2)
    p.tok_seq[1] = 2               # no such sequence
    p.tok_pos[2] = -1
    got, status = p.run(cuda_device, F32)
    assert status == csa.DEV_BAD_LAYOUT
    F.check(got, p.reference(tokens=[0]), F32, [0])
    assert (got[1:] == 0).all()
    p = F.PagedFp8(8, row_len=[32], tokens=[(0, 400)], heads=16, max_pages=2)
    p.row_len[0] = 33              # more rows than the table has room for
    got, status = p.run(cuda_device, F32)
    assert status == csa.DEV_CAPACITY
    p.row_len[0] = 32
    F.check(got, p.reference(), F32)


@BOTH
def test_attention_reads_nothing_else(cuda_device, dtype):
    p = F.PagedFp8(9, row_len=[83, 5], tokens=[(0, 290), (1, 17)], heads=16, page_rows=8)
    a, _ = p.run(cuda_device, dtype)
    n = 290 // 4                   # rows 72 .. 82 are held, but not visible to token 0
    j = torch.arange(n, 83)
    at = (p.table[0, j // 8].long(), j % 8)
    p.codes[at], p.scales[at] = 127, float("inf")
    x = torch.arange(290 - 127, 291)
    cap = p.swa_kv.shape[1]
    unseen = torch.ones(cap, dtype=torch.bool)
    unseen[x % cap] = False
    p.swa_codes[0, unseen], p.swa_scales[0, unseen] = 255, float("nan")
    p.swa_codes[1, 18:], p.swa_scales[1, 18:] = 127, float("inf")
    b, status = p.run(cuda_device, dtype)
    assert status == 0 and torch.equal(a, b)


def test_attention_cache_beyond_32_bit_offsets(cuda_device):
    dev = cuda_device
    p = F.PagedFp8(10, row_len=[150], tokens=[(0, 600)], heads=16, page_rows=64, window=0)
    pages, stride = 70000, 128
    cache = torch.zeros(pages, stride, H.HD, dtype=torch.uint8, device=dev)
    scales = torch.zeros(pages, 64, device=dev)
    far = torch.tensor([pages - 1, 0, pages // 2 + 1])
    cache[far.to(dev), :64] = p.codes[p.table[0, :3].long()].to(dev)
    scales[far.to(dev)] = p.scales[p.table[0, :3].long()].to(dev)
    table = torch.full_like(p.table, -1)
    table[0, :3] = far
    layout = csa.PagedLayoutFp8(p.tok_seq.to(dev), p.tok_pos.to(dev), p.row_len.to(dev), table.to(dev), 64)
    prm = csa.params(16, 1, 0, 4)
    out, status = torch.empty(1, 16, H.HD, device=dev), status_word(dev)
    csa.csa_paged_attention_fp8(layout, prm, cache.view(F8), scales, p.q.to(dev), out, status,
                                csa.paged_workspace(layout, prm))
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    F.check(out, p.reference(), F32)


@BOTH
def test_attention_long_rows_in_one_cta(cuda_device, dtype):
    # so many tokens that each is one CTA's work: long sums, held in f32
    dev, n, T = cuda_device, 20000, 320
    g = torch.Generator(device=dev).manual_seed(11)
    rows = torch.randn(n, H.HD, device=dev, generator=g)
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
    out = torch.empty(T, 64, H.HD, device=dev, dtype=dtype)
    csa.csa_paged_attention_fp8(layout, prm, cache, scales, q, out, status, csa.paged_workspace(layout, prm))
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    vals = F.values(*F.quantise(rows.double().cpu().numpy())).to(dev)
    for t in range(0, T, 37):
        v = vals[:int(pos[t]) // 4]
        ref = torch.softmax(prm.scale * q[t].double() @ v.T, 1) @ v
        assert (out[t].double() - ref).norm() <= F.REL[dtype] * ref.norm()


@BOTH
def test_attention_many_rows_of_little_weight(cuda_device, dtype):
    # one row whose logit stands 9 above 40,000 others that all hold the same
    # values: together they weigh as much as it does, each below 2^-12 of it
    dev, n = cuda_device, 40000
    g = torch.Generator(device=dev).manual_seed(23)
    common = torch.randn(H.HD, device=dev, generator=g)
    q = torch.randn(1, 64, H.HD, device=dev, generator=g).to(BF16)
    rows = common.repeat(n, 1)
    rows[n // 3] = 0.4 * q[0, 0].float() + 0.5 * torch.randn(H.HD, device=dev, generator=g)
    cache, scales = torch.zeros(n // 16, 16, H.HD, device=dev).to(F8), torch.zeros(n // 16, 16, device=dev)
    status = status_word(dev)
    slots = torch.arange(n, device=dev)
    csa.csa_paged_append_fp8(csa.AppendJobsFp8([csa.AppendJobFp8(rows, slots, cache, scales, 16)]), status)
    layout = csa.PagedLayoutFp8(torch.zeros(1, dtype=torch.int32, device=dev), torch.tensor([4 * n], device=dev),
                                torch.tensor([n], device=dev), torch.arange(n // 16, device=dev).int()[None], 16)
    prm = csa.params(64, 1, 0, 4)
    out = torch.empty(1, 64, H.HD, device=dev, dtype=dtype)
    csa.csa_paged_attention_fp8(layout, prm, cache, scales, q, out, status, csa.paged_workspace(layout, prm))
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    vals = F.values(*F.quantise(rows.double().cpu().numpy())).to(dev)
    w = torch.softmax(prm.scale * q[0].double() @ vals.T, 1)
    ref = w @ vals
    assert 0.05 < float(w[0, n // 3]) < 0.95
    # every row of the 39,999 is off alike, by 2^-9 (bf16: the weight's bound) or
    # 2^-18 of its weight and by 2^-24 of the largest: 39,999 of them add up
    tol = F.REL[dtype] + (2 ** -9 if dtype == BF16 else 2 ** -18) + n * 2 ** -24 * float(w[0, n // 3])
    err = (out[0].double() - ref).norm(dim=1) / ref.norm(dim=1)
    assert float(err.max()) <= tol, float(err.max())


@pytest.mark.parametrize("long", [150, 3000], ids=["whole", "cut"])
def test_attention_more_tokens_than_a_cta_lists(cuda_device, long):
    tokens = [(-1, -1)] * 8192
    for i in range(8192):
        if i % 41 == 7:
            tokens[i] = (0, 4 * (i % 150 + 1))
        elif i % 64 == 3:
            tokens[i] = (0, 3)
    tokens[5000] = (1, 4 * long)
    p = F.PagedFp8(long, row_len=[150, long], tokens=tokens, heads=65, window=0)
    for dtype in (F32, BF16):
        got, status = p.run(cuda_device, dtype, fill=7.5)
        assert status == 0
        assert bool((got[(p.tok_seq < 0).to(got.device)] == 7.5).all())
        seen = [t for t, (b, _) in enumerate(tokens) if b >= 0]
        F.check(got, p.reference(tokens=seen), dtype, seen)


@BOTH
@pytest.mark.parametrize("T", [1, 60, 152, 153, 400, 2000])
def test_attention_of_padding_and_of_tokens_without_rows(cuda_device, T, dtype):
    p = F.PagedFp8(T, row_len=[3], tokens=[(-1, -1) if t % 3 else (0, 2) for t in range(T)], heads=8, window=0)
    got, status = p.run(cuda_device, dtype)
    assert status == 0
    for r in range(3):
        assert (got[r::3] == (7 if r else 0)).all()


def test_attention_on_another_stream(cuda_device):
    p = F.PagedFp8(12, row_len=[500, 300], tokens=[(0, 2000), (1, 1200)], heads=64)
    a, _ = p.run(cuda_device, BF16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b, status = p.run(cuda_device, BF16, stream=s)
    assert status == 0 and torch.equal(a, b)


def test_attention_two_streams_at_once(cuda_device):
    dev = cuda_device
    ps = [F.PagedFp8(40 + i, row_len=[4000, 300 * i], tokens=[(0, 16000), (1, 1200 * i)], heads=64, page_rows=32)
          for i in range(2)]
    alone = [p.run(dev, F32)[0].clone() for p in ps]
    args, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for p in ps:
        layout, prm, codes, scales, q, _ = p.arguments(dev)
        args.append((layout, prm, codes, scales, q, torch.empty(2, 64, H.HD, device=dev), status_word(dev),
                     csa.paged_workspace(layout, prm)))
    torch.cuda.synchronize()
    for _ in range(20):
        for a, s in zip(args, streams):
            csa.csa_paged_attention_fp8(*a, stream=s)
    torch.cuda.synchronize()
    for a, want in zip(args, alone):
        assert int(a[6].item()) == 0 and torch.equal(a[5], want)


def test_attention_replayed_with_other_lengths(cuda_device):
    dev = cuda_device
    lens = [[3, 5], [6000, 0], [700, 900], [0, 0], [64, 6000]]
    ps = [F.PagedFp8(50 + i, row_len=n, tokens=[(0, 4 * n[0] + 1), (1, 4 * n[1] + 3)], heads=64, page_rows=32,
                     max_pages=200, spare_pages=250 - sum(-(-x // 32) for x in n)) for i, n in enumerate(lens)]
    parts = lambda p: (p.tok_seq, p.tok_pos, p.row_len, p.table, p.swa_codes, p.swa_scales, p.swa_first_pos,
                       p.codes, p.scales, p.q)
    b = [x.to(dev).clone() for x in parts(ps[0])]
    layout = csa.PagedLayoutFp8(*b[:4], 32, b[4].view(F8), b[5], b[6])
    prm = csa.params(64, 1, 128, 4)
    ws, out, status = csa.paged_workspace(layout, prm), torch.empty(2, 64, H.HD, device=dev), status_word(dev)
    call = lambda: csa.csa_paged_attention_fp8(layout, prm, b[7].view(F8), b[8], b[9], out, status, ws)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for p in ps:
        for buf, x in zip(b, parts(p)):
            buf.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        F.check(out, p.reference(), F32)


def test_append_and_read_replayed_on_another_stream(cuda_device):
    # one graph of both calls, other rows, slots and results at each replay; every
    # append overwrites codes and scales beside those that a replay before it read
    dev, n, page_rows = cuda_device, 700, 24
    g = torch.Generator().manual_seed(77)
    rows = torch.empty(n, 512, dtype=BF16, device=dev)
    slots, back = (torch.empty(n, dtype=torch.int64, device=dev) for _ in range(2))
    cache = torch.zeros(40, page_rows, 512, device=dev).to(F8)
    scales, out = torch.ones(40, page_rows, device=dev), torch.zeros(n, 512, device=dev)
    status, s = status_word(dev), torch.cuda.Stream()
    jobs = csa.AppendJobsFp8([csa.AppendJobFp8(rows, slots, cache, scales, page_rows)])
    held = np.zeros((40 * page_rows, 512), np.uint8), np.ones(40 * page_rows)

    def fill():
        x = torch.randn(n, 512, generator=g) * torch.exp2(torch.randint(-9, 9, (n, 1), generator=g).float())
        at, of = torch.randperm(40 * page_rows, generator=g)[:n], torch.randint(-1, 40 * page_rows, (n,), generator=g)
        rows.copy_(x)
        slots.copy_(at)
        back.copy_(of)
        held[0][at], held[1][at] = F.quantise(x.to(BF16).double().numpy())
        torch.cuda.synchronize()
        return of

    def calls():
        csa.csa_paged_append_fp8(jobs, status, stream=s)
        csa.csa_paged_read_fp8(cache, scales, back, out, status, page_rows, stream=s)

    fill()
    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        calls()
    want = out.cpu().double()
    for _ in range(4):
        of = fill()
        graph.replay()
        torch.cuda.synchronize()
        want[of >= 0] = F.values(*held)[of[of >= 0]]
        assert int(status.item()) == 0 and torch.equal(out.cpu().double(), want)


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("captured", [False, True])
def test_serving_loop(cuda_device, captured):
    # plan, quantising append (rows and window), attention over two interleaved layers'
    # pools, requests that grow, end and begin; then every held row read back
    dev = cuda_device
    torch.manual_seed(20)
    B, ratio, P, cap, heads, pages, layers = 5, 4, 3, 40, 16, 64, 2
    T, R = 64, 32
    i64 = lambda *x: torch.zeros(*x, dtype=torch.int64, device=dev)
    seq, pos = [i64(B), i64(B)], [torch.tensor([0, pages], device=dev), i64(2)]
    new_len = torch.zeros(B, dtype=torch.int32, device=dev)
    table = torch.full((B, 24), -1, dtype=torch.int32, device=dev)
    m = dict(table=table, free_ring=torch.randperm(pages, device=dev).int(), new_len=new_len, row_len=i64(B),
             swa_first_pos=i64(B), tok_off=i64(B + 1), row_off=i64(B + 1),
             tok_seq=torch.zeros(T, dtype=torch.int32, device=dev), tok_pos=i64(T), swa_slot=i64(T), row_slot=i64(R))
    plans = [csa.PagePlan(ratio=ratio, page_rows=P, swa_cap=cap, seq_len=seq[k], free_pos=pos[k],
                          seq_len_out=seq[1 - k], free_pos_out=pos[1 - k], **m) for k in (0, 1)]
    status = status_word(dev)
    pool = torch.full((pages, layers * P, H.HD), 127, dtype=torch.uint8, device=dev)
    pool_scales = torch.full((pages, layers * P), float("nan"), device=dev)
    rows = [torch.zeros(R, H.HD, dtype=BF16, device=dev) for _ in range(layers)]
    win, q = torch.zeros(T, H.HD, dtype=BF16, device=dev), torch.zeros(T, heads, H.HD, dtype=BF16, device=dev)
    swa, swa_scales = torch.zeros(B, cap, H.HD, device=dev).to(F8), torch.zeros(B, cap, device=dev)
    out = [torch.zeros(T, heads, H.HD, device=dev) for _ in range(layers)]
    part = [(pool.view(F8)[:, i * P:(i + 1) * P], pool_scales[:, i * P:(i + 1) * P]) for i in range(layers)]
    jobs = csa.AppendJobsFp8([csa.AppendJobFp8(rows[i], m["row_slot"], *part[i], P) for i in range(layers)]
                             + [csa.AppendJobFp8(win, m["swa_slot"], swa, swa_scales, cap)])
    layout = csa.PagedLayoutFp8(m["tok_seq"], m["tok_pos"], m["row_len"], table, P, swa, swa_scales,
                                m["swa_first_pos"])
    prm = csa.params(heads, 1, 16, ratio)
    ws = csa.paged_workspace(layout, prm)

    def step(k):
        csa.csa_page_plan(plans[k], status)
        csa.csa_paged_append_fp8(jobs, status)
        for i in range(layers):
            csa.csa_paged_attention_fp8(layout, prm, *part[i], q, out[i], status, ws)

    graphs = []
    if captured:
        step(0)
        torch.cuda.synchronize()
        for k in (0, 1):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                step(k)
            graphs.append(g)
    held = [0] * B
    kept = [[[] for _ in range(B)] for _ in range(layers)]
    near = [[] for _ in range(B)]
    steps = [[9, 0, 23, 0, 1], [1, 30, 1, 0, 1], [1, 1, 1, 4, 1], [1, 1, -1, 1, 3], [8, 1, 6, 1, -1],
             [1, 1, 1, 1, 0], [1, -1, 1, 20, 17], [1, 1, 1, 1, 1], [1, 1, 1, 1, 1], [2, 1, 12, 1, 1]]
    pack = lambda x: F.values(*F.quantise(x.double().cpu().numpy()[None]))[0]
    for n_step, new in enumerate(steps):
        k = n_step % 2
        new_len.copy_(torch.tensor(new, dtype=torch.int32))
        for buf in (*rows, win, q):
            buf.copy_(torch.randn(buf.shape, device=dev).to(BF16))
        for o in out:
            o.fill_(7.0)
        graphs[k].replay() if captured else step(k)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        r = t = 0
        first = list(held)
        for b, n in enumerate(new):
            if n < 0:
                held[b], near[b] = 0, []
                for x in kept:
                    x[b] = []
                continue
            near[b] += [pack(win[t + i]) for i in range(n)]
            for _ in range((held[b] + n) // ratio - held[b] // ratio):
                for x, src in zip(kept, rows):
                    x[b].append(pack(src[r]))
                r += 1
            held[b] += n
            t += n
        t = 0
        for b, n in enumerate(new):
            for p in range(first[b], first[b] + max(n, 0)):
                for i in range(layers):
                    seen = kept[i][b][:p // ratio] + near[b][max(0, p - 15):p + 1]
                    v = torch.stack(seen)
                    ref = torch.softmax(prm.scale * q[t].double().cpu() @ v.T, 1) @ v
                    assert (out[i][t].double().cpu() - ref).norm() <= F.REL[F32] * ref.norm()
                t += 1
        for o in out:
            assert (o[t:] == 7).all()
    # every row that is held, read back through the table
    for i in range(layers):
        slots = [int(table[b, g // P]) * P + g % P for b in range(B) for g in range(len(kept[i][b]))]
        want = torch.stack([x for b in kept[i] for x in b])
        got = torch.zeros(len(slots), H.HD, dtype=BF16, device=dev)
        csa.csa_paged_read_fp8(*part[i], torch.tensor(slots, device=dev), got, status, P)
        assert torch.equal(got.double().cpu(), want)


def test_read_feeds_the_gathered_attention(cuda_device):
    # selected rows of an 8-bit cache into the buffer that csa_sparse_mqa_decode attends:
    # the same rows through the table give the same result
    dev = cuda_device
    p = F.PagedFp8(60, row_len=[128], tokens=[(0, 512)], heads=16, page_rows=8, window=0)
    layout, prm, codes, scales, q, _ = p.arguments(dev)
    j = torch.arange(128)
    slots = (p.table[0, j // 8].long() * 8 + j % 8).to(dev)
    buf = torch.zeros(1, 128 + 128, H.HD, dtype=BF16, device=dev)
    status = status_word(dev)
    csa.csa_paged_read_fp8(codes, scales, slots, buf[0, :128], status, 8)
    gathered = csa.params(16, 128, 128, 4)
    one = csa.Layout(p.tok_seq.to(dev), p.tok_pos.to(dev), torch.tensor([0, 128], device=dev),
                     torch.zeros(1, 128, H.HD, dtype=BF16, device=dev), torch.zeros(1, dtype=torch.int64, device=dev),
                     128)
    a, b = torch.empty(1, 16, H.HD, device=dev), torch.empty(1, 16, H.HD, device=dev)
    csa.csa_sparse_mqa_decode(gathered, q, buf, torch.tensor([128], dtype=torch.int32, device=dev), a, status,
                              csa.workspace(one, gathered))
    csa.csa_paged_attention_fp8(layout, prm, codes, scales, q, b, status, csa.paged_workspace(layout, prm))
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    ref = p.reference()
    F.check(b, ref, F32)
    F.check(a, ref, F32, rel=H.REL[F32])


def test_binding_refuses_the_other_kind_of_layout(cuda_device):
    p = F.PagedFp8(61, row_len=[20], tokens=[(0, 80)], heads=16)
    layout, prm, codes, scales, q, _ = p.arguments(cuda_device)
    out, status = torch.empty(1, 16, H.HD, device=cuda_device), status_word(cuda_device)
    ws = csa.paged_workspace(layout, prm)
    with pytest.raises(ValueError, match="8-bit"):
        csa.csa_paged_attention(layout, prm, codes.float().to(BF16), q, out, status, ws)
    other = csa.PagedLayout(*layout.tensors[:4], 16)
    with pytest.raises(ValueError, match="PagedLayoutFp8"):
        csa.csa_paged_attention_fp8(other, prm, codes, scales, q, out, status, ws)
    with pytest.raises(ValueError, match="swa_scales"):
        csa.PagedLayoutFp8(*layout.tensors[:4], 16, layout.tensors[4], None, layout.tensors[5])
    with pytest.raises(ValueError, match="swa_kv"):
        csa.PagedLayoutFp8(*layout.tensors[:4], 16, layout.tensors[4].float().to(BF16), layout.swa_scales,
                           layout.tensors[5])
    with pytest.raises(ValueError, match="swa_scales"):
        csa.PagedLayoutFp8(*layout.tensors[:4], 16, layout.tensors[4], layout.swa_scales[:, 1:], layout.tensors[5])


def test_these_calls_under_the_checked_build(cuda_device):
    import os
    import subprocess
    import sys

    from sparse_compressed_kv_gb300 import build as B

    B.build(checks=True)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
                        os.path.join("tests", "test_gpu_paged_fp8.py"), "-k",
                        "test_append or test_read or random_shapes or bad_pages or lists or serving"],
                       cwd=root, env=dict(os.environ, CSA_CHECKS="1"), capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and " passed" in r.stdout, (r.stdout + r.stderr)[-3000:]
