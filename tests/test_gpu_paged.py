"""Paged caches on the GPU: the plan against Python integers, the append bit
for bit, the attention against float64, and the three as one serving loop."""
import numpy as np
import pytest
import torch

from sparse_compressed_kv_gb300 import csa
from tests import paged_helpers as H
from tests.gpu_helpers import Guarded

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


# ---------------------------------------------------------------- plan

def run_plan(device, *, ratio, page_rows, swa_cap, **case):
    t = H.plan_tensors(device, **case)
    guards = {k: Guarded(v.shape, v.dtype, device) for k, v in t.items() if v.numel()}
    for k, g in guards.items():
        g.t.copy_(t[k])
        t[k] = g.t
    status = torch.zeros(1, dtype=torch.int32, device=device)
    plan = csa.PagePlan(ratio=ratio, page_rows=page_rows, swa_cap=swa_cap, **t)
    want, bad = H.plan_reference(ratio=ratio, page_rows=page_rows, swa_cap=swa_cap, **case)
    for _ in range(2):      # a step planned twice gives the same result
        csa.csa_page_plan(plan, status)
        torch.cuda.synchronize()
        assert int(status.item()) == bad
        for k, v in want.items():
            assert t[k].tolist() == v, k
        assert t["seq_len"].tolist() == case["seq_len"]
        assert all(g.intact() for g in guards.values())
    return want


@pytest.mark.parametrize("seed,B,ctx,new,over,ratio,page_rows,swa_cap,head", [
    (1, 1, 0, 1, 0, 4, 16, 128, 0),            # a request's first token: no block yet
    (2, 1, 5000, 700, 0, 1, 1, 128, 3),        # a page per row
    (3, 7, 300, 40, 0.3, 4, 3, 16, 11),        # pages that are no power of two; the ring wraps
    (4, 33, 2000, 9, 0.2, 128, 2, 128, 100),
    (5, 600, 100, 3, 0.1, 4, 64, 8, 5),        # more requests than threads
    (6, 40, 900, 0, 0.5, 4, 8, 128, 1),        # nothing new, half of them over
    (7, 5, 70000, 60000, 0, 4, 64, 8192, 9),   # long prompts
    (8, 8192, 8, 2, 0.1, 4, 2, 4, 7),          # the most requests a plan takes
])
def test_plan(cuda_device, seed, B, ctx, new, over, ratio, page_rows, swa_cap, head):
    rng = np.random.default_rng(seed)
    seq_len = rng.integers(0, ctx + 1, B).tolist()
    new_len = rng.integers(0, new + 1, B).tolist() if B > 1 else [max(1, new)]
    new_len = [-1 if rng.random() < over else n for n in new_len]
    max_pages = max(-(-((s + max(n, 0)) // ratio) // page_rows) for s, n in zip(seq_len, new_len)) + 2
    need = sum(-(-((s + n) // ratio) // page_rows) + (-(s // ratio) // page_rows)
               for s, n in zip(seq_len, new_len) if n > 0)
    table, ring, pos = H.pool(seed, seq_len, ratio=ratio, page_rows=page_rows, max_pages=max_pages,
                              extra=need + 2, head=head)
    T = sum(n for n in new_len if n > 0)
    R = sum((s + n) // ratio - s // ratio for s, n in zip(seq_len, new_len) if n > 0)
    run_plan(cuda_device, ratio=ratio, page_rows=page_rows, swa_cap=swa_cap, seq_len=seq_len,
             new_len=new_len, table=table, free_ring=ring, free_pos=pos, tok_cap=T + 5, row_cap=R + 3)


BASE = dict(ratio=4, page_rows=2, swa_cap=8, seq_len=[20, 7, 0], new_len=[9, -1, 5],
            table=[[0, 1, 2, -1], [3, -1, -1, -1], [-1] * 4], free_ring=[4, 5, 6, -1, -1, -1, -1],
            free_pos=[0, 3], tok_cap=14, row_cap=4)


@pytest.mark.parametrize("changes,bits", [
    (dict(), 0),
    (dict(free_pos=[0, 1]), csa.DEV_CAPACITY),                      # a page short
    (dict(new_len=[13, -1, 5], tok_cap=20, row_cap=9), 0),      # 33 tokens: 8 blocks, all 4 pages
    (dict(new_len=[17, -1, 5], tok_cap=30, row_cap=9), csa.DEV_CAPACITY),   # 9 blocks: past max_pages
    (dict(tok_cap=13), csa.DEV_CAPACITY),
    (dict(row_cap=2), csa.DEV_CAPACITY),
    (dict(tok_cap=0, row_cap=0), csa.DEV_CAPACITY),
    (dict(new_len=[9, -2, 5]), csa.DEV_BAD_LENGTH),
    (dict(seq_len=[20, 7, -1]), csa.DEV_BAD_LENGTH),
    (dict(seq_len=[20, 7, 1 << 48]), csa.DEV_BAD_LENGTH),
    (dict(free_pos=[3, 0]), csa.DEV_BAD_LAYOUT),
    (dict(free_pos=[-1, 2]), csa.DEV_BAD_LAYOUT),
    (dict(free_pos=[0, 7]), csa.DEV_BAD_LAYOUT),                    # more free pages than there are
])
def test_plan_refused_as_a_whole(cuda_device, changes, bits):
    want = run_plan(cuda_device, **{**BASE, **changes})
    _, bad = H.plan_reference(**{**BASE, **changes})
    assert bad == bits
    if bits:
        assert want["table"] == BASE["table"] and want["free_ring"] == BASE["free_ring"]


def test_plan_without_buffers_for_maps(cuda_device):
    # requests that bring nothing need no token or row arrays
    run_plan(cuda_device, **{**BASE, "new_len": [0, -1, 0], "tok_cap": 0, "row_cap": 0})


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("n,width,pitch,page_rows,stride,pages", [
    (1, 1024, 1024, 64, 64, 2), (5, 16, 16, 1, 1, 40), (37, 80, 80, 3, 5, 21),
    (300, 256, 272, 16, 24, 30), (2000, 1024, 1024, 64, 192, 40), (64, 4112, 8192, 7, 7, 12),
    (0, 1024, 1024, 64, 64, 2),
])
def test_append(cuda_device, n, width, pitch, page_rows, stride, pages):
    g = torch.Generator().manual_seed(n + width)
    rows = torch.randint(0, 256, (max(n, 1), pitch), dtype=torch.uint8, generator=g)[:n, :width]
    slots = torch.randperm(pages * page_rows, generator=g)[:n].long()
    slots[torch.rand(n, generator=g) < 0.2] = -1
    cache = Guarded((pages, stride, width), torch.uint8, cuda_device)
    before = torch.randint(0, 256, cache.t.shape, dtype=torch.uint8, generator=g)
    cache.t.copy_(before)
    want = before.clone()
    for i, s in enumerate(slots.tolist()):
        if s >= 0:
            want[s // page_rows, s % page_rows] = rows[i]
    src = torch.empty(max(n, 1), pitch, dtype=torch.uint8, device=cuda_device)[:n, :width]
    src.copy_(rows)
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    jobs = csa.AppendJobs([csa.AppendJob(src, slots.to(cuda_device), cache.t, page_rows)])
    csa.csa_paged_append(jobs, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and cache.intact()
    assert torch.equal(cache.t.cpu(), want)


def test_append_several_caches_and_bad_slots(cuda_device):
    dev = cuda_device
    g = torch.Generator(device=dev).manual_seed(3)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    jobs, caches, wants = [], [], []
    for k, (n, width, dt) in enumerate([(33, 512, BF16), (33, 128, BF16), (50, 512, BF16), (9, 80, torch.uint8)]):
        rows = torch.randint(0, 100, (n, width), device=dev, generator=g).to(dt)
        slots = torch.randperm(96, device=dev, generator=g)[:n]
        cache = torch.full((12, 11, width), 7, dtype=dt, device=dev)
        want = cache.clone()
        want[slots // 8, slots % 8] = rows
        if k == 2:      # past the pool: skipped, and said so
            want[slots[4] // 8, slots[4] % 8] = 7
            slots[4] = 96
        jobs.append(csa.AppendJob(rows, slots, cache, 8))
        caches.append(cache)
        wants.append(want)
    csa.csa_paged_append(csa.AppendJobs(jobs), status)
    torch.cuda.synchronize()
    assert int(status.item()) == csa.DEV_BAD_INDEX
    for c, w in zip(caches, wants):
        assert torch.equal(c, w)


# ---------------------------------------------------------------- attention

CASES = {
    # one token, one row, no window
    "one-row": dict(row_len=[1], tokens=[(0, 4)], window=0, heads=1),
    # a window alone (no block is visible yet), and a position inside it
    "window-only": dict(row_len=[0, 1], tokens=[(0, 2), (1, 3)], heads=16),
    "tiny": dict(row_len=[256], tokens=[(0, 1024)], heads=16, page_rows=64),
    "ragged": dict(row_len=[300, 0, 64, 63, 65, 7], tokens=[(0, 1200), (1, 3), (2, 256), (3, 255),
                                                            (4, 260), (5, 30)], heads=64),
    # rows held that the token does not see yet, several tokens of one sequence
    "draft": dict(row_len=[130, 40], tokens=[(0, 516), (0, 517), (0, 518), (0, 519), (1, 161), (1, 162)],
                  heads=64, page_rows=24, gap=8),
    "odd-pages": dict(row_len=[201, 90], tokens=[(0, 805), (1, 370)], heads=24, page_rows=7, gap=2),
    "page-of-one": dict(row_len=[70], tokens=[(0, 300)], heads=8, page_rows=1),
    "page-of-two": dict(row_len=[333, 21], tokens=[(0, 128 * 333), (1, 128 * 21 + 5)], ratio=128,
                        heads=64, page_rows=2, sinks=True),
    "heads-128": dict(row_len=[500, 77], tokens=[(0, 2000), (1, 310)], heads=128, page_rows=32,
                      sinks=True),
    "heads-65": dict(row_len=[129], tokens=[(0, 516)], heads=65, page_rows=8),
    "no-window": dict(row_len=[128, 0, 64], tokens=[(0, 512), (1, 3), (2, 100)], window=0, heads=40,
                      page_rows=40, sinks=True),
    "long": dict(row_len=[5000], tokens=[(0, 20000)], heads=64, page_rows=64),
    "wide-window": dict(row_len=[30], tokens=[(0, 700)], window=600, heads=32, page_rows=8),
    "padding": dict(row_len=[100, 50], tokens=[(0, 400), (-1, -1), (1, 200), (-1, 7)], heads=16),
    "many": dict(row_len=[(37 * i) % 190 for i in range(200)],
                 tokens=[(i, 4 * ((37 * i) % 190) + i % 4) for i in range(200)], heads=16, page_rows=8),
}


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("name", CASES)
def test_attention(cuda_device, name, dtype):
    p = H.Paged(len(name), **CASES[name])
    got, status = p.run(cuda_device, dtype)
    assert status == 0
    seen = [t for t, b in enumerate(p.tok_seq.tolist()) if b >= 0]
    H.check(got, p.reference(), dtype, seen)
    for t, b in enumerate(p.tok_seq.tolist()):
        if b < 0:       # padding: the output is left as it was
            assert (got[t] == 7).all()
    again, _ = p.run(cuda_device, dtype)
    assert torch.equal(got, again)      # bit for bit


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_attention_peaked_and_large_logits(cuda_device, dtype):
    # logits up to several hundred, rising along the rows: the running maximum
    # moves many times, and far rows weigh nothing
    p = H.Paged(5, row_len=[640], tokens=[(0, 2560)], heads=64, page_rows=64, window=0)
    j = torch.arange(640)
    at = (p.table[0, j // 64].long(), j % 64)
    p.cache[at] = (p.cache[at].float() * (1 + j[:, None] / 40)).to(BF16)
    p.q *= 4
    ref = p.reference()
    got, status = p.run(cuda_device, dtype)
    assert status == 0
    # a weight's relative error is its logit's absolute error: 32 accumulation
    # steps of 2^-23 of a logit below 1000, so 0.004; the rest is as in REL
    l = p.scale * p.q[0].double() @ p.rows_of(0).T
    assert 100 < float(l.max()) < 1000
    err = (got.double().cpu() - ref).norm(dim=2)
    assert (err <= (H.REL[dtype] + 2 * 1000 * 32 * 2 ** -23) * ref.norm(dim=2)).all()


@pytest.mark.parametrize("scale", [0.0, -0.05])
def test_attention_other_scales(cuda_device, scale):
    p = H.Paged(6, row_len=[150], tokens=[(0, 600)], heads=64, page_rows=16)
    p.scale = scale
    got, status = p.run(cuda_device, F32)
    assert status == 0
    H.check(got, p.reference(), F32)


@pytest.mark.parametrize("page_rows", [16, 6])
def test_attention_bad_pages_lengths_and_window(cuda_device, page_rows):
    P = page_rows
    p = H.Paged(7, row_len=[100, 40, 30, 25], tokens=[(0, 400), (1, 160), (2, 120), (3, 100)], heads=16,
                page_rows=P, window=32)
    pages = p.cache.shape[0]
    p.table[0, 1] = pages          # past the pool
    p.table[0, 3] = -1
    p.swa_first_pos[1] = 150       # the ring lost positions 129 .. 149
    p.row_len[3] = -3              # read as 0
    lost = set(range(P, 2 * P)) | set(range(3 * P, 4 * P))
    first = 160 - 32 + 1
    gone = {0: lost, 1: {40 + i for i in range(150 - first)}, 2: None, 3: None}
    got, status = p.run(cuda_device, F32)
    assert status == csa.DEV_BAD_INDEX | csa.DEV_MISSING_SWA | csa.DEV_BAD_LENGTH
    p.table.clamp_(0, pages - 1)
    p.row_len.clamp_(min=0)
    p.cache.nan_to_num_(0.0)       # the reference reads lost rows before it drops them
    H.check(got, p.reference(lambda t: gone[t]), F32)


def test_attention_layout_errors(cuda_device):
    p = H.Paged(8, row_len=[20, 20], tokens=[(0, 80), (1, 80), (0, 60)], heads=16, max_pages=2)
    p.tok_seq[1] = 2               # no such sequence
    p.tok_pos[2] = -1
    got, status = p.run(cuda_device, F32)
    assert status == csa.DEV_BAD_LAYOUT
    H.check(got, _only(p, 0), F32, [0])
    assert (got[1:] == 0).all()
    p = H.Paged(8, row_len=[32], tokens=[(0, 400)], heads=16, max_pages=2)
    p.row_len[0] = 33              # more rows than the table has room for
    got, status = p.run(cuda_device, F32)
    assert status == csa.DEV_CAPACITY
    p.row_len[0] = 32
    H.check(got, p.reference(), F32)


def _only(p, t):
    ref = torch.zeros(len(p.tok_seq), p.heads, H.HD, dtype=torch.float64)
    l = p.scale * p.q[t].double() @ p.rows_of(t).T
    ref[t] = torch.softmax(l, 1) @ p.rows_of(t)
    return ref


def test_attention_reads_nothing_else(cuda_device):
    # every value outside the rows of the definition, infinities among them
    p = H.Paged(9, row_len=[83, 5], tokens=[(0, 290), (1, 17)], heads=16, page_rows=8)
    a, _ = p.run(cuda_device, F32)
    p.cache[p.cache.isnan()] = float("inf")
    n = 290 // 4                   # rows 72 .. 82 are held, but not visible to token 0
    j = torch.arange(n, 83)
    p.cache[p.table[0, j // 8].long(), j % 8] = float("nan")
    x = torch.arange(290 - 127, 291)
    cap = p.swa_kv.shape[1]
    unseen = torch.ones(cap, dtype=torch.bool)
    unseen[x % cap] = False
    p.swa_kv[0, unseen] = float("nan")
    p.swa_kv[1, 18:] = float("nan")
    b, status = p.run(cuda_device, F32)
    assert status == 0 and torch.equal(a, b)


def test_attention_cache_beyond_32_bit_offsets(cuda_device):
    # pages at the end of a pool of more than 4 GiB: 2.2 G values
    dev = cuda_device
    p = H.Paged(10, row_len=[150], tokens=[(0, 600)], heads=16, page_rows=64, window=0)
    pages, stride = 33700, 128
    cache = torch.empty(pages, stride, H.HD, dtype=BF16, device=dev)
    far = torch.tensor([pages - 1, 0, pages // 2 + 1])
    cache[far.to(dev), :64] = p.cache[p.table[0, :3].long()].to(dev)
    table = torch.full_like(p.table, -1)
    table[0, :3] = far
    layout = csa.PagedLayout(p.tok_seq.to(dev), p.tok_pos.to(dev), p.row_len.to(dev), table.to(dev), 64)
    prm = csa.params(16, 1, 0, 4)
    out = torch.empty(1, 16, H.HD, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    csa.csa_paged_attention(layout, prm, cache, p.q.to(dev), out, status, csa.paged_workspace(layout, prm))
    # and the append at the far end
    slots = torch.tensor([(pages - 1) * 64 + 63], device=dev)
    row = torch.full((1, H.HD), 3.0, dtype=BF16, device=dev)
    csa.csa_paged_append(csa.AppendJobs([csa.AppendJob(row, slots, cache, 64)]), status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    H.check(out, p.reference(), F32)
    assert (cache[pages - 1, 63] == 3).all()


def test_attention_long_rows_in_one_cta(cuda_device):
    # so many tokens that each is one CTA's work: long sums, held in f32
    dev, n, T = cuda_device, 20000, 320
    g = torch.Generator(device=dev).manual_seed(11)
    cache = torch.randn(n // 32, 32, H.HD, device=dev, generator=g).to(BF16)
    q = torch.randn(T, 64, H.HD, device=dev, generator=g).to(BF16)
    table = torch.randperm(n // 32, device=dev, generator=g).int()[None]
    pos = 4 * (n - torch.arange(T, device=dev) * 7)
    layout = csa.PagedLayout(torch.zeros(T, dtype=torch.int32, device=dev), pos,
                             torch.tensor([n], device=dev), table, 32)
    prm = csa.params(64, 1, 0, 4)
    ws = csa.paged_workspace(layout, prm)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    rows = cache[table[0].long()].reshape(-1, H.HD).double()
    for dtype in (F32, BF16):
        out = torch.empty(T, 64, H.HD, device=dev, dtype=dtype)
        csa.csa_paged_attention(layout, prm, cache, q, out, status, ws)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        for t in range(0, T, 37):
            m = int(pos[t]) // 4
            ref = torch.softmax(prm.scale * q[t].double() @ rows[:m].T, 1) @ rows[:m]
            assert (out[t].double() - ref).norm() <= H.REL[dtype] * ref.norm()


@pytest.mark.parametrize("T,n", [
    (100, 640),      # a whole token a CTA
    (60, 400),       # two CTAs a token, half of the columns each
    (30, 300),       # four
    (1, 20000),      # one token over all CTAs, three chunks each
    (160, 3000),     # long stretches, rounded into the partial on the way
], ids=str)
def test_attention_rising_maximum(cuda_device, T, n):
    # rows in steps of 48 whose logits rise by more than the rescaling's threshold,
    # so that what a CTA has accumulated is rescaled, and still counts
    dev = cuda_device
    g = torch.Generator(device=dev).manual_seed(T)
    rows = torch.randn(n, H.HD, device=dev, generator=g)
    rows = (rows * (2 + 2.2 * (torch.arange(n, device=dev) % 144 // 48))[:, None]).to(BF16)
    pages = -(-n // 16)
    table = torch.randperm(pages, device=dev, generator=g).int()[None]
    cache = torch.full((pages, 16, H.HD), float("nan"), device=dev, dtype=BF16)
    j = torch.arange(n, device=dev)
    cache[table[0, j // 16].long(), j % 16] = rows
    q = torch.randn(T, 64, H.HD, device=dev, generator=g).to(BF16)
    layout = csa.PagedLayout(torch.zeros(T, dtype=torch.int32, device=dev),
                             torch.full((T,), 4 * n, dtype=torch.int64, device=dev),
                             torch.tensor([n], device=dev), table, 16)
    prm = csa.params(64, 1, 0, 4)
    ws = csa.paged_workspace(layout, prm)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    for dtype in (F32, BF16):
        out = torch.empty(T, 64, H.HD, device=dev, dtype=dtype)
        csa.csa_paged_attention(layout, prm, cache, q, out, status, ws)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        for t in range(0, T, max(1, T // 12)):
            l = prm.scale * q[t].double() @ rows.double().T
            assert 20 < float(l.max()) < 40
            ref = torch.softmax(l, 1) @ rows.double()
            # a weight's relative error is its logit's absolute error: 32
            # accumulation steps of 2^-23 of at most 40, in weights and their sum
            tol = H.REL[dtype] + 2 * 40 * 32 * 2 ** -23
            err = (out[t].double() - ref).norm(dim=1) / ref.norm(dim=1)
            assert float(err.max()) <= tol, f"token {t}: off by {float(err.max()):.3e}"


@pytest.mark.parametrize("long", [150, 3000], ids=["whole", "cut"])
def test_attention_more_tokens_than_a_cta_lists(cuda_device, long):
    # mostly padding, so that one CTA's range holds more than a hundred tokens; real
    # ones and ones without rows among them, and one long enough to be cut
    dev, T, heads = cuda_device, 8192, 65
    g = torch.Generator(device=dev).manual_seed(long)
    n = [150, long]
    pages = [-(-x // 16) for x in n]
    table = torch.full((2, max(pages)), -1, dtype=torch.int32, device=dev)
    table[0, :pages[0]] = torch.arange(pages[0], device=dev)
    table[1, :pages[1]] = pages[0] + torch.arange(pages[1], device=dev)
    cache = torch.randn(sum(pages), 16, H.HD, device=dev, generator=g).to(BF16)
    q = torch.randn(T, heads, H.HD, device=dev, generator=g).to(BF16)
    i = torch.arange(T)
    seq, pos = torch.full((T,), -1, dtype=torch.int32), torch.full((T,), -1, dtype=torch.int64)
    real, empty = i % 41 == 7, i % 64 == 3
    seq[real | empty] = 0
    pos[real] = 4 * (i[real] % 150 + 1)
    pos[empty] = 3
    seq[5000], pos[5000] = 1, 4 * long
    layout = csa.PagedLayout(seq.to(dev), pos.to(dev), torch.tensor(n, device=dev), table, 16)
    prm = csa.params(heads, 1, 0, 4)
    ws = csa.paged_workspace(layout, prm)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    held = [cache[table[b, :pages[b]].long()].reshape(-1, H.HD)[:n[b]].double() for b in range(2)]
    for dtype in (F32, BF16):
        out = torch.full((T, heads, H.HD), 7.5, device=dev, dtype=dtype)
        csa.csa_paged_attention(layout, prm, cache, q, out, status, ws)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        assert bool((out[(seq < 0).to(dev)] == 7.5).all())
        for t in (seq >= 0).nonzero()[:, 0].tolist():
            rows = held[int(seq[t])][:int(pos[t]) // 4]
            if len(rows) == 0:
                assert bool((out[t] == 0).all())
                continue
            ref = torch.softmax(prm.scale * q[t].double() @ rows.T, 1) @ rows
            assert (out[t].double() - ref).norm() <= H.REL[dtype] * ref.norm(), t


def test_attention_on_another_stream(cuda_device):
    p = H.Paged(12, row_len=[500, 300], tokens=[(0, 2000), (1, 1200)], heads=64)
    a, _ = p.run(cuda_device, BF16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b, status = p.run(cuda_device, BF16, stream=s)
    assert status == 0 and torch.equal(a, b)


@pytest.mark.parametrize("seed", range(24))
def test_attention_random_shapes(cuda_device, seed):
    # token counts around the number of CTAs, any page size, heads and window
    rng = np.random.default_rng(100 + seed)
    B = int(rng.choice([1, 2, 5, 40, 151, 152, 153, 170]))
    new = int(rng.choice([1, 1, 2, 3]))
    ratio = int(rng.choice([1, 4, 128]))
    most = int(rng.choice([3, 70, 400, 1500])) if B < 100 else int(rng.choice([3, 70, 400]))
    ctx = [int(rng.integers(0, most + 1)) * ratio + int(rng.integers(0, ratio)) for _ in range(B)]
    p = H.Paged(seed, row_len=[(c + new) // ratio for c in ctx],
                tokens=[(b, ctx[b] + i) for b in range(B) for i in range(new)], ratio=ratio,
                page_rows=int(rng.choice([1, 2, 3, 8, 12, 16, 50, 64, 128])), gap=int(rng.choice([0, 8, 3])),
                heads=int(rng.choice([1, 3, 8, 16, 33, 64, 100])) if B < 100 else 8,
                window=int(rng.choice([0, 1, 20, 128])), sinks=bool(rng.integers(2)))
    dtype = [F32, BF16][seed % 2]
    got, status = p.run(cuda_device, dtype)
    assert status == 0
    tokens = sorted(set(rng.integers(0, B * new, 40).tolist()) | {0, B * new - 1})
    H.check(got, p.reference(tokens=tokens), dtype, tokens)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_attention_thousands_of_tokens_and_one_long(cuda_device, dtype):
    # so many short tokens that a CTA lists them in several turns, cut by a long one
    long = 30000
    tokens = [(0, 4 * (i % 13) + i % 4) for i in range(2500)] + [(1, 4 * long)] + \
             [(2, i % 4) if i % 3 else (-1, -1) for i in range(2600)]
    p = H.Paged(30, row_len=[12, long, 0], tokens=tokens, heads=8, page_rows=32, window=4, swa_cap=60)
    p.swa_first_pos[1] = 4 * long - 50
    got, status = p.run(cuda_device, dtype)
    assert status == 0
    check = [0, 1, 7, 51, 1234, 2499, 2500, 2502, 2503, 4000, 5098, 5099, 5100]
    check = [t for t in check if tokens[t][0] >= 0]
    H.check(got, p.reference(tokens=check), dtype, check)
    pad = torch.tensor([b < 0 for b, _ in tokens])
    assert (got.cpu()[pad] == 7).all() and not got.isnan().any()


def test_attention_far_positions(cuda_device):
    # positions past 2^32: their slots in the ring and their blocks
    far = (1 << 33) + 12345
    p = H.Paged(31, row_len=[90, 7], tokens=[(0, far), (1, far * 5)], heads=16, window=50)
    got, status = p.run(cuda_device, F32)
    assert status == 0
    H.check(got, p.reference(), F32)


def test_attention_shared_pages(cuda_device):
    # a prefix that two requests share: the same pages in two rows of the table
    p = H.Paged(32, row_len=[96, 96, 40], tokens=[(0, 400), (1, 390), (2, 170)], heads=32, page_rows=16)
    p.table[1, :4] = p.table[0, :4]
    p.table[2, :2] = p.table[0, 2:4]
    got, status = p.run(cuda_device, BF16)
    assert status == 0
    H.check(got, p.reference(), BF16)


def test_attention_two_streams_at_once(cuda_device):
    dev = cuda_device
    ps = [H.Paged(40 + i, row_len=[4000, 300 * i], tokens=[(0, 16000), (1, 1200 * i)], heads=64, page_rows=32)
          for i in range(2)]
    alone = [p.run(dev, F32)[0].clone() for p in ps]
    args, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for p in ps:
        layout = csa.PagedLayout(p.tok_seq.to(dev), p.tok_pos.to(dev), p.row_len.to(dev), p.table.to(dev),
                                 32, p.swa_kv.to(dev), p.swa_first_pos.to(dev))
        prm = csa.params(64, 1, 128, 4)
        args.append((layout, prm, p.cache.to(dev), p.q.to(dev), torch.empty(2, 64, H.HD, device=dev),
                     torch.zeros(1, dtype=torch.int32, device=dev), csa.paged_workspace(layout, prm)))
    torch.cuda.synchronize()
    for _ in range(20):
        for a, s in zip(args, streams):
            csa.csa_paged_attention(*a, stream=s)
    torch.cuda.synchronize()
    for a, want in zip(args, alone):
        assert int(a[5].item()) == 0 and torch.equal(a[4], want)


def test_attention_replayed_with_other_lengths(cuda_device):
    # captured once; lengths, tables and contents change between replays, from
    # whole tokens a CTA to one token cut over all of them
    dev = cuda_device
    lens = [[3, 5], [6000, 0], [700, 900], [0, 0], [64, 6000]]
    ps = [H.Paged(50 + i, row_len=n, tokens=[(0, 4 * n[0] + 1), (1, 4 * n[1] + 3)], heads=64, page_rows=32,
                  max_pages=200, spare_pages=250 - sum(-(-x // 32) for x in n)) for i, n in enumerate(lens)]
    bufs = [x.to(dev).clone() for x in (ps[0].tok_seq, ps[0].tok_pos, ps[0].row_len, ps[0].table,
                                        ps[0].swa_kv, ps[0].swa_first_pos, ps[0].cache, ps[0].q)]
    layout = csa.PagedLayout(*bufs[:4], 32, *bufs[4:6])
    prm = csa.params(64, 1, 128, 4)
    ws, out = csa.paged_workspace(layout, prm), torch.empty(2, 64, H.HD, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    csa.csa_paged_attention(layout, prm, bufs[6], bufs[7], out, status, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        csa.csa_paged_attention(layout, prm, bufs[6], bufs[7], out, status, ws)
    for p in ps:
        for b, x in zip(bufs, (p.tok_seq, p.tok_pos, p.row_len, p.table, p.swa_kv, p.swa_first_pos, p.cache, p.q)):
            b.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        H.check(out, p.reference(), F32)


# ---------------------------------------------------------------- as a serving loop

class Server:
    """Requests over one CSA-like layer: packed reference caches beside the
    paged ones."""

    def __init__(self, device, B, ratio, page_rows, swa_cap, heads=16, pages=64, max_pages=24,
                 tok_cap=64, row_cap=32, layers=2):
        i64 = lambda *x: torch.zeros(*x, dtype=torch.int64, device=device)
        self.dev, self.B, self.ratio, self.P, self.cap = device, B, ratio, page_rows, swa_cap
        self.heads, self.tok_cap, self.row_cap = heads, tok_cap, row_cap
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.seq = [i64(B), i64(B)]
        self.pos = [torch.tensor([0, pages], device=device), i64(2)]
        self.new_len = torch.zeros(B, dtype=torch.int32, device=device)
        self.table = torch.full((B, max_pages), -1, dtype=torch.int32, device=device)
        self.ring = torch.randperm(pages, device=device).int()
        self.row_len, self.first = i64(B), i64(B)
        self.tok_seq = torch.zeros(tok_cap, dtype=torch.int32, device=device)
        self.tok_pos, self.swa_slot, self.row_slot = i64(tok_cap), i64(tok_cap), i64(row_cap)
        self.tok_off, self.row_off = i64(B + 1), i64(B + 1)
        pool = torch.full((pages, layers * page_rows, H.HD), float("nan"), dtype=BF16, device=device)
        # two layers interleaved in one pool of pages: views with a stride
        self.pool = pool
        self.swa = torch.zeros(B, swa_cap, H.HD, dtype=BF16, device=device)
        self.rows = torch.zeros(row_cap, H.HD, dtype=BF16, device=device)
        self.win = torch.zeros(tok_cap, H.HD, dtype=BF16, device=device)
        self.q = torch.zeros(tok_cap, heads, H.HD, dtype=BF16, device=device)
        self.out = torch.zeros(tok_cap, heads, H.HD, device=device)
        self.plans = [csa.PagePlan(
            ratio=ratio, page_rows=page_rows, swa_cap=swa_cap, seq_len=self.seq[k],
            new_len=self.new_len, table=self.table, free_ring=self.ring, free_pos=self.pos[k],
            seq_len_out=self.seq[1 - k], row_len=self.row_len, swa_first_pos=self.first,
            free_pos_out=self.pos[1 - k], tok_off=self.tok_off, row_off=self.row_off,
            tok_seq=self.tok_seq, tok_pos=self.tok_pos, swa_slot=self.swa_slot,
            row_slot=self.row_slot) for k in (0, 1)]
        self.jobs = csa.AppendJobs([csa.AppendJob(self.rows, self.row_slot, pool, page_rows),
                                    csa.AppendJob(self.win, self.swa_slot, self.swa, swa_cap)])
        self.layout = csa.PagedLayout(self.tok_seq, self.tok_pos, self.row_len, self.table,
                                      page_rows, self.swa, self.first)
        self.prm = csa.params(heads, 1, 16, ratio)
        self.ws = csa.paged_workspace(self.layout, self.prm)

    def step(self, k):
        csa.csa_page_plan(self.plans[k], self.status)
        csa.csa_paged_append(self.jobs, self.status)
        csa.csa_paged_attention(self.layout, self.prm, self.pool, self.q, self.out, self.status,
                                self.ws)


def serve(device, captured):
    torch.manual_seed(20)
    B, ratio, P, cap = 5, 4, 3, 40
    s = Server(device, B, ratio, P, cap)
    steps = [[9, 0, 23, 0, 1], [1, 30, 1, 0, 1], [1, 1, 1, 4, 1], [1, 1, -1, 1, 3], [8, 1, 6, 1, -1],
             [1, 1, 1, 1, 0], [1, -1, 1, 20, 17], [1, 1, 1, 1, 1], [1, 1, 1, 1, 1], [2, 1, 12, 1, 1]]
    graphs = []
    if captured:
        s.step(0)                       # warm: nothing is new yet
        torch.cuda.synchronize()
        for k in (0, 1):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                s.step(k)
            graphs.append(g)
    held = [0] * B
    rows = [[] for _ in range(B)]       # the packed reference
    win = [[] for _ in range(B)]
    taken = []
    for i, new in enumerate(steps):
        k = i % 2
        s.new_len.copy_(torch.tensor(new, dtype=torch.int32))
        for buf in (s.rows, s.win, s.q):
            buf.copy_(torch.randn(buf.shape, device=device).to(BF16))
        s.out.fill_(7.0)
        graphs[k].replay() if captured else s.step(k)
        torch.cuda.synchronize()
        assert int(s.status.item()) == 0
        r = t = 0
        tok_seq, tok_pos = [], []
        for b, n in enumerate(new):
            if n < 0:
                held[b], rows[b], win[b] = 0, [], []
                continue
            for x in range(held[b], held[b] + n):
                win[b].append(s.win[t])
                tok_seq.append(b)
                tok_pos.append(x)
                t += 1
            for _ in range((held[b] + n) // ratio - held[b] // ratio):
                rows[b].append(s.rows[r].clone())
                r += 1
            win[b] = [w.clone() for w in win[b]]
            held[b] += n
        assert s.tok_seq[:t].tolist() == tok_seq and s.tok_pos[:t].tolist() == tok_pos
        assert (s.tok_seq[t:] == -1).all() and (s.out[t:] == 7).all()
        assert s.seq[1 - k].tolist() == held
        # the packed path on the same rows
        off = [0]
        for b in range(B):
            off.append(off[-1] + len(rows[b]))
        packed = torch.stack([x for b in rows for x in b] or [s.rows[0]])
        ring = torch.zeros_like(s.swa)
        for b in range(B):
            for x in range(max(0, held[b] - cap), held[b]):
                ring[b, x % cap] = win[b][x]
        first = torch.tensor([max(0, h - cap) for h in held], device=device)
        L = csa.Layout(s.tok_seq[:t].contiguous(), s.tok_pos[:t].contiguous(),
                       torch.tensor(off, device=device), ring, first, max(1, max(map(len, rows))),
                       packed.shape[0])
        ref = torch.empty(t, s.heads, H.HD, device=device)
        csa.csa_hca_decode(L, s.prm, packed, s.q[:t].contiguous(), ref, s.status,
                           csa.hca_workspace(L, s.prm))
        torch.cuda.synchronize()
        assert int(s.status.item()) == 0
        # both are f32 results of the same sums: each within REL of the value
        err = (s.out[:t] - ref).double().norm(dim=(1, 2))
        assert (err <= 2 * H.REL[F32] * ref.double().norm(dim=(1, 2))).all()
        taken.append(s.out[:t].clone())
    # no page is lost or held twice
    head, tail = s.pos[len(steps) % 2].tolist()
    free = [s.ring.tolist()[x % 64] for x in range(head, tail)]
    used = [p for b in range(B) for p in s.table[b, :-(-(held[b] // ratio) // P)].tolist()]
    assert sorted(free + used) == list(range(64))
    return taken


def test_serving_loop_matches_the_packed_path(cuda_device):
    serve(cuda_device, captured=False)


def test_serving_loop_captured(cuda_device):
    # two captured steps that share a workspace, replayed in turn
    serve(cuda_device, captured=True)


def test_paged_calls_under_the_checked_build(cuda_device):
    """The library with internal bounds checks: a failed one sets a status bit,
    and every test wants the status it expects."""
    import os
    import subprocess
    import sys

    from sparse_compressed_kv_gb300 import build as B

    B.build(checks=True)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
                        os.path.join("tests", "test_gpu_paged.py"), "-k",
                        "test_plan or test_append or random_shapes or bad_pages or thousands or serving"],
                       cwd=root, env=dict(os.environ, CSA_CHECKS="1"), capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and " passed" in r.stdout, (r.stdout + r.stderr)[-3000:]
