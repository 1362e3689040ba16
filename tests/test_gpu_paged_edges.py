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


@pytest.mark.parametrize("width,page_rows,gap", [(1024, 16, 0), (80, 3, 2)])
def test_append_to_one_layer_of_interleaved_pages(cuda_device, width, page_rows, gap):
    dev, pages, P, layers = cuda_device, 9, page_rows, 3
    g = torch.Generator(device=dev).manual_seed(width)
    pool = torch.randint(0, 256, (pages, layers * P + gap, width), dtype=torch.uint8, device=dev, generator=g)
    want, jobs, status = pool.clone(), [], torch.zeros(1, dtype=torch.int32, device=dev)
    for k in (0, 2):                # the layer between them, and the gap, stay as they are
        n = 2 * pages * P // 3
        rows = torch.randint(0, 256, (n, width), dtype=torch.uint8, device=dev, generator=g)
        slots = torch.randperm(pages * P, device=dev, generator=g)[:n]
        jobs.append(csa.AppendJob(rows, slots, pool[:, k * P:(k + 1) * P], P))
        want[slots // P, k * P + slots % P] = rows
    csa.csa_paged_append(csa.AppendJobs(jobs), status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and torch.equal(pool, want)


@pytest.mark.parametrize("page_rows", [16, 6])
def test_attention_over_one_layer_of_interleaved_pages(cuda_device, page_rows):
    # three layers' rows under the same page numbers; each call sees its own
    dev, P, layers = cuda_device, page_rows, 3
    ps = [H.Paged(60 + k, row_len=[210, 77], tokens=[(0, 850), (1, 320)], heads=24, page_rows=P, window=40)
          for k in range(layers)]
    pages = ps[0].cache.shape[0]
    pool = torch.full((pages, layers * P, H.HD), float("nan"), dtype=BF16, device=dev)
    for k, p in enumerate(ps):
        for b, n in enumerate([210, 77]):                   # one table for all layers
            j = torch.arange(n)
            pool[ps[0].table[b, j // P].long(), k * P + j % P] = p.cache[p.table[b, j // P].long(), j % P].to(dev)
    for k, p in enumerate(ps):
        layout = csa.PagedLayout(p.tok_seq.to(dev), p.tok_pos.to(dev), p.row_len.to(dev), ps[0].table.to(dev), P,
                                 p.swa_kv.to(dev), p.swa_first_pos.to(dev))
        prm = csa.params(24, 1, 40, 4)
        out, status = torch.empty(2, 24, H.HD, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
        csa.csa_paged_attention(layout, prm, pool[:, k * P:(k + 1) * P], p.q.to(dev), out, status,
                                csa.paged_workspace(layout, prm))
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        H.check(out, p.reference(), F32)


def test_serving_step_over_two_layers_of_interleaved_pages(cuda_device):
    # one plan a step for both layers; each layer's rows appended to and read from
    # its own half of every page
    dev, P, heads, ratio, cap, steps = cuda_device, 5, 16, 4, 24, [17, 1, 1, 30, 1, 4, 1]
    pages, tok_cap, row_cap = 20, 32, 10
    i64 = lambda *x: torch.zeros(*x, dtype=torch.int64, device=dev)
    seq, pos = [i64(1), i64(1)], [torch.tensor([0, pages], device=dev), i64(2)]
    new_len = torch.zeros(1, dtype=torch.int32, device=dev)
    table = torch.full((1, 8), -1, dtype=torch.int32, device=dev)
    ring = torch.randperm(pages, device=dev).int()
    row_len, first, tok_off, row_off = i64(1), i64(1), i64(2), i64(2)
    tok_seq = torch.zeros(tok_cap, dtype=torch.int32, device=dev)
    tok_pos, swa_slot, row_slot = i64(tok_cap), i64(tok_cap), i64(row_cap)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    plans = [csa.PagePlan(ratio=ratio, page_rows=P, swa_cap=cap, seq_len=seq[k], new_len=new_len, table=table,
                          free_ring=ring, free_pos=pos[k], seq_len_out=seq[1 - k], row_len=row_len,
                          swa_first_pos=first, free_pos_out=pos[1 - k], tok_off=tok_off, row_off=row_off,
                          tok_seq=tok_seq, tok_pos=tok_pos, swa_slot=swa_slot, row_slot=row_slot) for k in (0, 1)]
    pool = torch.full((pages, 2 * P, H.HD), float("nan"), dtype=BF16, device=dev)
    prm = csa.params(heads, 1, 16, ratio)
    parts = [pool[:, :P], pool[:, P:]]
    swa = [torch.zeros(1, cap, H.HD, dtype=BF16, device=dev) for _ in parts]
    held = [[], []]
    win = [[], []]
    for i, n in enumerate(steps):
        g = torch.Generator(device=dev).manual_seed(i)
        randn = lambda *x: torch.randn(*x, device=dev, generator=g).to(BF16)
        new_len.fill_(n)
        csa.csa_page_plan(plans[i % 2], status)
        T = sum(steps[:i + 1])
        for k, cache in enumerate(parts):
            rows, near, q = randn(row_cap, H.HD), randn(tok_cap, H.HD), randn(tok_cap, heads, H.HD)
            csa.csa_paged_append(csa.AppendJobs([csa.AppendJob(rows, row_slot, cache, P),
                                                 csa.AppendJob(near, swa_slot, swa[k], cap)]), status)
            layout = csa.PagedLayout(tok_seq, tok_pos, row_len, table, P, swa[k], first)
            out = torch.full((tok_cap, heads, H.HD), 7.0, device=dev)
            csa.csa_paged_attention(layout, prm, cache, q, out, status, csa.paged_workspace(layout, prm))
            held[k] += list(rows[:T // ratio - (T - n) // ratio].double())
            win[k] += list(near[:n].double())
            torch.cuda.synchronize()
            # the last token alone: older ones of a long step may have lost their window
            p = T - 1
            every = torch.stack(held[k][:p // ratio] + win[k][max(0, p - 15):p + 1])
            ref = torch.softmax(prm.scale * q[n - 1].double() @ every.T, 1) @ every
            assert (out[n - 1].double() - ref).norm() <= H.REL[F32] * ref.norm()
            assert (out[n:] == 7).all()
        # (the ring holds the newest 24 positions: a step of 30 tokens pushes out what
        # the first of them would see)
        lost = max(0, T - n - 15) < max(0, T - cap)
        assert int(status.item()) == (csa.DEV_MISSING_SWA if lost else 0)
        status.zero_()


def run_plan(device, *, ratio, page_rows, swa_cap, **case):
    t = H.plan_tensors(device, **case)
    status = torch.zeros(1, dtype=torch.int32, device=device)
    csa.csa_page_plan(csa.PagePlan(ratio=ratio, page_rows=page_rows, swa_cap=swa_cap, **t), status)
    torch.cuda.synchronize()
    want, bad = H.plan_reference(ratio=ratio, page_rows=page_rows, swa_cap=swa_cap, **case)
    return {k: t[k].tolist() for k in want}, int(status.item()), want, bad


@pytest.mark.parametrize("number", [-1, 9, 1 << 30, -(1 << 31)])
@pytest.mark.parametrize("new", [6, 30], ids=["few", "many"])
@pytest.mark.parametrize("where", ["old", "ring", "given-back"])
def test_plan_page_numbers_outside_the_pool(cuda_device, where, new, number):
    # request 0 holds 9 blocks in pages 0, 1, 2 (of 4 rows; the last holds one) and
    # brings some; request 1 ends and gives back pages 3 and 4
    table = [[0, 1, 2] + [-1] * 5, [3, 4] + [-1] * 6]
    ring = [5, 6, 7, 8] + [-1] * 5
    if where == "old":
        table[0][2] = number
    elif where == "ring":
        ring[0] = number
    else:
        table[1][1] = number
    case = dict(ratio=2, page_rows=4, swa_cap=8, seq_len=[18, 16], new_len=[new, -1], table=table, free_ring=ring,
                free_pos=[0, 4], tok_cap=45, row_cap=25)
    if where == "ring":
        case["new_len"][0] = new = max(new, 8)          # reaches the ring's first page
    got, status, want, bad = run_plan(cuda_device, **case)
    assert bad == 0 and status == csa.DEV_BAD_INDEX
    # the rows of that page have no slot; all else is as always, the number among it
    want["row_slot"] = [s if 0 <= s < 9 * 4 else -1 for s in want["row_slot"]]
    assert (-1 in want["row_slot"][:new // 2]) == (where != "given-back")
    assert got == want


def test_plan_leaves_other_numbers_alone(cuda_device):
    # a full old page, a table behind the request's pages and a ring behind the free
    # ones may hold anything
    case = dict(ratio=2, page_rows=4, swa_cap=8, seq_len=[16, 0], new_len=[4, 0], table=[[99, -5, -6], [77, -1, 55]],
                free_ring=[5, 1, -9, 1 << 30, 66, 7], free_pos=[0, 2], tok_cap=6, row_cap=4)
    got, status, want, bad = run_plan(cuda_device, **case)
    assert status == bad == 0 and got == want


def test_plan_with_a_shared_prefix(cuda_device):
    # two requests share the full pages 0 and 1; one of them ends as the header says:
    # by the caller, who puts back what the other does not hold
    step = dict(ratio=1, page_rows=2, swa_cap=4, tok_cap=4, row_cap=4)
    table, ring, N = [[0, 1, 2, -1], [0, 1, 3, -1]], [4, 5, 6, 7, -1, -1, -1, -1], 8
    got, status, want, bad = run_plan(cuda_device, seq_len=[6, 5], new_len=[1, 2], table=table, free_ring=ring,
                                      free_pos=[0, 4], **step)
    assert status == bad == 0 and got == want
    assert len(set(got["row_slot"][:3])) == 3 and got["table"] == [[0, 1, 2, 4], [0, 1, 3, 5]]
    head, tail = got["free_pos_out"]
    ring, own = got["free_ring"], [3, 5]
    for page in own:
        ring[tail % N] = page
        tail += 1
    got, status, want, bad = run_plan(cuda_device, seq_len=[got["seq_len_out"][0], 0], new_len=[1, 3],
                                      table=got["table"], free_ring=ring, free_pos=[head, tail], **step)
    assert status == bad == 0 and got == want
    head, tail = got["free_pos_out"]
    held = got["table"][0][:4] + got["table"][1][:2]
    free = [got["free_ring"][x % N] for x in range(head, tail)]
    assert sorted(held + free) == list(range(N))


@pytest.mark.parametrize("n", [1, 4, 40])
def test_attention_ring_for_several_tokens_a_step(cuda_device, n):
    # window + n - 1 slots hold every window of a step; one less loses a row of the first
    W, end = 20, 500 + n
    tokens = [(0, 500 + i) for i in range(n)]
    for cap, want in ((W + n - 1, 0), (W + n - 2, csa.DEV_MISSING_SWA)):
        if cap < W:
            continue
        p = H.Paged(70 + n, row_len=[end // 4], tokens=tokens, heads=16, window=W, swa_cap=cap)
        got, status = p.run(cuda_device, F32)
        assert status == want
        H.check(got, p.reference(lambda t: {(500 + t) // 4} if want and t == 0 else None), F32)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("row_len,tokens", [
    ([300], [(0, 1200)]),                                    # whole tokens
    ([20000], [(0, 80000)]),                                 # one token in many parts
    ([3000] * 14, [(b, 12000) for b in range(14)]),          # many tokens in a few parts
    ([9000] * 3, [(b, 36000) for b in range(3)]),            # a few tokens in many parts
], ids=["whole", "one", "many", "few"])
def test_attention_sinks_of_any_value(cuda_device, row_len, tokens, dtype):
    p = H.Paged(80, row_len=row_len, tokens=tokens, heads=9, page_rows=64, sinks=True)
    p.sinks[:] = torch.tensor([0.0, float("nan"), float("inf"), -float("inf"), 30.0, 80.0, -80.0, -1e30, 1e30])
    got, status = p.run(cuda_device, dtype)
    assert status == 0
    got, ref = got.double().cpu(), p.reference()
    assert got[:, 1].isnan().all() and ref[:, 1].isnan().all()
    for h in (2, 8):
        assert (got[:, h] == 0).all() and (ref[:, h] == 0).all()
    # the sink's logit has one rounding of its own, 2^-24 of 80 times log2 e or less
    for h in (0, 3, 4, 5, 6, 7):
        err = (got[:, h] - ref[:, h]).norm(dim=1)
        assert (err <= (H.REL[dtype] + 2 * 80 * 2 ** -23) * ref[:, h].norm(dim=1)).all(), h


# ---------------------------------------------------------------- long loops, wide sums

def test_append_of_more_pieces_than_a_pass_of_the_grid(cuda_device):
    # 1.25 M pieces of 16 bytes are one pass; the second pass begins inside a pair
    dev, P = cuda_device, 16
    g = torch.Generator(device=dev).manual_seed(1)
    jobs, caches, wants = [], [], []
    for n, width in ((9000, 80), (25000, 1024), (30000, 256)):
        rows = torch.randint(0, 256, (n, width), dtype=torch.uint8, device=dev, generator=g)
        pages = -(-n // P) + 3
        slots = torch.randperm(pages * P, device=dev, generator=g)[:n]
        slots[torch.rand(n, device=dev, generator=g) < 0.1] = -1
        cache = torch.randint(0, 256, (pages, P + 1, width), dtype=torch.uint8, device=dev, generator=g)
        want, keep = cache.clone(), slots >= 0
        want[slots[keep] // P, slots[keep] % P] = rows[keep]
        jobs.append(csa.AppendJob(rows, slots, cache, P))
        caches.append(cache)
        wants.append(want)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    csa.csa_paged_append(csa.AppendJobs(jobs), status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for c, w in zip(caches, wants):
        assert torch.equal(c, w)


def test_plan_gives_back_more_pages_than_a_pass_of_the_grid(cuda_device):
    seq_len = [60000, 5, 70001, 50000]
    table, ring, pos = H.pool(90, seq_len, ratio=1, page_rows=1, max_pages=70010, extra=40, head=123456)
    got, status, want, bad = run_plan(cuda_device, ratio=1, page_rows=1, swa_cap=16, seq_len=seq_len,
                                      new_len=[-1, 9, -1, -1], table=table, free_ring=ring, free_pos=pos, tok_cap=12,
                                      row_cap=12)
    assert status == bad == 0 and got == want


@pytest.mark.parametrize("B,new", [(3, [(1 << 31) - 1, (1 << 31) - 1, 7]), (8192, [1 << 19] * 8192)], ids=["few", "many"])
def test_plan_refuses_token_sums_past_32_bits(cuda_device, B, new):
    # the sum is 5 or 0 in 32 bits, what the maps would hold; blocks and pages are few
    assert sum(new) % (1 << 32) in (0, 5) and sum(new) >= 1 << 32
    table = [[-1, -1] for _ in range(B)]
    got, status, want, bad = run_plan(cuda_device, ratio=1 << 30, page_rows=1, swa_cap=16, seq_len=[0] * B, new_len=new,
                                      table=table, free_ring=[0, 1, 2, 3], free_pos=[0, 4], tok_cap=14, row_cap=4)
    assert status == bad == csa.DEV_CAPACITY and got == want
    assert got["seq_len_out"] == [0] * B and got["tok_seq"] == [-1] * 14


def test_plan_refuses_sums_of_given_back_pages_past_32_bits(cuda_device):
    # 8192 requests that hold 2^19 pages each: 0 in 32 bits.  (The table is 17 GB that
    # nothing reads, since the step is refused.)
    dev, B, n = cuda_device, 8192, 1 << 19
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB")
    t = H.plan_tensors(dev, seq_len=[n] * B, new_len=[-1] * B, table=[[0]] * B, free_ring=[3, 2, 1, 0], free_pos=[1, 2],
                       tok_cap=3, row_cap=2)
    t["table"] = torch.empty(B, n, dtype=torch.int32, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    csa.csa_page_plan(csa.PagePlan(ratio=1, page_rows=1, swa_cap=16, **t), status)
    torch.cuda.synchronize()
    assert int(status.item()) == csa.DEV_BAD_LAYOUT
    assert t["free_ring"].tolist() == [3, 2, 1, 0] and t["free_pos_out"].tolist() == [1, 2]
    assert (t["seq_len_out"] == n).all() and (t["row_len"] == n).all() and (t["tok_seq"] == -1).all()
    assert (t["tok_off"] == 0).all() and (t["row_off"] == 0).all() and (t["row_slot"] == -1).all()


# ---------------------------------------------------------------- every weight by itself

@pytest.mark.parametrize("T,n,heads", [(1, 512, 64), (40, 512, 64), (100, 512, 128), (330, 512, 64), (160, 4096, 64)], ids=str)
def test_attention_weights_element_by_element(cuda_device, T, n, heads):
    # Rows with one value each, so that an f32 output's column is the sum of n / 512
    # weights: a term of a weight that is lost in some tile, slice of rows or head
    # shows as 2^-8.  Relative bounds: two bf16 terms 2^-16; the logit (at most 6: a
    # product by the scale, a difference, 2^-24 of 9 each) and exp2 together 2^-20;
    # each sum of the denominator and of up to 16 terms a column, the partials and
    # the quotient, half a step to a step (2^-23) each: 40 of them.
    dev = cuda_device
    g = torch.Generator(device=dev).manual_seed(T + n)
    column = torch.cat([torch.randperm(H.HD, device=dev, generator=g) for _ in range(n // H.HD)])
    pages = n // 16
    table = torch.randperm(pages, device=dev, generator=g).int()[None]
    rows = torch.zeros(n, H.HD, dtype=BF16, device=dev)
    rows[torch.arange(n, device=dev), column] = 8.0
    cache = torch.empty(pages, 16, H.HD, dtype=BF16, device=dev)
    j = torch.arange(n, device=dev)
    cache[table[0, j // 16].long(), j % 16] = rows
    q = torch.randn(T, heads, H.HD, device=dev, generator=g).clamp_(-5.9, 5.9).to(BF16)
    layout = csa.PagedLayout(torch.zeros(T, dtype=torch.int32, device=dev),
                             torch.full((T,), 4 * n, dtype=torch.int64, device=dev), torch.tensor([n], device=dev),
                             table, 16)
    prm = csa.params(heads, 1, 0, 4, scale=0.125)
    out, status = torch.empty(T, heads, H.HD, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    csa.csa_paged_attention(layout, prm, cache, q, out, status, csa.paged_workspace(layout, prm))
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    l = q.double()[:, :, column]
    assert float(l.abs().max()) < 6
    w = torch.softmax(l, 2)
    ref = torch.zeros(T, heads, H.HD, dtype=torch.float64, device=dev).index_add_(2, column, 8 * w)
    err = ((out.double() - ref).abs() / ref).max()
    assert float(err) <= 2 ** -16 + 2 ** -20 + 40 * 2 ** -23, f"off by {float(err):.3e}"


# ---------------------------------------------------------------- prompts

@pytest.mark.parametrize("T,ctx,ratio,heads,dtype", [
    (700, 20000, 4, 64, F32), (1500, 6000, 4, 128, BF16), (4096, 30000, 128, 64, F32), (8192, 0, 4, 16, BF16),
    (8192, 1, 128, 8, F32),
], ids=str)
def test_attention_of_a_prompt_chunk(cuda_device, T, ctx, ratio, heads, dtype):
    # one request's chunk: every token sees the rows before it and its own window
    dev, P, W = cuda_device, 64, 128
    n, cap = (ctx + T) // ratio, W + T - 1
    g = torch.Generator(device=dev).manual_seed(T + ctx)
    pages = max(1, -(-n // P))
    table = torch.randperm(pages, device=dev, generator=g).int()[None]
    cache = torch.full((pages, P, H.HD), float("nan"), dtype=BF16, device=dev)
    rows = torch.randn(n, H.HD, device=dev, generator=g).to(BF16)
    j = torch.arange(n, device=dev)
    cache[table[0, j // P].long(), j % P] = rows
    ring = torch.randn(1, cap, H.HD, device=dev, generator=g).to(BF16)
    q = torch.randn(T, heads, H.HD, device=dev, generator=g).to(BF16)
    layout = csa.PagedLayout(torch.zeros(T, dtype=torch.int32, device=dev), ctx + torch.arange(T, device=dev),
                             torch.tensor([n], device=dev), table, P, ring,
                             torch.tensor([max(0, ctx + T - cap)], device=dev))
    prm = csa.params(heads, 1, W, ratio)
    out = torch.full((T, heads, H.HD), float("nan"), device=dev, dtype=dtype)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    csa.csa_paged_attention(layout, prm, cache, q, out, status, csa.paged_workspace(layout, prm))
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and bool(out.isfinite().all())
    for t in sorted({0, 1, 127, 128, T - 1} | set(range(0, T, T // 23))):
        p = ctx + t
        x = torch.arange(max(0, p - W + 1), p + 1, device=dev)
        every = torch.cat([rows[:p // ratio], ring[0, x % cap]]).double()
        ref = torch.softmax(prm.scale * q[t].double() @ every.T, 1) @ every
        assert (out[t].double() - ref).norm() <= H.REL[dtype] * ref.norm(), t


# ---------------------------------------------------------------- nothing to do, or next to it

@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 5, 151, 152, 153, 400, 8192])
def test_attention_of_padding_alone(cuda_device, T, dtype):
    p = H.Paged(100, row_len=[300, 0], tokens=[(-1, -1)] * T, heads=3, page_rows=8)
    got, status = p.run(cuda_device, dtype)
    assert status == 0 and (got == 7).all()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 60, 152, 153, 400, 2000])
def test_attention_of_tokens_without_rows(cuda_device, T, dtype):
    p = H.Paged(101, row_len=[300, 0], tokens=[(t % 2, 3) for t in range(T)], heads=66, page_rows=8, window=0,
                sinks=True)
    got, status = p.run(cuda_device, dtype)
    assert status == 0 and (got == 0).all()


def test_attention_without_tokens(cuda_device):
    p = H.Paged(102, row_len=[30], tokens=[], heads=3, page_rows=8)
    got, status = p.run(cuda_device, F32)
    assert status == 0 and got.numel() == 0


@pytest.mark.parametrize("page_rows", [1, 2, 8])
def test_attention_over_a_pool_of_one_page(cuda_device, page_rows):
    p = H.Paged(103, row_len=[page_rows], tokens=[(0, 4 * page_rows + 1)], heads=2, page_rows=page_rows, spare_pages=0,
                window=3)
    assert p.cache.shape[0] == 1
    got, status = p.run(cuda_device, F32)
    assert status == 0
    H.check(got, p.reference(), F32)


def test_a_refused_step_leaves_everything(cuda_device):
    # too few free pages: the maps are empty, so the append writes nothing and the
    # attention leaves its output, captured or not
    dev, P = cuda_device, 4
    t = H.plan_tensors(dev, seq_len=[6, 2], new_len=[30, 1], table=[[0] + [-1] * 9, [-1] * 10],
                       free_ring=[1, 2, -1], free_pos=[0, 2], tok_cap=40, row_cap=20)
    plan = csa.PagePlan(ratio=2, page_rows=P, swa_cap=16, **t)
    pool = torch.full((3, P, H.HD), float("nan"), dtype=BF16, device=dev)
    ring = torch.full((2, 16, H.HD), float("nan"), dtype=BF16, device=dev)
    jobs = csa.AppendJobs([csa.AppendJob(torch.ones(20, H.HD, dtype=BF16, device=dev), t["row_slot"], pool, P),
                           csa.AppendJob(torch.ones(40, H.HD, dtype=BF16, device=dev), t["swa_slot"], ring, 16)])
    layout = csa.PagedLayout(t["tok_seq"], t["tok_pos"], t["row_len"], t["table"], P, ring, t["swa_first_pos"])
    prm = csa.params(5, 1, 8, 2)
    q = torch.randn(40, 5, H.HD, device=dev).to(BF16)
    out, ws = torch.full((40, 5, H.HD), 7.0, device=dev), csa.paged_workspace(layout, prm)
    status = torch.zeros(1, dtype=torch.int32, device=dev)

    def step():
        csa.csa_page_plan(plan, status)
        csa.csa_paged_append(jobs, status)
        csa.csa_paged_attention(layout, prm, pool, q, out, status, ws)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for again in (lambda: None, g.replay):
        again()
        torch.cuda.synchronize()
        assert int(status.item()) == csa.DEV_CAPACITY
        assert pool.isnan().all() and ring.isnan().all() and (out == 7).all()
        assert t["seq_len_out"].tolist() == [6, 2] and t["free_ring"].tolist() == [1, 2, -1]
        status.zero_()


def test_these_calls_under_the_checked_build(cuda_device):
    """The library with internal bounds checks: a failed one sets a status bit, and
    every test wants the status it expects."""
    import os
    import subprocess
    import sys

    from sparse_compressed_kv_gb300 import build as B

    B.build(checks=True)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
                        os.path.join("tests", "test_gpu_paged_edges.py"), "-k",
                        "head_counts or interleaved or numbers or pieces or gives_back or prompt or element"],
                       cwd=root, env=dict(os.environ, CSA_CHECKS="1"), capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and " passed" in r.stdout, (r.stdout + r.stderr)[-3000:]
