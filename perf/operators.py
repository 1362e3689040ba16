"""The paged-cache operators as a serving step calls them: the page plan, the
append of new rows, and the attention of new tokens over paged rows.

Every state is synthetic: lengths come from the case, contents from the seed.
Rows and queries are N(0,1) rounded to bf16, as everywhere in this repository;
cache memory that no row was written to is NaN, since a server's pool holds
whatever was there before.
"""
from __future__ import annotations

import math
import random

import torch

own = False

HD = 512            # width of a compressed or window row
KEY_BYTES = 256     # an indexer key beside it
DEV = "cuda"


# ---------------------------------------------------------------- cases

def _plan(name, seqs, new_lo, new_hi, ctx_lo, ctx_hi, ratio, page_rows, swa_cap, over, lens=1):
    return dict(name=name, op="plan", seqs=seqs, new_lo=new_lo, new_hi=new_hi, ctx_lo=ctx_lo,
                ctx_hi=ctx_hi, ratio=ratio, page_rows=page_rows, swa_cap=swa_cap, over=over,
                lens=lens)


def _append(name, tokens, seqs, ratio, page_rows, gap, swa_cap, lens=1):
    return dict(name=name, op="append", tokens=tokens, seqs=seqs, ratio=ratio,
                page_rows=page_rows, gap=gap, swa_cap=swa_cap, lens=lens)


def _attn(name, seqs, new, ctx_lo, ctx_hi, ratio, page_rows, gap, heads, window, sinks, out,
          lens=1):
    return dict(name=name, op="attention", seqs=seqs, new=new, ctx_lo=ctx_lo, ctx_hi=ctx_hi,
                ratio=ratio, page_rows=page_rows, gap=gap, heads=heads, window=window,
                sinks=sinks, out=out, lens=lens)


def listed():
    return [
        # one decode step of a batch of 32 long contexts: one token each
        _plan("plan-decode-32", 32, 1, 1, 32768, 131072, 4, 64, 128, 0.0),
        # a busy server's decode step at ratio 128 with 256-token pages, some requests ending
        _plan("plan-decode-1024-hca", 1024, 1, 1, 100, 60000, 128, 2, 128, 0.03),
        # decode tokens and prefill chunks of many requests in one step
        _plan("plan-mixed-256", 256, 1, 2048, 0, 131072, 4, 64, 8192, 0.05),
        # what a decode step of 32 requests writes into one layer's caches
        _append("append-decode-32", 32, 32, 4, 64, 0, 128),
        # a 4096-token prefill chunk of one sequence
        _append("append-prefill-4096", 4096, 1, 4, 64, 0, 8192),
        # packed prompts of 16 requests, layers interleaved in the page pool
        _append("append-prompts-128k", 131072, 16, 4, 64, 64, 8192),
        # the smallest context: 256 rows and the window, 16 heads
        _attn("attn-tiny", 1, 1, 1024, 1024, 4, 64, 0, 16, 128, False, "f32"),
        # a layer of ratio 128 at one million tokens, batch 1
        _attn("attn-hca-1m", 1, 1, 1048576, 1048576, 128, 64, 0, 64, 128, False, "f32"),
        # ratio 128 in 256-token pages (two rows each), a batch of ragged contexts, with sinks
        _attn("attn-hca-batch128", 128, 1, 4096, 131072, 128, 2, 0, 64, 128, True, "bf16"),
        # every compressed row of one million tokens at ratio 4: the long axis
        _attn("attn-dense-1m", 1, 1, 1048576, 1048576, 4, 64, 0, 64, 128, False, "bf16"),
        # a ragged batch of 32 long contexts
        _attn("attn-batch32", 32, 1, 32768, 131072, 4, 64, 0, 64, 128, False, "bf16"),
        # four draft tokens a request, 128 heads, pages that end inside a tile
        _attn("attn-draft-h128", 16, 4, 1000, 40000, 4, 24, 8, 128, 128, True, "f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    lens = rng.randrange(2, 1 << 30)
    op = rng.choice(["plan", "append", "attention", "attention"])
    page_rows = rng.choice([1, 2, 3, 7, 8, 16, 24, 32, 40, 64, 100, 128, 256])
    if op == "plan":
        seqs = _log(rng, 1, 2048)
        new_hi = _log(rng, 1, max(1, min(4096, 400000 // seqs)))
        ratio = rng.choice([1, 4, 128])
        ctx_hi = _log(rng, 16, min(262144, 4000000 * page_rows * ratio // seqs))
        return dict(op="plan", seqs=seqs, new_lo=1, new_hi=new_hi, ctx_lo=ctx_hi // rng.choice([1, 4, 100]),
                    ctx_hi=ctx_hi, ratio=ratio, page_rows=page_rows,
                    swa_cap=rng.choice([128, 160, 1000, 8192]), over=rng.choice([0.0, 0.1, 0.5]),
                    lens=lens)
    if op == "append":
        seqs = _log(rng, 1, 256)
        ratio = rng.choice([1, 4, 128])
        return dict(op="append", tokens=_log(rng, seqs, 65536 if ratio == 1 else 131072),
                    seqs=seqs, ratio=ratio, page_rows=page_rows, gap=rng.choice([0, 0, 8, 64]),
                    swa_cap=rng.choice([128, 160, 1000, 8192]), lens=lens)
    heads = rng.choice([1, 8, 16, 24, 32, 40, 64, 64, 64, 96, 128])
    seqs, new = _log(rng, 1, 256), rng.choice([1, 1, 1, 2, 4])
    ratio = rng.choice([1, 4, 128])
    most = min(262144, 400000 * 64 // (max(64, heads) * seqs * new))   # rows a token
    ctx_hi = _log(rng, 2 * ratio, max(2, most) * ratio)
    return dict(op="attention", seqs=seqs, new=new, ctx_lo=ctx_hi // rng.choice([1, 3, 20]),
                ctx_hi=ctx_hi, ratio=ratio, page_rows=page_rows, gap=rng.choice([0, 0, 8, 5]),
                heads=heads, window=rng.choice([0, 1, 33, 128, 128, 200]),
                sinks=rng.random() < 0.3, out=rng.choice(["bf16", "f32"]), lens=lens)


# ---------------------------------------------------------------- host-side facts of a case

def _spread(rng, lo, hi):
    """Log-uniform between two lengths, zero included where the range starts there."""
    if lo >= hi:
        return hi
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo + 1), math.log(hi + 1)))) - 1))


def _plan_lengths(c):
    rng = random.Random(c["lens"])
    seq_len = [_spread(rng, c["ctx_lo"], c["ctx_hi"]) for _ in range(c["seqs"])]
    new_len = [_spread(rng, c["new_lo"], c["new_hi"]) for _ in range(c["seqs"])]
    for b in range(c["seqs"]):
        if rng.random() < c["over"]:
            new_len[b] = -1
    return seq_len, new_len


def _pages_of(tokens, c):
    return -(-(tokens // c["ratio"]) // c["page_rows"])


def _plan_sizes(c):
    seq_len, new_len = _plan_lengths(c)
    T = sum(max(n, 0) for n in new_len)
    R = sum((s + max(n, 0)) // c["ratio"] - s // c["ratio"] for s, n in zip(seq_len, new_len))
    need = sum(_pages_of(s + max(n, 0), c) - _pages_of(s, c) for s, n in zip(seq_len, new_len))
    rel = sum(_pages_of(s, c) for s, n in zip(seq_len, new_len) if n < 0)
    held = sum(_pages_of(s, c) for s in seq_len)
    widest = max(_pages_of(s + max(n, 0), c) for s, n in zip(seq_len, new_len))
    return seq_len, new_len, T, R, need, rel, held, max(1, widest) + 3


def _append_sizes(c):
    """Tokens of each request (ragged), the compressed rows they complete."""
    rng = random.Random(c["lens"])
    cut = sorted(rng.randrange(c["tokens"] + 1) for _ in range(c["seqs"] - 1))
    per = [b - a for a, b in zip([0] + cut, cut + [c["tokens"]])]
    return per, max(1, c["tokens"] // c["ratio"])


def _attn_lengths(c):
    rng = random.Random(c["lens"])
    return [_spread(rng, c["ctx_lo"], c["ctx_hi"]) for _ in range(c["seqs"])]


def _attn_sizes(c):
    ctx = _attn_lengths(c)
    end = [x + c["new"] for x in ctx]
    row_len = [e // c["ratio"] for e in end]
    pages = [-(-n // c["page_rows"]) for n in row_len]
    return ctx, end, row_len, pages


def work(case):
    c = case
    if c["op"] == "plan":
        _, _, T, R, need, rel, _, _ = _plan_sizes(c)
        B = c["seqs"]
        # lengths in; page ids moved; token and row maps, offsets and lengths out
        return {"bytes": B * (8 + 4) + 8 * (need + rel) + T * (4 + 8 + 8) + R * 8
                + (B + 1) * 16 + B * 24 + 32, "flops": 0}
    if c["op"] == "append":
        _, R = _append_sizes(c)
        return {"bytes": c["tokens"] * (2 * 2 * HD + 8) + R * (2 * 2 * HD + 2 * KEY_BYTES + 8),
                "flops": 0}
    ctx, end, row_len, _ = _attn_sizes(c)
    T, H = c["seqs"] * c["new"], c["heads"]
    rows, pairs = 0, 0
    for x, n in zip(ctx, row_len):
        last = x + c["new"] - 1
        rows += min(n, last // c["ratio"])
        if c["window"]:
            rows += last - max(0, x - c["window"] + 1) + 1
        for i in range(c["new"]):
            pairs += min(n, (x + i) // c["ratio"]) + min(c["window"], x + i + 1)
    return {"bytes": rows * 2 * HD + T * H * HD * (2 + (2 if c["out"] == "bf16" else 4)),
            "flops": 4 * pairs * H * HD}


# ---------------------------------------------------------------- states

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _i64(x):
    return torch.tensor(x, dtype=torch.int64, device=DEV)


def _prepare_plan(c, seed):
    seq_len, new_len, T, R, need, rel, held, max_pages = _plan_sizes(c)
    B = c["seqs"]
    g = _gen(seed)
    num_pages = held + need + 5
    perm = torch.randperm(num_pages, device=DEV, generator=g).int()
    # pages held, request after request; the rest of the pool waits in the free ring
    count = _i64([_pages_of(s, c) for s in seq_len])
    own_rows = torch.arange(max_pages, device=DEV)[None, :] < count[:, None]
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device=DEV)
    table[own_rows] = perm[:held]
    head = int(torch.randint(0, 1 << 20, (1,), device=DEV, generator=g))
    free = num_pages - held
    ring = torch.full((num_pages,), -1, dtype=torch.int32, device=DEV)
    ring[(head + torch.arange(free, device=DEV)) % num_pages] = perm[held:]
    tok_cap, row_cap = T + 3, R + 2
    s = dict(case=c, seq_len=_i64(seq_len), new_len=_i32(new_len), table=table, free_ring=ring,
             free_pos=_i64([head, head + free]), tok_cap=tok_cap, row_cap=row_cap)
    for name, n, dt in (("seq_len_out", B, torch.int64), ("row_len", B, torch.int64),
                        ("swa_first_pos", B, torch.int64), ("free_pos_out", 2, torch.int64),
                        ("tok_off", B + 1, torch.int64), ("row_off", B + 1, torch.int64),
                        ("tok_seq", tok_cap, torch.int32), ("tok_pos", tok_cap, torch.int64),
                        ("swa_slot", tok_cap, torch.int64), ("row_slot", row_cap, torch.int64)):
        s[name] = torch.full((n,), -9, dtype=dt, device=DEV)
    if own:
        from sparse_compressed_kv_gb300 import csa
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        s["plan"] = csa.PagePlan(
            ratio=c["ratio"], page_rows=c["page_rows"], swa_cap=c["swa_cap"],
            **{k: s[k] for k in ("seq_len", "new_len", "table", "free_ring", "free_pos",
                                 "seq_len_out", "row_len", "swa_first_pos", "free_pos_out",
                                 "tok_off", "row_off", "tok_seq", "tok_pos", "swa_slot",
                                 "row_slot")})
    return s


PLAN_OUTPUTS = ("table", "free_ring", "free_pos_out", "seq_len_out", "row_len", "swa_first_pos",
                "tok_off", "row_off", "tok_seq", "tok_pos", "swa_slot", "row_slot")


def _prepare_append(c, seed):
    per, R = _append_sizes(c)
    T, P, g = c["tokens"], c["page_rows"], _gen(seed)
    stride = P + c["gap"]
    num_pages = -(-R // P) + 4
    randn = lambda *shape: torch.randn(*shape, device=DEV, generator=g).to(torch.bfloat16)
    pages = torch.randperm(num_pages, device=DEV, generator=g)
    r = torch.arange(R, device=DEV)
    row_slot = pages[r // P] * P + r % P
    # the ring keeps each request's newest swa_cap tokens; older ones get no slot
    cap = c["swa_cap"]
    start = torch.randint(0, 1 << 20, (c["seqs"],), device=DEV, generator=g)
    n = _i64(per)
    seq = torch.repeat_interleave(torch.arange(c["seqs"], device=DEV), n)
    i = torch.arange(T, device=DEV) - (torch.cumsum(n, 0) - n)[seq]
    swa_slot = torch.where(i >= n[seq] - cap, seq * cap + (start[seq] + i) % cap, -1)
    s = dict(case=c, rows=randn(R, HD), keys=randn(R, KEY_BYTES // 2), window=randn(T, HD),
             row_slot=row_slot, swa_slot=swa_slot,
             comp_kv=torch.zeros(num_pages, stride, HD, dtype=torch.bfloat16, device=DEV),
             k_idx=torch.zeros(num_pages, stride, KEY_BYTES // 2, dtype=torch.bfloat16, device=DEV),
             swa_kv=torch.zeros(c["seqs"], cap, HD, dtype=torch.bfloat16, device=DEV))
    if own:
        from sparse_compressed_kv_gb300 import csa
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        s["jobs"] = csa.AppendJobs([
            csa.AppendJob(s["rows"], row_slot, s["comp_kv"], page_rows=P),
            csa.AppendJob(s["keys"], row_slot, s["k_idx"], page_rows=P),
            csa.AppendJob(s["window"], swa_slot, s["swa_kv"], page_rows=cap)])
    return s


def _prepare_attention(c, seed):
    ctx, end, row_len, pages = _attn_sizes(c)
    B, new, P, W, g = c["seqs"], c["new"], c["page_rows"], c["window"], _gen(seed)
    stride, T, H = P + c["gap"], c["seqs"] * c["new"], c["heads"]
    num_pages, max_pages = sum(pages) + 3, max(1, max(pages)) + 1
    randn = lambda *shape: torch.randn(*shape, device=DEV, generator=g, dtype=torch.bfloat16)
    count = _i64(pages)
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device=DEV)
    held = torch.arange(max_pages, device=DEV)[None, :] < count[:, None]
    table[held] = torch.randperm(num_pages, device=DEV, generator=g)[:sum(pages)].int()
    cache = torch.full((num_pages, stride, HD), float("nan"), dtype=torch.bfloat16, device=DEV)
    n = _i64(row_len)
    total = sum(row_len)
    seq = torch.repeat_interleave(torch.arange(B, device=DEV), n)
    j = torch.arange(total, device=DEV) - (torch.cumsum(n, 0) - n)[seq]
    at = table[seq, j // P].long() * stride + j % P
    cache.view(-1, HD)[at] = randn(total, HD)
    cap = max(1, W) + new + 5
    s = dict(case=c, table=table, cache=cache, row_len=n,
             tok_seq=torch.arange(B, device=DEV, dtype=torch.int32).repeat_interleave(new),
             tok_pos=(_i64(ctx)[:, None] + torch.arange(new, device=DEV)[None, :]).reshape(-1),
             swa_kv=randn(B, cap, HD), swa_first_pos=(_i64(end) - cap).clamp_min(0),
             q=randn(T, H, HD),
             sinks=torch.randn(H, device=DEV, generator=g) if c["sinks"] else None,
             out=torch.empty(T, H, HD, device=DEV,
                             dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32))
    if own:
        from sparse_compressed_kv_gb300 import csa
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        s["layout"] = csa.PagedLayout(s["tok_seq"], s["tok_pos"], s["row_len"], s["table"],
                                      page_rows=P, swa_kv=s["swa_kv"],
                                      swa_first_pos=s["swa_first_pos"])
        s["prm"] = csa.params(H, 1, W, c["ratio"])
        s["ws"] = csa.paged_workspace(s["layout"], s["prm"])
    return s


def prepare(case, seed):
    return {"plan": _prepare_plan, "append": _prepare_append,
            "attention": _prepare_attention}[case["op"]](case, seed)


# ---------------------------------------------------------------- plain forms

def _plain_plan(s):
    c = s["case"]
    B, P, ratio, cap = c["seqs"], c["page_rows"], c["ratio"], c["swa_cap"]
    table, ring = s["table"], s["free_ring"]
    N = ring.numel()
    seq_len, new = s["seq_len"], s["new_len"].long()
    over = new < 0
    new = new.clamp_min(0)
    end = torch.where(over, 0, seq_len + new)
    old_rows = seq_len // ratio
    rows = end // ratio
    old_pages = (old_rows + P - 1) // P
    need = torch.where(over, 0, (rows + P - 1) // P - old_pages)
    rel = torch.where(over, old_pages, 0)
    add = torch.where(over, 0, rows - old_rows)
    zero = torch.zeros(1, dtype=torch.int64, device=DEV)
    offsets = lambda x: torch.cat([zero, torch.cumsum(x, 0)])
    tok_off, row_off = offsets(new), offsets(add)
    head, tail = s["free_pos"][0], s["free_pos"][1]
    col = torch.arange(table.shape[1], device=DEV)[None, :]
    gone = table[(col < old_pages[:, None]) & over[:, None]]
    fresh = (col >= old_pages[:, None]) & (col < (old_pages + need)[:, None])
    table[fresh] = ring[(head + torch.arange(int(need.sum()), device=DEV)) % N]
    ring[(tail + torch.arange(gone.numel(), device=DEV)) % N] = gone
    t = torch.arange(s["tok_cap"], device=DEV)
    b = torch.searchsorted(tok_off[1:], t, right=True)
    real, b = b < B, b.clamp_max(B - 1)
    pos = seq_len[b] + t - tok_off[b]
    s["tok_seq"].copy_(torch.where(real, b, -1))
    s["tok_pos"].copy_(torch.where(real, pos, -1))
    s["swa_slot"].copy_(torch.where(real & (pos >= end[b] - cap), b * cap + pos % cap, -1))
    r = torch.arange(s["row_cap"], device=DEV)
    b = torch.searchsorted(row_off[1:], r, right=True)
    real, b = b < B, b.clamp_max(B - 1)
    block = torch.where(real, old_rows[b] + r - row_off[b], 0)
    s["row_slot"].copy_(torch.where(real, table[b, block // P].long() * P + block % P, -1))
    s["tok_off"].copy_(tok_off)
    s["row_off"].copy_(row_off)
    s["seq_len_out"].copy_(end)
    s["row_len"].copy_(rows)
    s["swa_first_pos"].copy_((end - cap).clamp_min(0))
    s["free_pos_out"].copy_(s["free_pos"] + torch.stack([need.sum(), rel.sum()]))


def _plain_append(s):
    P, cap = s["case"]["page_rows"], s["case"]["swa_cap"]
    slot = s["row_slot"]
    s["comp_kv"][slot // P, slot % P] = s["rows"]
    s["k_idx"][slot // P, slot % P] = s["keys"]
    keep = s["swa_slot"] >= 0
    slot = s["swa_slot"][keep]
    s["swa_kv"][slot // cap, slot % cap] = s["window"][keep]


def _plain_attention(s):
    c = s["case"]
    P, W, ratio = c["page_rows"], c["window"], c["ratio"]
    stride, cap = s["cache"].shape[1], s["swa_kv"].shape[1]
    b, p = s["tok_seq"].long(), s["tok_pos"]
    n = torch.minimum(s["row_len"][b], p // ratio)
    most = s["table"].shape[1] * P
    j = torch.arange(most, device=DEV)[None, :]
    real = j < n[:, None]
    page = s["table"][b].long()[:, torch.arange(most, device=DEV) // P].clamp_min(0)
    rows = s["cache"].view(-1, HD)[page * stride + j % P].float()
    x = p[:, None] - W + 1 + torch.arange(W, device=DEV)[None, :]
    local = s["swa_kv"].view(-1, HD)[b[:, None] * cap + x % cap].float()
    rows = torch.cat([rows.masked_fill_(~real[:, :, None], 0.0), local], 1)
    real = torch.cat([real, x >= 0], 1)
    logits = torch.matmul(s["q"].float(), rows.transpose(1, 2)) * HD ** -0.5
    logits = logits.masked_fill(~real[:, None, :], float("-inf"))
    top = logits.amax(2, keepdim=True) if logits.shape[2] else logits.new_full(logits.shape[:2] + (1,), -math.inf)
    top = torch.where(top == -math.inf, 0.0, top)
    e = torch.exp(logits - top)
    z = e.sum(2, keepdim=True)
    if s["sinks"] is not None:
        z = z + torch.exp(s["sinks"][None, :, None] - top)
    empty = ~real.any(1)
    o = torch.matmul(e, rows) / torch.where(empty[:, None, None], 1.0, z)
    s["out"].copy_(o)


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        from sparse_compressed_kv_gb300 import csa
        if op == "plan":
            csa.csa_page_plan(s["plan"], s["status"])
        elif op == "append":
            csa.csa_paged_append(s["jobs"], s["status"])
        else:
            csa.csa_paged_attention(s["layout"], s["prm"], s["cache"], s["q"], s["out"], s["status"],
                                    s["ws"], sinks=s["sinks"])
    else:
        {"plan": _plain_plan, "append": _plain_append, "attention": _plain_attention}[op](s)
    if op == "plan":
        return {k: s[k] for k in PLAN_OUTPUTS}
    if op == "append":
        return {k: s[k] for k in ("comp_kv", "k_idx", "swa_kv")}
    return s["out"]


# ---------------------------------------------------------------- from the definitions

def _exact_plan(s):
    c = s["case"]
    P, ratio, cap = c["page_rows"], c["ratio"], c["swa_cap"]
    seq_len, new_len = s["seq_len"].tolist(), s["new_len"].tolist()
    table, ring = s["table"].tolist(), s["free_ring"].tolist()
    head, tail = s["free_pos"].tolist()
    N = len(ring)
    o = {k: [] for k in ("seq_len_out", "row_len", "swa_first_pos", "tok_seq", "tok_pos",
                         "swa_slot", "row_slot")}
    tok_off, row_off, freed = [0], [0], []
    for b, (have, add) in enumerate(zip(seq_len, new_len)):
        pages = -(-(have // ratio) // P)
        if add < 0:
            freed += table[b][:pages]
            end = 0
        else:
            end = have + add
            for x in range(have, end):
                o["tok_seq"].append(b)
                o["tok_pos"].append(x)
                o["swa_slot"].append(b * cap + x % cap if x >= end - cap else -1)
            for g in range(have // ratio, end // ratio):
                if g // P >= pages:
                    table[b][pages] = ring[head % N]
                    head, pages = head + 1, pages + 1
                o["row_slot"].append(table[b][g // P] * P + g % P)
        tok_off.append(len(o["tok_seq"]))
        row_off.append(len(o["row_slot"]))
        o["seq_len_out"].append(end)
        o["row_len"].append(end // ratio)
        o["swa_first_pos"].append(max(0, end - cap))
    for page in freed:
        ring[tail % N] = page
        tail += 1
    for k in ("tok_seq", "tok_pos", "swa_slot"):
        o[k] += [-1] * (s["tok_cap"] - len(o[k]))
    o["row_slot"] += [-1] * (s["row_cap"] - len(o["row_slot"]))
    o |= dict(table=table, free_ring=ring, free_pos_out=[head, tail], tok_off=tok_off,
              row_off=row_off)
    return {k: torch.tensor(o[k], dtype=s[k].dtype) for k in PLAN_OUTPUTS}


def _exact_append(s):
    P, cap = s["case"]["page_rows"], s["case"]["swa_cap"]
    done = {}
    for name, rows, slots, n in (("comp_kv", "rows", "row_slot", P), ("k_idx", "keys", "row_slot", P),
                                 ("swa_kv", "window", "swa_slot", cap)):
        to = s[name].double().cpu()
        src, at = s[rows].double().cpu(), s[slots].cpu()
        took = (at >= 0).nonzero().flatten()
        flat = to.view(-1, to.shape[-1])
        flat.index_copy_(0, at[took] // n * to.shape[1] + at[took] % n, src[took])
        done[name] = to
    return done


def _exact_attention(s):
    c = s["case"]
    P, W, ratio = c["page_rows"], c["window"], c["ratio"]
    cap = s["swa_kv"].shape[1]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    row_len, pos = s["row_len"].tolist(), s["tok_pos"].tolist()
    for t, b in enumerate(s["tok_seq"].tolist()):
        seen = min(row_len[b], pos[t] // ratio)
        block = torch.arange(seen, device=DEV)
        held = s["cache"][s["table"][b, block // P].long(), block % P]
        near = torch.arange(max(0, pos[t] - W + 1), pos[t] + 1, device=DEV) if W else block[:0]
        rows = torch.cat([held, s["swa_kv"][b, near % cap]]).double()
        if not rows.shape[0]:
            continue
        l = s["q"][t].double() @ rows.T / math.sqrt(HD)
        every = l if s["sinks"] is None else torch.cat([l, s["sinks"].double()[:, None]], 1)
        out[t] = torch.exp(l - torch.logsumexp(every, 1, keepdim=True)) @ rows
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return _exact_plan(s)
    if case["op"] == "append":
        return _exact_append(s) if case["tokens"] <= 32768 else None
    return _exact_attention(s)
