"""The 8-bit paged caches as a serving step calls them: rows quantised as they
are appended (e4m3 codes and one power-of-two scale a row), rows read back by
slot, and the attention of new tokens over the 8-bit rows in place.

Every state is synthetic: lengths come from the case, contents from the seed.
Rows are N(0,1) times a magnitude of their own (2 to the power of N(0,1)/2, so
that scales differ from row to row), queries N(0,1), both rounded to bf16.
Cache memory that no row was written to is NaN where a call reads the cache.
"""
from __future__ import annotations

import math
import random

import torch

own = False

HD = 512            # width of a compressed or window row
DEV = "cuda"
F8 = torch.float8_e4m3fn
TOP = 448.0         # the largest e4m3 value
KMAX = 60           # scales are 2^-60 .. 2^60
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def _append(name, tokens, seqs, ratio, page_rows, gap, swa_cap, rows, lens=1):
    return dict(name=name, op="append", tokens=tokens, seqs=seqs, ratio=ratio, page_rows=page_rows,
                gap=gap, swa_cap=swa_cap, rows=rows, lens=lens)


def _read(name, rows, pool, run, page_rows, gap, out, lens=1):
    return dict(name=name, op="read", rows=rows, pool=pool, run=run, page_rows=page_rows, gap=gap,
                out=out, lens=lens)


def _attn(name, seqs, new, ctx_lo, ctx_hi, ratio, page_rows, gap, heads, window, sinks, out, lens=1):
    return dict(name=name, op="attention", seqs=seqs, new=new, ctx_lo=ctx_lo, ctx_hi=ctx_hi,
                ratio=ratio, page_rows=page_rows, gap=gap, heads=heads, window=window, sinks=sinks,
                out=out, lens=lens)


def listed():
    return [
        # what a decode step of 32 requests writes into one layer's caches
        _append("append8-decode-32", 32, 32, 4, 64, 0, 128, "bf16"),
        # a 4096-token prefill chunk of one sequence, rows still in f32
        _append("append8-prefill-4096", 4096, 1, 4, 64, 0, 8192, "f32"),
        # packed prompts of 16 requests, layers interleaved in the page pool
        _append("append8-prompts-128k", 131072, 16, 4, 64, 64, 8192, "bf16"),
        # one token's 1024 selected rows out of a one-million-token context, scattered
        _read("read8-topk-1024", 1024, 262144, 1, 64, 0, "bf16"),
        # every row of a 524,288-token context back in f32, pages that are no power of two
        _read("read8-context-131072", 131072, 140000, 24, 24, 8, "f32"),
        # the smallest context: 256 rows and the window, 16 heads
        _attn("attn8-tiny", 1, 1, 1024, 1024, 4, 64, 0, 16, 128, False, "f32"),
        # a layer of ratio 128 at one million tokens, batch 1
        _attn("attn8-hca-1m", 1, 1, 1048576, 1048576, 128, 64, 0, 64, 128, False, "bf16"),
        # ratio 128 in 256-token pages (two rows each), a batch of ragged contexts, with sinks
        _attn("attn8-hca-batch128", 128, 1, 4096, 131072, 128, 2, 0, 64, 128, True, "bf16"),
        # every compressed row of one million tokens at ratio 4: the long axis
        _attn("attn8-dense-1m", 1, 1, 1048576, 1048576, 4, 64, 0, 64, 128, False, "bf16"),
        # a ragged batch of 32 long contexts
        _attn("attn8-batch32", 32, 1, 32768, 131072, 4, 64, 0, 64, 128, False, "bf16"),
        # four draft tokens a request, 128 heads, pages that end inside a tile
        _attn("attn8-draft-h128", 16, 4, 1000, 40000, 4, 24, 8, 128, 128, True, "f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    lens = rng.randrange(2, 1 << 30)
    op = rng.choice(["append", "read", "attention", "attention"])
    page_rows = rng.choice([1, 2, 3, 7, 8, 16, 24, 32, 40, 64, 100, 128, 256])
    gap = rng.choice([0, 0, 8, 5, 64])
    if op == "append":
        seqs = _log(rng, 1, 256)
        ratio = rng.choice([1, 4, 128])
        rows = rng.choice(["bf16", "bf16", "f32"])
        most = 131072 >> (ratio == 1) >> (rows == "f32")
        return dict(op="append", tokens=_log(rng, seqs, most), seqs=seqs, ratio=ratio,
                    page_rows=page_rows, gap=gap, swa_cap=rng.choice([128, 160, 1000, 8192]),
                    rows=rows, lens=lens)
    if op == "read":
        rows = _log(rng, 1, 131072)
        return dict(op="read", rows=rows, pool=rows + _log(rng, 1, 131072),
                    run=rng.choice([1, 1, 7, page_rows]), page_rows=page_rows, gap=min(gap, page_rows),
                    out=rng.choice(["bf16", "bf16", "f32"]), lens=lens)
    heads = rng.choice([1, 8, 16, 24, 32, 40, 64, 64, 64, 96, 128])
    seqs, new = _log(rng, 1, 256), rng.choice([1, 1, 1, 2, 4])
    ratio = rng.choice([1, 4, 128])
    most = min(262144, 400000 * 64 // (max(64, heads) * seqs * new))   # rows a token
    ctx_hi = _log(rng, 2 * ratio, max(2, most) * ratio)
    return dict(op="attention", seqs=seqs, new=new, ctx_lo=ctx_hi // rng.choice([1, 3, 20]),
                ctx_hi=ctx_hi, ratio=ratio, page_rows=page_rows, gap=min(gap, 8), heads=heads,
                window=rng.choice([0, 1, 33, 128, 128, 200]), sinks=rng.random() < 0.3,
                out=rng.choice(["bf16", "bf16", "f32"]), lens=lens)


# ---------------------------------------------------------------- host-side facts of a case

def _spread(rng, lo, hi):
    """Log-uniform between two lengths, zero included where the range starts there."""
    if lo >= hi:
        return hi
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo + 1), math.log(hi + 1)))) - 1))


def _append_sizes(c):
    """Tokens of each request (ragged), the compressed rows they complete."""
    rng = random.Random(c["lens"])
    cut = sorted(rng.randrange(c["tokens"] + 1) for _ in range(c["seqs"] - 1))
    per = [b - a for a, b in zip([0] + cut, cut + [c["tokens"]])]
    return per, max(1, c["tokens"] // c["ratio"])


def _attn_sizes(c):
    rng = random.Random(c["lens"])
    ctx = [_spread(rng, c["ctx_lo"], c["ctx_hi"]) for _ in range(c["seqs"])]
    end = [x + c["new"] for x in ctx]
    row_len = [e // c["ratio"] for e in end]
    pages = [-(-n // c["page_rows"]) for n in row_len]
    return ctx, end, row_len, pages


def work(case):
    c = case
    if c["op"] == "append":
        _, R = _append_sizes(c)
        width = 4 if c["rows"] == "f32" else 2
        return {"bytes": (c["tokens"] + R) * (width * HD + 8 + HD + 4), "flops": 0}
    if c["op"] == "read":
        width = 4 if c["out"] == "f32" else 2
        return {"bytes": c["rows"] * (HD + 4 + 8 + width * HD), "flops": 0}
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
    return {"bytes": rows * (HD + 4) + T * H * HD * (2 + (2 if c["out"] == "bf16" else 4)),
            "flops": 4 * pairs * H * HD}


# ---------------------------------------------------------------- the 8-bit form of a row, plainly

def _quantise(rows):
    """Rows [n, width] to e4m3 codes and f32 scales 2^k, k the least with
    amax <= 448 * 2^k (a row of zeros: the smallest scale)."""
    x = rows.float()
    mant, exp = torch.frexp(x.abs().amax(1))          # amax = mant 2^exp, mant in [0.5, 1)
    k = (exp - 9 + (mant > TOP / 512).int()).clamp(-KMAX, KMAX)
    k = torch.where(mant == 0, -KMAX, k).int()
    power = lambda e: ((e + 127) << 23).view(torch.float32)      # 2^e, exactly
    return (x * power(-k)[:, None]).to(F8), power(k)


# ---------------------------------------------------------------- states

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _i64(x):
    return torch.tensor(x, dtype=torch.int64, device=DEV)


def _rows(g, n, dtype=torch.bfloat16):
    x = torch.randn(n, HD, device=DEV, generator=g)
    x *= torch.exp2(torch.randn(n, 1, device=DEV, generator=g) / 2)
    return x.to(dtype)


def _prepare_append(c, seed):
    per, R = _append_sizes(c)
    T, P, g = c["tokens"], c["page_rows"], _gen(seed)
    stride = P + c["gap"]
    num_pages = -(-R // P) + 4
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
    dt = TYPES[c["rows"]]
    s = dict(case=c, rows=_rows(g, R, dt), window=_rows(g, T, dt), row_slot=row_slot,
             swa_slot=swa_slot, comp_kv=torch.zeros(num_pages, stride, HD, device=DEV).to(F8),
             comp_scale=torch.zeros(num_pages, stride, device=DEV),
             swa_kv=torch.zeros(c["seqs"], cap, HD, device=DEV).to(F8),
             swa_scale=torch.zeros(c["seqs"], cap, device=DEV))
    if own:
        from sparse_compressed_kv_gb300 import csa
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        s["jobs"] = csa.AppendJobsFp8([
            csa.AppendJobFp8(s["rows"], row_slot, s["comp_kv"], s["comp_scale"], page_rows=P),
            csa.AppendJobFp8(s["window"], swa_slot, s["swa_kv"], s["swa_scale"], page_rows=cap)])
    return s


def _prepare_read(c, seed):
    P, g, rng = c["page_rows"], _gen(seed), random.Random(c["lens"])
    stride = P + c["gap"]
    num_pages = -(-c["pool"] // P)
    codes = torch.full((num_pages, stride, HD), float("nan"), device=DEV).to(F8)
    scale = torch.full((num_pages, stride), float("nan"), device=DEV)
    for a in range(0, num_pages, max(1, 65536 // P)):
        b = min(num_pages, a + max(1, 65536 // P))
        x, k = _quantise(_rows(g, (b - a) * P))
        codes[a:b, :P], scale[a:b, :P] = x.view(b - a, P, HD), k.view(b - a, P)
    # runs of neighbouring rows, in random order; a few entries name no row
    starts = num_pages * P // c["run"]
    first = torch.randperm(starts, device=DEV, generator=g)[:-(-c["rows"] // c["run"])] * c["run"]
    slots = (first[:, None] + torch.arange(c["run"], device=DEV)[None, :]).reshape(-1)[:c["rows"]]
    if slots.numel() < c["rows"]:
        slots = slots.repeat(-(-c["rows"] // slots.numel()))[:c["rows"]]
    slots = slots.contiguous()
    if c["rows"] > 4:
        slots[rng.randrange(c["rows"])] = -1
    s = dict(case=c, codes=codes, scale=scale, slots=slots,
             out=torch.zeros(c["rows"], HD, device=DEV, dtype=TYPES[c["out"]]))
    if own:
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    return s


def _prepare_attention(c, seed):
    ctx, end, row_len, pages = _attn_sizes(c)
    B, new, P, W, g = c["seqs"], c["new"], c["page_rows"], c["window"], _gen(seed)
    stride, T, H = P + c["gap"], c["seqs"] * c["new"], c["heads"]
    num_pages, max_pages = sum(pages) + 3, max(1, max(pages)) + 1
    count = _i64(pages)
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device=DEV)
    held = torch.arange(max_pages, device=DEV)[None, :] < count[:, None]
    table[held] = torch.randperm(num_pages, device=DEV, generator=g)[:sum(pages)].int()
    codes = torch.full((num_pages, stride, HD), float("nan"), device=DEV).to(F8)
    scale = torch.full((num_pages, stride), float("nan"), device=DEV)
    n = _i64(row_len)
    total = sum(row_len)
    seq = torch.repeat_interleave(torch.arange(B, device=DEV), n)
    j = torch.arange(total, device=DEV) - (torch.cumsum(n, 0) - n)[seq]
    at = table[seq, j // P].long() * stride + j % P
    flat = codes.view(torch.uint8).view(-1, HD)
    for a in range(0, total, 131072):
        x, k = _quantise(_rows(g, min(131072, total - a)))
        flat[at[a:a + 131072]] = x.view(torch.uint8)
        scale.view(-1)[at[a:a + 131072]] = k
    cap = max(1, W) + new + 5
    near, near_scale = _quantise(_rows(g, B * cap))
    s = dict(case=c, table=table, codes=codes, scale=scale, row_len=n,
             tok_seq=torch.arange(B, device=DEV, dtype=torch.int32).repeat_interleave(new),
             tok_pos=(_i64(ctx)[:, None] + torch.arange(new, device=DEV)[None, :]).reshape(-1),
             swa_kv=near.view(B, cap, HD), swa_scale=near_scale.view(B, cap),
             swa_first_pos=(_i64(end) - cap).clamp_min(0),
             q=torch.randn(T, H, HD, device=DEV, generator=g, dtype=torch.bfloat16),
             sinks=torch.randn(H, device=DEV, generator=g) if c["sinks"] else None,
             out=torch.empty(T, H, HD, device=DEV, dtype=TYPES[c["out"]]))
    if own:
        from sparse_compressed_kv_gb300 import csa
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        s["layout"] = csa.PagedLayoutFp8(s["tok_seq"], s["tok_pos"], s["row_len"], s["table"],
                                         page_rows=P, swa_kv=s["swa_kv"], swa_scales=s["swa_scale"],
                                         swa_first_pos=s["swa_first_pos"])
        s["prm"] = csa.params(H, 1, W, c["ratio"])
        s["ws"] = csa.paged_workspace(s["layout"], s["prm"])
    return s


def prepare(case, seed):
    return {"append": _prepare_append, "read": _prepare_read,
            "attention": _prepare_attention}[case["op"]](case, seed)


# ---------------------------------------------------------------- plain forms

def _plain_append(s):
    for rows, slots, to, scales, n in (
            ("rows", "row_slot", "comp_kv", "comp_scale", s["case"]["page_rows"]),
            ("window", "swa_slot", "swa_kv", "swa_scale", s["case"]["swa_cap"])):
        keep = s[slots] >= 0
        at = s[slots][keep]
        codes, k = _quantise(s[rows][keep])
        s[to].view(torch.uint8)[at // n, at % n] = codes.view(torch.uint8)
        s[scales][at // n, at % n] = k


def _plain_read(s):
    P = s["case"]["page_rows"]
    keep = s["slots"] >= 0
    at = s["slots"][keep]
    codes = s["codes"].view(torch.uint8)[at // P, at % P].view(F8)
    s["out"][keep] = (codes.float() * s["scale"][at // P, at % P][:, None]).to(s["out"].dtype)


def _plain_attention(s):
    c = s["case"]
    P, W, ratio = c["page_rows"], c["window"], c["ratio"]
    stride, cap = s["codes"].shape[1], s["swa_kv"].shape[1]
    b, p = s["tok_seq"].long(), s["tok_pos"]
    n = torch.minimum(s["row_len"][b], p // ratio)
    most = s["table"].shape[1] * P
    j = torch.arange(most, device=DEV)[None, :]
    real = j < n[:, None]
    page = s["table"][b].long()[:, torch.arange(most, device=DEV) // P].clamp_min(0)
    at = page * stride + j % P
    values = lambda codes, scale, i: (codes.view(torch.uint8).view(-1, HD)[i].view(F8).float()
                                      * scale.view(-1)[i][:, :, None])
    rows = values(s["codes"], s["scale"], at).masked_fill_(~real[:, :, None], 0.0)
    x = p[:, None] - W + 1 + torch.arange(W, device=DEV)[None, :]
    rows = torch.cat([rows, values(s["swa_kv"], s["swa_scale"], b[:, None] * cap + x % cap)], 1)
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
    s["out"].copy_(torch.matmul(e, rows) / torch.where(empty[:, None, None], 1.0, z))


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        from sparse_compressed_kv_gb300 import csa
        if op == "append":
            csa.csa_paged_append_fp8(s["jobs"], s["status"])
        elif op == "read":
            csa.csa_paged_read_fp8(s["codes"], s["scale"], s["slots"], s["out"], s["status"],
                                   page_rows=s["case"]["page_rows"])
        else:
            csa.csa_paged_attention_fp8(s["layout"], s["prm"], s["codes"], s["scale"], s["q"],
                                        s["out"], s["status"], s["ws"], sinks=s["sinks"])
    else:
        {"append": _plain_append, "read": _plain_read, "attention": _plain_attention}[op](s)
    if op == "append":
        return {k: s[k] for k in ("comp_kv", "comp_scale", "swa_kv", "swa_scale")}
    return s["out"]


# ---------------------------------------------------------------- from the definitions

def _exact_codes(x):
    """float64 rows to the nearest e4m3 values (ties to even) and scales."""
    # the powers of two, exactly (the device's own power function may be off)
    power = torch.tensor([2.0 ** e for e in range(-KMAX, KMAX + 1)], dtype=torch.float64, device=x.device)
    k = torch.searchsorted(TOP * power, x.abs().amax(1)).clamp_max(2 * KMAX)     # amax <= 448 2^k
    y = x / power[k][:, None]
    # the step of e4m3 next to y: 2^-9 up to 2^-5, and twice as much from each power of two on
    above = torch.bucketize(y.abs(), power[KMAX - 5:KMAX + 9], right=True)
    step = power[KMAX - 9:KMAX + 6][above]
    return torch.round(y / step) * step, power[k]


def _exact_append(s):
    done = {}
    for rows, slots, to, scales, n in (
            ("rows", "row_slot", "comp_kv", "comp_scale", s["case"]["page_rows"]),
            ("window", "swa_slot", "swa_kv", "swa_scale", s["case"]["swa_cap"])):
        took = (s[slots] >= 0).nonzero().flatten()
        at = s[slots][took]
        codes, k = _exact_codes(s[rows][took].double())
        flat, flat_k = s[to].double().view(-1, HD), s[scales].double().view(-1)
        i = at // n * s[to].shape[1] + at % n
        done[to] = flat.index_copy(0, i, codes).view(s[to].shape)
        done[scales] = flat_k.index_copy(0, i, k).view(s[scales].shape)
    return done


def _exact_read(s):
    P, stride = s["case"]["page_rows"], s["codes"].shape[1]
    out = s["out"].double()
    took = (s["slots"] >= 0).nonzero().flatten()
    i = s["slots"][took] // P * stride + s["slots"][took] % P
    out[took] = s["codes"].double().view(-1, HD).index_select(0, i) * s["scale"].double().view(-1, 1)[i]
    return out


def _exact_attention(s):
    c = s["case"]
    P, W, ratio = c["page_rows"], c["window"], c["ratio"]
    cap = s["swa_kv"].shape[1]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    codes, near_codes = s["codes"].view(torch.uint8), s["swa_kv"].view(torch.uint8)
    row_len, pos = s["row_len"].tolist(), s["tok_pos"].tolist()
    for t, b in enumerate(s["tok_seq"].tolist()):
        block = torch.arange(min(row_len[b], pos[t] // ratio), device=DEV)
        page = s["table"][b, block // P].long()
        near = torch.arange(max(0, pos[t] - W + 1), pos[t] + 1, device=DEV) if W else block[:0]
        c8 = torch.cat([codes[page, block % P], near_codes[b, near % cap]]).view(F8).double()
        k = torch.cat([s["scale"][page, block % P], s["swa_scale"][b, near % cap]]).double()
        if not c8.shape[0]:
            continue
        rows = c8 * k[:, None]
        l = s["q"][t].double() @ rows.T / math.sqrt(HD)
        every = l if s["sinks"] is None else torch.cat([l, s["sinks"].double()[:, None]], 1)
        out[t] = torch.exp(l - torch.logsumexp(every, 1, keepdim=True)) @ rows
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "read": _exact_read,
            "attention": _exact_attention}[case["op"]](s)
