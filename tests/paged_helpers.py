"""Plain implementations of the paged-cache calls, from their definitions:
Python integers for the plan, float64 for the attention."""
from __future__ import annotations

import numpy as np
import torch

from sparse_compressed_kv_gb300 import csa

HD = 512


# ---------------------------------------------------------------- plan

def plan_reference(*, ratio, page_rows, swa_cap, seq_len, new_len, table, free_ring, free_pos,
                   tok_cap, row_cap):
    """The outputs of one plan as lists, and the status bits it raises."""
    B, N = len(seq_len), len(free_ring)
    table, ring = [list(r) for r in table], list(free_ring)
    max_pages = len(table[0])
    pages_of = lambda tokens: -(-(tokens // ratio) // page_rows)
    bad = 0
    if any(s < 0 or s >= 1 << 48 or n < -1 for s, n in zip(seq_len, new_len)):
        bad |= csa.DEV_BAD_LENGTH
    fine = [(s, n) for s, n in zip(seq_len, new_len) if 0 <= s < 1 << 48 and n >= -1]
    if any(max(pages_of(s), pages_of(s + n)) > max_pages for s, n in fine):
        bad |= csa.DEV_CAPACITY
    need = sum(pages_of(s + n) - pages_of(s) for s, n in fine if n >= 0)
    rel = sum(pages_of(s) for s, n in fine if n < 0)
    head, tail = free_pos
    if not (0 <= head <= tail <= head + N):
        bad |= csa.DEV_BAD_LAYOUT
    elif need > tail - head:
        bad |= csa.DEV_CAPACITY
    elif tail + rel - head > N:
        bad |= csa.DEV_BAD_LAYOUT
    if sum(n for _, n in fine if n > 0) > tok_cap or \
            sum((s + n) // ratio - s // ratio for s, n in fine if n > 0) > row_cap:
        bad |= csa.DEV_CAPACITY
    o = dict(seq_len_out=[], row_len=[], swa_first_pos=[], tok_off=[0], row_off=[0], tok_seq=[],
             tok_pos=[], swa_slot=[], row_slot=[])
    freed = []
    for b in range(B):
        end = seq_len[b]
        if not bad and new_len[b] < 0:
            freed += table[b][:pages_of(end)]
            end = 0
        elif not bad:
            have, held = end, pages_of(end)
            end += new_len[b]
            for p in range(have, end):
                o["tok_seq"].append(b)
                o["tok_pos"].append(p)
                o["swa_slot"].append(b * swa_cap + p % swa_cap if p >= end - swa_cap else -1)
            for g in range(have // ratio, end // ratio):
                if g // page_rows == held:
                    table[b][held] = ring[head % N]
                    head, held = head + 1, held + 1
                o["row_slot"].append(table[b][g // page_rows] * page_rows + g % page_rows)
        o["tok_off"].append(len(o["tok_seq"]))
        o["row_off"].append(len(o["row_slot"]))
        o["seq_len_out"].append(end)
        o["row_len"].append(end // ratio if end > 0 else 0)
        o["swa_first_pos"].append(max(0, end - swa_cap))
    for page in freed:
        ring[tail % N] = page
        tail += 1
    for k, cap in (("tok_seq", tok_cap), ("tok_pos", tok_cap), ("swa_slot", tok_cap),
                   ("row_slot", row_cap)):
        o[k] += [-1] * (cap - len(o[k]))
    return dict(o, table=table, free_ring=ring, free_pos_out=[head, tail]), bad


def plan_tensors(device, *, seq_len, new_len, table, free_ring, free_pos, tok_cap, row_cap):
    B = len(seq_len)
    i64 = lambda x: torch.tensor(x, dtype=torch.int64, device=device)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=device)
    fill = lambda n, dt: torch.full((n,), -9, dtype=dt, device=device)
    return dict(seq_len=i64(seq_len), new_len=i32(new_len), table=i32(table),
                free_ring=i32(free_ring), free_pos=i64(free_pos),
                seq_len_out=fill(B, torch.int64), row_len=fill(B, torch.int64),
                swa_first_pos=fill(B, torch.int64), free_pos_out=fill(2, torch.int64),
                tok_off=fill(B + 1, torch.int64), row_off=fill(B + 1, torch.int64),
                tok_seq=fill(tok_cap, torch.int32), tok_pos=fill(tok_cap, torch.int64),
                swa_slot=fill(tok_cap, torch.int64), row_slot=fill(row_cap, torch.int64))


def pool(seed, seq_len, *, ratio, page_rows, max_pages, extra, head=0):
    """A consistent pool: a table with the requests' pages in random order, and
    the free ring with `extra` pages, starting at `head`."""
    rng = np.random.default_rng(seed)
    held = [-(-(s // ratio) // page_rows) for s in seq_len]
    N = sum(held) + extra
    perm = rng.permutation(N).tolist()
    table, at = [], 0
    for n in held:
        table.append(perm[at:at + n] + [-5] * (max_pages - n))
        at += n
    ring = [-7] * N
    for i, page in enumerate(perm[at:]):
        ring[(head + i) % N] = page
    return table, ring, [head, head + extra]


# ---------------------------------------------------------------- attention

def bf16(gen, *shape):
    return torch.randn(*shape, generator=gen).to(torch.bfloat16)


class Paged:
    """A paged cache on the CPU, its window rings, and one query per token.
    Memory that belongs to no row is NaN."""

    def __init__(self, seed, *, row_len, tokens, ratio=4, page_rows=16, gap=0, heads=16, window=128,
                 swa_cap=None, sinks=False, spare_pages=2, max_pages=None, value=1.0):
        g = torch.Generator().manual_seed(seed)
        self.ratio, self.page_rows, self.heads, self.window = ratio, page_rows, heads, window
        B = len(row_len)
        pages = [-(-n // page_rows) for n in row_len]
        num_pages = sum(pages) + spare_pages
        max_pages = max_pages or max(1, max(pages)) + 1
        perm = torch.randperm(num_pages, generator=g)
        self.table = torch.full((B, max_pages), -1, dtype=torch.int32)
        self.cache = torch.full((num_pages, page_rows + gap, HD), float("nan"), dtype=torch.bfloat16)
        at = 0
        for b, n in enumerate(row_len):
            own = perm[at:at + pages[b]]
            at += pages[b]
            self.table[b, :pages[b]] = own.int()
            r = torch.arange(n)
            self.cache[own[r // page_rows], r % page_rows] = bf16(g, n, HD) * value
        # tokens: (sequence, position) pairs; a sequence -1 is padding
        self.tok_seq = torch.tensor([b for b, _ in tokens], dtype=torch.int32)
        self.tok_pos = torch.tensor([p for _, p in tokens], dtype=torch.int64)
        self.row_len = torch.tensor(row_len, dtype=torch.int64)
        ends = [max([p + 1 for q, p in tokens if q == b], default=0) for b in range(B)]
        cap = swa_cap or max(1, window) + 7
        self.swa_kv = bf16(g, B, cap, HD)
        self.swa_first_pos = torch.tensor([max(0, e - cap) for e in ends], dtype=torch.int64)
        self.q = bf16(g, len(tokens), heads, HD)
        self.sinks = torch.randn(heads, generator=g) if sinks else None
        self.scale = HD ** -0.5

    def rows_of(self, t):
        """The rows token t attends, as the definition lists them."""
        b, p = int(self.tok_seq[t]), int(self.tok_pos[t])
        n = min(int(self.row_len[b]), p // self.ratio)
        j = torch.arange(n)
        held = self.cache[self.table[b, j // self.page_rows].long(), j % self.page_rows]
        x = torch.arange(max(0, p - self.window + 1), p + 1) if self.window else j[:0]
        return torch.cat([held, self.swa_kv[b, x % self.swa_kv.shape[1]]]).double()

    def reference(self, skip=lambda t: None, tokens=None):
        """float64 [T, H, 512]; `skip(t)` names rows that token t does not see."""
        out = torch.full((len(self.tok_seq), self.heads, HD), float("nan"), dtype=torch.float64)
        for t, b in enumerate(self.tok_seq.tolist()):
            if b < 0 or (tokens is not None and t not in tokens):
                continue
            rows, gone = self.rows_of(t), skip(t)
            if gone is not None:
                rows = rows[[i for i in range(len(rows)) if i not in gone]]
            if not len(rows):
                out[t] = 0
                continue
            l = self.scale * self.q[t].double() @ rows.T
            every = l if self.sinks is None else torch.cat([l, self.sinks.double()[:, None]], 1)
            out[t] = torch.exp(l - torch.logsumexp(every, 1, keepdim=True)) @ rows
        return out

    def run(self, device, out_dtype, fill=7.0, stream=None):
        """The GPU's output (guarded), the status word and the guard's state."""
        from tests.gpu_helpers import Guarded
        to = lambda x: None if x is None else x.to(device)
        ring = dict(swa_kv=to(self.swa_kv), swa_first_pos=to(self.swa_first_pos)) if self.window else {}
        layout = csa.PagedLayout(to(self.tok_seq), to(self.tok_pos), to(self.row_len),
                                 to(self.table), self.page_rows, **ring)
        prm = csa.params(self.heads, 1, self.window, self.ratio, self.scale)
        out = Guarded((len(self.tok_seq), self.heads, HD), out_dtype, device, fill)
        ws = Guarded((csa.csa_paged_workspace_size(layout, prm),), torch.uint8, device, 0xEE)
        status = torch.zeros(1, dtype=torch.int32, device=device)
        cache, q, sinks = to(self.cache), to(self.q), to(self.sinks)
        csa.csa_paged_attention(layout, prm, cache, q, out.t, status, ws.t, sinks=sinks,
                                stream=stream)
        torch.cuda.synchronize()
        assert out.intact() and ws.intact(), "guard band overwritten"
        return out.t, int(status.item())


# Relative 2-norm error of a token's output, for random rows (their rounding
# errors add like the rows themselves, in squares).
#   bf16: the weights rounded to bf16 (half a step: 2^-8) and the output
#     rounded to bf16 (2^-8): at most sqrt(2) 2^-8.
#   f32: weights as two bf16 terms (2^-8 of 2^-8); sums of 16 products at a
#     time into a truncating f32 accumulator, one step (2^-23) each: 32 of
#     them in a logit of magnitude at most 6 (six sigma), which is the weight's
#     relative error; at most 160 of them (2560 rows) in an output before
#     partial sums are added with rounding, each half a step on average.
REL = {torch.bfloat16: 2 ** 0.5 * 2 ** -8,
       torch.float32: 2 ** -16 + 6 * 32 * 2 ** -23 + 128 * 2 ** -23}


def check(got, ref, dtype, tokens=None):
    got = got.double().cpu()
    for t in range(len(ref)) if tokens is None else tokens:
        norm = ref[t].norm()
        err = (got[t] - ref[t]).norm()
        assert err <= REL[dtype] * norm, f"token {t}: off by {float(err / norm):.3e}"
