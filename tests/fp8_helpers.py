"""Plain implementations of the 8-bit paged-cache calls, from their
definitions: the format's 127 magnitudes as a table, float64 for the rest."""
from __future__ import annotations

import numpy as np
import torch

from sparse_compressed_kv_gb300 import csa
from tests import paged_helpers as H

F8 = torch.float8_e4m3fn
HD = H.HD

# magnitudes of codes 0 .. 126 (4 exponent bits of bias 7, 3 mantissa bits; 127 is NaN)
E4M3 = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) for c in range(127)])


def quantise(rows) -> tuple:
    """Float64 rows [n, width] -> codes uint8 [n, width], scales float64 [n]."""
    x = np.asarray(rows, dtype=np.float64)
    top = np.where(np.isfinite(x), np.abs(x), 0).max(axis=1, initial=0.0)
    k = np.full(len(x), -60)
    for e in range(-60, 60):                    # the least k with top <= 448 2^k
        k[top > 448 * 2.0 ** e] = e + 1
    with np.errstate(invalid="ignore"):
        y = np.abs(x) / (2.0 ** k)[:, None]
    hi = np.searchsorted(E4M3, np.where(np.isfinite(y), y, 0), side="left").clip(0, 126)
    lo = (hi - 1).clip(0)
    with np.errstate(invalid="ignore"):
        up, down = E4M3[hi] - y, y - E4M3[lo]
        code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
        code = np.where(np.isfinite(y) & (y <= 448), code, 127)
    sign = np.where(np.isnan(x), 0, np.signbit(x))
    return (code + 128 * sign).astype(np.uint8), 2.0 ** k


def values(codes, scales):
    """Codes uint8 [..., width] and scales [...] -> float64."""
    c = torch.as_tensor(codes).long()
    table = torch.tensor(np.append(E4M3, np.nan))
    v = table[c & 127] * torch.where(c >= 128, -1.0, 1.0).double()
    return v * torch.as_tensor(scales).double()[..., None]


class PagedFp8(H.Paged):
    """A paged 8-bit cache on the CPU.  Rows differ in magnitude by up to
    2^spread; `cache` and `swa_kv` hold the values that the codes stand for."""

    def __init__(self, seed, *, spread=2.0, row_len, **kw):
        super().__init__(seed, row_len=row_len, **kw)
        g = torch.Generator().manual_seed(seed + 1)
        self.codes, self.scales = self._pack(self.cache, g, spread)
        self.swa_codes, self.swa_scales = self._pack(self.swa_kv, g, spread)
        self.requantised()

    @staticmethod
    def _pack(rows, g, spread):
        flat = rows.reshape(-1, HD).double()
        flat = flat * torch.exp2(spread * (torch.rand(len(flat), 1, generator=g).double() - 0.5))
        codes, scales = quantise(flat.numpy())
        unwritten = flat.isnan().all(1).numpy()
        scales[unwritten] = np.nan
        return (torch.from_numpy(codes).view(rows.shape),
                torch.from_numpy(scales).float().view(rows.shape[:-1]))

    def requantised(self):
        """The values again, after a test changed codes or scales."""
        self.cache = values(self.codes, self.scales)
        self.swa_kv = values(self.swa_codes, self.swa_scales)

    def arguments(self, device):
        to = lambda x: None if x is None else x.to(device)
        f8 = lambda x: x.to(device).view(F8)
        ring = dict(swa_kv=f8(self.swa_codes), swa_scales=to(self.swa_scales),
                    swa_first_pos=to(self.swa_first_pos)) if self.window else {}
        layout = csa.PagedLayoutFp8(to(self.tok_seq), to(self.tok_pos), to(self.row_len), to(self.table),
                                    self.page_rows, **ring)
        prm = csa.params(self.heads, 1, self.window, self.ratio, self.scale)
        return layout, prm, f8(self.codes), to(self.scales), to(self.q), to(self.sinks)

    def run(self, device, out_dtype, fill=7.0, stream=None):
        from tests.gpu_helpers import Guarded
        layout, prm, codes, scales, q, sinks = self.arguments(device)
        out = Guarded((len(self.tok_seq), self.heads, HD), out_dtype, device, fill)
        ws = Guarded((csa.csa_paged_workspace_size(layout, prm),), torch.uint8, device, 0xEE)
        status = torch.zeros(1, dtype=torch.int32, device=device)
        csa.csa_paged_attention_fp8(layout, prm, codes, scales, q, out.t, status, ws.t, sinks=sinks,
                                    stream=stream)
        torch.cuda.synchronize()
        assert out.intact() and ws.intact(), "guard band overwritten"
        return out.t, int(status.item())


# Relative 2-norm error of a token's output, for random rows (their rounding
# errors add like the rows themselves, in squares; rows differ in magnitude by
# at most 4 and logits stay below 12).
#   bf16: a weight off by at most 2^-9, the output rounded to bf16 (2^-8).
#   f32: a weight off by at most 2^-18.  Its logit: 16 products of 32 columns into
#     an f32 accumulator, one step (2^-23) each, and products with the scales.
#     The query: a value below 2^-2 where its head's largest is brought to 224
#     (3.5: 2^-8, one value in 300) is off by 2^-10, 2^-17.8 of the largest; two of
#     512, times a row's values (2.5 times a magnitude of 2) and the scale 512^-.5: at
#     most 2^-17.  The output: sums of
#     32 rows, six terms each, at most 1,728 rows before they are added, rounded, to the partial:
#     324 steps, half of 2^-23 each on average.
REL = {torch.bfloat16: (2 ** -18 + 2 ** -16) ** 0.5,
       torch.float32: 2 ** -18 + 12 * 19 * 2 ** -23 + 2 ** -17 + 162 * 2 ** -23}


def check(got, ref, dtype, tokens=None, rel=None):
    got = got.double().cpu()
    for t in range(len(ref)) if tokens is None else tokens:
        norm = ref[t].norm()
        err = (got[t] - ref[t]).norm()
        assert err <= (rel or REL[dtype]) * norm, f"token {t}: off by {float(err / norm):.3e}"
