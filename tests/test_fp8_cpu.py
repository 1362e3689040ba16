"""8-bit paged caches on the CPU: argument errors are decided before anything is
launched, the binding refuses wrong tensors, and the tests' reference is what
the format says."""
import ctypes

import numpy as np
import pytest
import torch

from sparse_compressed_kv_gb300 import build as B
from sparse_compressed_kv_gb300 import csa
from tests import fp8_helpers as F

INVALID, UNSUPPORTED, CAPACITY, WORKSPACE = 1, 2, 3, 7
PTR = 1 << 20
BIG = 1 << 24


@pytest.fixture(scope="module")
def lib():
    B.build()
    return csa.load()


def test_reference_is_the_format():
    # torch's own view of the 256 codes, and its rounding of values
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double()
    got = F.values(codes[:, None], torch.ones(256))[:, 0]
    assert torch.equal(got.nan_to_num(999), want.nan_to_num(999))
    g = torch.Generator().manual_seed(1)
    x = torch.randn(500, 64, generator=g) * torch.exp2(torch.randint(-8, 8, (500, 64), generator=g).float())
    c, k = F.quantise(x.double().numpy())
    y = (x.double() / torch.from_numpy(k)[:, None])
    assert float(y.abs().max()) <= 448 and (y.abs().amax(1) > 224).all()
    assert torch.equal(torch.from_numpy(c), y.float().to(torch.float8_e4m3fn).view(torch.uint8))


def test_reference_at_the_borders():
    top = [448.0, 448.0000001, 449, 896, 224, 0, 2.0 ** 70, 2.0 ** -100, 448 * 2.0 ** 60]
    c, k = F.quantise(np.array([[t] * 16 for t in top]))
    assert np.log2(k).tolist() == [0, 1, 1, 1, -1, -60, 60, -60, 60]
    assert c[:, 0].tolist() == [126, 118, 118, 126, 126, 0, 127, 0, 126]
    c, k = F.quantise(np.array([[np.inf, -np.inf, np.nan, 1.0, -0.0] + [0] * 11]))
    assert c[0, :5].tolist() == [127, 255, 127, 126 - 6, 128] and k[0] == 2.0 ** -8


def job(**changes):
    return csa.csa_append_fp8_job_t(**{**dict(
        rows=PTR, slots=PTR + BIG, num_rows=3, row_pitch=1024, type=1, width=512, page_rows=16,
        num_pages=4, page_stride=16, scale_stride=16, cache=PTR + 2 * BIG, scales=PTR + 3 * BIG), **changes})


STATUS = PTR + 4 * BIG


@pytest.mark.parametrize("changes,code", [
    (dict(num_rows=-1), INVALID), (dict(width=0), INVALID), (dict(width=24), INVALID),
    (dict(page_rows=0), INVALID), (dict(num_pages=0), INVALID), (dict(page_stride=15), INVALID),
    (dict(scale_stride=15), INVALID), (dict(row_pitch=1008), INVALID), (dict(row_pitch=1032), INVALID),
    (dict(type=2), INVALID), (dict(type=-1), INVALID), (dict(type=0), INVALID),     # f32: a row is 2048 bytes
    (dict(rows=None), INVALID), (dict(slots=None), INVALID), (dict(cache=None), INVALID),
    (dict(scales=None), INVALID), (dict(rows=PTR + 8), INVALID), (dict(cache=PTR + 8), INVALID),
    (dict(slots=PTR + 4), INVALID), (dict(scales=PTR + 2), INVALID),
    (dict(width=1040, row_pitch=2080), UNSUPPORTED), (dict(num_pages=1 << 31), UNSUPPORTED),
    (dict(num_pages=1 << 28), UNSUPPORTED), (dict(num_rows=1 << 31), UNSUPPORTED),
    (dict(page_stride=1 << 31), UNSUPPORTED), (dict(scale_stride=1 << 31), UNSUPPORTED),
    (dict(row_pitch=1 << 31), UNSUPPORTED),
    # what is read under what is written
    (dict(rows=PTR + 2 * BIG + 512), INVALID), (dict(rows=PTR + 3 * BIG), INVALID),
    (dict(slots=PTR + 2 * BIG), INVALID), (dict(slots=PTR + 3 * BIG + 248), INVALID),
    (dict(cache=STATUS - 512 * 64 + 512), INVALID), (dict(scales=STATUS - 252), INVALID),
])
def test_append_refusals(lib, changes, code):
    jobs = (csa.csa_append_fp8_job_t * 2)(job(), job(**changes))
    assert lib.csa_paged_append_fp8(jobs, 2, STATUS, None) == code


def test_append_refuses_rows_under_another_jobs_cache(lib):
    jobs = (csa.csa_append_fp8_job_t * 2)(job(), job(cache=PTR + 8 * BIG, scales=PTR + 9 * BIG, rows=PTR + 2 * BIG))
    assert lib.csa_paged_append_fp8(jobs, 2, STATUS, None) == INVALID


def test_append_counts(lib):
    jobs = (csa.csa_append_fp8_job_t * 5)(*[job() for _ in range(5)])
    assert lib.csa_paged_append_fp8(jobs, 0, STATUS, None) == INVALID
    assert lib.csa_paged_append_fp8(jobs, 5, STATUS, None) == UNSUPPORTED
    assert lib.csa_paged_append_fp8(None, 1, STATUS, None) == INVALID
    assert lib.csa_paged_append_fp8(jobs, 1, None, None) == INVALID
    assert lib.csa_paged_append_fp8(jobs, 1, STATUS + 2, None) == INVALID
    empty = (csa.csa_append_fp8_job_t * 1)(job(num_rows=0, rows=None, slots=None, cache=None, scales=None))
    assert lib.csa_paged_append_fp8(empty, 1, STATUS, None) == 0


def read(**changes):
    return csa.csa_read_fp8_t(**{**dict(
        cache=PTR, scales=PTR + BIG, slots=PTR + 2 * BIG, num_rows=3, width=512, page_rows=16, num_pages=4,
        page_stride=16, scale_stride=16, type=1, out_pitch=1024, out=PTR + 3 * BIG), **changes})


@pytest.mark.parametrize("changes,code", [
    (dict(num_rows=-1), INVALID), (dict(width=8), INVALID), (dict(page_rows=0), INVALID),
    (dict(num_pages=0), INVALID), (dict(page_stride=15), INVALID), (dict(scale_stride=15), INVALID),
    (dict(type=2), INVALID), (dict(type=0), INVALID), (dict(out_pitch=1016), INVALID),
    (dict(out_pitch=1000), INVALID), (dict(cache=None), INVALID), (dict(scales=None), INVALID),
    (dict(slots=None), INVALID), (dict(out=None), INVALID), (dict(cache=PTR + 8), INVALID),
    (dict(out=PTR + 8), INVALID), (dict(slots=PTR + 4), INVALID), (dict(scales=PTR + 2), INVALID),
    (dict(width=1040, out_pitch=2080), UNSUPPORTED), (dict(num_pages=1 << 28), UNSUPPORTED),
    (dict(num_rows=1 << 31), UNSUPPORTED), (dict(page_stride=1 << 31), UNSUPPORTED),
    (dict(out_pitch=1 << 31), UNSUPPORTED),
    (dict(out=PTR), INVALID), (dict(out=PTR + BIG), INVALID), (dict(out=PTR + 2 * BIG), INVALID),
    (dict(out=STATUS - 1024), INVALID),
])
def test_read_refusals(lib, changes, code):
    assert lib.csa_paged_read_fp8(ctypes.byref(read(**changes)), STATUS, None) == code


def test_read_null_arguments(lib):
    assert lib.csa_paged_read_fp8(None, STATUS, None) == INVALID
    assert lib.csa_paged_read_fp8(ctypes.byref(read()), None, None) == INVALID
    none = read(num_rows=0, cache=None, scales=None, slots=None, out=None)
    assert lib.csa_paged_read_fp8(ctypes.byref(none), STATUS, None) == 0


NAMES = ("tok_seq", "tok_pos", "row_len", "table", "swa_kv", "swa_first_pos")


def attend(lib, P=None, null=(), **changes):
    at = {n: PTR + BIG * i for i, n in enumerate(NAMES + ("cache", "scales", "swa_scales", "q", "sinks", "out",
                                                          "status", "ws"))}
    a = {**dict(num_seqs=2, num_tokens=3, page_rows=16, max_pages=8, swa_cap=128, num_pages=16, page_stride=16,
                scale_stride=16, out_type=0, ws_bytes=1 << 40), **at, **changes, **{n: None for n in null}}
    L = csa.csa_paged_layout_t(**{n: a[n] for n in NAMES + ("num_seqs", "num_tokens", "page_rows", "max_pages",
                                                            "swa_cap")})
    return lib.csa_paged_attention_fp8(
        ctypes.byref(L), ctypes.byref(P or csa.params(16, 1)), a["cache"], a["scales"], a["swa_scales"],
        a["num_pages"], a["page_stride"], a["scale_stride"], a["q"], a["sinks"], a["out_type"], a["out"],
        a["status"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("changes,code", [
    (dict(num_seqs=0), INVALID), (dict(num_tokens=-1), INVALID), (dict(page_rows=0), INVALID),
    (dict(max_pages=0), INVALID), (dict(num_tokens=8193), UNSUPPORTED), (dict(max_pages=1 << 27), UNSUPPORTED),
    (dict(num_pages=0), INVALID), (dict(page_stride=15), INVALID), (dict(scale_stride=15), INVALID),
    (dict(num_pages=1 << 31), UNSUPPORTED), (dict(num_pages=1 << 28), UNSUPPORTED),
    (dict(scale_stride=1 << 31), UNSUPPORTED), (dict(out_type=2), INVALID), (dict(swa_cap=127), CAPACITY),
    (dict(num_seqs=1 << 24), UNSUPPORTED), (dict(ws_bytes=100), WORKSPACE), (dict(ws=PTR + 13 * BIG + 128), INVALID),
    (dict(scales=PTR + 2), INVALID), (dict(swa_scales=PTR + 2), INVALID), (dict(cache=PTR + 8), INVALID),
    (dict(q=PTR + 8), INVALID), (dict(swa_kv=PTR + 8), INVALID),
] + [(dict(null=(n,)), WORKSPACE if n == "ws" else INVALID) for n in NAMES + ("cache", "scales", "swa_scales", "q",
                                                                           "out", "status", "ws")])
def test_attention_refusals(lib, changes, code):
    assert attend(lib, **changes) == code


@pytest.mark.parametrize("changes,code", [
    (dict(hd=256), UNSUPPORTED), (dict(n_heads=0), INVALID), (dict(n_heads=129), UNSUPPORTED),
    (dict(window=-1), INVALID), (dict(ratio=0), INVALID), (dict(scale=float("nan")), INVALID),
])
def test_attention_param_refusals(lib, changes, code):
    P = csa.params(16, 1)
    for k, v in changes.items():
        setattr(P, k, v)
    assert attend(lib, P=P) == code


@pytest.mark.parametrize("written", ["out", "ws", "status"])
def test_attention_refuses_outputs_over_inputs(lib, written):
    where = {n: PTR + BIG * i for i, n in enumerate(NAMES + ("cache", "scales", "swa_scales", "q", "sinks", "out",
                                                             "status", "ws"))}
    for n in NAMES + ("swa_scales", "q", "sinks", "out", "status", "ws"):
        if n != written:
            assert attend(lib, **{written: where[n]}) == INVALID, n


def test_attention_of_no_tokens_launches_nothing(lib):
    assert attend(lib, num_tokens=0, null=("q", "out", "tok_seq", "tok_pos")) == 0


F8, BF = torch.float8_e4m3fn, torch.bfloat16


@pytest.mark.parametrize("change,what", [
    (dict(rows=torch.zeros(3, 512, dtype=torch.float16)), "rows"),
    (dict(rows=torch.zeros(3, 4, 128, dtype=BF)), "rows"),
    (dict(rows=torch.zeros(3, 256, dtype=BF)), "values"),
    (dict(cache=torch.zeros(4, 16, 512, dtype=BF)), "float8"),
    (dict(cache=torch.zeros(4, 16 * 512).to(F8)), "float8"),
    (dict(scales=torch.zeros(4, 16, dtype=BF)), "scales"),
    (dict(scales=torch.zeros(4, 16, 1)), "scales"),
    (dict(scales=torch.zeros(3, 16)), "scales"),
    (dict(scales=torch.zeros(4, 15)), "page"),
    (dict(scales=torch.zeros(4, 32)[:, ::2]), "page"),
    (dict(cache=torch.zeros(4, 15, 512).to(F8)), "page"),
    (dict(rows=torch.zeros(512, 3, dtype=BF).T), "contiguous"),
    (dict(), "GPU"),
])
def test_binding_refuses(change, what):
    a = {**dict(rows=torch.zeros(3, 512, dtype=BF), cache=torch.zeros(4, 16, 512).to(F8),
                scales=torch.zeros(4, 16)), **change}
    with pytest.raises(ValueError, match=what):
        csa.AppendJobFp8(a["rows"], torch.zeros(3, dtype=torch.int64), a["cache"], a["scales"], 16)


@pytest.mark.parametrize("change,what", [
    (dict(out=torch.zeros(3, 512, dtype=torch.float16)), "out"), (dict(out=torch.zeros(3, 256)), "values"),
    (dict(out=torch.zeros(4, 512)), "slots"), (dict(slots=torch.zeros(3, dtype=torch.int32)), "slots"),
    (dict(out=torch.zeros(512, 3).T), "contiguous"), (dict(out=torch.zeros(1, 512).expand(3, 512)), "overlap"),
])
def test_binding_refuses_reads(change, what):
    a = {**dict(out=torch.zeros(3, 512), slots=torch.zeros(3, dtype=torch.int64)), **change}
    with pytest.raises(ValueError, match=what):
        csa.csa_paged_read_fp8(torch.zeros(4, 16, 512).to(F8), torch.zeros(4, 16), a["slots"], a["out"], None, 16)
