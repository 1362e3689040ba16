"""ctypes binding of libcsa.so (see include/csa.h) -- argument marshalling only.

Every function here takes torch tensors that already live on the current CUDA
device, turns them into the C ABI's plain pointers and sizes, and calls the
entry point of the same name on torch's current stream.  No step of the
computation runs in Python, and there is no fallback: if libcsa.so is missing
or the GPU is not an sm_103 part, the calls raise.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# CSA_CHECKS=1 in the environment selects the build with internal bounds
# checks (libcsa_checks.so: same entry points, CSA_DEV_CHECK on a failed check)
LIB_PATH = os.path.join(_HERE, "libcsa_checks.so" if os.environ.get("CSA_CHECKS") == "1"
                        else "libcsa.so")

CSA_OK = 0
STATUS_NAMES = {
    0: "CSA_OK", 1: "CSA_ERR_INVALID_ARGUMENT", 2: "CSA_ERR_UNSUPPORTED", 3: "CSA_ERR_CAPACITY",
    4: "CSA_ERR_CUDA", 5: "CSA_ERR_DEVICE_FAULT", 6: "CSA_ERR_TIMEOUT", 7: "CSA_ERR_WORKSPACE",
}
DEV_BAD_INDEX, DEV_MISSING_SWA, DEV_BAD_LAYOUT = 0x01, 0x02, 0x04
DEV_CAPACITY, DEV_BAD_LENGTH, DEV_TIMEOUT = 0x08, 0x10, 0x20
DEV_CHECK = 0x40

EXPORTS = ("csa_status_string", "csa_abi_version", "csa_workspace_size", "csa_indexer_scores",
           "csa_topk", "csa_indexer_topk", "csa_gather_mixed", "csa_sparse_mqa_decode", "csa_decode",
           "csa_hca_workspace_size", "csa_hca_decode", "csa_fp4_quantize_keys",
           "csa_indexer_scores_fp4", "csa_decode_fp4", "csa_shard_workspace_size",
           "csa_shard_candidates", "csa_shard_merge", "csa_shard_attention", "csa_window_attention",
           "csa_shard_combine", "csa_page_plan", "csa_paged_append", "csa_paged_workspace_size",
           "csa_paged_attention", "csa_paged_append_fp8", "csa_paged_read_fp8",
           "csa_paged_attention_fp8")
MAX_APPEND_JOBS = 4  # csa_paged_append's limit (include/csa.h)
MAX_SHARDS = 8  # csa_shard_merge's limit (include/csa.h)
FP4_ROW = 80  # bytes per MXFP4 key row (include/csa.h)


class CsaError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn}: {STATUS_NAMES.get(code, code)}")
        self.code = code


class csa_layout_t(ctypes.Structure):
    _fields_ = [
        ("num_seqs", ctypes.c_int32), ("num_tokens", ctypes.c_int32),
        ("total_comp_rows", ctypes.c_int64), ("max_comp_rows", ctypes.c_int64),
        ("tok_seq", ctypes.c_void_p), ("tok_pos", ctypes.c_void_p), ("comp_off", ctypes.c_void_p),
        ("swa_kv", ctypes.c_void_p), ("swa_cap", ctypes.c_int32),
        ("swa_first_pos", ctypes.c_void_p),
    ]


class csa_params_t(ctypes.Structure):
    _fields_ = [
        ("n_ih", ctypes.c_int32), ("ihd", ctypes.c_int32), ("hd", ctypes.c_int32),
        ("n_heads", ctypes.c_int32), ("top_k", ctypes.c_int32), ("window", ctypes.c_int32),
        ("ratio", ctypes.c_int32), ("scale", ctypes.c_float),
    ]


class csa_page_plan_t(ctypes.Structure):
    _fields_ = [
        ("num_seqs", ctypes.c_int32), ("ratio", ctypes.c_int32), ("page_rows", ctypes.c_int32),
        ("max_pages", ctypes.c_int32), ("num_pages", ctypes.c_int64), ("tok_cap", ctypes.c_int64),
        ("row_cap", ctypes.c_int64), ("swa_cap", ctypes.c_int32),
    ] + [(name, ctypes.c_void_p) for name in (
        "seq_len", "new_len", "table", "free_ring", "free_pos", "seq_len_out", "row_len",
        "swa_first_pos", "free_pos_out", "tok_off", "row_off", "tok_seq", "tok_pos", "swa_slot",
        "row_slot")]


class csa_append_job_t(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_void_p), ("slots", ctypes.c_void_p), ("num_rows", ctypes.c_int64),
        ("row_pitch", ctypes.c_int64), ("row_bytes", ctypes.c_int32), ("page_rows", ctypes.c_int32),
        ("num_pages", ctypes.c_int64), ("page_stride", ctypes.c_int64), ("cache", ctypes.c_void_p),
    ]


class csa_paged_layout_t(ctypes.Structure):
    _fields_ = [
        ("num_seqs", ctypes.c_int32), ("num_tokens", ctypes.c_int32), ("page_rows", ctypes.c_int32),
        ("max_pages", ctypes.c_int32), ("tok_seq", ctypes.c_void_p), ("tok_pos", ctypes.c_void_p),
        ("row_len", ctypes.c_void_p), ("table", ctypes.c_void_p), ("swa_kv", ctypes.c_void_p),
        ("swa_cap", ctypes.c_int32), ("swa_first_pos", ctypes.c_void_p),
    ]


class csa_append_fp8_job_t(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_void_p), ("slots", ctypes.c_void_p), ("num_rows", ctypes.c_int64),
        ("row_pitch", ctypes.c_int64), ("type", ctypes.c_int), ("width", ctypes.c_int32),
        ("page_rows", ctypes.c_int32), ("num_pages", ctypes.c_int64),
        ("page_stride", ctypes.c_int64), ("scale_stride", ctypes.c_int64),
        ("cache", ctypes.c_void_p), ("scales", ctypes.c_void_p),
    ]


class csa_read_fp8_t(ctypes.Structure):
    _fields_ = [
        ("cache", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("slots", ctypes.c_void_p),
        ("num_rows", ctypes.c_int64), ("width", ctypes.c_int32), ("page_rows", ctypes.c_int32),
        ("num_pages", ctypes.c_int64), ("page_stride", ctypes.c_int64),
        ("scale_stride", ctypes.c_int64), ("type", ctypes.c_int), ("out_pitch", ctypes.c_int64),
        ("out", ctypes.c_void_p),
    ]


_lib = None


def load() -> ctypes.CDLL:
    """Load libcsa.so, or libcsa_checks.so under CSA_CHECKS=1 (built by
    sparse_compressed_kv_gb300.build); raise if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{os.path.basename(LIB_PATH)} not found at {LIB_PATH}: run the "
                           "build (python -m sparse_compressed_kv_gb300.build --all) first")
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.c_void_p
    L = ctypes.POINTER(csa_layout_t)
    Pm = ctypes.POINTER(csa_params_t)
    i32, i64, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    lib.csa_status_string.argtypes = [ctypes.c_int]
    lib.csa_status_string.restype = ctypes.c_char_p
    lib.csa_abi_version.restype = i32
    lib.csa_workspace_size.argtypes = [L, Pm, ctypes.POINTER(sz)]
    lib.csa_indexer_scores.argtypes = [L, Pm, P, P, P, P, i64, P, P]
    lib.csa_topk.argtypes = [L, Pm, P, i64, P, P, P, P, sz, P]
    lib.csa_indexer_topk.argtypes = [L, Pm, P, P, P, P, P, P, P, sz, P]
    lib.csa_gather_mixed.argtypes = [L, Pm, P, P, P, P, P, P, P]
    lib.csa_sparse_mqa_decode.argtypes = [i32, Pm, P, P, P, P, P, P, P, sz, P]
    lib.csa_decode.argtypes = [L, Pm, P, P, P, P, P, P, P, P, P, P, sz, P]
    lib.csa_hca_workspace_size.argtypes = [L, Pm, ctypes.POINTER(sz)]
    lib.csa_hca_decode.argtypes = [L, Pm, P, P, P, P, P, P, sz, P]
    lib.csa_fp4_quantize_keys.argtypes = [i64, P, P, P]
    lib.csa_indexer_scores_fp4.argtypes = [L, Pm, P, P, P, P, i64, P, P]
    lib.csa_decode_fp4.argtypes = [L, Pm, P, P, P, P, P, P, P, P, P, P, sz, P]
    lib.csa_shard_workspace_size.argtypes = [L, Pm, i64, i64, ctypes.POINTER(sz)]
    lib.csa_shard_candidates.argtypes = [L, Pm, i64, i64, P, P, P, P, P, P, P, P, sz, P]
    lib.csa_shard_merge.argtypes = [i32, i32, i32, ctypes.POINTER(i64), P, P, P, P, P, P, P, P, P]
    lib.csa_shard_attention.argtypes = [L, Pm, i64, i64, P, P, P, P, P, P, P, P, sz, P]
    lib.csa_window_attention.argtypes = [L, Pm, P, P, P, P, P, sz, P]
    lib.csa_shard_combine.argtypes = [i32, i32, i32, P, P, P, P, P, P]
    lib.csa_page_plan.argtypes = [ctypes.POINTER(csa_page_plan_t), P, P]
    lib.csa_paged_append.argtypes = [ctypes.POINTER(csa_append_job_t), i32, P, P]
    Lp = ctypes.POINTER(csa_paged_layout_t)
    lib.csa_paged_workspace_size.argtypes = [Lp, Pm, ctypes.POINTER(sz)]
    lib.csa_paged_attention.argtypes = [Lp, Pm, P, i64, i64, P, P, ctypes.c_int, P, P, P, sz, P]
    lib.csa_paged_append_fp8.argtypes = [ctypes.POINTER(csa_append_fp8_job_t), i32, P, P]
    lib.csa_paged_read_fp8.argtypes = [ctypes.POINTER(csa_read_fp8_t), P, P]
    lib.csa_paged_attention_fp8.argtypes = [Lp, Pm, P, P, P, i64, i64, i64, P, P, ctypes.c_int, P, P, P, sz, P]
    for fn in EXPORTS[2:]:
        getattr(lib, fn).restype = ctypes.c_int
    _lib = lib
    return lib


def _p(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(fn: str, code: int):
    if code != CSA_OK:
        raise CsaError(fn, code)


def params(n_heads: int, top_k: int, window: int = 128, ratio: int = 4,
           scale: Optional[float] = None, n_ih: int = 64, ihd: int = 128,
           hd: int = 512) -> csa_params_t:
    return csa_params_t(n_ih, ihd, hd, n_heads, top_k, window, ratio,
                        float(scale if scale is not None else hd ** -0.5))


class Layout:
    """Device-side layout arrays plus the host-side sizes of csa_layout_t."""

    def __init__(self, tok_seq, tok_pos, comp_off, swa_kv, swa_first_pos,
                 max_comp_rows: int, total_comp_rows: Optional[int] = None,
                 swa_cap: Optional[int] = None):
        self.tok_seq = tok_seq
        self.tok_pos = tok_pos
        self.comp_off = comp_off
        self.swa_kv = swa_kv
        self.swa_first_pos = swa_first_pos
        self.max_comp_rows = int(max_comp_rows)
        self.total_comp_rows = int(total_comp_rows if total_comp_rows is not None
                                   else max_comp_rows)
        self.swa_cap = int(swa_cap if swa_cap is not None else swa_kv.shape[1])

    def c(self) -> csa_layout_t:
        return csa_layout_t(
            int(self.comp_off.shape[0] - 1), int(self.tok_seq.shape[0]), self.total_comp_rows,
            self.max_comp_rows, _p(self.tok_seq), _p(self.tok_pos), _p(self.comp_off),
            _p(self.swa_kv), self.swa_cap, _p(self.swa_first_pos))


def status_string(code: int) -> str:
    return load().csa_status_string(code).decode()


def abi_version() -> int:
    return int(load().csa_abi_version())


def csa_workspace_size(layout: Layout, prm: csa_params_t) -> int:
    n = ctypes.c_size_t(0)
    lc = layout.c()
    _check("csa_workspace_size", load().csa_workspace_size(ctypes.byref(lc), ctypes.byref(prm),
                                                           ctypes.byref(n)))
    return int(n.value)


def workspace(layout: Layout, prm: csa_params_t, device=None) -> torch.Tensor:
    """A zero-filled workspace of csa_workspace_size bytes (allocated by torch)."""
    return torch.zeros(csa_workspace_size(layout, prm), dtype=torch.uint8,
                       device=device or layout.tok_seq.device)


def csa_indexer_scores(layout: Layout, prm: csa_params_t, q_idx, w_idx, k_idx, scores,
                       dev_status, stream=None):
    lc = layout.c()
    _check("csa_indexer_scores", load().csa_indexer_scores(
        ctypes.byref(lc), ctypes.byref(prm), _p(q_idx), _p(w_idx), _p(k_idx), _p(scores),
        int(scores.shape[1]), _p(dev_status), _stream(stream)))


def csa_topk(layout: Layout, prm: csa_params_t, scores, idx, n_sel, dev_status, ws,
             stream=None):
    lc = layout.c()
    _check("csa_topk", load().csa_topk(
        ctypes.byref(lc), ctypes.byref(prm), _p(scores), int(scores.shape[1]), _p(idx),
        _p(n_sel), _p(dev_status), _p(ws), int(ws.numel()), _stream(stream)))


def csa_indexer_topk(layout: Layout, prm: csa_params_t, q_idx, w_idx, k_idx, idx, n_sel,
                     dev_status, ws, stream=None):
    lc = layout.c()
    _check("csa_indexer_topk", load().csa_indexer_topk(
        ctypes.byref(lc), ctypes.byref(prm), _p(q_idx), _p(w_idx), _p(k_idx), _p(idx), _p(n_sel),
        _p(dev_status), _p(ws), int(ws.numel()), _stream(stream)))


def csa_gather_mixed(layout: Layout, prm: csa_params_t, idx, n_sel, comp_kv, kv_buf, kv_len,
                     dev_status, stream=None):
    lc = layout.c()
    _check("csa_gather_mixed", load().csa_gather_mixed(
        ctypes.byref(lc), ctypes.byref(prm), _p(idx), _p(n_sel), _p(comp_kv), _p(kv_buf),
        _p(kv_len), _p(dev_status), _stream(stream)))


def csa_sparse_mqa_decode(prm: csa_params_t, q, kv_buf, kv_len, out, dev_status, ws,
                          sinks=None, stream=None):
    _check("csa_sparse_mqa_decode", load().csa_sparse_mqa_decode(
        int(q.shape[0]), ctypes.byref(prm), _p(q), _p(kv_buf), _p(kv_len), _p(sinks), _p(out),
        _p(dev_status), _p(ws), int(ws.numel()), _stream(stream)))


def csa_decode(layout: Layout, prm: csa_params_t, q_idx, w_idx, k_idx, comp_kv, q, out,
               dev_status, ws, idx_out=None, sinks=None, stream=None):
    lc = layout.c()
    _check("csa_decode", load().csa_decode(
        ctypes.byref(lc), ctypes.byref(prm), _p(q_idx), _p(w_idx), _p(k_idx), _p(comp_kv), _p(q),
        _p(sinks), _p(out), _p(idx_out), _p(dev_status), _p(ws), int(ws.numel()),
        _stream(stream)))


def csa_hca_workspace_size(layout: Layout, prm: csa_params_t) -> int:
    n = ctypes.c_size_t(0)
    lc = layout.c()
    _check("csa_hca_workspace_size", load().csa_hca_workspace_size(
        ctypes.byref(lc), ctypes.byref(prm), ctypes.byref(n)))
    return int(n.value)


def hca_workspace(layout: Layout, prm: csa_params_t, device=None) -> torch.Tensor:
    return torch.zeros(csa_hca_workspace_size(layout, prm), dtype=torch.uint8,
                       device=device or layout.tok_seq.device)


def csa_hca_decode(layout: Layout, prm: csa_params_t, comp_kv, q, out, dev_status, ws,
                   sinks=None, stream=None):
    lc = layout.c()
    _check("csa_hca_decode", load().csa_hca_decode(
        ctypes.byref(lc), ctypes.byref(prm), _p(comp_kv), _p(q), _p(sinks), _p(out),
        _p(dev_status), _p(ws), int(ws.numel()), _stream(stream)))


def csa_fp4_quantize_keys(k_idx, k_fp4, stream=None):
    """bf16 keys [R, 128] -> MXFP4 rows [R, 80] uint8 (both on the GPU)."""
    _check("csa_fp4_quantize_keys", load().csa_fp4_quantize_keys(
        int(k_idx.shape[0]), _p(k_idx), _p(k_fp4), _stream(stream)))


def csa_indexer_scores_fp4(layout: Layout, prm: csa_params_t, q_idx, w_idx, k_fp4, scores,
                           dev_status, stream=None):
    lc = layout.c()
    _check("csa_indexer_scores_fp4", load().csa_indexer_scores_fp4(
        ctypes.byref(lc), ctypes.byref(prm), _p(q_idx), _p(w_idx), _p(k_fp4), _p(scores),
        int(scores.shape[1]), _p(dev_status), _stream(stream)))


def csa_decode_fp4(layout: Layout, prm: csa_params_t, q_idx, w_idx, k_fp4, comp_kv, q, out,
                   dev_status, ws, idx_out=None, sinks=None, stream=None):
    lc = layout.c()
    _check("csa_decode_fp4", load().csa_decode_fp4(
        ctypes.byref(lc), ctypes.byref(prm), _p(q_idx), _p(w_idx), _p(k_fp4), _p(comp_kv), _p(q),
        _p(sinks), _p(out), _p(idx_out), _p(dev_status), _p(ws), int(ws.numel()),
        _stream(stream)))


# ---------------------------------------------------------------- sharded decode

def csa_shard_workspace_size(layout: Layout, prm: csa_params_t, lo: int, hi: int) -> int:
    n = ctypes.c_size_t(0)
    lc = layout.c()
    _check("csa_shard_workspace_size", load().csa_shard_workspace_size(
        ctypes.byref(lc), ctypes.byref(prm), int(lo), int(hi), ctypes.byref(n)))
    return int(n.value)


def csa_shard_candidates(layout: Layout, prm: csa_params_t, lo: int, hi: int, q_idx, w_idx,
                         k_idx_shard, cand_score, cand_idx, n_cand, dev_status, ws, stream=None):
    lc = layout.c()
    _check("csa_shard_candidates", load().csa_shard_candidates(
        ctypes.byref(lc), ctypes.byref(prm), int(lo), int(hi), _p(q_idx), _p(w_idx),
        _p(k_idx_shard), _p(cand_score), _p(cand_idx), _p(n_cand), _p(dev_status), _p(ws),
        int(ws.numel()), _stream(stream)))


def csa_shard_merge(bounds, cand_score, cand_idx, n_cand, idx, n_sel, shard_idx, shard_nsel,
                    dev_status, stream=None):
    """cand_* [G, T, top_k], n_cand [G, T] -> idx [T, top_k], n_sel [T],
    shard_idx [G, T, top_k], shard_nsel [G, T]; bounds: G + 1 ints (host)."""
    G, T, K = (int(x) for x in cand_idx.shape)
    b = (ctypes.c_int64 * (G + 1))(*[int(x) for x in bounds])
    _check("csa_shard_merge", load().csa_shard_merge(
        T, K, G, b, _p(cand_score), _p(cand_idx), _p(n_cand), _p(idx), _p(n_sel), _p(shard_idx),
        _p(shard_nsel), _p(dev_status), _stream(stream)))


def csa_shard_attention(layout: Layout, prm: csa_params_t, lo: int, hi: int, shard_idx,
                        shard_nsel, comp_kv_shard, q, part_o, part_ml, dev_status, ws,
                        stream=None):
    lc = layout.c()
    _check("csa_shard_attention", load().csa_shard_attention(
        ctypes.byref(lc), ctypes.byref(prm), int(lo), int(hi), _p(shard_idx), _p(shard_nsel),
        _p(comp_kv_shard), _p(q), _p(part_o), _p(part_ml), _p(dev_status), _p(ws),
        int(ws.numel()), _stream(stream)))


def csa_window_attention(layout: Layout, prm: csa_params_t, q, part_o, part_ml, dev_status, ws,
                         stream=None):
    lc = layout.c()
    _check("csa_window_attention", load().csa_window_attention(
        ctypes.byref(lc), ctypes.byref(prm), _p(q), _p(part_o), _p(part_ml), _p(dev_status),
        _p(ws), int(ws.numel()), _stream(stream)))


def csa_shard_combine(part_o, part_ml, out, dev_status, sinks=None, stream=None):
    """part_o [P, T, H, 512], part_ml [P, T, H, 2] -> out [T, H, 512]."""
    P, T, H, _ = (int(x) for x in part_o.shape)
    _check("csa_shard_combine", load().csa_shard_combine(
        P, T, H, _p(part_o), _p(part_ml), _p(sinks), _p(out), _p(dev_status), _stream(stream)))


# ---------------------------------------------------------------- paged caches

def _arg(name: str, t, dtype, shape=None, contiguous=True) -> int:
    """A tensor argument's address, its type, shape and device checked."""
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on the GPU")
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} lives on {t.device}, not on the current device")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _device_stream(fn: str, index: int, stream=None) -> int:
    """The stream's address for a call on tensors of device `index`, which has
    to be the current one.  (These calls take a few microseconds on the GPU:
    torch.cuda.current_stream's object alone would cost three.)"""
    if index != torch.cuda.current_device():
        raise ValueError(f"{fn}: tensors live on cuda:{index}, not on the current device")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    own = getattr(stream, "device_index", index)     # (any object with a cuda_stream will do)
    if own != index:
        raise ValueError(f"{fn}: the stream belongs to cuda:{own}, not cuda:{index}")
    return stream.cuda_stream


def _ptr(t, index: int, contiguous=True) -> int:
    if t.get_device() != index or index < 0:         # (a host tensor's is -1)
        raise ValueError(f"tensor must live on cuda:{index}")
    if contiguous and not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _page_stride(cache, page_rows: int) -> int:
    """Rows from a page to the next of a cache [num_pages, rows, *row], which
    is a whole pool or one layer's part of a pool that several share
    (pool[:, first:first + page_rows]): the rows of a page are dense, the pages
    any whole number of rows apart."""
    shape = cache.shape
    rows = shape[1]
    if rows < page_rows:
        raise ValueError(f"a page of cache holds {rows} rows, not {page_rows}")
    if cache.is_contiguous():
        return rows
    want, width = [], 1
    for n in reversed(shape[1:]):
        want.insert(0, width)
        width *= n
    row = width // max(rows, 1)
    dense = all(n == 1 or s == w for n, s, w in zip(shape[1:], cache.stride()[1:], want))
    apart = cache.stride(0) if shape[0] > 1 else width
    if not dense or row == 0 or apart % row or apart < width:
        raise ValueError("cache must have dense pages, a whole number of rows apart, got shape "
                         f"{tuple(shape)} and stride {cache.stride()}")
    return apart // row


class PagePlan:
    """csa_page_plan's arguments: the sizes are taken from the tensors, which
    the object keeps alive (it is made once and used every step)."""

    def __init__(self, *, ratio: int, page_rows: int, swa_cap: int, seq_len, new_len, table,
                 free_ring, free_pos, seq_len_out, row_len, swa_first_pos, free_pos_out, tok_off,
                 row_off, tok_seq, tok_pos, swa_slot, row_slot):
        i32, i64 = torch.int32, torch.int64
        B, (tok_cap,), (row_cap,) = int(seq_len.shape[0]), tok_seq.shape, row_slot.shape
        if table.dim() != 2 or table.shape[0] != B:
            raise ValueError(f"table must have shape ({B}, max_pages), got {tuple(table.shape)}")
        if free_ring.dim() != 1:
            raise ValueError("free_ring must have one dimension")
        want = dict(seq_len=(i64, (B,)), new_len=(i32, (B,)), table=(i32, None),
                    free_ring=(i32, None), free_pos=(i64, (2,)), seq_len_out=(i64, (B,)),
                    row_len=(i64, (B,)), swa_first_pos=(i64, (B,)), free_pos_out=(i64, (2,)),
                    tok_off=(i64, (B + 1,)), row_off=(i64, (B + 1,)), tok_seq=(i32, None),
                    tok_pos=(i64, (tok_cap,)), swa_slot=(i64, (tok_cap,)), row_slot=(i64, None))
        given = dict(seq_len=seq_len, new_len=new_len, table=table, free_ring=free_ring,
                     free_pos=free_pos, seq_len_out=seq_len_out, row_len=row_len,
                     swa_first_pos=swa_first_pos, free_pos_out=free_pos_out, tok_off=tok_off,
                     row_off=row_off, tok_seq=tok_seq, tok_pos=tok_pos, swa_slot=swa_slot,
                     row_slot=row_slot)
        at = {k: _arg(k, given[k], *want[k]) for k in want}
        self.tensors, self.device = given, seq_len.device.index
        self.c = csa_page_plan_t(num_seqs=B, ratio=ratio, page_rows=page_rows,
                                 max_pages=int(table.shape[1]), num_pages=int(free_ring.shape[0]),
                                 tok_cap=tok_cap, row_cap=row_cap, swa_cap=swa_cap, **at)
        self.ref = ctypes.byref(self.c)


def csa_page_plan(plan: PagePlan, dev_status, stream=None):
    s = _device_stream("csa_page_plan", plan.device, stream)
    _check("csa_page_plan", load().csa_page_plan(plan.ref, _ptr(dev_status, plan.device), s))


class AppendJob:
    """Rows [n, ...] (dense within a row, any pitch) to slots [n] of a cache
    [num_pages, at least page_rows, ...] whose rows have the same bytes: a
    whole pool, or one layer's part of it (pool[:, first:first + page_rows])."""

    def __init__(self, rows, slots, cache, page_rows: int):
        n = int(rows.shape[0])
        if cache.dim() < 2 or cache.dtype != rows.dtype or cache.shape[2:] != rows.shape[1:]:
            raise ValueError(f"cache must be {rows.dtype} [num_pages, rows of a page, "
                             f"*{tuple(rows.shape[1:])}], got {cache.dtype} {tuple(cache.shape)}")
        if n and not rows[0].is_contiguous():
            raise ValueError("a row must be contiguous")
        apart = _page_stride(cache, page_rows)
        size = rows.element_size()
        width = size * (rows[0].numel() if n else cache[0, 0].numel())
        pitch = rows.stride(0) * size if n > 1 else width
        self.tensors, self.device = (rows, slots, cache), cache.device.index
        self.c = csa_append_job_t(
            rows=_arg("rows", rows, rows.dtype, contiguous=False),
            slots=_arg("slots", slots, torch.int64, (n,)), num_rows=n, row_pitch=pitch,
            row_bytes=width, page_rows=page_rows, num_pages=int(cache.shape[0]),
            page_stride=apart, cache=_arg("cache", cache, cache.dtype, contiguous=False))


class AppendJobs:
    """Up to four AppendJob for one launch."""

    def __init__(self, jobs):
        self.jobs = list(jobs)
        if not 1 <= len(self.jobs) <= MAX_APPEND_JOBS:
            raise ValueError(f"1 to {MAX_APPEND_JOBS} jobs, got {len(self.jobs)}")
        self.device = self.jobs[0].device
        if any(j.device != self.device for j in self.jobs):
            raise ValueError(f"jobs on devices {[j.device for j in self.jobs]}: one call runs on one")
        self.c = (csa_append_job_t * len(self.jobs))(*[j.c for j in self.jobs])


def csa_paged_append(jobs: AppendJobs, dev_status, stream=None):
    s = _device_stream("csa_paged_append", jobs.device, stream)
    _check("csa_paged_append", load().csa_paged_append(jobs.c, len(jobs.jobs),
                                                       _ptr(dev_status, jobs.device), s))


class PagedLayout:
    """csa_paged_attention's layout: tokens [T] of sequences [B], the block
    table [B, max_pages], the window ring [B, swa_cap, 512] (None without a
    window).  Keeps its tensors alive; made once for buffers that stay."""

    ring_type = torch.bfloat16

    def __init__(self, tok_seq, tok_pos, row_len, table, page_rows: int, swa_kv=None,
                 swa_first_pos=None):
        T, B = int(tok_seq.shape[0]), int(row_len.shape[0])
        if table.dim() != 2 or table.shape[0] != B:
            raise ValueError(f"table must have shape ({B}, max_pages), got {tuple(table.shape)}")
        ring = {}
        if swa_kv is not None:
            if swa_kv.dim() != 3 or swa_kv.shape[0] != B or swa_kv.shape[2] != 512:
                raise ValueError(f"swa_kv must have shape ({B}, swa_cap, 512), "
                                 f"got {tuple(swa_kv.shape)}")
            if swa_first_pos is None:
                raise ValueError("swa_kv needs swa_first_pos")
            ring = dict(swa_kv=_arg("swa_kv", swa_kv, self.ring_type), swa_cap=int(swa_kv.shape[1]),
                        swa_first_pos=_arg("swa_first_pos", swa_first_pos, torch.int64, (B,)))
        self.tensors = (tok_seq, tok_pos, row_len, table, swa_kv, swa_first_pos)
        self.device, self.num_tokens = row_len.device.index, T
        self.c = csa_paged_layout_t(
            num_seqs=B, num_tokens=T, page_rows=page_rows, max_pages=int(table.shape[1]),
            tok_seq=_arg("tok_seq", tok_seq, torch.int32, (T,)),
            tok_pos=_arg("tok_pos", tok_pos, torch.int64, (T,)),
            row_len=_arg("row_len", row_len, torch.int64, (B,)),
            table=_arg("table", table, torch.int32), **ring)
        self.ref = ctypes.byref(self.c)


def csa_paged_workspace_size(layout: PagedLayout, prm: csa_params_t) -> int:
    n = ctypes.c_size_t(0)
    _check("csa_paged_workspace_size", load().csa_paged_workspace_size(
        ctypes.byref(layout.c), ctypes.byref(prm), ctypes.byref(n)))
    return int(n.value)


def paged_workspace(layout: PagedLayout, prm: csa_params_t, device=None) -> torch.Tensor:
    return torch.empty(csa_paged_workspace_size(layout, prm), dtype=torch.uint8,
                       device=device or torch.device("cuda", layout.device))


def csa_paged_attention(layout: PagedLayout, prm: csa_params_t, cache, q, out, dev_status, ws,
                        sinks=None, stream=None):
    """cache bf16 [num_pages, at least page_rows, 512] (a whole pool, or one
    layer's part of it, as for AppendJob), q bf16 [T, H, 512], out f32 or bf16
    [T, H, 512]."""
    dev = layout.device
    s = _device_stream("csa_paged_attention", dev, stream)
    if cache.dtype != torch.bfloat16 or q.dtype != torch.bfloat16:
        raise ValueError("cache and q must be bfloat16")
    if layout.ring_type is not torch.bfloat16:
        raise ValueError("layout is one of 8-bit rows")
    if out.dtype != torch.float32 and out.dtype != torch.bfloat16:
        raise ValueError("out must be float32 or bfloat16")
    shape = (layout.num_tokens, prm.n_heads, prm.hd)
    if q.shape != shape or out.shape != shape:
        raise ValueError(f"q and out must have shape {shape}")
    if cache.dim() != 3 or cache.shape[2] != prm.hd:
        raise ValueError(f"cache must have shape (num_pages, rows of a page, {prm.hd})")
    if sinks is not None and (sinks.dtype != torch.float32 or sinks.shape != (prm.n_heads,)):
        raise ValueError(f"sinks must be float32 [{prm.n_heads}]")
    _check("csa_paged_attention", load().csa_paged_attention(
        layout.ref, ctypes.byref(prm), _ptr(cache, dev, contiguous=False), cache.shape[0],
        cache.shape[1] if cache.is_contiguous() else _page_stride(cache, layout.c.page_rows), _ptr(q, dev),
        None if sinks is None else _ptr(sinks, dev), 1 if out.dtype == torch.bfloat16 else 0,
        _ptr(out, dev), _ptr(dev_status, dev), _ptr(ws, dev), ws.numel(), s))


# ---------------------------------------------------------------- 8-bit paged caches

_FP8_TYPES = {torch.float32: 0, torch.bfloat16: 1}      # csa_type_t


def _fp8_pool(cache, scales, page_rows: int) -> tuple:
    """The shape, and the page strides (rows), of a cache float8_e4m3fn [num_pages, at least
    page_rows, width] and of its scales float32 [num_pages, at least page_rows]:
    each a whole pool, or one layer's part of it."""
    pool, beside = cache.shape, scales.shape
    if cache.dtype != torch.float8_e4m3fn or len(pool) != 3:
        raise ValueError("cache must be float8_e4m3fn [num_pages, rows of a page, width], "
                         f"got {cache.dtype} {tuple(pool)}")
    if scales.dtype != torch.float32 or len(beside) != 2 or beside[0] != pool[0]:
        raise ValueError(f"scales must be float32 [{pool[0]}, rows of a page], "
                         f"got {scales.dtype} {tuple(beside)}")
    return pool, _page_stride(cache, page_rows), _page_stride(scales, page_rows)


class AppendJobFp8:
    """Rows [n, width] (bfloat16 or float32, dense within a row, any pitch) to
    slots [n] of a cache float8_e4m3fn [num_pages, at least page_rows, width]
    and its scales float32 [num_pages, at least page_rows]: a whole pool, or
    one layer's part of it (pool[:, first:first + page_rows])."""

    def __init__(self, rows, slots, cache, scales, page_rows: int):
        if rows.dim() != 2 or rows.dtype not in _FP8_TYPES:
            raise ValueError(f"rows must be bfloat16 or float32 [n, width], got {rows.dtype} {tuple(rows.shape)}")
        n, width = (int(x) for x in rows.shape)
        pool, apart, scales_apart = _fp8_pool(cache, scales, page_rows)
        if pool[2] != width:
            raise ValueError(f"cache rows hold {pool[2]} values, rows {width}")
        if n and not rows[0].is_contiguous():
            raise ValueError("a row must be contiguous")
        size = rows.element_size()
        self.tensors, self.device = (rows, slots, cache, scales), cache.device.index
        self.c = csa_append_fp8_job_t(
            rows=_arg("rows", rows, rows.dtype, contiguous=False),
            slots=_arg("slots", slots, torch.int64, (n,)), num_rows=n,
            row_pitch=rows.stride(0) * size if n > 1 else width * size, type=_FP8_TYPES[rows.dtype],
            width=width, page_rows=page_rows, num_pages=pool[0], page_stride=apart,
            scale_stride=scales_apart, cache=_arg("cache", cache, cache.dtype, contiguous=False),
            scales=_arg("scales", scales, torch.float32, contiguous=False))


class AppendJobsFp8:
    """Up to four AppendJobFp8 for one launch."""

    def __init__(self, jobs):
        self.jobs = list(jobs)
        if not 1 <= len(self.jobs) <= MAX_APPEND_JOBS:
            raise ValueError(f"1 to {MAX_APPEND_JOBS} jobs, got {len(self.jobs)}")
        self.device = self.jobs[0].device
        if any(j.device != self.device for j in self.jobs):
            raise ValueError(f"jobs on devices {[j.device for j in self.jobs]}: one call runs on one")
        self.c = (csa_append_fp8_job_t * len(self.jobs))(*[j.c for j in self.jobs])


def csa_paged_append_fp8(jobs: AppendJobsFp8, dev_status, stream=None):
    s = _device_stream("csa_paged_append_fp8", jobs.device, stream)
    _check("csa_paged_append_fp8", load().csa_paged_append_fp8(jobs.c, len(jobs.jobs),
                                                               _ptr(dev_status, jobs.device), s))


def csa_paged_read_fp8(cache, scales, slots, out, dev_status, page_rows: int, stream=None):
    """Rows `slots` [n] of an 8-bit cache (as for AppendJobFp8) into out [n,
    width], bfloat16 or float32, dense within a row."""
    shape, kind = out.shape, _FP8_TYPES.get(out.dtype)
    if len(shape) != 2 or kind is None:
        raise ValueError(f"out must be bfloat16 or float32 [n, width], got {out.dtype} {tuple(shape)}")
    n, width = shape
    pool, apart, scales_apart = _fp8_pool(cache, scales, page_rows)
    if pool[2] != width:
        raise ValueError(f"cache rows hold {pool[2]} values, out {width}")
    if slots.dtype != torch.int64 or slots.shape != (n,):
        raise ValueError(f"slots must be int64 [{n}], got {slots.dtype} {tuple(slots.shape)}")
    if n and width > 1 and out.stride(1) != 1:
        raise ValueError("a row must be contiguous")
    size, dev = out.element_size(), out.get_device()
    pitch = out.stride(0) * size if n > 1 else width * size
    if pitch < width * size:
        raise ValueError("rows of out must not overlap")
    s = _device_stream("csa_paged_read_fp8", dev, stream)
    # (by position: names take a microsecond more, a tenth of the call)
    r = csa_read_fp8_t(_ptr(cache, dev, False), _ptr(scales, dev, False), _ptr(slots, dev), n, width,
                       page_rows, pool[0], apart, scales_apart, kind, pitch, _ptr(out, dev, False))
    _check("csa_paged_read_fp8", load().csa_paged_read_fp8(ctypes.byref(r), _ptr(dev_status, dev), s))


class PagedLayoutFp8(PagedLayout):
    """csa_paged_attention_fp8's layout: PagedLayout with the window ring in
    8 bits, swa_kv float8_e4m3fn [B, swa_cap, 512] and swa_scales float32 [B,
    swa_cap] (None without a window)."""

    ring_type = torch.float8_e4m3fn

    def __init__(self, tok_seq, tok_pos, row_len, table, page_rows: int, swa_kv=None,
                 swa_scales=None, swa_first_pos=None):
        super().__init__(tok_seq, tok_pos, row_len, table, page_rows, swa_kv, swa_first_pos)
        self.swa_scales, self.swa_scales_at = swa_scales, None
        if swa_kv is not None:
            if swa_scales is None:
                raise ValueError("swa_kv needs swa_scales")
            self.swa_scales_at = _arg("swa_scales", swa_scales, torch.float32, swa_kv.shape[:2])


def csa_paged_attention_fp8(layout: PagedLayoutFp8, prm: csa_params_t, cache, scales, q, out,
                            dev_status, ws, sinks=None, stream=None):
    """cache float8_e4m3fn [num_pages, at least page_rows, 512] and scales
    float32 [num_pages, at least page_rows] (whole pools, or one layer's part
    of them), q bf16 [T, H, 512], out f32 or bf16 [T, H, 512], ws
    paged_workspace(layout, prm)."""
    dev = layout.device
    s = _device_stream("csa_paged_attention_fp8", dev, stream)
    if not isinstance(layout, PagedLayoutFp8):
        raise ValueError("layout must be a PagedLayoutFp8")
    if q.dtype != torch.bfloat16:
        raise ValueError("q must be bfloat16")
    if out.dtype not in _FP8_TYPES:
        raise ValueError("out must be float32 or bfloat16")
    shape = (layout.num_tokens, prm.n_heads, prm.hd)
    if q.shape != shape or out.shape != shape:
        raise ValueError(f"q and out must have shape {shape}")
    pool, apart, scales_apart = _fp8_pool(cache, scales, layout.c.page_rows)
    if pool[2] != prm.hd:
        raise ValueError(f"cache must have shape (num_pages, rows of a page, {prm.hd})")
    if sinks is not None and (sinks.dtype != torch.float32 or sinks.shape != (prm.n_heads,)):
        raise ValueError(f"sinks must be float32 [{prm.n_heads}]")
    _check("csa_paged_attention_fp8", load().csa_paged_attention_fp8(
        layout.ref, ctypes.byref(prm), _ptr(cache, dev, contiguous=False),
        _ptr(scales, dev, contiguous=False), layout.swa_scales_at, pool[0], apart, scales_apart,
        _ptr(q, dev), None if sinks is None else _ptr(sinks, dev), _FP8_TYPES[out.dtype], _ptr(out, dev),
        _ptr(dev_status, dev), _ptr(ws, dev), ws.numel(), s))
