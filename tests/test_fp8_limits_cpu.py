"""The longest token that the 8-bit paged attention takes: decided before anything is
launched (a workspace that is too small ends the call behind that check)."""
import pytest

from sparse_compressed_kv_gb300 import csa
from tests.test_fp8_cpu import UNSUPPORTED, WORKSPACE, attend, lib  # noqa: F401


@pytest.mark.parametrize("page_rows,max_pages,window,code", [
    (65535, 32767, (1 << 31) - 65 - 65535 * 32767, WORKSPACE),
    (65535, 32767, (1 << 31) - 64 - 65535 * 32767, UNSUPPORTED),
    (1 << 30, 1, (1 << 30) - 65, WORKSPACE), (1 << 30, 1, (1 << 30) - 64, UNSUPPORTED),
    (1, (1 << 31) - 65, 0, WORKSPACE), (1, (1 << 31) - 64, 0, UNSUPPORTED),
])
def test_attention_longest_token(lib, page_rows, max_pages, window, code):  # noqa: F811
    got = attend(lib, P=csa.params(16, 1, window, 1), num_seqs=1, num_tokens=1, page_rows=page_rows,
                 max_pages=max_pages, swa_cap=max(1, window), num_pages=1, page_stride=page_rows,
                 scale_stride=page_rows, ws_bytes=100)
    assert got == code
