"""The bytes that bench.py's roofline counts for an FFN call (CPU only)."""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)
import bench  # noqa: E402


@pytest.mark.parametrize("N,d,esize", [(1024, 2048, 2), (16640, 2880, 2), (7, 64, 4)])
def test_rows_of_the_tokens_type_go_in_and_out(N, d, esize):
    assert bench.ffn_call_bytes(5, 1000, N, d, esize, False) == 5 * 1000 + 2 * N * d * esize


@pytest.mark.parametrize("N,d,blocks", [(1024, 2048, 16), (16640, 2880, 23), (7, 64, 1)])
def test_block_scaled_calls_read_codes_and_scales(N, d, blocks):
    """One byte a value and four a block of 128 columns in, bf16 out: the bf16 rows are read by the call before."""
    assert bench.ffn_call_bytes(5, 1000, N, d, 2, True) == 5 * 1000 + N * (d + 4 * blocks) + N * d * 2
