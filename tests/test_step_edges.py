"""Calls around a decode step on the CPU, at the edges of what they accept."""
import ctypes

import pytest

import sparse_attention_kv_swap_gb300 as pkg
from sparse_attention_kv_swap_gb300 import binding as B


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_kv_swap_gb300 import build
    build.build()
    return B.load_library()


@pytest.mark.parametrize("batch,steps,heads", [
    (2 ** 31 - 1, 1, 1), (2 ** 31 - 256, 1, 1), (1, 2 ** 31 - 1, 1), (2 ** 24, 1, 128),
    (2 ** 31 - 1, 2 ** 31 - 1, 128), (2 ** 30, 2 ** 28, 64)])  # products beyond 63 bits
def test_attend_prefix_refuses_rows_beyond_32_bits(lib, batch, steps, heads):
    """With the rows that a last tile lacks, and whatever their product overflows to."""
    fmt = pkg.make_kv_format(1, 32, 16)
    args = B._HsPrefixArgs(q_dev=0x20000, out_dev=0x20000, dtype=B.HS_DTYPE_BF16, batch=batch,
                           steps=steps, num_heads=heads, num_requests=1, max_seq_len=64,
                           num_prefixes=0)
    call = lib.hs_attend_prefix(ctypes.byref(fmt), ctypes.byref(args), None)
    assert call == B.HS_ERR_UNSUPPORTED
    with pytest.raises(pkg.HsError):
        pkg.hs_prefix_workspace_bytes(fmt, batch, steps, heads, 1)


def test_prefix_workspace_of_many_rows(lib):
    fmt = pkg.make_kv_format(1, 32, 16)
    assert pkg.hs_prefix_workspace_bytes(fmt, 2 ** 31 - 4097, 1, 1, 1) > 0
