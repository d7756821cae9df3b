"""Limits of the paged cache's calls and its pages that are settled on the host."""

import ctypes

import pytest

from test_kv_host import UNS, _pool

cpa = pytest.importorskip("context_long_sequence_zigzag_gb300")


def test_reserve_refuses_tables_whose_pages_pass_32_bits():
    """Demands and releases of a batch are summed in 32 bits: 4096 sequences of 2^20 pages are past that."""
    lib = cpa._lib
    for B, columns, page_size in ((4096, 1 << 20, 1), (4096, (1 << 18) + 1, 16), (2, (1 << 29) + 1, 1)):
        pool = _pool(page_size=page_size)
        assert lib.cp_pages_reserve(ctypes.byref(pool), B, columns, 256, 256, 256, 256, None) == UNS
