"""Limits of the paged cache's calls and its pages that are settled on the host."""

import ctypes
from types import SimpleNamespace

import pytest
import torch

from test_kv_host import OK, UNS, _pool

cpa = pytest.importorskip("context_long_sequence_zigzag_gb300")


def test_reserve_refuses_tables_whose_pages_pass_32_bits():
    """Demands and releases of a batch are summed in 32 bits: 4096 sequences of 2^20 pages are past that."""
    lib = cpa._lib
    for B, columns, page_size in ((4096, 1 << 20, 1), (4096, (1 << 18) + 1, 16), (2, (1 << 29) + 1, 1)):
        pool = _pool(page_size=page_size)
        assert lib.cp_pages_reserve(ctypes.byref(pool), B, columns, 256, 256, 256, 256, None) == UNS


@pytest.mark.parametrize("name", ["cp_kv_workspace_size", "cp_kv4_workspace_size"])
def test_workspace_is_sized_for_the_caches_device(monkeypatch, name):
    """The size goes by the current device's SMs: it is asked for with the cache's device current."""
    current = ["cuda:0"]

    class On:
        def __init__(self, device):
            self.device = str(device)

        def __enter__(self):
            current.append(self.device)

        def __exit__(self, *_):
            current.pop()

    asked = []
    monkeypatch.setattr(cpa.torch.cuda, "device", On)
    monkeypatch.setattr(cpa._lib, name, lambda *_: asked.append(current[-1]) or OK)
    getattr(cpa, name)(SimpleNamespace(ptr=None, device=torch.device("cuda", 1)), 2)
    assert asked == ["cuda:1"]
