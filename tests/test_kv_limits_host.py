"""Limits of the paged cache's calls and its pages that are settled on the host."""

import ctypes
from types import SimpleNamespace

import pytest
import torch

from test_kv_host import OK, UNS, _cache, _pool

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


def test_clusters_only_where_they_fit_the_gpu_at_once():
    """Few short runs take clusters of four to eight CTAs, and no workspace, as long as all CTAs are resident: two an
    SM, but one of fp32 heads of 192 with more than 16 rows (152 SMs)."""
    n = ctypes.c_size_t(0)

    def size(dtype, seqs, d_qk, n_q):
        c = _cache(num_seqs=seqs, hq=32, hkv=8, d_qk=d_qk, dtype=dtype)
        assert cpa._lib.cp_kv_workspace_size(ctypes.byref(c), n_q, ctypes.byref(n)) == OK
        return n.value

    f32, bf16 = cpa.CP_DT_F32, cpa.CP_DT_BF16
    assert size(f32, 5, 192, 8) > 0 and size(f32, 4, 192, 8) == 0  # 32 rows: 160 and 128 CTAs
    for other in ((f32, 192, 4), (f32, 128, 8), (bf16, 192, 8), (bf16, 192, 16)):
        assert size(other[0], 9, *other[1:]) == 0 and size(other[0], 10, *other[1:]) > 0  # 288 and 320 CTAs


def test_build_checks_the_registers_of_kernels_that_hand_them_over():
    """The attention's launcher refuses a kernel of other than 128 registers a thread: a build with one fails."""
    build = pytest.importorskip("context_long_sequence_zigzag_gb300.build")
    log = """ptxas info    : Compiling entry function '_ZN6cpattn14kv_join_kernelILi8EEEvi' for 'sm_103a'
ptxas info    : Used 48 registers, used 1 barriers
ptxas info    : Compiling entry function '_ZN6cpattn14kv_attn_kernelILi1EEEvi' for 'sm_103a'
ptxas info    : Function properties for _ZN6cpattn14kv_attn_kernelILi1EEEvi
    8 bytes stack frame, 8 bytes spill stores, 8 bytes spill loads
ptxas info    : Used %d registers, used 1 barriers
"""
    build.check_registers(log % 128)
    with pytest.raises(RuntimeError, match="120 registers"):
        build.check_registers(log % 120)
