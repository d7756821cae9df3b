"""The binding of the 4-bit cache and the key weights, without a GPU."""

import os
import subprocess
import sys

import pytest
import torch

cpa = pytest.importorskip("context_long_sequence_zigzag_gb300")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_import_takes_no_private_name_of_a_cuda_build():
    """A torch built without CUDA lacks the raw stream's query: the host-side calls still answer."""
    code = """
import torch
if hasattr(torch._C, "_cuda_getCurrentRawStream"):
    del torch._C._cuda_getCurrentRawStream
import context_long_sequence_zigzag_gb300 as cpa
assert cpa.cp_kv4_block_bytes(128, 128) == 9216
assert cpa.cp_workspace_size(cpa.Problem(1024, 8, 2, 128, 128, 4), cpa.CP_OP_FWD) > 0
"""
    done = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=240)
    assert done.returncode == 0, done.stderr[-2000:]


def test_key_weights_need_tensors_on_a_gpu():
    T, prob = 8, cpa.Problem(8, 2, 2, 64, 64, 1)
    q, k, lse = torch.zeros(T, 2, 64).bfloat16(), torch.zeros(T, 2, 64).bfloat16(), torch.zeros(2, T)
    for ws in (None, torch.zeros(1 << 20, dtype=torch.uint8)):
        with pytest.raises(ValueError, match="CUDA device"):
            cpa.cp_attn_key_weights(prob, q, k, lse, ws=ws)
    with pytest.raises(ValueError, match="CUDA device"):
        cpa.cp_attn_key_weights(prob, None, k, lse)


def test_key_weights_without_memory_for_the_plan():
    """A host that cannot hold the tile plan: a status, not the end of the process."""
    code = """
import resource, context_long_sequence_zigzag_gb300 as cpa
prob = cpa.Problem(1 << 30, 2, 2, 128, 128, 1, "contiguous")
size = next(int(x.split()[1]) for x in open("/proc/self/status") if x.startswith("VmSize")) << 10
resource.setrlimit(resource.RLIMIT_AS, (size + (64 << 20),) * 2)
for last in (0, 16):
    status = cpa._lib.cp_attn_key_weights(prob.ptr, last, 256, 256, 256, 256, 256, 0, None)
    assert status == cpa.CP_ERR_UNSUPPORTED, status
"""
    done = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=240)
    assert done.returncode == 0, (done.returncode, done.stderr[-2000:])
