"""Calls of the paged cache and its pages at sizes and forms where their kernels go other ways: against the float64
oracle, with the tolerances derived in test_gpu_kv.py unless a test says otherwise."""

import math

import numpy as np
import pytest
import torch

import oracle
from test_gpu_kv import BF, WIDE, Held, f64

pytestmark = pytest.mark.gpu

cpa = pytest.importorskip("context_long_sequence_zigzag_gb300")


@pytest.fixture(autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    assert cpa.cp_device_status() == 0


# ---------------------------------------------------------------- attention: the probabilities' terms
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("hq,hkv,d_qk,d_v,n_q", [(8, 2, 128, 128, 1), (16, 1, 64, 64, 1), (4, 2, 192, 128, 8), (32, 1, 128, 64, 1)])
def test_probabilities_are_two_terms(hq, hkv, d_qk, d_v, n_q, wide):
    """bf16 caches, up to 32 rows a kv head, O in fp32 for a join: a probability is two terms of bf16.  The first is cut
    off (below 2^-7 of it), the second rounded (2^-8 of that), and 2^-20 is added: off by 2^-15 + 2^-20.  The product
    takes two tensor-core steps where test_gpu_kv.py counts one: n 2^-26."""
    h = Held([700, 33, 1, 2000], hq, hkv, d_qk, d_v, BF, 64, n_q, seed=30, columns=WIDE // 64 + 1 if wide else None)
    o, lse = (f64(x) for x in h.run(part=True))
    for b, n in enumerate(h.lengths):
        k, v, q = f64(h.k[b]), f64(h.v[b]), f64(h.q[b])
        for t in range(n_q):
            at = np.arange(max(n - (n_q - 1 - t), 0))
            for x in range(hq):
                c = h.kv_of(x)
                want, want_lse = oracle.kv_attention(q[t:t + 1, x], k[:, c], v[:, c], [at], h.scale)
                if not len(at):
                    continue
                score = 2.0 ** -18 * h.scale * (np.abs(k[at, c]) @ np.abs(q[t, x])).max()
                p = np.exp(k[at, c] @ q[t, x] * h.scale - want_lse[0])
                room = (p @ np.abs(v[at, c])) * (2 * score + len(at) * 2.0 ** -26 + 2.0 ** -18 + 2.0 ** -15 + 2.0 ** -20)
                assert np.all(np.abs(o[b, t, x] - want[0]) <= room), (b, t, x)


@pytest.mark.parametrize("n_q", [1, 4, 8])
def test_an_infinite_value_stays_one(n_q):
    """bf16 caches: an infinite value that a query sees comes out as it is, whatever its probability's bits (an 8-bit
    one, whose second term would be 0, among them)."""
    h = Held([65, 300], 8, 1, 64, 64, BF, 64, n_q, seed=31)
    h.v[0][3, :, 5], h.v[1][290, :, 6] = math.inf, -math.inf
    h.k[0].zero_()  # (all probabilities alike: exactly 1 before the division)
    for b in range(2):
        h.put(b)
    for part in (False, True):
        o, _ = h.run(part=part)
        sees = [t for t in range(n_q) if 300 - (n_q - 1 - t) > 290]
        assert (o[0, :, :, 5] == math.inf).all() and (o[1, sees, :, 6] == -math.inf).all()
        assert o[0, ..., :5].isfinite().all() and o[1, ..., 7:].isfinite().all()
