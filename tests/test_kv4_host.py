"""Host-side checks of the 4-bit key/value cache: the oracle's format, and the
calls' refusals (everything here is refused or answered before GPU work)."""

import ctypes
import math

import numpy as np
import pytest

import oracle

cpa = pytest.importorskip("context_long_sequence_zigzag_gb300")


@pytest.mark.parametrize("d_qk,d_v", [(64, 64), (128, 128), (192, 128), (128, 64)])
def test_oracle_format_round_trip_and_error(d_qk, d_v):
    rng = np.random.RandomState(1)
    k, v = rng.randn(64, d_qk) * 3 + 1, rng.randn(64, d_v)
    k[3], v[5, :64] = 2.5, 0.0  # groups of one value
    parts = oracle.kv4_quantise(k), oracle.kv4_quantise(v)
    block = oracle.kv4_pack(*parts)
    assert block.shape[0] == oracle.kv4_block_bytes(d_qk, d_v) == cpa.cp_kv4_block_bytes(d_qk, d_v)
    for (codes, low, scale), got, x in zip(parts, oracle.kv4_unpack(block, d_qk, d_v), (k, v)):
        for a, b in zip((codes, low, scale), got):
            assert np.array_equal(a, b)
        # half a step, and the scale's rounding at the top of the range (15 steps of half a unit of 2^-8)
        step = np.repeat(scale, 64, -1)
        assert np.all(np.abs(oracle.kv4_values(codes, low, scale) - x) <= step * (0.5 + 15 * 2.0 ** -8) + 1e-12)
        assert np.all(low <= x.reshape(64, -1, 64).min(-1))


def test_oracle_keep():
    assert oracle.kv4_keep([5, 1, 5, 5], 4, 2, 0) == [0, 2]
    assert oracle.kv4_keep([5, 1, 7, math.nan, 0], 5, 3, 1) == [2, 3, 4]
    assert oracle.kv4_keep([1, 2], 2, 5, 5) == [0, 1]
    assert oracle.kv4_keep([9, 9, 9], 3, 2, 2) == [1, 2]


def test_oracle_key_weights_sum_to_the_queries():
    rng = np.random.RandomState(2)
    T, cu = 20, [0, 13, 20]
    q, k, v = rng.randn(T, 4, 8), rng.randn(T, 2, 8), rng.randn(T, 2, 8)
    for last in (None, 3, 100):
        ref_lse = oracle.attn_forward(q, k, v, cu, 0.3)[1]
        w = oracle.attn_key_weights(q, k, ref_lse, cu, 0.3, last=last)
        # every counted query's probabilities sum to 1, over 2 heads a kv head
        want = [2 * min(n, last or n) for n in (13, 7)]
        assert np.allclose([[w[c, :13].sum(), w[c, 13:].sum()] for c in range(2)], [want, want])


def _desc(**kw):
    base = dict(num_seqs=2, hq=8, hkv=2, d_qk=128, d_v=128, gqa=0, dtype=cpa.CP_DT_BF16, scale=0.1, num_pages=4,
                max_pages=2, pages=4096, weights=8192, page_table=64)
    base.update(kw)
    return cpa.cp_kv4_t(**base)


@pytest.mark.parametrize("change,status", [
    ({}, cpa.CP_OK),
    ({"hq": 6, "hkv": 4}, cpa.CP_ERR_INVALID_ARG),
    ({"hkv": 0}, cpa.CP_ERR_INVALID_ARG),
    ({"num_seqs": -1}, cpa.CP_ERR_INVALID_ARG),
    ({"d_qk": 96}, cpa.CP_ERR_UNSUPPORTED),
    ({"d_v": 192}, cpa.CP_ERR_UNSUPPORTED),
    ({"d_v": 0}, cpa.CP_ERR_INVALID_ARG),
    ({"gqa": 2}, cpa.CP_ERR_INVALID_ARG),
    ({"dtype": 7}, cpa.CP_ERR_INVALID_ARG),
    ({"scale": math.nan}, cpa.CP_ERR_INVALID_ARG),
    ({"scale": 0.0}, cpa.CP_ERR_INVALID_ARG),
    ({"pages": None}, cpa.CP_ERR_INVALID_ARG),
    ({"pages": 4104}, cpa.CP_ERR_INVALID_ARG),
    ({"page_table": 66}, cpa.CP_ERR_INVALID_ARG),
    ({"weights": 8196}, cpa.CP_ERR_INVALID_ARG),
    ({"num_pages": -1}, cpa.CP_ERR_INVALID_ARG),
    ({"max_pages": 1 << 25}, cpa.CP_ERR_UNSUPPORTED),
    ({"num_seqs": 4097}, cpa.CP_ERR_UNSUPPORTED),
    ({"num_seqs": 0, "pages": None, "page_table": None}, cpa.CP_OK),
    ({"weights": None}, cpa.CP_OK),
])
def test_validate(change, status):
    assert cpa._lib.cp_kv4_validate(ctypes.byref(_desc(**change))) == status


def test_calls_refuse_before_gpu_work():
    lib, c = cpa._lib, _desc()
    ref, bad, uns, wsp = ctypes.byref(c), cpa.CP_ERR_INVALID_ARG, cpa.CP_ERR_UNSUPPORTED, cpa.CP_ERR_WORKSPACE
    assert lib.cp_kv4_validate(None) == bad
    assert lib.cp_kv4_append(None, 16, 16, None, 4, None, 16, 16, 4, None) == bad
    assert lib.cp_kv4_append(ref, None, 16, None, 4, None, 16, 16, 4, None) == bad
    assert lib.cp_kv4_append(ref, 24, 16, None, 4, None, 16, 16, 4, None) == bad  # k not 16-byte aligned
    assert lib.cp_kv4_append(ref, 16, 16, None, 3, None, 16, 16, 4, None) == bad  # fewer rows than tokens
    assert lib.cp_kv4_append(ref, 16, 16, None, 4, None, 16, 16, -1, None) == bad
    assert lib.cp_kv4_append(ref, 16, 16, None, 0, None, 16, 16, 0, None) == cpa.CP_OK  # nothing to do
    assert lib.cp_kv4_read(ref, 16, 16, 4, None, 16, None) == bad
    assert lib.cp_kv4_read(ref, None, 16, 4, 16, 16, None) == bad
    n = ctypes.c_size_t(0)
    assert lib.cp_kv4_workspace_size(ref, 1, 1, ctypes.byref(n)) == cpa.CP_OK and n.value % 256 == 0
    assert lib.cp_kv4_workspace_size(ref, 0, 0, ctypes.byref(n)) == bad
    assert lib.cp_kv4_workspace_size(ref, 17, 0, ctypes.byref(n)) == uns
    assert lib.cp_kv4_workspace_size(ref, 1, 2, ctypes.byref(n)) == bad
    assert lib.cp_kv4_workspace_size(ref, 1, 0, None) == bad
    attn = lambda c, n_q=1, q=256, lens=256, o=256, f=0, lse=256, acc=0, ws=256, b=1 << 40: lib.cp_kv4_attn(  # noqa: E731
        ctypes.byref(c), n_q, q, lens, o, f, lse, acc, ws, b, None)
    assert attn(c, n_q=0) == bad and attn(c, n_q=17) == uns
    assert attn(c, q=None) == bad and attn(c, o=None) == bad and attn(c, lse=None) == bad and attn(c, lens=None) == bad
    assert attn(c, f=2) == bad and attn(c, acc=2) == bad
    assert attn(_desc(weights=None), acc=1) == bad
    assert attn(c, ws=None) == wsp and attn(c, ws=128) == wsp and attn(c, b=0) == wsp
    assert attn(_desc(num_seqs=0), q=None) == cpa.CP_OK
    to = _desc(page_table=128)
    evict = lambda c, to, lens=4096, budget=64, recent=8, new=8192, kept=16384: lib.cp_kv4_evict(  # noqa: E731
        ctypes.byref(c), lens, budget, recent, ctypes.byref(to), new, kept, None)
    assert evict(c, _desc(d_v=64)) == bad and evict(c, _desc(num_seqs=3)) == bad and evict(c, _desc(hq=2, hkv=1)) == bad
    assert evict(c, to, budget=0) == bad and evict(c, to, budget=129) == bad
    assert evict(c, to, recent=65) == bad and evict(c, to, recent=-1) == bad
    assert evict(c, to, lens=None) == bad and evict(c, to, new=None) == bad and evict(c, to, kept=None) == bad
    assert evict(c, to, new=4096) == bad and evict(c, to, new=4100) == bad  # the new lengths over the old ones
    assert evict(c, c) == bad  # onto itself
    assert evict(_desc(weights=None), to) == bad and evict(c, _desc(page_table=128, weights=None)) == bad


def test_key_weights_refusals_and_workspace():
    p = cpa.Problem(1024, 8, 2, 128, 128, 4, "zigzag")
    lib = cpa._lib
    f = lambda last=0, q=256, k=256, l=256, w=256, ws=256, b=1 << 40: lib.cp_attn_key_weights(  # noqa: E731
        p.ptr, last, q, k, l, w, ws, b, None)
    assert f(last=-1) == cpa.CP_ERR_INVALID_ARG
    assert f(q=None) == f(k=None) == f(l=None) == f(w=None) == f(w=8) == cpa.CP_ERR_INVALID_ARG
    assert f(ws=None) == f(ws=64) == f(b=0) == cpa.CP_ERR_WORKSPACE
    assert lib.cp_attn_key_weights(None, 0, 256, 256, 256, 256, 256, 1 << 40, None) == cpa.CP_ERR_INVALID_ARG
    q = cpa.Problem(0, 8, 2, 128, 128, 4, "zigzag")
    assert lib.cp_attn_key_weights(q.ptr, 0, None, None, None, None, None, 0, None) == cpa.CP_OK
    assert cpa.cp_workspace_size(p, cpa.CP_OP_KEY_WEIGHTS) > 0


def test_python_checks_its_tensors():
    import torch

    with pytest.raises(ValueError):  # not on a GPU
        cpa.Kv4Cache(torch.zeros(1, 2, cpa.cp_kv4_block_bytes(128, 128), dtype=torch.uint8),
                     torch.zeros(1, 1, dtype=torch.int32), 2, 2, 128, 128)
    with pytest.raises(cpa.CpError):
        cpa.cp_kv4_block_bytes(96, 128)
    with pytest.raises(ValueError):
        cpa.cp_attn_key_weights(cpa.Problem(8, 2, 2, 64, 64, 1), torch.zeros(8, 2, 64), torch.zeros(8, 2, 64),
                                torch.zeros(2, 8), last=0)
