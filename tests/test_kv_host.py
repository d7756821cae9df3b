"""Host-side checks of rotary positions, the paged cache in the model's own type and its pages: the oracle, and the
calls' refusals (everything here is refused or answered before GPU work)."""

import ctypes
import math

import numpy as np
import pytest
import torch

import oracle

cpa = pytest.importorskip("context_long_sequence_zigzag_gb300")

OK, BAD, UNS, WSP = cpa.CP_OK, cpa.CP_ERR_INVALID_ARG, cpa.CP_ERR_UNSUPPORTED, cpa.CP_ERR_WORKSPACE


# ---------------------------------------------------------------- the oracle
def test_oracle_rope_is_a_rotation_by_relative_position():
    rng = np.random.RandomState(0)
    q, k = rng.randn(1, 1, 12), rng.randn(1, 1, 12)
    f = 10.0 ** -np.arange(4)
    for adjacent in (False, True):
        turn = lambda x, p, inv=False: oracle.rope(x, p * f[None], 2, adjacent, inverse=inv)  # noqa: E731
        assert np.allclose((turn(q, 700) * turn(k, 690)).sum(), (turn(q, 10) * k).sum())
        assert np.allclose(turn(turn(q, 5), 5, True), q)
        assert np.array_equal(turn(q, 5)[..., [0, 1, 10, 11]], q[..., [0, 1, 10, 11]])
    # by hand: a quarter turn of one pair
    assert np.allclose(oracle.rope([[[1.0, 2.0]]], np.array([[math.pi / 2]])), [[[-2.0, 1.0]]])
    assert np.allclose(oracle.rope([[[1.0, 2.0]]], np.array([[math.pi / 2]]), factor=3.0), [[[-6.0, 3.0]]])


def test_oracle_attention():
    rng = np.random.RandomState(1)
    q, k, v = rng.randn(3, 4), rng.randn(5, 4), rng.randn(5, 2)
    o, lse = oracle.kv_attention(q, k, v, [np.arange(5), np.arange(1), np.arange(0)], 0.5)
    s = np.exp(k @ q[0] * 0.5)
    assert np.allclose(o[0], s @ v / s.sum()) and np.allclose(lse[0], np.log(s.sum()))
    assert np.allclose(o[1], v[0]) and np.allclose(lse[1], q[1] @ k[0] * 0.5)
    assert np.all(o[2] == 0) and lse[2] == -np.inf


def test_oracle_pages_by_hand():
    # pages of 4: sequences of 6 (pages 5, 3), 8 (5, 1), 0
    pool = oracle.Pages([0, 1, 0, 1, 0, 2, 0], 4)
    table = [[5, 3], [5, 1], [-1, -1]]
    rows, n, counts, pairs = pool.fork(table, [6, 8, 0], [0, 0, -1, 1, 0, 2])
    # 0 keeps page 3, its twins get 0 and 2; the page 1 stays whole with its one child
    assert rows == [[5, 3], [5, 0], [], [5, 1], [5, 2], []] and n == [6, 6, 0, 8, 6, 0]
    assert pairs == [(3, 0), (3, 2)] and pool.refs == [1, 1, 1, 1, 0, 4, 0] and counts == [5, 0]
    rows, counts = pool.reserve([r + [-1] * (4 - len(r)) for r in rows], n, [2, 3, 5, 1, 0, 0])
    assert rows == [[5, 3], [5, 0, 4], [6, -1], [5, 1, -1], [5, 2], []] and counts == [7, 2]
    rows, counts = pool.reserve([r + [-1] * (4 - len(r)) for r in rows], [8, 9, 1, 9, 6, 0], [-5, -9, 0, 3, 4, 0])
    assert rows == [[5], [], [6], [5, 1, -1], [5, 2, 0], []] and counts == [5, 0]
    pool = oracle.Pages([0, 3, 0, 0, 1, 2], 4)
    assert pool.compact() == ([-1, 1, -1, -1, 0, 2], [(4, 0), (5, 2)]) and pool.refs == [1, 3, 2, 0, 0, 0]
    # a page that another sequence holds whole is not written: both of these get copies
    pool = oracle.Pages([2, 1, 0, 0], 4)
    rows, n, counts, pairs = pool.fork([[0], [0, 1]], [2, 7], [0, 1, 1])
    assert rows == [[2], [0, 1], [0, 3]] and pairs == [(0, 2), (1, 3)]


# ---------------------------------------------------------------- frequencies
def test_turns():
    rng = np.random.RandomState(2)
    f = [0.0, 1.0, -1.0, 2 * math.pi, 1e-30, 5e-324, 4294967295.5, -123456.789, 2.0 ** -40, math.nextafter(1, 0)]
    f += list(np.exp(rng.uniform(-30, 22, 200)))
    assert cpa.cp_rope_turns(f) == oracle.rope_turns(f)
    assert cpa.cp_rope_turns(torch.tensor([1.0, 0.5], dtype=torch.float64)) == oracle.rope_turns([1.0, 0.5])
    for bad in (math.inf, math.nan, 2.0 ** 32, -2.0 ** 32):
        with pytest.raises(cpa.CpError):
            cpa.cp_rope_turns([1.0, bad])
    lib, one = cpa._lib, (ctypes.c_double * 1)(1.0)
    assert lib.cp_rope_turns(None, 1, one) == lib.cp_rope_turns(one, 1, None) == lib.cp_rope_turns(one, -1, one) == BAD
    assert lib.cp_rope_turns(None, 0, None) == OK


# ---------------------------------------------------------------- refusals
def _rope(**kw):
    base = dict(first=0, dims=128, pairing=0, axes=1, factor=1.0, turns=256, axis=None)
    base.update(kw)
    return cpa.cp_rope_t(**base)


@pytest.mark.parametrize("change,status", [
    ({"dims": 0}, BAD), ({"dims": 3}, BAD), ({"dims": -2}, BAD), ({"dims": 514}, UNS), ({"dims": 130}, BAD),
    ({"first": -1}, BAD), ({"first": 2}, BAD), ({"first": 2147483647, "dims": 2}, BAD), ({"axes": 0}, BAD),
    ({"axes": 5}, UNS), ({"axes": 3}, BAD), ({"pairing": 2}, BAD), ({"factor": math.inf}, BAD),
    ({"factor": math.nan}, BAD), ({"turns": None}, BAD), ({"turns": 260}, BAD), ({"axis": 258}, BAD)])
def test_rope_descriptor(change, status):
    lib, r = cpa._lib, _rope(**change)
    assert lib.cp_rope(ctypes.byref(r), 4, 256, 2, 128, 1, 2, 1 << 20, 1 << 21, 0, None, None, 0, None) == status
    c = _cache(d_qk=128)
    assert lib.cp_kv_append(ctypes.byref(c), 256, 256, 4, None, 256, 256, 4, ctypes.byref(r), 256, 2, None) == status


def test_rope_refuses_before_gpu_work():
    lib, r = cpa._lib, _rope()
    M = 1 << 20

    def f(T=4, pos=256, stride=1, d=128, dt=1, hq=2, q=M, qo=2 * M, hkv=1, k=3 * M, ko=4 * M, inv=0, r=r):
        return lib.cp_rope(None if r is None else ctypes.byref(r), T, pos, stride, d, dt, hq, q, qo, hkv, k, ko, inv, None)

    assert f(r=None) == f(T=-1) == f(T=1 << 31) == f(d=0) == f(hq=-1) == f(hkv=-1) == f(dt=2) == f(inv=2) == BAD
    assert f(d=132) == BAD  # rows of 264 bytes
    assert f(d=2048) == f(hq=1025) == f(hkv=1025) == UNS
    assert f(stride=0) == f(pos=None) == f(pos=258) == BAD
    assert f(q=None) == f(qo=None) == f(k=None) == f(ko=None) == f(q=M + 8) == f(ko=M + 8) == BAD
    n = 4 * 2 * 128 * 2
    assert f(qo=M + n - 16) == f(qo=M - n + 16) == BAD  # over its own input, but not in place
    assert f(qo=3 * M) == f(ko=M + 16) == f(ko=2 * M) == BAD  # over the other's input, or output
    assert f(T=0, q=None) == OK and f(hq=0, hkv=0, q=None, k=None, pos=None) == OK


def _cache(**kw):
    base = dict(num_seqs=2, hq=8, hkv=2, d_qk=128, d_v=128, gqa=0, dtype=cpa.CP_DT_BF16, scale=0.1, page_size=64,
                num_pages=4, max_pages=2, k_pages=4096, v_pages=8192, page_table=64)
    base.update(kw)
    return cpa.cp_kv_t(**base)


@pytest.mark.parametrize("change,status", [
    ({}, OK), ({"hq": 6, "hkv": 4}, BAD), ({"hkv": 0}, BAD), ({"num_seqs": -1}, BAD), ({"d_qk": 96}, UNS),
    ({"d_v": 192}, UNS), ({"d_v": 0}, BAD), ({"gqa": 2}, BAD), ({"dtype": 7}, BAD), ({"scale": math.nan}, BAD),
    ({"scale": 0.0}, BAD), ({"scale": 2e38}, UNS), ({"k_pages": None}, BAD), ({"v_pages": None}, BAD), ({"k_pages": 4104}, BAD),
    ({"page_table": 66}, BAD), ({"num_pages": -1}, BAD), ({"max_pages": -1}, BAD), ({"page_size": 0}, BAD),
    ({"page_size": 8}, UNS), ({"page_size": 48}, UNS), ({"page_size": 256}, UNS), ({"page_size": 16}, OK),
    ({"max_pages": 1 << 25}, UNS), ({"num_pages": 1 << 25}, UNS), ({"num_seqs": 4097}, UNS), ({"hq": 2048}, UNS),
    ({"num_seqs": 0, "k_pages": None, "v_pages": None, "page_table": None}, OK)])
def test_cache_descriptor(change, status):
    assert cpa._lib.cp_kv_validate(ctypes.byref(_cache(**change))) == status


def test_cache_calls_refuse_before_gpu_work():
    lib, c = cpa._lib, _cache()
    ref = ctypes.byref(c)
    assert lib.cp_kv_validate(None) == BAD

    def add(c=ref, k=256, v=256, n=4, rows=None, cu=256, start=256, tokens=4):
        return lib.cp_kv_append(c, k, v, n, rows, cu, start, tokens, None, None, 0, None)

    assert add(c=None) == add(k=None) == add(v=None) == add(k=264) == add(cu=None) == add(start=None) == BAD
    assert add(n=3) == add(n=-1) == add(tokens=-1) == add(n=1 << 31) == add(rows=258) == BAD
    assert add(tokens=0, k=None) == OK
    n = ctypes.c_size_t(0)
    assert lib.cp_kv_workspace_size(ref, 1, ctypes.byref(n)) == OK and n.value % 256 == 0
    assert lib.cp_kv_workspace_size(ref, 0, ctypes.byref(n)) == lib.cp_kv_workspace_size(ref, 1, None) == BAD
    assert lib.cp_kv_workspace_size(ref, 17, ctypes.byref(n)) == UNS

    def attn(c=c, n_q=1, q=256, lens=256, o=256, f=0, lse=256, ws=256, b=1 << 40):
        return lib.cp_kv_attn(ctypes.byref(c), n_q, q, lens, o, f, lse, ws, b, None)

    assert attn(n_q=0) == attn(q=None) == attn(o=None) == attn(lse=None) == attn(lens=None) == attn(f=2) == BAD
    assert attn(n_q=17) == UNS and attn(c=_cache(d_qk=80)) == UNS
    wide = _cache(max_pages=100)
    assert attn(wide, ws=None) == attn(wide, ws=128) == attn(wide, b=0) == WSP
    assert lib.cp_kv_workspace_size(ctypes.byref(wide), 1, ctypes.byref(n)) == OK and n.value > 0
    small = n.value
    for more in (_cache(max_pages=1000), _cache(max_pages=100, num_seqs=4000), _cache(max_pages=100, hq=256)):
        assert lib.cp_kv_workspace_size(ctypes.byref(more), 16, ctypes.byref(n)) == OK and n.value >= small
    assert attn(_cache(num_seqs=0), q=None) == OK


def _pool(num_pages=8, page_size=64, refs=256, base=(4096, 8192), size=(64, 32), n=None):
    pool = cpa.cp_pages_t(num_pages=num_pages, page_size=page_size, refs=refs, num_buffers=len(base) if n is None else n)
    pool.keep = ((ctypes.c_void_p * max(len(base), 1))(*base), (ctypes.c_int64 * max(len(size), 1))(*size))
    pool.base = ctypes.cast(pool.keep[0], ctypes.POINTER(ctypes.c_void_p))
    pool.bytes = ctypes.cast(pool.keep[1], ctypes.POINTER(ctypes.c_int64))
    return pool


@pytest.mark.parametrize("kw,status", [
    ({}, OK), ({"num_pages": -1}, BAD), ({"page_size": 0}, BAD), ({"refs": None}, BAD), ({"refs": 258}, BAD),
    ({"n": -1}, BAD), ({"n": 129}, UNS), ({"num_pages": (1 << 24) + 1}, UNS), ({"size": (64, 24)}, BAD),
    ({"size": (0, 32)}, BAD), ({"size": (64, 1 << 40)}, UNS), ({"base": (4096, 8200)}, BAD), ({"base": (None, 16)}, BAD),
    ({"base": (), "size": ()}, OK), ({"num_pages": 0, "refs": None, "base": (None, None)}, OK)])
def test_pool_descriptor(kw, status):
    assert cpa._lib.cp_pages_validate(ctypes.byref(_pool(**kw))) == status


def test_page_calls_refuse_before_gpu_work():
    lib, pool = cpa._lib, _pool()
    ref = ctypes.byref(pool)
    n = ctypes.c_size_t(0)
    assert lib.cp_pages_validate(None) == lib.cp_pages_workspace_size(ref, -1, ctypes.byref(n)) == BAD
    assert lib.cp_pages_workspace_size(ref, 4097, ctypes.byref(n)) == UNS
    assert lib.cp_pages_workspace_size(ref, 5, ctypes.byref(n)) == OK and n.value % 256 == 0

    def reserve(p=ref, B=2, cols=3, t=256, lens=256, extra=256, counts=256):
        return lib.cp_pages_reserve(p, B, cols, t, lens, extra, counts, None)

    assert reserve(p=None) == reserve(B=-1) == reserve(cols=-1) == reserve(t=None) == reserve(lens=None) == BAD
    assert reserve(extra=None) == reserve(counts=None) == reserve(t=258) == BAD
    assert reserve(B=4097) == reserve(cols=1 << 26) == UNS

    def fork(p=ref, B=2, cols=3, t=1024, lens=256, m=2, mcols=3, par=512, nt=2048, nl=4096, counts=256, ws=256, b=1 << 30):
        return lib.cp_pages_fork(p, B, cols, t, lens, m, mcols, par, nt, nl, counts, ws, b, None)

    assert fork(p=None) == fork(B=-1) == fork(m=-1) == fork(t=None) == fork(lens=None) == fork(par=None) == BAD
    assert fork(nt=None) == fork(nl=None) == fork(counts=None) == BAD
    assert fork(nt=1024) == fork(nt=1040) == fork(nl=256) == fork(nl=260) == fork(nl=512) == BAD  # onto the old ones
    assert fork(m=4097) == UNS and fork(ws=None) == fork(ws=264) == fork(b=16) == WSP

    def pack(p=ref, B=2, cols=3, t=1024, lens=256, nt=2048, moved=4096, counts=256, ws=256, b=1 << 30):
        return lib.cp_pages_compact(p, B, cols, t, lens, nt, moved, counts, ws, b, None)

    assert pack(p=None) == pack(t=None) == pack(nt=None) == pack(nt=1028) == pack(lens=None) == pack(moved=None) == BAD
    assert pack(counts=None) == BAD and pack(ws=None) == pack(b=0) == WSP

    def copy(p=pool, to=pool, m=3, src=256, dst=256):
        return lib.cp_pages_copy(ctypes.byref(p), ctypes.byref(to), m, src, dst, None)

    assert copy(m=-1) == copy(src=None) == copy(dst=258) == copy(to=_pool(size=(64, 48))) == BAD
    assert copy(to=_pool(base=(4096,), size=(64,))) == BAD
    assert copy(m=0, src=None) == OK and copy(_pool(base=(), size=()), _pool(base=(), size=())) == OK


def test_python_checks_its_tensors():
    f32, i32 = torch.float32, torch.int32
    with pytest.raises(ValueError):  # not on a GPU
        cpa.KvCache(torch.zeros(1, 2, 64, 128), torch.zeros(1, 2, 64, 128), torch.zeros(1, 1, dtype=i32), 2)
    with pytest.raises(ValueError):
        cpa.KvCache(torch.zeros(1, 2, 64, 128, dtype=torch.float16), torch.zeros(1, 2, 64, 128), torch.zeros(1, 1, dtype=i32), 2)
    with pytest.raises(ValueError):
        cpa.PagePool(torch.zeros(3, dtype=i32), [torch.zeros(3, 16)])
    with pytest.raises(ValueError):
        cpa.PagePool(None, [])
    for kw in ({"axis": [0]}, {"axis": [0, 4]}, {"axis": [0, -1]}, {"first": -1}, {"factor": math.inf}, {"device": "cpu"}):
        with pytest.raises(ValueError):
            cpa.Rope([1.0, 0.5], **kw)
    with pytest.raises(ValueError):
        cpa.Rope([], device="cpu")
    with pytest.raises(ValueError):
        cpa.cp_rope(None, None, torch.zeros(1, 1, 8, dtype=f32))
