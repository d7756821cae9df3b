"""Calls of the paged cache and its pages at sizes and forms where their kernels go other ways: against the float64
oracle, with the tolerances derived in test_gpu_kv.py unless a test says otherwise."""

import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
from test_gpu_kv import BF, F32, WIDE, Held, check_rope, f64, ints, pool_of, randn

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


# ---------------------------------------------------------------- attention: clusters or even shares
def test_attn_where_clusters_do_not_fit():
    """fp32 heads of 192 with 32 rows: one CTA an SM, so that 40 clusters of four do not fit and shares are even."""
    h = Held([70, 0, 200, 31, 129], 32, 8, 192, 128, F32, 64, 8, seed=32)
    assert cpa.cp_kv_workspace_size(h.cache, 8) > 0
    h.check(*h.run())


def test_a_cache_without_columns_or_pages():
    """A table of no columns: every sequence is empty, and neither pages nor a table have to be there.  A pool of no
    pages: every slot is absent."""
    c = cpa.cp_kv_t(num_seqs=2, hq=4, hkv=2, d_qk=64, d_v=64, gqa=0, dtype=cpa.CP_DT_F32, scale=0.1, page_size=64,
                    num_pages=4, max_pages=0, k_pages=None, v_pages=None, page_table=None)
    q, lengths = torch.ones(2, 1, 4, 64, device="cuda"), ints([0, 0])
    o, lse = torch.ones(2, 1, 4, 64, device="cuda"), torch.ones(4, 2, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    assert cpa._lib.cp_kv_attn(ctypes.byref(c), 1, q.data_ptr(), lengths.data_ptr(), o.data_ptr(), 0, lse.data_ptr(),
                               None, 0, stream) == cpa.CP_OK
    assert (o == 0).all() and (lse == -math.inf).all()
    cache = cpa.KvCache(torch.ones(4, 2, 64, 64, device="cuda"), torch.ones(4, 2, 64, 64, device="cuda"),
                        torch.empty(2, 0, dtype=torch.int32, device="cuda"), 4)
    o, lse = cpa.cp_kv_attn(cache, q, ints([0, 3]))  # (a length that the table does not hold)
    assert cpa.cp_device_status() == 0x302 and (o == 0).all() and (lse == -math.inf).all()
    for columns in (2, WIDE // 64 + 1):
        none = torch.empty(0, 2, 64, 64, device="cuda")
        cache = cpa.KvCache(none, none, torch.zeros(2, columns, dtype=torch.int32, device="cuda"), 4)
        o, lse = cpa.cp_kv_attn(cache, q, ints([0, 0]))
        assert cpa.cp_device_status() == 0 and (o == 0).all() and (lse == -math.inf).all()
        k = torch.ones(2, 2, 64, device="cuda")
        cpa.cp_kv_append(cache, k, k, ints([0, 1, 2]), ints([0, 70]))
        assert cpa.cp_device_status() == 0x301
        o, lse = cpa.cp_kv_attn(cache, q, ints([1, 71]))
        assert cpa.cp_device_status() == 0x301 and (o == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("hq,n_q,gqa", [(8, 1, "blocked"), (24, 9, "interleaved"), (128, 3, "blocked")])
def test_attn_in_clusters_of_four(hq, n_q, gqa, dtype):
    """Six sequences of eight kv heads in a short table: 48 runs (96 of fp32 with 48 rows, in even shares)."""
    h = Held([1, 64, 290, 0, 131, 33], hq, 8, 64, 64, dtype, 32, n_q, gqa, seed=33)
    assert (cpa.cp_kv_workspace_size(h.cache, n_q) == 0) == (dtype == BF or hq * n_q <= 8 * 32)
    h.check(*h.run())


# ---------------------------------------------------------------- tiles of several tokens
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,hq,hkv,d,first,pairs,adjacent", [
    (20011, 2, 1, 64, 0, 32, False), (20011, 1, 2, 64, 16, 16, True), (20011, 3, 1, 32, 3, 11, False),
    (50003, 1, 0, 16, 0, 1, True), (39001, 5, 3, 128, 64, 32, False)])
def test_rope_of_many_tokens(T, hq, hkv, d, first, pairs, adjacent, dtype):
    """Tiles of 8 to 20 tokens, the last one with fewer; with and without channels that only move."""
    rng = np.random.RandomState(T)
    q, k = randn(rng, (T, hq, d), dtype), randn(rng, (T, hkv, d), dtype)
    f = 10000.0 ** (-np.arange(pairs) / pairs)
    pos = rng.randint(0, 1 << 17, (T, 2))
    axis = rng.randint(0, 2, pairs)
    axis[0] = 1
    rope = cpa.Rope(f, axis=axis, first=first, pairing="adjacent" if adjacent else "halves")
    angle = pos[:, axis] * f[None]
    for inverse in (False, True):
        out = cpa.cp_rope(rope, ints(pos.tolist()), q, k if hkv else None, inverse=inverse)
        for got, x in zip(out if hkv else (out,), (q, k)):
            check_rope(got, x, angle, first, adjacent, 1.0, inverse)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pairs,first,adjacent", [(32, 0, False), (16, 32, True), (21, 3, False)])
def test_append_of_many_tokens(pairs, first, adjacent, dtype):
    """Tiles of 16 tokens, the last one with fewer and in part behind the last sequence."""
    rng = np.random.RandomState(34)
    start, counts, hkv, d, page = [7, 0, 100], [39000, 0, 1010], 2, 64, 16
    n, after = sum(counts), [a + m for a, m in zip(start, counts)]
    pages, table = pool_of(after, page, rng)
    k, v = randn(rng, (n + 9, hkv, d), dtype), randn(rng, (n + 9, hkv, d), dtype)
    kp, vp = (torch.full((pages, hkv, page, d), 7.0, dtype=dtype, device="cuda") for _ in range(2))
    f = 1000.0 ** (-np.arange(pairs) / pairs)
    rope = cpa.Rope(f, first=first, pairing="adjacent" if adjacent else "halves")
    cpa.cp_kv_append(cpa.KvCache(kp, vp, ints(table.tolist()), hkv), k, v, ints([0, 39000, 39000, n]), ints(start), rope=rope)
    slot = np.concatenate([np.arange(a, b) for a, b in zip(start, after)])
    at = table[np.repeat(np.arange(3), counts), slot // page], slot % page
    got_k, got_v = f64(kp).transpose(0, 2, 1, 3), f64(vp).transpose(0, 2, 1, 3)
    assert np.array_equal(got_v[at], f64(v)[:n])
    check_rope(torch.from_numpy(got_k[at]).to(dtype), k[:n], slot[:, None] * f[None], first, adjacent, 1.0, False)
    mark = np.ones((pages, page), bool)
    mark[at] = False
    assert np.all(got_k[mark] == 7) and np.all(got_v[mark] == 7)


# ---------------------------------------------------------------- pages taken back
@pytest.mark.parametrize("B,most,shared", [(1, 40000, 0), (7, 9000, 3000), (1500, 60, 20), (4096, 9, 0)])
def test_reserve_takes_many_pages_back(B, most, shared):
    """Thousands of entries go at once, of one sequence or of all, some of pages that others hold; others grow."""
    rng = np.random.RandomState(B)
    held = rng.randint(shared, most + 1, B)
    held[0] = most
    rows, at = [], shared
    for n in held:
        rows.append(list(range(shared)) + list(range(at, at + n - shared)))
        at += n - shared
    pages, columns, page = at + 50, most + 2, 16
    order = rng.permutation(pages)
    rows = [[int(order[p]) for p in r] for r in rows]
    refs = np.zeros(pages, int)
    np.add.at(refs, np.concatenate([np.array(r, int) for r in rows]), 1)
    lengths = [int(n) * page - int(rng.randint(0, page)) if n else 0 for n in held]
    extra = [int(-rng.randint(0, 2 * n + 2)) if rng.rand() < 0.7 else int(rng.randint(0, page)) for n in lengths]
    extra[0] = 5 - lengths[0]
    extra = [min(x, columns * page - n) for x, n in zip(extra, lengths)]
    table = np.full((B, columns), -7)
    for b, r in enumerate(rows):
        table[b, :len(r)] = r
    pool = cpa.PagePool(ints(refs.tolist()), [], page)
    t = ints(table.tolist())
    counts = cpa.cp_pages_reserve(pool, t, ints(lengths), ints(extra))
    # in arrays: sequences let go first, then the lowest free pages go to the lowest sequence
    needs = np.array([-(-max(n + x, 0) // page) for n, x in zip(lengths, extra)])
    for b, r in enumerate(rows):
        np.subtract.at(refs, np.array(r[needs[b]:], int), 1)
        table[b, needs[b]:len(r)] = -1
    free = np.flatnonzero(refs == 0)
    taken = 0
    for b, r in enumerate(rows):
        n = max(needs[b] - len(r), 0)
        table[b, len(r):len(r) + n] = free[taken:taken + n]
        taken += n
    refs[free[:taken]] = 1
    assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(pool.refs.cpu().numpy(), refs)
    assert counts.tolist() == [int((refs != 0).sum()), 0]


def test_reserve_takes_a_long_sequence_back_in_parallel():
    """65536 pages of one sequence: one after another in a thread they would take 5 ms; shared among the 8192 threads of
    the call a few dozen microseconds."""
    pages = 1 << 16
    pool = cpa.PagePool(torch.empty(pages, dtype=torch.int32, device="cuda"), [], 16)
    table = torch.empty(1, pages, dtype=torch.int32, device="cuda")
    lengths, extra, best = ints([pages * 16]), ints([-pages * 16]), 1e9
    for _ in range(4):
        pool.refs.fill_(1)
        torch.arange(pages, out=table[0])
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        counts = cpa.cp_pages_reserve(pool, table, lengths, extra)
        b.record()
        torch.cuda.synchronize()
        assert counts.tolist() == [0, 0] and (table == -1).all() and not pool.refs.any()
        best = min(best, a.elapsed_time(b))
    assert best < 2.0
