"""GPU parity of the 4-bit key/value cache: append, read, attention, eviction
and a prompt's key weights against the float64 oracle.

Tolerances, derived from the arithmetic (u = 2^-24, the half step of fp32):
* codes (for the held scales), lows, kept slots, moved bytes: equal.  Scales:
  (max - low) / 15 in fp32 (4 u = 2^-22), rounded to bf16 (half a step, 2^-8).
* scores: fp32 sums of exact products of magnitude at most (16 + n) s |q|, and
  low |q|; d / 16 tensor-core adds a group and a few FMAs, each off by at most
  2 u of the running magnitude: SCORE = 2^-19 * scale * sum |q| (31 s + |low|)
  covers 16 such steps.  bf16 queries are taken as two e4m3 terms of a row
  scaled to a largest channel of 128 .. 256: four bits each, so exact where the
  second's last bit is at least 2^-9, and off by at most 2^-10 below (channels
  under 2^-9 of the largest): 2^-17 of the largest at most, with codes up to
  15.  TINY = scale * 2^-17 max |q| * 15 s * (number of such channels).
* lse: the scores' error, 2^-22 for the sum and log of it (relative to
  max(1, |lse|)).
* probabilities: relative error SCORE + 2^-20.  Weights: that of the sum.
* o: sum p s (n - 8) and sum p (low + 8 s) with those probabilities, in bf16
  caches with p s rounded to bf16, each by at most 2^-8 of itself: together
  2^-8 of sum p s |n - 8| = sum p |v - (low + 8 s)|; and rounded to bf16
  (2^-8 of o).
"""

import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

cpa = pytest.importorskip("context_long_sequence_zigzag_gb300")


@pytest.fixture(autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    assert cpa.cp_device_status() == 0


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def f64(t):
    return t.detach().cpu().double().numpy()


class Filled:
    """A pool of random held tokens, the table of some sequences, and what the pages hold."""

    def __init__(self, lengths, hq, hkv, d_qk, d_v, dtype=torch.bfloat16, seed=0, max_pages=None, extra_pages=2,
                 gqa="blocked", scale=None, pages_of=None):
        rng = np.random.RandomState(seed)
        need = [-(-n // 64) for n in lengths]
        self.max_pages = max(need + [1]) if max_pages is None else max_pages
        self.num_pages = sum(need) + extra_pages
        lead = (self.num_pages, hkv, 64)

        def held(d, spread):
            low = oracle.bf16_values(oracle.bf16_bits(-np.abs(rng.randn(*lead, d // 64)) * spread - 0.5))
            step = oracle.bf16_values(oracle.bf16_bits(rng.uniform(0.05, 0.3, lead + (d // 64,))))
            return rng.randint(0, 16, lead + (d,)).astype(np.uint8), low, step

        self.k, self.v = held(d_qk, 2.0), held(d_v, 1.0)
        order = rng.permutation(self.num_pages)
        # entries past a sequence's pages are never read: junk
        table = rng.randint(-5, 1 << 20, (len(lengths), self.max_pages))
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        self.table = table
        self.lengths, self.hq, self.hkv, self.d_qk, self.d_v, self.dtype = lengths, hq, hkv, d_qk, d_v, dtype
        self.gqa = gqa
        self.scale = d_qk ** -0.5 if scale is None else scale
        self.pages = torch.from_numpy(oracle.kv4_pack(self.k, self.v)).cuda()
        self.w0 = rng.rand(self.num_pages, hkv, 64).astype(np.float32)
        self.weights = torch.from_numpy(self.w0).cuda()
        self.cache = cpa.Kv4Cache(self.pages, ints(table.tolist()).reshape(len(lengths), self.max_pages), hq, hkv, d_qk,
                                  d_v, self.weights, self.scale, gqa, dtype)

    def kv_of(self, h):
        return h % self.hkv if self.gqa == "interleaved" else h // (self.hq // self.hkv)

    def sequence(self, b, which):
        """(values, lows, scales) of sequence b, [slots, hkv, ...]."""
        ids = self.table[b, :-(-self.lengths[b] // 64)]
        codes, low, step = (x[ids].transpose(0, 2, 1, 3).reshape(64 * len(ids), self.hkv, x.shape[-1])
                            for x in which)
        return oracle.kv4_values(codes, low, step), low, step


def check_attn(c, n_q=1, seed=1, part=False, q=None, accumulate=True, **kw):
    B = len(c.lengths)
    rng = np.random.RandomState(seed)
    if q is None:
        q = torch.from_numpy(rng.randn(B, n_q, c.hq, c.d_qk).astype(np.float32)).to(c.dtype).cuda()
    o, lse = cpa.cp_kv4_attn(c.cache, q, ints(c.lengths), accumulate=accumulate, part=part, **kw)
    torch.cuda.synchronize()
    o, lse, qn = f64(o), f64(lse), f64(q)
    assert o.shape == (B, n_q, c.hq, c.d_v) and lse.shape == (c.hq, B * n_q)
    want_w, tol_w = c.w0.astype(np.float64), 2.0 ** -23 * np.ones_like(c.w0)
    for b, n in enumerate(c.lengths):
        k, kl, ks = c.sequence(b, c.k)
        v, vl, vs = c.sequence(b, c.v)
        ref_o, ref_lse, ref_w = oracle.kv4_attention(qn[b], k, v, n, c.scale, c.kv_of)
        low = oracle.kv4_attention(qn[b], k, np.repeat(vl, 64, -1), n, c.scale, c.kv_of)[0]
        off = oracle.kv4_attention(qn[b], k, np.abs(v - np.repeat(vl + 8 * vs, 64, -1)), n, c.scale, c.kv_of)[0]
        for h in range(c.hq):
            g = c.kv_of(h)
            mag = (31 * ks[:n, g] + np.abs(kl[:n, g])).max(0) if n else np.zeros(c.d_qk // 64)
            qa = np.abs(qn[b, :, h])
            score = 2.0 ** -19 * c.scale * (qa.reshape(n_q, -1, 64).sum(-1) @ mag)  # [n_q]
            if c.dtype == torch.bfloat16 and n:
                top = qa.max(-1)
                tiny = ((qa > 0) & (qa < 2.0 ** -9 * top[:, None])).sum(-1)
                score = score + c.scale * 2.0 ** -17 * top * 15 * ks[:n, g].max() * tiny
            for t in range(n_q):
                if n - (n_q - 1 - t) <= 0:
                    assert lse[h, b * n_q + t] == -math.inf and not o[b, t, h].any()
                    continue
                assert abs(lse[h, b * n_q + t] - ref_lse[h, t]) <= score[t] + 2.0 ** -22 * max(1, abs(ref_lse[h, t]))
                above = ref_o[t, h] - low[t, h]  # sum p (v - low) >= 0
                tol = 2 * (score[t] + 2.0 ** -19) * (above + np.abs(low[t, h]))
                if c.dtype == torch.bfloat16:
                    tol = tol + 2.0 ** -8 * off[t, h] + (0 if part else 2.0 ** -8 * np.abs(ref_o[t, h]))
                err = np.abs(o[b, t, h] - ref_o[t, h])
                assert np.all(err <= tol), (b, t, h, (err - tol).max())
        ids = c.table[b, :-(-n // 64)]
        ref_w = ref_w.reshape(len(ids), 64, c.hkv).transpose(0, 2, 1)
        want_w[ids] += ref_w
        tol_w[ids] += (score.max() * 2 + 2.0 ** -19) * (ref_w + c.w0[ids])
    if accumulate:
        assert np.all(np.abs(f64(c.weights) - want_w) <= tol_w)
    else:
        assert np.array_equal(c.weights.cpu().numpy(), c.w0)
    return o, lse


# ---------------------------------------------------------------- attention
@pytest.mark.parametrize("d_qk,d_v", [(128, 128), (64, 64), (192, 128), (128, 64), (64, 128), (192, 64)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attn_head_dims(d_qk, d_v, dtype):
    check_attn(Filled([1, 63, 64, 65, 0, 300], 4, 2, d_qk, d_v, dtype, seed=3))


@pytest.mark.parametrize("hq,hkv,gqa", [(1, 1, "blocked"), (8, 8, "blocked"), (7, 1, "blocked"), (12, 3, "interleaved"),
                                        (18, 2, "blocked"), (40, 1, "blocked"), (16, 2, "interleaved")])
def test_attn_heads(hq, hkv, gqa):
    check_attn(Filled([33, 200, 2], hq, hkv, 128, 128, seed=4, gqa=gqa))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n_q", [1, 2, 3, 5, 16])
def test_attn_several_queries(n_q, dtype):
    """Early queries of a short sequence see nothing; the others see one slot fewer each."""
    check_attn(Filled([1, 2, 4, 0, 66, 130], 4, 2, 128, 128, dtype, seed=5), n_q=n_q)


@pytest.mark.parametrize("n", list(range(1, 5)) + [31, 32, 33, 95, 96, 97, 1000, 5000])
def test_attn_lengths(n):
    check_attn(Filled([n], 4, 1, 128, 128, seed=n))


def test_attn_many_sequences():
    rng = np.random.RandomState(6)
    check_attn(Filled([int(x) for x in rng.randint(0, 150, 211)], 2, 1, 64, 64, seed=7))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attn_long_sequence(dtype):
    check_attn(Filled([40001, 3], 8, 2, 128, 128, dtype, seed=8), n_q=2)


def test_attn_without_weights_leaves_them_and_a_cache_needs_none():
    c = Filled([70, 9], 4, 2, 128, 128, seed=9)
    check_attn(c, accumulate=False)
    bare = cpa.Kv4Cache(c.pages, c.cache.page_table, 4, 2, 128, 128)
    q = torch.randn(2, 1, 4, 128, device="cuda").bfloat16()
    a, b = cpa.cp_kv4_attn(bare, q, ints(c.lengths)), cpa.cp_kv4_attn(c.cache, q, ints(c.lengths))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    with pytest.raises(cpa.CpError):
        cpa.cp_kv4_attn(bare, q, ints(c.lengths), accumulate=True)


@pytest.mark.parametrize("spread", [1e-30, 1e-3, 1e25])
def test_attn_query_magnitudes(spread):
    """Queries far from 1, rows with one channel far above the others, rows of zeros."""
    c = Filled([300, 40], 4, 2, 128, 128, seed=19, scale=0.1 / spread)
    q = torch.randn(2, 2, 4, 128, device="cuda")
    q[0, 0, :2, 5] = 3000.0
    q[1, 1, 3] = 0.0
    q[0, 1, 1, :64] *= 1e-4
    check_attn(c, n_q=2, q=(q * spread).bfloat16())


def test_attn_infinite_query_gives_nan():
    c = Filled([100], 2, 1, 128, 128, seed=20)
    q = torch.randn(1, 1, 2, 128, device="cuda").bfloat16()
    ref = cpa.cp_kv4_attn(c.cache, q, ints([100]))
    q[0, 0, 1, 3] = math.inf
    o, lse = cpa.cp_kv4_attn(c.cache, q, ints([100]))
    assert torch.isnan(o[0, 0, 1]).all() and torch.isnan(lse[1, 0])
    assert torch.equal(o[0, 0, 0], ref[0][0, 0, 0]) and torch.equal(lse[0], ref[1][0])


def test_attn_thousands_of_sequences():
    """More sequences than leave room for eight rows' partials of the widest heads in shared memory."""
    rng = np.random.RandomState(21)
    lengths = [int(x) for x in rng.randint(0, 40, 1500)]
    c = Filled(lengths, 8, 1, 192, 128, seed=22)
    q = torch.from_numpy(rng.randn(1500, 1, 8, 192).astype(np.float32)).bfloat16().cuda()
    o, lse = cpa.cp_kv4_attn(c.cache, q, ints(lengths), accumulate=True)
    some = [0, 1, 700, 1498, 1499]
    for b in some:
        part = Filled.__new__(Filled)
        part.__dict__.update(c.__dict__, lengths=[lengths[b]], table=c.table[b:b + 1], weights=torch.from_numpy(c.w0).cuda())
        part.cache = cpa.Kv4Cache(c.pages, ints(part.table.tolist()).reshape(1, -1), 8, 1, 192, 128, part.weights)
        o1, lse1 = check_attn(part, q=q[b:b + 1].contiguous())
        ids = c.table[b, :-(-lengths[b] // 64)]
        assert np.abs(f64(c.weights)[ids] - f64(part.weights)[ids]).max(initial=0) < 1e-4
        assert np.abs(f64(o[b]) - o1[0]).max() < 0.05


def test_attn_large_scores():
    """Scores in the hundreds: only differences from the maximum may be exponentiated."""
    check_attn(Filled([500], 4, 2, 128, 128, torch.float32, seed=10, scale=4.0), accumulate=False)


def test_attn_rising_scores():
    """Every sub-block raises the maximum."""
    c = Filled([700], 2, 1, 64, 64, torch.float32, seed=11, scale=1.0)
    ids = c.table[0, :11]
    c.k[0][:] = 15
    for p, page in enumerate(ids):
        c.k[1][page] = 0.0
        c.k[2][page] = (np.arange(64) + 64 * p + 1)[None, :, None] / 1024.0
    c.k[2][:] = oracle.bf16_values(oracle.bf16_bits(c.k[2]))
    c.pages.copy_(torch.from_numpy(oracle.kv4_pack(c.k, c.v)))
    check_attn(c, q=torch.full((1, 1, 2, 64), 0.5, device="cuda"))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attn_nan_behind_the_end_and_in_unseen_slots(dtype):
    """NaN parameters past a sequence's end, and in the slots that only later queries see, reach nothing else."""
    c = Filled([75, 6], 4, 2, 128, 128, dtype, seed=12)
    q = torch.randn(2, 3, 4, 128, device="cuda").to(dtype)
    ref = cpa.cp_kv4_attn(c.cache, q, ints(c.lengths))
    page, row = int(c.table[0, 1]), 75 % 64
    c.k[2][page, :, row:] = math.nan
    c.v[1][page, :, row:] = math.nan
    c.v[2][page, :, row:] = math.nan
    c.k[1][page, 0, row - 1] = math.nan  # slot 74, head 0: the last query's alone
    c.v[2][page, 0, row - 1] = math.nan
    c.v[2][page, 1, row - 2] = math.nan  # slot 73, head 1 (values only): the last two's
    c.pages.copy_(torch.from_numpy(oracle.kv4_pack(c.k, c.v)))
    o, lse = cpa.cp_kv4_attn(c.cache, q, ints(c.lengths))
    got, want = torch.isnan(o).any(-1), torch.zeros(2, 3, 4, dtype=torch.bool, device="cuda")
    want[0, 2, :2] = True
    want[0, 1:, 2:] = True
    assert torch.equal(got, want)
    assert torch.equal(o[~want], ref[0][~want])
    nan_lse = torch.isnan(lse).view(4, 2, 3)
    assert nan_lse.sum() == 2 and bool(nan_lse[:2, 0, 2].all())


def test_attn_nothing_but_nan():
    """A sequence whose only visible keys are NaN gives NaN, not the empty result."""
    c = Filled([1, 40], 2, 1, 64, 64, seed=18)
    c.k[1][c.table[0, 0]] = math.nan
    c.k[1][c.table[1, 0]] = math.nan
    c.pages.copy_(torch.from_numpy(oracle.kv4_pack(c.k, c.v)))
    o, lse = cpa.cp_kv4_attn(c.cache, torch.ones(2, 1, 2, 64, device="cuda").bfloat16(), ints(c.lengths))
    assert torch.isnan(o).all() and torch.isnan(lse).all()


def test_attn_partials_join_to_the_whole():
    """A sequence cut over two caches (context-parallel ranks): the partial results join in cp_lse_merge."""
    c = Filled([128 + 71], 8, 2, 128, 128, seed=13)
    q = torch.randn(1, 1, 8, 128, device="cuda").bfloat16()
    whole = cpa.cp_kv4_attn(c.cache, q, ints([199]), part=True)
    parts = []
    for first, n in ((0, 128), (2, 71)):
        table = c.cache.page_table[:, first:first + 2].contiguous()
        part = cpa.Kv4Cache(c.pages, table, 8, 2, 128, 128)
        parts.append(cpa.cp_kv4_attn(part, q, ints([n]), part=True))
    prob = cpa.Problem(1, 8, 2, 128, 128, 1)
    o, lse = cpa.cp_lse_merge(prob, parts[0][0].view(1, 8, 128), parts[0][1], parts[1][0].view(1, 8, 128), parts[1][1])
    # both sides are off by SCORE (steps <= 0.3, lows above -10, |q| <= 5 a channel) and 2^-8 of sum p (v - low) <= 15 * 0.3
    score = 2.0 ** -19 * 128 ** -0.5 * float(q.abs().sum(-1).max()) * (31 * 0.31 + 10)
    assert (lse - whole[1]).abs().max() < 2 * score + 1e-5
    assert (o.view(-1) - whole[0].view(-1)).abs().max() < 2 * (2.0 ** -8 * 4.7 + 4 * score * 5)


def test_attn_repeats_bit_for_bit_and_in_a_graph():
    c = Filled([2000, 17, 0, 900], 8, 2, 128, 128, seed=14)
    q = torch.randn(4, 2, 8, 128, device="cuda").bfloat16()
    lens = ints(c.lengths)
    ref = [t.clone() for t in cpa.cp_kv4_attn(c.cache, q, lens, accumulate=True)] + [c.weights.clone()]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    o, lse = torch.empty_like(ref[0]), torch.empty_like(ref[1])
    ws = torch.empty(cpa.cp_kv4_workspace_size(c.cache, 2, True), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        cpa.cp_kv4_attn(c.cache, q, lens, accumulate=True, o=o, lse=lse, ws=ws)
    for _ in range(3):
        c.weights.copy_(torch.from_numpy(c.w0))
        ws.fill_(0xff)  # what a workspace held before does not matter
        graph.replay()
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1]) and torch.equal(c.weights, ref[2])
    lens.copy_(ints([1900, 0, 20, 900]))  # other lengths, same graph
    c.table[2, 0] = c.table[1, 0]
    c.cache.page_table.copy_(ints(c.table.tolist()))
    graph.replay()
    o2, lse2 = cpa.cp_kv4_attn(c.cache, q, lens)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_two_graphs_and_two_streams_at_once():
    """Captured calls with workspaces of their own run side by side; a workspace may serve one after the other."""
    c = Filled([3000, 500], 8, 2, 128, 128, seed=23)
    q = [torch.randn(2, 1, 8, 128, device="cuda").bfloat16() for _ in range(2)]
    lens = ints(c.lengths)
    ref = [cpa.cp_kv4_attn(c.cache, x, lens) for x in q]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for share in (False, True):
        ws = [torch.empty(cpa.cp_kv4_workspace_size(c.cache), dtype=torch.uint8, device="cuda") for _ in range(2)]
        if share:
            ws[1] = ws[0]
        out, graphs = [], []
        for i in range(2):
            o, lse, g = torch.empty_like(ref[i][0]), torch.empty_like(ref[i][1]), torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(g, stream=streams[i]):
                cpa.cp_kv4_attn(c.cache, q[i], lens, o=o, lse=lse, ws=ws[i])
            out.append((o, lse))
            graphs.append(g)
        torch.cuda.synchronize()
        for _ in range(20):
            for i in range(2):
                with torch.cuda.stream(streams[0 if share else i]):
                    graphs[i].replay()
        torch.cuda.synchronize()
        for a, b in zip(out, ref):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_key_weights_refuse_capture():
    T = 256
    q, k = torch.randn(T, 2, 128, device="cuda").bfloat16(), torch.randn(T, 2, 128, device="cuda").bfloat16()
    prob = cpa.Problem(T, 2, 2, 128, 64, 1, "contiguous")
    lse = torch.zeros(2, T, device="cuda")
    ws = torch.empty(cpa.cp_workspace_size(prob, cpa.CP_OP_KEY_WEIGHTS), dtype=torch.uint8, device="cuda")
    for last in (None, 16):
        w = cpa.cp_attn_key_weights(prob, q, k, lse, last=last, ws=ws)
        torch.cuda.synchronize()
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            with pytest.raises(cpa.CpError) as e:
                cpa.cp_attn_key_weights(prob, q, k, lse, last=last, w=w, ws=ws)
            torch.empty(1, device="cuda").zero_()  # the capture itself goes on
        assert e.value.status == cpa.CP_ERR_UNSUPPORTED


def test_attn_on_another_stream():
    c = Filled([3000], 8, 2, 128, 128, seed=15)
    q = torch.randn(1, 1, 8, 128, device="cuda").bfloat16()
    ref = cpa.cp_kv4_attn(c.cache, q, ints([3000]))
    side = torch.cuda.Stream()
    lens = ints([3000])
    side.wait_stream(torch.cuda.current_stream())
    got = [cpa.cp_kv4_attn(c.cache, q, lens, stream=side) for _ in range(4)]
    got.append(cpa.cp_kv4_attn(c.cache, q, lens, stream=side.cuda_stream))
    side.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, ref))


def test_buffers_made_for_another_stream_wait_for_their_last_use():
    """The outputs made here may take memory that work queued on the current stream still writes."""
    c = Filled([3000], 8, 2, 128, 128, seed=24)
    q, lens = torch.randn(1, 1, 8, 128, device="cuda").bfloat16(), ints([3000])
    ref = cpa.cp_kv4_attn(c.cache, q, lens)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        old = torch.empty_like(ref[0])
        torch.cuda._sleep(20_000_000)  # cycles: some 10 ms
        old.fill_(7.0)
        del old
        got = cpa.cp_kv4_attn(c.cache, q, lens, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_default_stream_by_its_handle():
    c = Filled([3000], 8, 2, 128, 128, seed=24)
    q, lens = torch.randn(1, 1, 8, 128, device="cuda").bfloat16(), ints([3000])
    ref = cpa.cp_kv4_attn(c.cache, q, lens)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        old = torch.empty_like(ref[0])
        torch.cuda._sleep(20_000_000)
        old.fill_(7.0)
        del old
        got = cpa.cp_kv4_attn(c.cache, q, lens, stream=0)  # on the default stream, after what this one holds
    torch.cuda.synchronize()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_attn_many_rows():
    """2048 rows of a kv head: 128 passes (256 in fp32)."""
    check_attn(Filled([70, 9], 256, 2, 64, 64, seed=25), n_q=16)
    check_attn(Filled([70, 9], 256, 2, 64, 64, seed=25, dtype=torch.float32), n_q=16)


def test_first_calls_are_captured():
    """Nothing has to run once before a capture: a process whose first calls are captured."""
    code = """
import torch, context_long_sequence_zigzag_gb300 as cpa
n = cpa.cp_kv4_block_bytes(128, 128)
ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
make = lambda t: cpa.Kv4Cache(torch.zeros(4, 2, n, dtype=torch.uint8, device="cuda"), ints(t), 4, 2, 128, 128,
                              torch.zeros(4, 2, 64, device="cuda"))
a, b = make([[2, 0]]), make([[1]])
k, v, q = (torch.randn(100, 2, 128, device="cuda").bfloat16() for _ in range(3))
cu, start, lens = ints([0, 100]), ints([0]), ints([100])
q = q.view(-1)[:512].view(1, 1, 4, 128)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    cpa.cp_kv4_append(a, k, v, cu, start)
    o, lse = cpa.cp_kv4_attn(a, q, lens, accumulate=True)
    new, kept = cpa.cp_kv4_evict(a, lens, 64, 8, b)
g.replay()
torch.cuda.synchronize()
assert abs(float(a.weights.sum()) - 4) < 1e-4 and new.tolist() == [64] and int((kept >= 0).sum()) == 128
"""
    done = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=240)
    assert done.returncode == 0, done.stderr[-2000:]


def test_decode_step_in_a_graph():
    """Append, attention with weights, eviction and read in one graph, replayed with other lengths and values."""
    B, hkv, d = 3, 2, 64

    def caches():
        c = Filled([150, 64, 20], 4, hkv, d, d, seed=26)
        ids = torch.arange(B * 2, dtype=torch.int32, device="cuda").view(B, 2)
        block = cpa.cp_kv4_block_bytes(d, d)
        return c, cpa.Kv4Cache(torch.zeros(B * 2, hkv, block, dtype=torch.uint8, device="cuda"), ids, 4, hkv, d, d,
                               torch.zeros(B * 2, hkv, 64, device="cuda"))

    (c1, to1), (c2, to2) = caches(), caches()
    k, v, q = (torch.randn(B, 1, h, d, device="cuda").bfloat16() for h in (hkv, hkv, 4))
    cu, start, lens = ints([0, 1, 2, 3]), ints([149, 62, 18]), ints([150, 63, 19])
    cu_read, zeros = ints([0, 40, 80, 120]), ints([0, 0, 0])

    def step(c, to):
        cpa.cp_kv4_append(c.cache, k.view(B, hkv, d), v.view(B, hkv, d), cu, start)
        o, lse = cpa.cp_kv4_attn(c.cache, q, lens, accumulate=True)
        new, kept = cpa.cp_kv4_evict(c.cache, lens, 100, 10, to)
        rk, rv = cpa.cp_kv4_read(to, cu_read, zeros, 120)
        return o, lse, new, kept, rk, rv

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(c1, to1)
    for n in ([150, 63, 19], [100, 64, 20], [128, 1, 2]):
        lens.copy_(ints(n))
        start.copy_(ints([x - 1 for x in n]))
        k.normal_(), v.normal_(), q.normal_()
        graph.replay()
        want = step(c2, to2)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.equal(c1.pages, c2.pages) and torch.equal(c1.weights, c2.weights)
        assert torch.equal(to1.pages, to2.pages) and torch.equal(to1.weights, to2.weights)


def test_attn_shared_prefix_pages():
    """Two sequences over the same page: both add to its weights."""
    c = Filled([64, 64], 4, 2, 128, 128, seed=16)
    c.table[1, 0] = c.table[0, 0]
    c.cache.page_table.copy_(ints(c.table.tolist()))
    check_attn(c)


def test_bad_pages_and_lengths_are_recorded_not_followed():
    """A page outside the pool counts as absent, a length outside the table is clamped."""
    c = Filled([130, 64], 4, 2, 128, 128, seed=17)
    q = torch.randn(2, 1, 4, 128, device="cuda").bfloat16()
    table = c.cache.page_table.clone()
    gone = cpa.Kv4Cache(c.pages, table[:, [0, 2, 1]].contiguous(), 4, 2, 128, 128)
    want = cpa.cp_kv4_attn(gone, q, ints([66, 0]))
    bad = table.clone()
    bad[0, 1] = c.num_pages
    got = cpa.cp_kv4_attn(cpa.Kv4Cache(c.pages, bad, 4, 2, 128, 128), q, ints([130, -7]))
    assert cpa.cp_device_status() & 0x300 == 0x300
    score = 2.0 ** -19 * 128 ** -0.5 * float(q.abs().sum(-1).max()) * (31 * 0.31 + 10)  # as above
    assert (got[1][:, 0] - want[1][:, 0]).abs().max() < 2 * score + 1e-5
    assert (got[0][0].float() - want[0][0].float()).abs().max() < 2 * (2.0 ** -8 * (4.7 + 5) + 4 * score * 5)
    assert not got[0][1].any() and torch.isneginf(got[1][:, 1]).all()


# ---------------------------------------------------------------- append and read
def empty_cache(num_pages, table, hq, hkv, d_qk, d_v, dtype):
    pages = torch.full((num_pages, hkv, cpa.cp_kv4_block_bytes(d_qk, d_v)), 0xA5, dtype=torch.uint8, device="cuda")
    weights = torch.full((num_pages, hkv, 64), -1.0, device="cuda")
    return cpa.Kv4Cache(pages, ints(table), hq, hkv, d_qk, d_v, weights, dtype=dtype)


def check_held(x, held):
    """codes, lows and scales that the cache holds of x [tokens, hkv, d]."""
    codes, low, step = held
    assert np.array_equal(low, oracle.kv4_quantise(x)[1])
    span = (x.reshape(low.shape + (64,)).max(-1) - low) / 15
    assert np.all(np.abs(step - span) <= (2.0 ** -8 + 2.0 ** -22) * span)
    assert np.array_equal(codes, oracle.kv4_codes(x, low, step))


@pytest.mark.parametrize("d_qk,d_v", [(128, 128), (64, 64), (192, 128), (128, 64)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_and_read(d_qk, d_v, dtype):
    rng = np.random.RandomState(20)
    hkv, counts, start = 3, [70, 0, 1, 5], [60, 3, 63, 0]
    cu, n = [0, 70, 70, 71, 76], 76
    table = [[4, 0, 9], [8, 8, 8], [1, 2, 7], [3, 5, 5]]
    cache = empty_cache(10, table, hkv, hkv, d_qk, d_v, dtype)
    before = cache.pages.clone()
    pad = 4  # rows behind the last sequence
    k = torch.from_numpy((rng.randn(n + pad, hkv, d_qk) * 2 + 1).astype(np.float32)).to(dtype).cuda()
    v = torch.from_numpy(rng.randn(n + pad, hkv, d_v).astype(np.float32)).to(dtype).cuda()
    k[5, 1] = 3.0       # one value: scale 0
    v[6, 2, :64] = 0.0
    k[7, 0, 3], k[8, 1, 9], v[9, 2, 0] = math.nan, math.inf, -math.inf
    w = torch.rand(hkv, n + pad, device="cuda")
    rows = ints(rng.permutation(n + pad)[:n + pad].tolist())
    cpa.cp_kv4_append(cache, k, v, ints(cu), ints(start), w=w, rows=rows)
    rk, rv = torch.full((n + pad, hkv, d_qk), 7.0, dtype=dtype, device="cuda"), torch.full((n + pad, hkv, d_v), 7.0, dtype=dtype, device="cuda")
    cpa.cp_kv4_read(cache, ints(cu), ints(start), n + pad, k=rk, v=rv)
    r = rows.long()
    touched = torch.zeros(10, 64, dtype=torch.bool)
    blocks = oracle.kv4_unpack  # one block at a time
    for b in range(4):
        for i in range(counts[b]):
            slot = start[b] + i
            page, row, t = table[b][slot // 64], slot % 64, cu[b] + i
            touched[page, row] = True
            src = int(r[t])
            assert torch.equal(cache.weights[page, :, row], w[:, src])
            for h in range(hkv):
                for held, x, back in zip(blocks(cache.pages[page, h].cpu().numpy(), d_qk, d_v), (k, v), (rk, rv)):
                    one = f64(x[src, h])
                    got = f64(back[t, h])
                    for g in range(len(one) // 64):
                        s = slice(64 * g, 64 * g + 64)
                        if not np.isfinite(one[s]).all():
                            assert np.isnan(got[s]).all()
                            continue
                        c, lo, st = held[0][row, s], held[1][row, g:g + 1], held[2][row, g:g + 1]
                        check_held(one[s], (c, lo, st))
                        want = torch.from_numpy(oracle.kv4_values(c, lo, st).astype(np.float32)).to(dtype)
                        assert np.array_equal(got[s], f64(want))
    # rows behind the last sequence and slots that no token went to stay as they were
    assert (rk[n:] == 7).all() and (rv[n:] == 7).all()
    assert (cache.weights.transpose(1, 2)[~touched.cuda()] == -1).all()
    for page in range(10):
        a, b = (oracle.kv4_unpack(x[page, 0].cpu().numpy(), d_qk, d_v) for x in (cache.pages, before))
        rest = ~touched[page].numpy()
        for p, q in zip(a, b):
            assert all(np.array_equal(x[rest], y[rest], equal_nan=True) for x, y in zip(p, q))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_rounds_halves_and_borders_exactly(dtype):
    """Values at and next to the borders between codes, for many scales and offsets."""
    rng = np.random.RandomState(21)
    x = []
    for _ in range(200):
        step = oracle.bf16_values(oracle.bf16_bits(np.float32(2.0 ** rng.uniform(-10, 10))))
        low = oracle.bf16_values(oracle.bf16_bits(np.float32(rng.randn() * step * 20)))
        g = low + step * (rng.randint(0, 15, 64) + 0.5)
        g[0], g[1] = low, low + 15 * step
        g[2:20] = np.nextafter(g[2:20].astype(np.float32), np.float32(1e30))
        g[20:40] = np.nextafter(g[20:40].astype(np.float32), np.float32(-1e30))
        x.append(g)
    x = torch.from_numpy(np.stack(x).astype(np.float32)).to(dtype).view(-1, 1, 64)
    cache = empty_cache(4, [[0, 1, 2, 3]], 1, 1, 64, 64, dtype)
    cpa.cp_kv4_append(cache, x.cuda(), x.cuda(), ints([0, 200]), ints([0]))
    held = [oracle.kv4_unpack(cache.pages[p, 0].cpu().numpy(), 64, 64) for p in range(4)]
    for which in range(2):
        codes, low, step = (np.concatenate([h[which][i] for h in held])[:200] for i in range(3))
        check_held(f64(x).reshape(200, 64), (codes, low, step))


def test_append_extremes():
    """The largest finite values, subnormal steps, and a constant offset far above the spread."""
    x = torch.zeros(4, 1, 64)
    x[0] = torch.linspace(-3.38e38, 3.38e38, 64, dtype=torch.float64)
    x[1] = torch.linspace(0, 1e-38, 64, dtype=torch.float64)
    x[2] = 1000.0 + torch.linspace(0, 1, 64)
    x[3] = -3.4028e38  # below bf16's lowest: reads as NaN, as an infinity does
    cache = empty_cache(1, [[0]], 1, 1, 64, 64, torch.float32)
    cpa.cp_kv4_append(cache, x.cuda(), x.cuda(), ints([0, 4]), ints([0]))
    k, v = cpa.cp_kv4_read(cache, ints([0, 4]), ints([0]), 4)
    assert torch.isnan(k[3]).all() and torch.isnan(v[3]).all()
    for i, tol in ((0, 6.8e38 / 15), (1, 1e-38 / 15), (2, 4.0 / 15)):  # half a step, doubled; low in bf16: 4 below 1000
        assert (k[i, 0].cpu().double() - x[i, 0].double()).abs().max() <= tol * 0.6
        assert torch.equal(k[i], v[i])
    assert (cache.weights[0, 0, :4] == 0).all()


def test_append_and_read_keep_out_of_what_is_not_theirs():
    cache = empty_cache(3, [[0, 3], [-1, 1]], 2, 2, 64, 64, torch.bfloat16)
    before = cache.pages.clone()
    k = torch.randn(6, 2, 64, device="cuda").bfloat16()
    # page 3 and page -1 are outside the pool, slot 128 outside the table, row 9 outside k
    for cu, start, rows in (([0, 3, 3], [64, 0], None), ([0, 0, 2], [0, 5], None), ([0, 0, 2], [0, 128], None),
                            ([0, 2, 2], [-2, 0], None), ([0, 1, 1], [0, 0], [9]), ([0, 1, 1], [0, 0], [-1])):
        cpa.cp_kv4_append(cache, k, k, ints(cu), ints(start), rows=None if rows is None else ints(rows))
        assert torch.equal(cache.pages, before), (cu, start, rows)
        assert cpa.cp_device_status() & 0x300 == 0x300
    out = torch.full((6, 2, 64), 5.0, device="cuda").bfloat16()
    cpa.cp_kv4_read(cache, ints([0, 3, 3]), ints([64, 0]), 6, k=out, v=out.clone())
    assert (out == 5).all() and cpa.cp_device_status() & 0x300 == 0x300


# ---------------------------------------------------------------- eviction
def check_evict(c, budget, recent, weights=None, to_pages=None):
    if weights is not None:
        c.w0 = weights.astype(np.float32)
        c.weights.copy_(torch.from_numpy(c.w0))
    B, need = len(c.lengths), -(-budget // 64)
    n_pages = B * need + 1 if to_pages is None else to_pages
    ids = np.random.RandomState(1).permutation(n_pages)[:B * need].reshape(B, need)
    to = cpa.Kv4Cache(torch.full((n_pages,) + tuple(c.pages.shape[1:]), 0x5A, dtype=torch.uint8, device="cuda"),
                      ints(ids.tolist()).reshape(B, need), c.hq, c.hkv, c.d_qk, c.d_v,
                      torch.full((n_pages, c.hkv, 64), -3.0, device="cuda"), dtype=c.dtype)
    before = c.pages.clone()
    new, kept = cpa.cp_kv4_evict(c.cache, ints(c.lengths), budget, recent, to)
    assert new.tolist() == [min(n, budget) for n in c.lengths]
    assert torch.equal(c.pages, before) and np.array_equal(c.weights.cpu().numpy(), c.w0, equal_nan=True)
    kept, w_to = kept.cpu().numpy(), to.weights.cpu().numpy()
    blocks = to.pages.cpu().numpy()
    blank = oracle.kv4_unpack(np.full(blocks.shape[2], 0x5A, np.uint8), c.d_qk, c.d_v)
    for b, n in enumerate(c.lengths):
        src = c.table[b]
        for h in range(c.hkv):
            w = np.concatenate([c.w0[src[p], h] for p in range(-(-n // 64))] + [np.zeros(0, np.float32)])[:n]
            want = oracle.kv4_keep(w.tolist(), n, budget, recent)
            assert kept[b, h].tolist() == want + [-1] * (budget - len(want))
            j = np.array(want, int)
            page = src[j // 64]
            flat = lambda parts: [x[page, h, j % 64] for x in parts]  # noqa: E731
            got = [oracle.kv4_unpack(blocks[p, h], c.d_qk, c.d_v) for p in ids[b]]
            for which, held in ((0, c.k), (1, c.v)):
                for i, x in enumerate(flat(held)):
                    out = np.concatenate([g[which][i] for g in got])
                    assert np.array_equal(out[:len(j)], x)
                    rest = np.concatenate([blank[which][i]] * need)[len(j):]  # slots behind: as they were
                    assert np.array_equal(out[len(j):], rest, equal_nan=True)
            out = np.concatenate([w_to[p, h] for p in ids[b]])
            assert np.array_equal(out[:len(j)], w[j], equal_nan=True) and (out[len(j):] == -3).all()


@pytest.mark.parametrize("budget,recent", [(1, 0), (1, 1), (64, 10), (65, 65), (100, 0), (100, 99), (1000, 3), (300, 300)])
def test_evict(budget, recent):
    check_evict(Filled([0, 1, 63, 64, 65, 101, 300, 1000, 1001], 2, 2, 128, 128, seed=30), budget, recent)


@pytest.mark.parametrize("d_qk,d_v,hkv", [(64, 64, 1), (192, 128, 3), (128, 64, 2)])
def test_evict_head_dims(d_qk, d_v, hkv):
    check_evict(Filled([500, 77], hkv, hkv, d_qk, d_v, seed=31), 90, 20)


@pytest.mark.parametrize("kind", ["equal", "few", "special", "signed", "close"])
def test_evict_ties_and_special_weights(kind):
    c = Filled([900, 130, 2500], 2, 2, 64, 64, seed=32)
    rng = np.random.RandomState(33)
    w = {"equal": np.ones_like(c.w0), "few": rng.randint(0, 3, c.w0.shape),
         "special": rng.choice([0.0, -0.0, 1.0, math.inf, -math.inf, math.nan, 1e-45], c.w0.shape),
         "signed": rng.randn(*c.w0.shape), "close": 1 + rng.randint(0, 4, c.w0.shape) * 2.0 ** -23}[kind]
    check_evict(c, 128, 30, weights=w)


def test_evict_long():
    check_evict(Filled([50000, 4097, 40], 2, 2, 64, 64, seed=34), 4096, 512)


def test_evict_rows_longer_than_shared_memory():
    """450,000 slots a row: their keys are read again in every pass."""
    n, budget, recent = 450_000, 1000, 100
    pages = -(-n // 64)
    rng = np.random.RandomState(36)
    table, w = rng.permutation(pages), rng.rand(pages, 1, 64).astype(np.float32)
    block = cpa.cp_kv4_block_bytes(64, 64)
    blank = lambda m: torch.zeros(m, 1, block, dtype=torch.uint8, device="cuda")  # noqa: E731
    c = cpa.Kv4Cache(blank(pages), ints([table.tolist()]), 1, 1, 64, 64, torch.from_numpy(w).cuda())
    to = cpa.Kv4Cache(blank(16), ints([list(range(16))]), 1, 1, 64, 64, torch.zeros(16, 1, 64, device="cuda"))
    new, kept = cpa.cp_kv4_evict(c, ints([n]), budget, recent, to)
    held = w[table].reshape(-1)[:n]
    want = oracle.kv4_keep(held.tolist(), n, budget, recent)
    assert new.tolist() == [budget] and kept[0, 0].tolist() == want
    assert np.array_equal(to.weights.cpu().numpy().reshape(-1)[:budget], held[want])


def test_evict_within_one_pool():
    """Another table of the same pool."""
    c = Filled([200], 1, 1, 64, 64, seed=35, extra_pages=4)
    free = [p for p in range(c.num_pages) if p not in c.table[0, :4]][:2]
    to = cpa.Kv4Cache(c.pages, ints([free]), 1, 1, 64, 64, c.weights)
    new, kept = cpa.cp_kv4_evict(c.cache, ints([200]), 100, 40, to)
    a, _ = cpa.cp_kv4_read(to, ints([0, 100]), ints([0]), 100)
    b, _ = cpa.cp_kv4_read(c.cache, ints([0, 200]), ints([0]), 200)
    assert new.tolist() == [100] and torch.equal(a[:, 0], b[kept[0, 0].long(), 0])


# ---------------------------------------------------------------- a prompt's key weights
def check_key_weights(lengths, hq, hkv, d, C, layout, last=None, dtype=torch.bfloat16, causal=True, gqa="blocked", seed=40,
                      spread=1.0):
    rng = np.random.RandomState(seed)
    cu = np.concatenate([[0], np.cumsum(lengths)]).tolist()
    T = cu[-1]
    q, k = (torch.from_numpy((rng.randn(T, h, d) * spread).astype(np.float32)).to(dtype) for h in (hq, hkv))
    perm = torch.from_numpy(oracle.shard_order(cu, C, layout))
    prob = cpa.Problem(T, hq, hkv, d, 64, C, layout, cu, causal, None, gqa, dtype)
    qn, kn = f64(q), f64(k)
    lse = oracle.attn_forward(qn, kn, np.zeros((T, hkv, 8)), cu, d ** -0.5, causal=causal,
                              gqa=gqa)[1].astype(np.float32)
    dev = lambda x: x.index_select(0, perm).contiguous().cuda()  # noqa: E731
    w = cpa.cp_attn_key_weights(prob, dev(q), dev(k), torch.from_numpy(lse)[:, perm].contiguous().cuda(), last=last)
    torch.cuda.synchronize()
    got = np.zeros((hkv, T))
    got[:, perm.numpy()] = f64(w)
    want = oracle.attn_key_weights(qn, kn, lse.astype(np.float64), cu, d ** -0.5, causal, last, gqa == "interleaved")
    # a probability's relative error: d / 16 tensor-core adds (or d / 32 fp32 adds and 5 of a warp's sum) of terms up to
    # |q||k| scale, the difference from lse and the exponential; the sums of at most 128-term parts
    big = np.abs(qn).max() * np.abs(kn).max() * d ** 0.5
    tol = 2.0 ** -23 * (d / 16 * big + 64 + np.abs(lse).max() * 4)
    assert np.all(np.abs(got - want) <= tol * want + 1e-30), (np.abs(got - want) / np.maximum(want, 1e-30)).max() / tol
    return w


@pytest.mark.parametrize("layout", ["contiguous", "zigzag", "striped"])
@pytest.mark.parametrize("C", [1, 2, 4])
@pytest.mark.parametrize("last", [None, 1, 50, 200])
def test_key_weights_layouts(layout, C, last):
    check_key_weights([700, 1, 129, 64], 4, 2, 128, C, layout, last)


@pytest.mark.parametrize("d,dtype", [(128, torch.bfloat16), (192, torch.bfloat16), (64, torch.bfloat16),
                                     (64, torch.float32), (128, torch.float32)])
def test_key_weights_dims(d, dtype):
    check_key_weights([515, 130], 4, 4, d, 2, "zigzag", None, dtype)
    check_key_weights([515, 130], 4, 4, d, 2, "zigzag", 33, dtype)


@pytest.mark.parametrize("hq,hkv,gqa", [(6, 2, "interleaved"), (7, 1, "blocked"), (3, 3, "blocked")])
@pytest.mark.parametrize("last", [None, 32])
def test_key_weights_heads(hq, hkv, gqa, last):
    check_key_weights([300, 45], hq, hkv, 128, 2, "zigzag", last, gqa=gqa)


def test_key_weights_not_causal_and_packed():
    check_key_weights([100, 300, 7, 260], 4, 2, 128, 2, "contiguous", causal=False)
    check_key_weights([100, 300, 7, 260], 4, 2, 128, 2, "zigzag", 40, causal=False)
    rng = np.random.RandomState(41)
    lengths = [int(x) for x in rng.randint(1, 400, 30)]
    check_key_weights(lengths, 4, 2, 128, 4, "zigzag")
    check_key_weights(lengths, 4, 2, 128, 4, "zigzag", 20)
    check_key_weights(lengths, 2, 2, 192, 2, "striped")


def test_key_weights_excluded_queries_and_debug_checks():
    """lse = +inf leaves a query out; plans of windows pass the plan checks."""
    T, cu = 400, [0, 400]
    q, k = torch.randn(T, 2, 128, device="cuda").bfloat16(), torch.randn(T, 2, 128, device="cuda").bfloat16()
    prob = cpa.Problem(T, 2, 2, 128, 64, 1, "contiguous", cu)
    lse = torch.from_numpy(oracle.attn_forward(f64(q), f64(k), np.zeros((T, 2, 8)), cu, 128 ** -0.5)[1]).float().cuda()
    some = lse.clone()
    some[:, :350] = math.inf
    old = cpa.cp_set_debug_checks(True)
    try:
        a = cpa.cp_attn_key_weights(prob, q, k, some)
        b = cpa.cp_attn_key_weights(prob, q, k, lse, last=50)
        torch.cuda.synchronize()
    finally:
        cpa.cp_set_debug_checks(old)
    assert (a - b).abs().max() <= 1e-6 * b.max()
    assert (a.sum() - 100).abs() < 1e-3  # 2 heads, 50 queries


@pytest.mark.parametrize("last", [None, 20, 16])
def test_key_weights_infinite_key(last):
    """A key of -inf under positive queries has scores of -inf: weight 0, and no other key changes."""
    T, cu = 300, [0, 300]
    q, k = torch.rand(T, 2, 128).bfloat16() + 0.5, torch.randn(T, 2, 128).bfloat16()
    k[37] = -math.inf
    lse = oracle.attn_forward(f64(q), f64(k), np.zeros((T, 2, 8)), cu, 128 ** -0.5)[1]
    want = oracle.attn_key_weights(f64(q), f64(k), lse, cu, 128 ** -0.5, True, last)
    prob = cpa.Problem(T, 2, 2, 128, 64, 1, "contiguous", cu)
    w = f64(cpa.cp_attn_key_weights(prob, q.cuda(), k.cuda(), torch.from_numpy(lse).float().cuda(), last=last))
    assert (w[:, 37] == 0).all() and (want[:, 37] == 0).all()
    # (check_key_weights' bound with |q| <= 1.5, |k| < 5, |lse| < 7: 2^-23 (8 * 85 + 64 + 28) = 9.2e-5)
    assert np.all(np.abs(w - want) <= 1e-4 * want + 1e-30)


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prompt_then_decode_with_eviction(dtype):
    """A packed prompt in zigzag shards through cp_attn_fwd, its keys' weights, the cache, eviction, and decoding steps
    that append, attend and add to the weights; each step against the oracle on what the cache holds."""
    rng = np.random.RandomState(50)
    lengths, hq, hkv, d, C, budget, recent = [330, 97], 4, 2, 64, 2, 128, 32
    cu = [0, 330, 427]
    T = cu[-1]
    q, k, v = (torch.from_numpy(rng.randn(T, h, d).astype(np.float32)).to(dtype).cuda() for h in (hq, hkv, hkv))
    prob = cpa.Problem(T, hq, hkv, d, d, C, "zigzag", cu, dtype=dtype)
    qs, ks, vs = (cpa.cp_shard_permute(prob, x) for x in (q, k, v))
    o, lse = cpa.cp_attn_fwd(prob, qs, ks, vs)
    w = cpa.cp_attn_key_weights(prob, qs, ks, lse)
    # the sharded row of every token, by the same permutation
    at = torch.arange(T, dtype=torch.int32, device="cuda").view(T, 1).expand(T, 4).contiguous()
    rows = cpa.cp_shard_permute(prob, at, inverse=True)[:, 0].contiguous()
    assert torch.equal(ks[rows.long()], k)
    block = cpa.cp_kv4_block_bytes(d, d)
    make = lambda table, n: cpa.Kv4Cache(torch.zeros(n, hkv, block, dtype=torch.uint8, device="cuda"), ints(table), hq,  # noqa: E731
                                         hkv, d, d, torch.zeros(n, hkv, 64, device="cuda"), dtype=dtype)
    full = make([[0, 1, 2, 3, 4, 5], [6, 7, -1, -1, -1, -1]], 8)
    cpa.cp_kv4_append(full, ks, vs, ints(cu), ints([0, 0]), w=w, rows=rows)
    small = make([[5, 1, 3], [2, 0, 4]], 6)
    lens, kept = cpa.cp_kv4_evict(full, ints(lengths), budget, recent, small)
    assert lens.tolist() == [128, 97] and kept[0, :, 96:].tolist() == [list(range(298, 330))] * 2
    wn = f64(w[:, rows.long()])
    for h in range(hkv):
        assert kept[0, h].tolist() == oracle.kv4_keep(wn[h, :330].tolist(), 330, budget, recent)
    held = [128, 97]
    for step in range(3):
        n_q = step + 1
        qd, kd, vd = (torch.from_numpy(rng.randn(2 * n_q, h, d).astype(np.float32)).to(dtype).cuda() for h in (hq, hkv, hkv))
        cpa.cp_kv4_append(small, kd, vd, ints([0, n_q, 2 * n_q]), ints(held))
        held = [n + n_q for n in held]
        before = small.weights.clone()
        od, _ = cpa.cp_kv4_attn(small, qd.view(2, n_q, hq, d), ints(held), accumulate=True)
        exact = cpa.Kv4Cache(small.pages, small.page_table, hq, hkv, d, d, dtype=torch.float32)  # values read as they are
        rk, rv = cpa.cp_kv4_read(exact, ints([0, held[0], sum(held)]), ints([0, 0]), sum(held))
        added = (small.weights - before)[small.page_table.long()].transpose(1, 2).flatten(2)  # [2, hkv, slots]
        for b in range(2):
            s = slice(0, held[0]) if b == 0 else slice(held[0], None)
            ref = oracle.kv4_attention(f64(qd.view(2, n_q, hq, d)[b]), f64(rk[s]), f64(rv[s]), held[b], d ** -0.5, lambda h: h // 2)
            # a group's range is at most 2 max |x|, its step a 15th of that: 31 s + |low| <= 31 / 7.5 + 1 times max |x|
            score = 2.0 ** -19 * d ** -0.5 * float(qd.abs().sum(-1).max()) * 5.2 * float(rk.abs().max())
            top = float(rv.abs().max())
            tol = 2 * (score + 2.0 ** -19) * 3 * top + (2.0 ** -8 * 3 * top if dtype == torch.bfloat16 else 0)
            assert np.abs(f64(od[b]) - ref[0]).max() < tol
            # (each probability at most 1, over 2 heads and n_q queries; sums of up to a few hundred lose 2^-23 of that)
            assert np.abs(f64(added[b, :, :held[b]]) - ref[2].T).max() < 2 * n_q * (2 * score + 2.0 ** -19) + 2.0 ** -23 * 700
            assert not added[b, :, held[b]:].any()
