"""The 4-bit cache and the key weights at the limits of what their calls
accept: the widest caches, queries and keys that are not numbers, rows that see
nothing, pages that are not there."""

import math

import numpy as np
import pytest
import torch

import oracle
from test_gpu_kv4 import Filled, check_attn, f64, ints

pytestmark = pytest.mark.gpu

cpa = pytest.importorskip("context_long_sequence_zigzag_gb300")


@pytest.fixture(autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    assert cpa.cp_device_status() == 0


def test_append_and_read_of_the_widest_cache():
    """1024 heads of 192 + 128, more tokens than an SM's CTAs hold one each: one call gives what many short ones give."""
    hkv, d_qk, d_v, n, chunk = 1024, 192, 128, 12800, 512
    pages = n // 64
    torch.manual_seed(60)
    k, v = (torch.randn(n, hkv, d, device="cuda", dtype=torch.bfloat16) for d in (d_qk, d_v))
    table = ints([torch.randperm(pages).tolist()])
    make = lambda: cpa.Kv4Cache(torch.zeros(pages, hkv, cpa.cp_kv4_block_bytes(d_qk, d_v), dtype=torch.uint8,  # noqa: E731
                                            device="cuda"), table, hkv, hkv, d_qk, d_v)
    whole, pieces = make(), make()
    cpa.cp_kv4_append(whole, k, v, ints([0, n]), ints([0]))
    for i in range(0, n, chunk):
        cpa.cp_kv4_append(pieces, k[i:i + chunk], v[i:i + chunk], ints([0, chunk]), ints([i]))
    assert torch.equal(whole.pages, pieces.pages)
    rk, rv = cpa.cp_kv4_read(whole, ints([0, n]), ints([0]), n)
    for i in range(0, n, chunk):
        ck, cv = cpa.cp_kv4_read(pieces, ints([0, chunk]), ints([i]), chunk)
        assert torch.equal(rk[i:i + chunk], ck) and torch.equal(rv[i:i + chunk], cv)
    # a group's range is below 14, its step below 0.94: half of it, 15 roundings of the scale (2^-8), the value's own (2^-8
    # of 7) and the difference's: 0.94 (0.5 + 15 / 256) + 0.03 + 0.01 < 0.6
    assert (rk - k).abs().max() <= 0.6 and (rv - v).abs().max() <= 0.6
    torch.cuda.empty_cache()


@pytest.mark.parametrize("graph", [False, True])
def test_evictions_in_a_row_through_the_same_buffers(graph):
    """The move starts while the selection runs: it has to see this call's kept slots and lengths, not the last call's,
    which lie in the same buffers."""
    B, hkv, d, budget, recent, slots = 8, 4, 64, 200, 16, 1024
    pages, need = B * slots // 64, -(-budget // 64)
    torch.manual_seed(61)
    block = cpa.cp_kv4_block_bytes(d, d)
    table = torch.randperm(pages, device="cuda").int().view(B, -1)
    weights = torch.rand(pages, hkv, 64, device="cuda")
    full = cpa.Kv4Cache(torch.randint(0, 256, (pages, hkv, block), dtype=torch.uint8, device="cuda"), table, hkv, hkv, d, d,
                        weights)
    small = cpa.Kv4Cache(torch.zeros(B * need, hkv, block, dtype=torch.uint8, device="cuda"),
                         torch.arange(B * need, device="cuda").int().view(B, need), hkv, hkv, d, d,
                         torch.zeros(B * need, hkv, 64, device="cuda"))
    lens, new, kept = ints([0] * B), ints([0] * B), torch.zeros(B, hkv, budget, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            cpa.cp_kv4_evict(full, lens, budget, recent, small, new_lengths=new, kept=kept)
    for i in range(30):
        n = torch.randint(0, slots + 1, (B,)).int()
        lens.copy_(n)
        weights.uniform_()
        small.weights.fill_(-1.0)
        new.fill_(-1), kept.fill_(-1)
        if graph:
            g.replay()
        else:
            cpa.cp_kv4_evict(full, lens, budget, recent, small, new_lengths=new, kept=kept)
        want_n = n.clamp(max=budget)
        assert torch.equal(new.cpu(), want_n)
        held = weights[table.long()].transpose(1, 2).flatten(2)  # [B, hkv, slots]
        moved = small.weights.view(B, need, hkv, 64).transpose(1, 2).flatten(2)[..., :budget]
        behind = torch.arange(budget, device="cuda").view(1, 1, -1) >= want_n.cuda().view(-1, 1, 1)
        assert torch.equal(kept < 0, behind.expand_as(kept))
        assert torch.equal(moved, held.gather(2, kept.clamp(min=0).long()).masked_fill(behind, -1.0))
        for b in (0, B - 1):
            for h in range(hkv):
                keep = oracle.kv4_keep(held[b, h, :int(n[b])].tolist(), int(n[b]), budget, recent)
                assert kept[b, h, :len(keep)].tolist() == keep


# (9 to 16 rows of a kv head in bf16 take two column tiles, cuts of the long sequence meet in the second kernel; the
# scores are small, so that no row's rescaling depends on the others' values)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (4, 2), (6, 2)])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_attn_queries_that_are_no_numbers_stay_in_what_they_see(dtype, hq, hkv, bad):
    """Rows that see nothing give o = 0 and lse = -inf whatever they hold; a row of NaN is NaN, and so are the weights of
    the slots that it sees; nothing else changes."""
    n_q, lengths = 5, [3, 70, 20000, 0, 96]
    rng = np.random.RandomState(70)
    q = torch.from_numpy(rng.randn(5, n_q, hq, 128).astype(np.float32)).to(dtype).cuda()
    nan_rows = [(0, 0), (0, 1), (1, 0), (2, 1), (3, 2), (4, 4)]  # (sequence, query)
    runs = []
    for value in (0.0, bad):
        c = Filled(lengths, hq, hkv, 128, 128, dtype, seed=71, scale=0.002)
        x = q.clone()
        for b, t in nan_rows:
            x[b, t, :, 7] = value
        o, lse = cpa.cp_kv4_attn(c.cache, x, ints(lengths), accumulate=True)
        plain = cpa.cp_kv4_attn(c.cache, x, ints(lengths))
        assert torch.equal(o.nan_to_num(9.0), plain[0].nan_to_num(9.0))
        assert torch.equal(lse.nan_to_num(9.0), plain[1].nan_to_num(9.0))
        runs.append((o, lse.view(hq, 5, n_q), c.weights.cpu()))
    (o0, lse0, w0), (o, lse, w) = runs
    for b, n in enumerate(lengths):
        seen = [max(0, n - (n_q - 1 - t)) for t in range(n_q)]
        first = 0  # slots from here on are seen by no row of NaN
        for t in range(n_q):
            if seen[t] == 0:
                assert not o[b, t].any() and torch.isneginf(lse[:, b, t]).all()
            elif (b, t) in nan_rows:
                assert torch.isnan(o[b, t]).all() and torch.isnan(lse[:, b, t]).all()
                first = max(first, seen[t])
            else:
                assert torch.equal(o[b, t], o0[b, t]) and torch.equal(lse[:, b, t], lse0[:, b, t])
        ids = c.table[b, :-(-n // 64)]
        flat = [x[ids].transpose(0, 1).reshape(hkv, -1) for x in (w, w0)]
        assert torch.isnan(flat[0][:, :first]).all() and torch.equal(flat[0][:, first:], flat[1][:, first:])
    assert not torch.isnan(w0).any() and not torch.isnan(o0).any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attn_scores_of_next_to_nothing(dtype):
    """Queries near the smallest numbers and a scale near none: uniform weights, and unseen slots stay unseen."""
    c = Filled([1, 40, 300], 4, 2, 128, 128, dtype, seed=72, scale=1e-12)
    q = (torch.randn(3, 3, 4, 128, generator=torch.Generator().manual_seed(73)) * 1e-37).to(dtype).cuda()
    check_attn(c, n_q=3, q=q)


@pytest.mark.parametrize("exponent", [-9, -8, -7, -5, -3, -2])
def test_attn_small_channels_beside_a_large_one(exponent):
    """Every significand of a bf16 query channel far below the row's largest (128): off by at most 2^-17 of that, and
    not at all from 2^-9 of it on.  The large channel's key is 0 and the others' all 15, so that the errors add up."""
    c = Filled([1], 128, 1, 128, 128, seed=74, scale=0.01)
    page = c.table[0, 0]
    c.k[0][page], c.k[1][page], c.k[2][page] = 15, 0.0, 1.0
    c.k[0][page, :, :, 0] = 0
    c.pages.copy_(torch.from_numpy(oracle.kv4_pack(c.k, c.v)))
    x = (1 + torch.arange(128) / 128.0) * 2.0 ** exponent
    q = x.view(1, 1, 128, 1).repeat(1, 1, 1, 128)
    q[..., 0] = 128.0
    assert torch.equal(q.bfloat16().float(), q)
    _, lse = check_attn(c, q=q.bfloat16().cuda(), accumulate=False)
    # one slot: lse is the score.  127 channels of x 15 scale; fp32 sums of d / 16 terms
    exact = x.double().numpy() * 127 * 15 * 0.01
    most = 127 * 15 * 0.01 * 2.0 ** -10 if exponent < -2 else 0.0
    assert np.abs(lse[:, 0] - exact).max() <= most + 2.0 ** -19 * 31 * 0.01 * float(q.sum(-1).max())


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("lengths,last", [([1100, 130, 40], None), ([1100, 130, 40], 30), ([1100, 130, 40], 64),
                                          ([640], 32), ([640], 400)])
@pytest.mark.parametrize("d,dtype", [(128, torch.bfloat16), (192, torch.bfloat16), (64, torch.bfloat16),
                                     (128, torch.float32)])
@pytest.mark.parametrize("causal", [True, False])
def test_key_weights_of_queries_left_out(d, dtype, causal, lengths, last, bad):
    """lse = +inf leaves a query out whatever it holds, wherever its step lies: inside, on the diagonal, gathered."""
    hq, hkv = 4, 2
    rng = np.random.RandomState(80)
    cu = np.concatenate([[0], np.cumsum(lengths)]).tolist()
    T = cu[-1]
    q, k = (torch.from_numpy(rng.randn(T, h, d).astype(np.float32)).to(dtype) for h in (hq, hkv))
    lse = oracle.attn_forward(f64(q), f64(k), np.zeros((T, hkv, 8)), cu, d ** -0.5, causal=causal)[1].astype(np.float32)
    out = [(T - 1, h) for h in range(hq)] + [(T - 2, 1), (T - 20, 0), (600, 2), (600, 3), (3, 1)]  # (row, head)
    for i, h in out:
        lse[h, i] = math.inf
    perm = torch.from_numpy(oracle.shard_order(cu, 2, "zigzag"))
    prob = cpa.Problem(T, hq, hkv, d, 64, 2, "zigzag", cu, causal, dtype=dtype)
    dev = lambda x: x.index_select(0, perm).contiguous().cuda()  # noqa: E731
    lse_d = torch.from_numpy(lse)[:, perm].contiguous().cuda()
    want = oracle.attn_key_weights(f64(q), f64(k), lse.astype(np.float64), cu, d ** -0.5, causal, last)
    w = cpa.cp_attn_key_weights(prob, dev(q), dev(k), lse_d, last=last)
    got = np.zeros((hkv, T))
    got[:, perm.numpy()] = f64(w)
    # check_key_weights' bound
    big = float(q.abs().max() * k.abs().max()) * d ** 0.5
    tol = 2.0 ** -23 * (d / 16 * big + 64 + np.abs(lse[np.isfinite(lse)]).max() * 4)
    assert np.all(np.abs(got - want) <= tol * want + 1e-30)
    for i, h in out:
        q[i, h, 5] = bad
    assert torch.equal(cpa.cp_attn_key_weights(prob, dev(q), dev(k), lse_d, last=last), w)


def test_append_scales_halfway_between_two():
    """Ranges of 15 times a number halfway between two bf16 scales: to the even one, as (max - low) / 15 rounds."""
    half = torch.arange(257, 512, 2, dtype=torch.float64) / 512  # 9 bits, the last one set
    tokens = half.numel() * 3
    x = torch.zeros(tokens, 1, 64)
    x[:, 0, 17] = (15 * torch.cat([half, half * 2.0 ** 9, half * 2.0 ** -11])).float()
    assert torch.equal(x[:, 0, 17].double() / 15, torch.cat([half, half * 2.0 ** 9, half * 2.0 ** -11]))  # exact
    pages = -(-tokens // 64)
    block = cpa.cp_kv4_block_bytes(64, 64)
    cache = cpa.Kv4Cache(torch.zeros(pages, 1, block, dtype=torch.uint8, device="cuda"), ints([list(range(pages))]), 1, 1, 64,
                         64, dtype=torch.float32)
    cpa.cp_kv4_append(cache, x.cuda(), x.cuda(), ints([0, tokens]), ints([0]))
    held = [oracle.kv4_unpack(cache.pages[p, 0].cpu().numpy(), 64, 64) for p in range(pages)]
    want = (x[:, 0, 17].double() / 15).float().bfloat16().double().numpy()
    for which in range(2):
        step = np.concatenate([h[which][2] for h in held])[:tokens, 0]
        assert np.array_equal(step, want)


@pytest.mark.parametrize("n_q", [1, 3])
def test_attn_of_the_same_pages_in_fp32(n_q):
    """The pages do not depend on the descriptor's dtype: one of FP32 over pages of a BF16 cache gives FP32 results."""
    c = Filled([700, 33, 0], 8, 2, 128, 128, torch.bfloat16, seed=75)
    q = torch.randn(3, n_q, 8, 128, generator=torch.Generator().manual_seed(76)).bfloat16().cuda()
    check_attn(c, n_q=n_q, q=q, part=True, accumulate=False)
    c.dtype = torch.float32
    c.cache = cpa.Kv4Cache(c.pages, c.cache.page_table, 8, 2, 128, 128, c.weights, c.scale, "blocked", torch.float32)
    check_attn(c, n_q=n_q, q=q.float(), part=True)


@pytest.mark.parametrize("spread", [1e-37, 1e-20, 1e20, 1e36])
def test_attn_scale_against_the_queries_magnitude(spread):
    """The scale times the queries is what counts, whatever either is."""
    c = Filled([300, 40], 4, 2, 128, 128, seed=77, scale=0.1 / spread)
    q = torch.randn(2, 2, 4, 128, generator=torch.Generator().manual_seed(78)) * spread
    check_attn(c, n_q=2, q=q.bfloat16().cuda())
