"""Cases of the serving operators: a key/value cache held in 4 bits, attention over it, eviction by attention weight.

``run`` computes an operator in its plain form (elementary torch operations, fp32) where ``own`` is false, and makes
the package's call where it is true.  Both take the same state.

Cache format.  A page holds 64 tokens.  A page's block of one key/value head is two sub-blocks of 32 tokens, each
    K codes [32][d_qk / 2]   V codes [32][d_v / 2]   K parameters [32][2][d_qk / 64]   V scales [32][d_v / 64]
    V lows [d_v / 64][32]
with parameters in bf16 (K: the scales, then the lows).  A channel group is 64 channels; value = scale * code + low.
Eight channels 8w .. 8w+7 share a 32-bit word, channel 8w+i in bits 4i; word w of a K row lies at position
(w % 4) * (d / 32) + w / 4 of the row, of a V row at (w % 8) * (d / 64) + w / 8.
"""

import math

import numpy as np
import torch

own = False

PAGE = 64
SUB = 32
GROUP = 64


# ---------------------------------------------------------------- cases
def _append(name, batch, new, hkv, d_qk, d_v, dtype, cp, held, lens_seed):
    return {"name": name, "op": "append", "batch": batch, "new": new, "hkv": hkv, "d_qk": d_qk, "d_v": d_v,
            "dtype": dtype, "cp": cp, "held": held, "lens_seed": lens_seed}


def _attn(name, batch, tokens, ragged, hq, hkv, d_qk, d_v, dtype, n_q, weights, lens_seed):
    return {"name": name, "op": "attn", "batch": batch, "tokens": tokens, "ragged": ragged, "hq": hq, "hkv": hkv,
            "d_qk": d_qk, "d_v": d_v, "dtype": dtype, "n_q": n_q, "weights": weights, "lens_seed": lens_seed}


def _evict(name, batch, tokens, ragged, hkv, d_qk, d_v, budget, recent, lens_seed):
    return {"name": name, "op": "evict", "batch": batch, "tokens": tokens, "ragged": ragged, "hkv": hkv,
            "d_qk": d_qk, "d_v": d_v, "budget": budget, "recent": recent, "lens_seed": lens_seed}


def _keyw(name, tokens, seqs, hq, hkv, d_qk, cp, layout, last, dtype, lens_seed):
    return {"name": name, "op": "keyw", "tokens": tokens, "seqs": seqs, "hq": hq, "hkv": hkv, "d_qk": d_qk,
            "cp": cp, "layout": layout, "last": last, "dtype": dtype, "lens_seed": lens_seed}


def listed():
    return [
        # one decoding step's new tokens of 32 requests: launch latency counts
        _append("append 1 x 32", 32, 1, 8, 128, 128, "bf16", 1, 4096, 1),
        # a 64K prompt, straight out of its 8 zigzag shards, with its keys' weights
        _append("append prompt 64K", 1, 65536, 8, 128, 128, "bf16", 8, 0, 2),
        # one request answering from a 16K prompt: the latency of a single decoding step
        _attn("attn 1 x 16K", 1, 16384, False, 32, 8, 128, 128, "bf16", 1, False, 3),
        # eight requests of 1 to 64K tokens in one batch
        _attn("attn 8 x ragged 64K", 8, 65536, True, 32, 8, 128, 128, "bf16", 1, False, 4),
        # heads of their own keys (192 wide, values 128), 128K tokens
        _attn("attn mla 128K", 1, 131072, False, 64, 64, 192, 128, "bf16", 1, False, 5),
        # fp32 queries, 64-wide heads, short ragged requests
        _attn("attn f32 d64", 5, 1999, True, 8, 4, 64, 64, "f32", 1, False, 6),
        # decoding that also sums the attention weight of every held token
        _attn("attn weights 4 x 64K", 4, 65536, False, 16, 4, 128, 128, "bf16", 1, True, 7),
        # four speculated tokens a request, checked in one pass
        _attn("attn weights spec 4", 16, 8191, True, 32, 8, 128, 128, "bf16", 4, True, 8),
        # a 64K prompt cut to 4K tokens before decoding
        _evict("evict 64K to 4K", 1, 65536, False, 8, 128, 128, 4096, 512, 9),
        # 32 requests that have outgrown their budget by two pages
        _evict("evict 32 x 4224", 32, 4224, False, 8, 128, 128, 4096, 256, 10),
        # every key's weight over all queries of a 16K prompt in two zigzag shards
        _keyw("key weights 16K", 16384, 1, 32, 8, 128, 2, "zigzag", 0, "bf16", 11),
        # the weights that the last 64 queries of a 64K prompt give
        _keyw("key weights 64K last 64", 65536, 1, 32, 8, 128, 8, "zigzag", 64, "bf16", 12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "evict", "keyw"])
    lens_seed = rng.randrange(1 << 30)
    d_qk, d_v = rng.choice([(128, 128), (128, 128), (64, 64), (192, 128)])
    hkv = rng.choice([1, 2, 4, 8])
    if op == "append":
        batch = _log(rng, 1, 64)
        new = 1 if rng.random() < 0.4 else _log(rng, 2, max(2, 65536 // batch))
        case = _append("", batch, new, hkv, d_qk, d_v, rng.choice(["bf16", "bf16", "f32"]),
                       rng.choice([1, 2, 4]), rng.randrange(0, 3000), lens_seed)
    elif op == "attn":
        batch = _log(rng, 1, 64)
        tokens = _log(rng, 16, max(16, min(131072, 4194304 // (batch * hkv))))
        n_q = rng.choice([1, 1, 1, 2, 3, 4, 8])
        case = _attn("", batch, tokens, rng.random() < 0.7, hkv * rng.choice([1, 2, 4, 7, 8]), hkv, d_qk, d_v,
                     rng.choice(["bf16", "bf16", "bf16", "f32"]), n_q, rng.random() < 0.4, lens_seed)
    elif op == "evict":
        batch = _log(rng, 1, 32)
        tokens = _log(rng, 100, max(100, min(131072, 1048576 // (batch * hkv))))
        budget = max(2, int(tokens * rng.uniform(0.03, 1.1)))
        case = _evict("", batch, tokens, rng.random() < 0.5, hkv, d_qk, d_v, budget, rng.randrange(0, budget),
                      lens_seed)
    else:
        last = rng.choice([0, 0, 1, 16, 32, 64, 100, 256])
        tokens = _log(rng, 200, 8192 if last == 0 else 65536)
        case = _keyw("", tokens, rng.choice([1, 1, 2, 5]), hkv * rng.choice([1, 2, 4]), hkv, rng.choice([128, 128, 192]),
                     rng.choice([1, 2, 4, 8]), rng.choice(["contiguous", "zigzag", "striped"]), last, "bf16", lens_seed)
    del case["name"]
    return case


def _lengths(case):
    """Tokens that every sequence of the case holds before the call."""
    n, b = case["tokens"], case["batch"]
    if not case["ragged"]:
        return [n] * b
    rs = np.random.RandomState(case["lens_seed"])
    got = [int(x) for x in np.exp(rs.uniform(0.0, math.log(n), b)).round().clip(1, n)]
    got[rs.randint(b)] = n
    return got


def _splits(case):
    """Lengths of the packed sequences of a prompt."""
    cuts = np.sort(np.random.RandomState(case["lens_seed"]).randint(0, case["tokens"] + 1, case["seqs"] - 1))
    return [int(x) for x in np.diff(np.concatenate([[0], cuts, [case["tokens"]]]))]


def _sharded(lengths, cp, layout):
    """Global row, sequence and position of every row of the sharded order."""
    rows, start = [], 0
    per_rank = [[] for _ in range(cp)]
    for s, n in enumerate(lengths):
        at = np.arange(n)
        for r in range(cp):
            if layout == "striped":
                mine = at[r::cp]
            elif layout == "contiguous":
                mine = at[r * n // cp:(r + 1) * n // cp]
            else:
                m = 2 * cp
                other = m - 1 - r
                mine = np.concatenate([at[r * n // m:(r + 1) * n // m], at[other * n // m:(other + 1) * n // m]])
            per_rank[r].append(np.stack([start + mine, np.full(len(mine), s), mine]))
        start += n
    for r in range(cp):
        rows += per_rank[r]
    return np.concatenate(rows, axis=1) if rows else np.zeros((3, 0), np.int64)


# ---------------------------------------------------------------- the packed format, plainly
def _sizes(d_qk, d_v):
    parts = [SUB * d_qk // 2, SUB * d_v // 2, SUB * d_qk // GROUP * 4, SUB * d_v // GROUP * 2, SUB * d_v // GROUP * 2]
    return parts, sum(parts)


def _word_at(d, lanes, device):
    w = torch.arange(d // 8, device=device)
    return (w % lanes) * (d // (8 * lanes)) + w // lanes


def _quantise(x):
    """Codes [..., d] (uint8), scales and lows [..., d / 64] (bf16) of x [..., d]; the codes' borders in 64 bits."""
    g = x.float().unflatten(-1, (-1, GROUP))
    low = g.amin(-1).bfloat16()
    low = torch.where(low.float() > g.amin(-1), torch.nextafter(low, torch.full_like(low, -math.inf)), low)
    scale = ((0.5 * g.amax(-1) - 0.5 * low.float()) / 7.5).bfloat16()
    s = scale.float().unsqueeze(-1)
    n = ((g.double() - low.double().unsqueeze(-1)) / torch.where(s > 0, s, torch.ones_like(s))).round().clamp(0, 15)
    return torch.where(s > 0, n, torch.zeros_like(n)).flatten(-2).to(torch.uint8), scale, low


def _dequantise(codes, scale, low):
    g = codes.unflatten(-1, (-1, GROUP)).float()
    return (g * scale.float().unsqueeze(-1) + low.float().unsqueeze(-1)).flatten(-2)


def _pack_codes(codes, lanes):
    d = codes.shape[-1]
    w = codes.unflatten(-1, (d // 8, 8))
    out = torch.empty_like(w)
    out[..., _word_at(d, lanes, codes.device), :] = w
    out = out.flatten(-2)
    return out[..., 0::2] | (out[..., 1::2] << 4)


def _unpack_codes(b, lanes):
    d = 2 * b.shape[-1]
    n = torch.stack([b & 15, b >> 4], -1).flatten(-2).unflatten(-1, (d // 8, 8))
    return n[..., _word_at(d, lanes, b.device), :].flatten(-2)


def _pack_pages(k, v):
    """Blocks [pages, heads, bytes] of k, v [pages, heads, 64, d]."""
    at = lambda x: x.unflatten(2, (2, SUB))  # noqa: E731
    (kc, ks, kl), (vc, vs, vl) = (_quantise(at(x)) for x in (k, v))
    raw = lambda x: x.contiguous().view(torch.uint8).flatten(3)  # noqa: E731
    parts = [_pack_codes(kc, 4).flatten(3), _pack_codes(vc, 8).flatten(3), raw(torch.cat([ks, kl], -1)), raw(vs),
             raw(vl.transpose(-1, -2))]
    return torch.cat(parts, -1).flatten(2)


def _values(pages, table, d_qk, d_v):
    """k [B, heads, P * 64, d_qk] and v in fp32 of the pages that a table names."""
    parts, sub = _sizes(d_qk, d_v)
    b = pages[table.clamp(min=0).long()].unflatten(-1, (2, sub))  # [B, P, heads, 2, sub]
    kc, vc, kp, vs, vl = b.split(parts, -1)
    half = lambda x: x.contiguous().view(torch.bfloat16)  # noqa: E731
    kp = half(kp).unflatten(-1, (SUB, 2, d_qk // GROUP))
    k = _dequantise(_unpack_codes(kc.unflatten(-1, (SUB, -1)), 4), kp[..., 0, :], kp[..., 1, :])
    v = _dequantise(_unpack_codes(vc.unflatten(-1, (SUB, -1)), 8), half(vs).unflatten(-1, (SUB, -1)),
                    half(vl).unflatten(-1, (-1, SUB)).transpose(-1, -2))
    flat = lambda x: x.permute(0, 2, 1, 3, 4, 5).flatten(2, 4)  # noqa: E731
    return flat(k), flat(v)


# ---------------------------------------------------------------- states
def _dtype(case):
    return torch.float32 if case.get("dtype") == "f32" else torch.bfloat16


def _keys(gen, shape):
    """Keys as projections give them: some channels with an offset and a spread of their own."""
    d = shape[-1]
    spread = torch.exp(0.5 * torch.randn(d, generator=gen, device="cuda"))
    offset = torch.randn(d, generator=gen, device="cuda")
    return torch.randn(shape, generator=gen, device="cuda") * spread + offset


def _table(gen, lengths, columns):
    """A pool's size and a table [B, columns] of its pages in no order; -1 where a sequence has none."""
    need = [-(-n // PAGE) for n in lengths]
    total = sum(need) + 3
    ids = torch.randperm(total, generator=gen, device="cuda")[:sum(need)].to(torch.int32)
    table = torch.full((len(lengths), columns), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return total, table


def _filled(gen, total, hkv, d_qk, d_v):
    """A pool of `total` pages, every slot holding a token."""
    some = max(1, (1 << 22) // (hkv * PAGE))
    spread = torch.exp(0.5 * torch.randn(d_qk, generator=gen, device="cuda"))
    offset = torch.randn(d_qk, generator=gen, device="cuda")
    got = []
    for at in range(0, total, some):
        n = min(some, total - at)
        k = torch.randn(n, hkv, PAGE, d_qk, generator=gen, device="cuda") * spread + offset
        v = torch.randn(n, hkv, PAGE, d_v, generator=gen, device="cuda")
        got.append(_pack_pages(k.bfloat16(), v.bfloat16()))
    return torch.cat(got)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cu(counts):
    return _ints(np.concatenate([[0], np.cumsum(counts)]).tolist())


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = {"case": case}
    op = case["op"]
    if op == "append":
        hkv, d_qk, d_v = case["hkv"], case["d_qk"], case["d_v"]
        start, counts = _append_rows(case)
        total, s["table"] = _table(gen, [a + n for a, n in zip(start, counts)], max(-(-(a + n) // PAGE) for a, n in zip(start, counts)))
        n = sum(counts)
        s["k"] = _keys(gen, (n, hkv, d_qk)).to(_dtype(case))
        s["v"] = torch.randn(n, hkv, d_v, generator=gen, device="cuda").to(_dtype(case))
        s["w"] = torch.rand(hkv, n, generator=gen, device="cuda") ** 4
        s["pages"] = torch.zeros(total, hkv, 2 * _sizes(d_qk, d_v)[1], dtype=torch.uint8, device="cuda")
        s["weights"] = torch.zeros(total, hkv, PAGE, device="cuda")
        s["cu"], s["start"] = _cu(counts), _ints(start)
        order = _sharded(counts, case["cp"], "zigzag")[0]
        s["rows"] = _ints(np.argsort(order).tolist())  # the sharded row of every token
        s["seq"] = torch.repeat_interleave(torch.arange(len(counts), device="cuda"), torch.tensor(counts, device="cuda"))
        s["slot"] = torch.cat([torch.arange(a, a + m, device="cuda") for a, m in zip(start, counts)])
    elif op == "attn":
        hq, hkv, d_qk, d_v = case["hq"], case["hkv"], case["d_qk"], case["d_v"]
        lengths = _lengths(case)
        total, s["table"] = _table(gen, lengths, -(-max(lengths) // PAGE))
        s["pages"] = _filled(gen, total, hkv, d_qk, d_v)
        s["q"] = torch.randn(case["batch"], case["n_q"], hq, d_qk, generator=gen, device="cuda").to(_dtype(case))
        s["lengths"] = _ints(lengths)
        s["weights"] = torch.rand(total, hkv, PAGE, generator=gen, device="cuda")
        s["sums"] = s["weights"].clone()
    elif op == "evict":
        hkv, d_qk, d_v = case["hkv"], case["d_qk"], case["d_v"]
        lengths = _lengths(case)
        after = [min(n, case["budget"]) for n in lengths]
        total, s["table"] = _table(gen, lengths, -(-max(lengths) // PAGE))
        s["pages"] = _filled(gen, total, hkv, d_qk, d_v)
        s["weights"] = torch.rand(total, hkv, PAGE, generator=gen, device="cuda") ** 8
        to, s["to_table"] = _table(gen, after, -(-case["budget"] // PAGE))
        s["to_pages"] = torch.zeros(to, hkv, s["pages"].shape[2], dtype=torch.uint8, device="cuda")
        s["to_weights"] = torch.zeros(to, hkv, PAGE, device="cuda")
        s["lengths"], s["cu"], s["zero"] = _ints(lengths), _cu(after), _ints([0] * len(lengths))
        s["seq"] = torch.repeat_interleave(torch.arange(len(after), device="cuda"), torch.tensor(after, device="cuda"))
        s["slot"] = torch.cat([torch.arange(n, device="cuda") for n in after])
    else:
        hq, hkv, d = case["hq"], case["hkv"], case["d_qk"]
        lengths = _splits(case)
        _, seq, pos = (torch.from_numpy(x).cuda() for x in _sharded(lengths, case["cp"], case["layout"]))
        n = case["tokens"]
        s["q"] = torch.randn(n, hq, d, generator=gen, device="cuda").to(_dtype(case))
        s["k"] = _keys(gen, (n, hkv, d)).to(_dtype(case))
        s["seq"], s["pos"] = seq, pos
        near = pos >= torch.tensor(lengths, device="cuda")[seq] - (case["last"] or n)
        s["queries"] = near.nonzero()[:, 0]
        s["lse"] = torch.zeros(hq, n, device="cuda")
        some = max(1, (1 << 31) // (n * hq))
        for at in range(0, len(s["queries"]), some):
            i = s["queries"][at:at + some]
            x = _pair_scores(s["q"][i], s["k"], seq[i], pos[i], seq, pos, d ** -0.5)
            s["lse"][:, i] = torch.logsumexp(x, -1).unflatten(1, (hq // hkv, -1)).flatten(0, 1)
        s["lengths"] = lengths
    return s


def _append_rows(case):
    """Tokens held before, and tokens that come, for every sequence."""
    rs = np.random.RandomState(case["lens_seed"])
    b, new = case["batch"], case["new"]
    start = [int(x) for x in rs.randint(0, case["held"] + 1, b)]
    counts = [new] * b if new == 1 or b == 1 else [int(x) for x in rs.randint(0, new + 1, b - 1)] + [new]
    return start, counts


# ---------------------------------------------------------------- one pass
def run(s):
    return {"append": _run_append, "attn": _run_attn, "evict": _run_evict, "keyw": _run_keyw}[s["case"]["op"]](s)


def _cache(s, hq, pages="pages", table="table", weights="weights"):
    """The package's handle of a state's pages, which a program keeps."""
    name = "handle of " + pages
    if name not in s:
        import context_long_sequence_zigzag_gb300 as cpa

        c = s["case"]
        s["package"] = cpa
        s[name] = cpa.Kv4Cache(s[pages], s[table], hq, c["hkv"], c["d_qk"], c["d_v"], weights=s.get(weights),
                               dtype=_dtype(c))
    return s["package"], s[name]


def _run_append(s):
    """Rows of k, v and their weights into the cache; what the cache then holds of them."""
    case = s["case"]
    if own:
        cpa, cache = _cache(s, case["hkv"])
        cpa.cp_kv4_append(cache, s["k"], s["v"], s["cu"], s["start"], w=s["w"], rows=s["rows"])
        k, v = cpa.cp_kv4_read(cache, s["cu"], s["start"], s["k"].shape[0])
        return {"k": k, "v": v, "weights": s["weights"]}
    rows = s["rows"].long()
    k, v = (_dequantise(*_quantise(s[x][rows])).to(_dtype(case)) for x in ("k", "v"))
    page = s["table"][s["seq"], s["slot"] // PAGE].long()
    weights = s["weights"].clone()
    weights[page, :, s["slot"] % PAGE] = s["w"][:, rows].t()
    return {"k": k, "v": v, "weights": weights}


def _run_attn(s):
    """One decoding step: the newest n_q queries of every sequence against the tokens it holds."""
    case = s["case"]
    if own:
        cpa, cache = _cache(s, case["hq"], weights="sums")
        if case["weights"]:
            s["sums"].copy_(s["weights"])
        o, lse = cpa.cp_kv4_attn(cache, s["q"], s["lengths"], accumulate=case["weights"])
        return {"o": o, "lse": lse, "weights": s["sums"]} if case["weights"] else {"o": o, "lse": lse}
    hkv, n_q, b = case["hkv"], case["n_q"], case["batch"]
    g = case["hq"] // hkv
    k, v = _values(s["pages"], s["table"], case["d_qk"], case["d_v"])
    q = s["q"].float().unflatten(2, (hkv, g)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [B, hkv, n_q * g, d]
    x = (q * case["d_qk"] ** -0.5) @ k.transpose(-1, -2)
    at = torch.arange(k.shape[2], device="cuda")
    behind = (n_q - 1 - torch.arange(n_q, device="cuda")).repeat_interleave(g)
    seen = (at < (s["lengths"][:, None, None] - behind[:, None]))[:, None]
    x = torch.where(seen, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    held = (at < s["lengths"][:, None])[:, None, :, None]
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    o = p @ torch.where(held, v, torch.zeros_like(v))
    o = o.unflatten(2, (n_q, g)).permute(0, 2, 1, 3, 4).flatten(2, 3).to(_dtype(case))
    lse = (top + torch.log(total)).squeeze(-1).unflatten(2, (n_q, g)).permute(1, 3, 0, 2).reshape(case["hq"], b * n_q)
    if not case["weights"]:
        return {"o": o, "lse": lse}
    given = p.sum(2).unflatten(2, (-1, PAGE)).transpose(1, 2).flatten(0, 1)  # [B * P, hkv, 64]
    weights = s["weights"].index_add(0, s["table"].clamp(min=0).flatten().long(), given)
    return {"o": o, "lse": lse, "weights": weights}


def _run_evict(s):
    """The kept tokens of every sequence and head in pages of their own."""
    case = s["case"]
    budget, recent, hkv = case["budget"], case["recent"], case["hkv"]
    if own:
        cpa, cache = _cache(s, hkv)
        _, to = _cache(s, hkv, "to_pages", "to_table", "to_weights")
        after, kept = cpa.cp_kv4_evict(cache, s["lengths"], budget, recent, to)
        k, v = cpa.cp_kv4_read(to, s["cu"], s["zero"], s["seq"].shape[0])
        return {"after": after, "kept": kept, "k": k, "v": v, "weights": s["to_weights"]}
    table = s["table"].clamp(min=0).long()
    w = s["weights"][table].transpose(1, 2).flatten(2)  # [B, hkv, slots]
    slots = w.shape[2]
    at = torch.arange(slots, device="cuda")
    n = s["lengths"][:, None, None]
    w = torch.where(at < n - recent, w, torch.where(at < n, math.inf, -math.inf))
    order = torch.sort(w, dim=-1, descending=True, stable=True)[1][..., :budget]
    after = torch.minimum(s["lengths"], torch.full_like(s["lengths"], budget))
    rank = torch.arange(order.shape[2], device="cuda")
    kept = torch.sort(torch.where(rank < after[:, None, None], order, slots), -1)[0]
    kept = torch.nn.functional.pad(kept, (0, budget - kept.shape[2]), value=slots)
    k, v = _values(s["pages"], s["table"], case["d_qk"], case["d_v"])
    from_slot = kept[s["seq"], :, s["slot"]]  # [rows, hkv]
    head = torch.arange(hkv, device="cuda")
    seq = s["seq"][:, None]
    k, v = (x[seq, head, from_slot].bfloat16() for x in (k, v))
    page = s["to_table"][s["seq"], s["slot"] // PAGE].long()
    weights = s["to_weights"].clone()
    weights[page, :, s["slot"] % PAGE] = s["weights"][table[seq, from_slot // PAGE], head, from_slot % PAGE]
    kept = torch.where(kept < slots, kept, -1).to(torch.int32)
    return {"after": after, "kept": kept, "k": k, "v": v, "weights": weights}


def _pair_scores(q, k, q_seq, q_pos, k_seq, k_pos, scale):
    """scale q.k where the query sees the key, else -inf: [hkv, G * queries, keys] in fp32."""
    hq, hkv = q.shape[1], k.shape[1]
    x = q.float().mul(scale).unflatten(1, (hkv, hq // hkv)).permute(1, 2, 0, 3).flatten(1, 2) @ k.float().permute(1, 2, 0)
    seen = (q_seq[:, None] == k_seq) & (q_pos[:, None] >= k_pos)
    return x.unflatten(1, (hq // hkv, -1)).masked_fill_(~seen, -math.inf).flatten(1, 2)


def _run_keyw(s):
    """Every key's attention weight, summed over the queries that count and the heads that share it."""
    case = s["case"]
    if own:
        if "problem" not in s:
            import context_long_sequence_zigzag_gb300 as cpa

            s["package"] = cpa
            s["problem"] = cpa.Problem(case["tokens"], case["hq"], case["hkv"], case["d_qk"], 128, case["cp"],
                                       case["layout"], np.concatenate([[0], np.cumsum(s["lengths"])]).tolist(), dtype=_dtype(case))
        return s["package"].cp_attn_key_weights(s["problem"], s["q"], s["k"], s["lse"], last=case["last"] or None)
    i = s["queries"]
    x = _pair_scores(s["q"][i], s["k"], s["seq"][i], s["pos"][i], s["seq"], s["pos"], case["d_qk"] ** -0.5)
    lse = s["lse"][:, i].unflatten(0, (case["hkv"], -1)).flatten(1, 2)
    return x.sub_(lse[..., None]).exp_().sum(1)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "keyw":
        pairs = 0
        for n in _splits(case):
            m = min(n, case["last"] or n)
            pairs += m * (n - m) + m * (m + 1) // 2
        queries = sum(min(n, case["last"] or n) for n in _splits(case))
        elt = 2 if case["dtype"] == "bf16" else 4
        moved = case["tokens"] * case["hkv"] * (case["d_qk"] * elt + 4) + queries * case["hq"] * (case["d_qk"] * elt + 4)
        return {"bytes": moved, "flops": 2.0 * pairs * case["hq"] * case["d_qk"]}
    hkv, d_qk, d_v = case["hkv"], case["d_qk"], case["d_v"]
    held = _sizes(d_qk, d_v)[1] / SUB  # bytes of one token's head
    if op == "append":
        tokens = sum(_append_rows(case)[1])
        elt = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": tokens * hkv * (2 * elt * (d_qk + d_v) + held + 8) + 4 * tokens, "flops": 0.0}
    lengths = _lengths(case)
    if op == "attn":
        elt = 2 if case["dtype"] == "bf16" else 4
        rows = case["batch"] * case["n_q"] * case["hq"]
        per = held + (8 if case["weights"] else 0)
        return {"bytes": sum(lengths) * hkv * per + rows * (elt * (d_qk + d_v) + 4),
                "flops": 2.0 * sum(lengths) * case["n_q"] * case["hq"] * (d_qk + d_v)}
    kept = sum(min(n, case["budget"]) for n in lengths)
    return {"bytes": sum(lengths) * hkv * 4 + kept * hkv * (2 * held + 8 + 2 * (d_qk + d_v)), "flops": 0.0}


# ---------------------------------------------------------------- from the definitions, in 64 bits
def _held_64(blocks, d, off, lanes, where):
    """Channels of packed rows by their bytes: blocks [..., bytes] (two sub-blocks), slots 0 .. 63 -> [..., 64, d] in 64 bits.

    where(slot, group) -> byte offsets of a group's scale and low inside a sub-block."""
    dev = blocks.device
    sub = blocks.shape[-1] // 2
    slot = torch.arange(PAGE, device=dev)[:, None]
    ch = torch.arange(d, device=dev)
    word = ch // 8
    spot = (word % lanes) * (d // (8 * lanes)) + word // lanes
    base = (slot // SUB) * sub
    byte = base + off + (slot % SUB) * (d // 2) + spot * 4 + (ch % 8) // 2
    code = (blocks[..., byte].to(torch.int16) >> (4 * (ch % 2)).to(torch.int16)) & 15
    two = []
    for at in where(slot % SUB, ch // GROUP):
        bits = blocks[..., base + at].to(torch.int32) | (blocks[..., base + at + 1].to(torch.int32) << 8)
        two.append((bits << 16).view(torch.float32).double())
    return two[0] * code + two[1]


def _kv_64(pages, d_qk, d_v):
    o1 = SUB * d_qk // 2
    o2 = o1 + SUB * d_v // 2
    o3 = o2 + SUB * 4 * (d_qk // GROUP)
    o4 = o3 + SUB * 2 * (d_v // GROUP)
    nk, nv = d_qk // GROUP, d_v // GROUP
    k = _held_64(pages, d_qk, 0, 4, lambda t, g: (o2 + (t * 2 * nk + g) * 2, o2 + (t * 2 * nk + nk + g) * 2))
    v = _held_64(pages, d_v, o1, 8, lambda t, g: (o3 + (t * nv + g) * 2, o4 + (g * SUB + t) * 2))
    return k, v


def _round_64(x):
    """The values that x [..., d] (64 bits) is held as."""
    g = x.unflatten(-1, (-1, GROUP))
    low, high = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    near = low.float().bfloat16()
    under = torch.nextafter(near, torch.full_like(near, -math.inf))
    near = torch.where(near.double() > low, under, near).double()
    step = ((high - near) / 15).float().bfloat16().double()
    code = torch.where(step > 0, ((g - near) / step.clamp(min=1e-300)).round().clamp(0, 15), torch.zeros_like(g))
    return (near + step * code).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "append":
        rows = s["rows"].long()
        weights = s["weights"].double()
        weights[s["table"][s["seq"], s["slot"] // PAGE].long(), :, s["slot"] % PAGE] = s["w"].double()[:, rows].t()
        return {"k": _round_64(s["k"][rows].double()), "v": _round_64(s["v"][rows].double()), "weights": weights}
    if op == "attn":
        return _exact_attn(case, s)
    if op == "evict":
        return _exact_evict(case, s)
    hq, hkv, n = case["hq"], case["hkv"], case["tokens"]
    group = hq // hkv
    out = torch.zeros(hkv, n, dtype=torch.float64, device="cuda")
    some = max(1, (1 << 29) // n)
    for h in range(hq):
        keys = s["k"][:, h // group].double()
        for at in range(0, len(s["queries"]), some):
            i = s["queries"][at:at + some]
            p = torch.exp(s["q"][i, h].double() @ keys.t() / math.sqrt(case["d_qk"]) - s["lse"][h, i].double()[:, None])
            p[(s["seq"][i][:, None] != s["seq"]) | (s["pos"][i][:, None] < s["pos"])] = 0.0
            out[h // group] += p.sum(0)
    return out


def _exact_attn(case, s):
    hq, hkv, n_q = case["hq"], case["hkv"], case["n_q"]
    group = hq // hkv
    lengths = _lengths(case)
    o = torch.zeros(case["batch"], n_q, hq, case["d_v"], dtype=torch.float64, device="cuda")
    lse = torch.full((hq, case["batch"], n_q), -math.inf, dtype=torch.float64, device="cuda")
    weights = s["weights"].double()
    for b, n in enumerate(lengths):
        ids = s["table"][b, :-(-n // PAGE)].long()
        for h in range(hkv):
            k, v = (x.flatten(0, 1)[:n] for x in _kv_64(s["pages"][ids, h], case["d_qk"], case["d_v"]))
            for t in range(n_q):
                m = n - (n_q - 1 - t)
                if m <= 0:
                    continue
                x = s["q"][b, t, h * group:(h + 1) * group].double() @ k[:m].t() / math.sqrt(case["d_qk"])
                p = torch.softmax(x, -1)
                o[b, t, h * group:(h + 1) * group] = p @ v[:m]
                lse[h * group:(h + 1) * group, b, t] = torch.logsumexp(x, -1)
                at = torch.arange(m, device="cuda")
                weights[ids[at // PAGE], h, at % PAGE] += p.sum(0)
    got = {"o": o, "lse": lse.flatten(1)}
    return {**got, "weights": weights} if case["weights"] else got


def _exact_evict(case, s):
    budget, recent = case["budget"], case["recent"]
    lengths = _lengths(case)
    after = [min(n, budget) for n in lengths]
    kept = np.full((case["batch"], case["hkv"], budget), -1, np.int32)
    weights = s["to_weights"].double()
    ks, vs = [], []
    for b, n in enumerate(lengths):
        ids = s["table"][b, :-(-n // PAGE)].long()
        k, v = (x.transpose(1, 2).flatten(0, 1) for x in _kv_64(s["pages"][ids], case["d_qk"], case["d_v"]))
        w = s["weights"][ids].transpose(1, 2).flatten(0, 1)[:n].cpu().numpy()
        row = torch.arange(after[b], device="cuda")
        for h in range(case["hkv"]):
            old = max(0, n - recent)
            best = np.lexsort((np.arange(old), -w[:old, h].astype(np.float64)))[:after[b] - (n - old)]
            kept[b, h, :after[b]] = np.sort(np.concatenate([best, np.arange(old, n)]))
        slot = torch.from_numpy(kept[b, :, :after[b]].astype(np.int64)).cuda().t()
        head = torch.arange(case["hkv"], device="cuda")
        ks.append(k[slot, head])
        vs.append(v[slot, head])
        weights[s["to_table"][b, row // PAGE].long(), :, row % PAGE] = torch.from_numpy(w).cuda()[slot, head].double()
    return {"after": _ints(after), "kept": torch.from_numpy(kept), "k": torch.cat(ks), "v": torch.cat(vs), "weights": weights}
