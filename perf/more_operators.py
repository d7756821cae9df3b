"""Cases of the serving operators around a paged key/value cache in the model's own type: rotary positions, tokens into
the cache, attention of the newest tokens over it, and the sharing of its pages between sequences.

``run`` computes an operator in its plain form (elementary torch operations, fp32) where ``own`` is false, and makes
the package's call where it is true.  Both take the same state.

Cache.  k_pages [pages, hkv, page_size, d_qk], v_pages [pages, hkv, page_size, d_v]; token j of sequence b is row
j % page_size of page page_table[b][j / page_size].  refs[p] counts the sequences that hold page p; 0 is free.
"""

import math

import numpy as np
import torch

own = False


# ---------------------------------------------------------------- cases
def _rope(name, tokens, hq, hkv, d, first, dims, sections, pairing, dtype, inverse, far):
    return {"name": name, "op": "rope", "tokens": tokens, "hq": hq, "hkv": hkv, "d": d, "first": first, "dims": dims,
            "sections": sections, "pairing": pairing, "dtype": dtype, "inverse": inverse, "far": far}


def _append(name, batch, new, hkv, d_qk, d_v, dtype, page, cp, held, dims, lens_seed):
    return {"name": name, "op": "append", "batch": batch, "new": new, "hkv": hkv, "d_qk": d_qk, "d_v": d_v,
            "dtype": dtype, "page": page, "cp": cp, "held": held, "dims": dims, "lens_seed": lens_seed}


def _attn(name, batch, tokens, ragged, hq, hkv, d_qk, d_v, dtype, n_q, page, lens_seed):
    return {"name": name, "op": "attn", "batch": batch, "tokens": tokens, "ragged": ragged, "hq": hq, "hkv": hkv,
            "d_qk": d_qk, "d_v": d_v, "dtype": dtype, "n_q": n_q, "page": page, "lens_seed": lens_seed}


def _fork(name, groups, beams, prefix, layers, hkv, d, page, lens_seed):
    return {"name": name, "op": "fork", "groups": groups, "beams": beams, "prefix": prefix, "layers": layers,
            "hkv": hkv, "d": d, "page": page, "lens_seed": lens_seed}


def _compact(name, batch, tokens, layers, hkv, d, page, pages, lens_seed):
    return {"name": name, "op": "compact", "batch": batch, "tokens": tokens, "layers": layers, "hkv": hkv, "d": d,
            "page": page, "pages": pages, "lens_seed": lens_seed}


def listed():
    return [
        # queries and keys of one decoding step of 32 requests: launch latency counts
        _rope("rope step 32", 32, 32, 8, 128, 0, 128, "64", "halves", "bf16", False, 131072),
        # queries and keys of a 64K prompt
        _rope("rope prompt 64K", 65536, 32, 8, 128, 0, 128, "64", "halves", "bf16", False, 65536),
        # the gradient through the positions of a video's tokens (time, height, width), in training
        _rope("rope video gradient", 20011, 16, 4, 128, 0, 128, "16 24 24", "adjacent", "f32", True, 4096),
        # one decoding step's new tokens of 32 requests, keys rotated on the way
        _append("append 1 x 32", 32, 1, 8, 128, 128, "bf16", 64, 1, 4096, 128, 1),
        # a 64K prompt, straight out of its 8 zigzag shards
        _append("append prompt 64K", 1, 65536, 8, 128, 128, "bf16", 64, 8, 0, 128, 2),
        # one request in a short chat: the latency of a single decoding step
        _attn("attn 1 x 4K", 1, 4096, False, 32, 8, 128, 128, "bf16", 1, 64, 3),
        # sixteen requests of 1 to 32K tokens in one batch, in small pages
        _attn("attn 16 x ragged 32K", 16, 32768, True, 32, 8, 128, 128, "bf16", 1, 16, 4),
        # heads of their own keys (192 wide, values 128), 128K tokens
        _attn("attn mla 128K", 1, 131072, False, 64, 64, 192, 128, "bf16", 1, 64, 5),
        # four speculated tokens a request, checked in one pass, in fp32
        _attn("attn f32 spec 4", 5, 1999, True, 8, 4, 64, 64, "f32", 4, 64, 6),
        # a beam search's step of one request: 4 beams change parents and get room for a token, one layer's cache
        _fork("fork 1 x 4", 1, 4, 700, 1, 8, 128, 64, 7),
        # the same of 16 requests with 8 beams, 4 layers' caches in one page table
        _fork("fork 16 x 8", 16, 8, 1000, 4, 8, 128, 64, 8),
        # a pool whose requests have come and gone, packed to its front
        _compact("compact 768 pages", 24, 1500, 2, 8, 128, 64, 768, 9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "append", "attn", "attn", "attn", "fork", "compact"])
    lens_seed = rng.randrange(1 << 30)
    d_qk, d_v = rng.choice([(128, 128), (128, 128), (64, 64), (192, 128)])
    hkv = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 64, 128])
    if op == "rope":
        hq = hkv * rng.choice([1, 2, 4, 7])
        dims = rng.choice([d_qk, d_qk, 64, 32])
        axes = rng.choice([1, 1, 2, 3])
        cuts = sorted(rng.sample(range(1, dims // 2), axes - 1))
        case = _rope("", _log(rng, 1, 65536), hq, hkv, d_qk, rng.choice([0, d_qk - dims]), dims,
                     " ".join(str(b - a) for a, b in zip([0] + cuts, cuts + [dims // 2])), rng.choice(["halves", "adjacent"]),
                     rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.5, _log(rng, 64, 1000000))
    elif op == "append":
        batch = _log(rng, 1, 64)
        new = 1 if rng.random() < 0.4 else _log(rng, 2, max(2, 65536 // batch))
        case = _append("", batch, new, hkv, d_qk, d_v, rng.choice(["bf16", "bf16", "f32"]), page,
                       rng.choice([1, 2, 4]), rng.randrange(0, 3000), rng.choice([0, 64, d_qk]), lens_seed)
    elif op == "attn":
        batch = _log(rng, 1, 64)
        tokens = _log(rng, 1, max(16, min(131072, 4194304 // (batch * hkv))))
        case = _attn("", batch, tokens, rng.random() < 0.7, hkv * rng.choice([1, 2, 4, 7, 8]), hkv, d_qk, d_v,
                     rng.choice(["bf16", "bf16", "bf16", "f32"]), rng.choice([1, 1, 1, 2, 3, 4, 8]), page, lens_seed)
    elif op == "fork":
        case = _fork("", _log(rng, 1, 16), rng.choice([2, 3, 4, 8]), _log(rng, 10, 1000), rng.choice([1, 2, 4]), hkv,
                     rng.choice([64, 128]), page, lens_seed)
    else:
        tokens = _log(rng, 20, 1500)
        batch = _log(rng, 2, 24)
        case = _compact("", batch, tokens, rng.choice([1, 2]), hkv, rng.choice([64, 128]), page, 0, lens_seed)
        case["pages"] = int(sum(-(-n // page) for n in _spread(case)) * rng.uniform(1.05, 2.5)) + 3
    del case["name"]
    return case


def _sections(case):
    """Pairs of channels that turn with each axis' position."""
    return [int(x) for x in case["sections"].split()]


def _dtype(case):
    return torch.float32 if case.get("dtype") == "f32" else torch.bfloat16


def _elt(case):
    return 4 if case.get("dtype") == "f32" else 2


def _lengths(case):
    """Tokens that every sequence of an attention case holds."""
    n, b = case["tokens"], case["batch"]
    if not case["ragged"]:
        return [n] * b
    rs = np.random.RandomState(case["lens_seed"])
    got = [int(x) for x in np.exp(rs.uniform(0.0, math.log(max(n, 2)), b)).round().clip(1, n)]
    got[rs.randint(b)] = n
    return got


def _append_rows(case):
    """Tokens held before, and tokens that come, for every sequence."""
    rs = np.random.RandomState(case["lens_seed"])
    b, new = case["batch"], case["new"]
    start = [int(x) for x in rs.randint(0, case["held"] + 1, b)]
    counts = [new] * b if new == 1 or b == 1 else [int(x) for x in rs.randint(0, new + 1, b - 1)] + [new]
    return start, counts


def _beams(case):
    """Held tokens, shared tokens (whole pages of the group's prompt) and the parent of every beam of a fork case."""
    rs = np.random.RandomState(case["lens_seed"])
    lengths, shared, parents = [], [], []
    for g in range(case["groups"]):
        prompt = int(rs.randint(case["prefix"] // 2, case["prefix"] + 1))
        for _ in range(case["beams"]):
            lengths.append(prompt + int(rs.randint(1, 2 * case["page"])))
            shared.append(prompt // case["page"] * case["page"])
        order = g * case["beams"] + rs.randint(0, case["beams"], case["beams"])
        parents += [int(x) for x in order]
    if case["groups"] > 1:  # one request has ended: its beams let go of their pages
        at = int(rs.randint(case["groups"])) * case["beams"]
        parents[at:at + case["beams"]] = [-1] * case["beams"]
    return lengths, shared, parents


def _spread(case):
    """Tokens of every sequence of a compaction."""
    rs = np.random.RandomState(case["lens_seed"])
    return [int(x) for x in rs.randint(0, case["tokens"] + 1, case["batch"])]


def _zigzag_rows(lengths, cp):
    """Row of every token (sequences one after another) in the order of cp zigzag shards."""
    start, per_rank = 0, [[] for _ in range(cp)]
    for n in lengths:
        cut = [j * n // (2 * cp) for j in range(2 * cp + 1)]
        for r in range(cp):
            for c in (r, 2 * cp - 1 - r):
                per_rank[r].append(start + np.arange(cut[c], cut[c + 1]))
        start += n
    return np.argsort(np.concatenate([x for rank in per_rank for x in rank])) if start else np.zeros(0, np.int64)


# ---------------------------------------------------------------- states
def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cu(counts):
    return _ints(np.concatenate([[0], np.cumsum(counts)]).tolist())


def _table(gen, lengths, page, columns):
    """A pool's size and a table [B, columns] of its pages in no order; -1 where a sequence has none."""
    need = torch.tensor([-(-n // page) for n in lengths], device="cuda")
    total = int(need.sum()) + 3
    ids = torch.randperm(total, generator=gen, device="cuda")[:total - 3].to(torch.int32)
    table = torch.full((len(lengths), columns), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(columns, device="cuda") < need[:, None]] = ids
    return total, table


def _inv_freq(pairs):
    """Frequencies of the pairs of one axis, in 64 bits."""
    return 10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / max(pairs, 1))


def _random(gen, shape, dtype, scale=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype).mul_(scale)


def _layers(gen, case, pages):
    """K and V pages of every layer."""
    shape = (pages, case["hkv"], case["page"], case["d"])
    return [_random(gen, shape, torch.bfloat16) for _ in range(2 * case["layers"])]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = {"case": case}
    op = case["op"]
    if op == "rope":
        n, axes = case["tokens"], len(_sections(case))
        s["inv_freq"] = torch.cat([_inv_freq(m) for m in _sections(case)])
        s["axis"] = torch.repeat_interleave(torch.arange(axes), torch.tensor(_sections(case)))
        s["positions"] = torch.randint(0, case["far"], (n, axes), generator=gen, device="cuda", dtype=torch.int32)
        s["q"] = _random(gen, (n, case["hq"], case["d"]), _dtype(case))
        s["k"] = _random(gen, (n, case["hkv"], case["d"]), _dtype(case))
    elif op == "append":
        hkv, page = case["hkv"], case["page"]
        start, counts = _append_rows(case)
        after = [a + m for a, m in zip(start, counts)]
        total, s["table"] = _table(gen, after, page, max(-(-m // page) for m in after))
        n = sum(counts)
        s["k"] = _random(gen, (n, hkv, case["d_qk"]), _dtype(case))
        s["v"] = _random(gen, (n, hkv, case["d_v"]), _dtype(case))
        s["k_pages"] = torch.zeros(total, hkv, page, case["d_qk"], dtype=_dtype(case), device="cuda")
        s["v_pages"] = torch.zeros(total, hkv, page, case["d_v"], dtype=_dtype(case), device="cuda")
        s["cu"], s["start"] = _cu(counts), _ints(start)
        s["rows"] = _ints(_zigzag_rows(counts, case["cp"]).tolist())  # the sharded row of every token
        s["inv_freq"] = _inv_freq(case["dims"] // 2)
        s["seq"] = torch.repeat_interleave(torch.arange(len(counts), device="cuda"), torch.tensor(counts, device="cuda"))
        s["slot"] = torch.cat([torch.arange(a, b, device="cuda") for a, b in zip(start, after)])
        # positions go with the rows of k: a token's slot, at the row that the token is in
        s["positions"] = torch.zeros(n, 1, dtype=torch.int32, device="cuda")
        s["positions"][s["rows"].long(), 0] = s["slot"].to(torch.int32)
    elif op == "attn":
        lengths, page = _lengths(case), case["page"]
        total, s["table"] = _table(gen, lengths, page, -(-max(lengths) // page))
        # keys as projections give them: some channels with an offset and a spread of their own
        spread = torch.exp(0.5 * torch.randn(case["d_qk"], generator=gen, device="cuda"))
        offset = torch.randn(case["d_qk"], generator=gen, device="cuda")
        k = _random(gen, (total, case["hkv"], page, case["d_qk"]), _dtype(case))
        s["k_pages"] = k.mul_(spread.to(k.dtype)).add_(offset.to(k.dtype))
        s["v_pages"] = _random(gen, (total, case["hkv"], page, case["d_v"]), _dtype(case))
        s["q"] = _random(gen, (case["batch"], case["n_q"], case["hq"], case["d_qk"]), _dtype(case))
        s["lengths"] = _ints(lengths)
    elif op == "fork":
        lengths, shared, parents = _beams(case)
        page = case["page"]
        columns = max(-(-n // page) for n in lengths) + 1
        rows, pages = np.full((len(lengths), columns), -1), 0
        for b, (n, m) in enumerate(zip(lengths, shared)):
            held, common = -(-n // page), m // page
            if b % case["beams"] == 0:
                prompt, pages = np.arange(pages, pages + common), pages + common
            rows[b, :common] = prompt
            rows[b, common:held], pages = np.arange(pages, pages + held - common), pages + held - common
        total = pages + 2 * len(lengths)
        at = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
        table = torch.from_numpy(rows).cuda()
        s["table"] = torch.where(table < 0, -1, at[table.clamp(min=0)]).to(torch.int32)
        s["refs"] = torch.bincount(s["table"][s["table"] >= 0].long(), minlength=total).to(torch.int32)
        s["lengths"], s["parents"] = _ints(lengths), _ints(parents)
        s["extra"] = _ints([int(p >= 0) for p in parents])
        s["layers"] = _layers(gen, case, total)
    else:
        lengths = _spread(case)
        page = case["page"]
        _, table = _table(gen, lengths, page, max(1, max(-(-n // page) for n in lengths)))
        at = torch.randperm(case["pages"], generator=gen, device="cuda").to(torch.int32)
        s["table"] = torch.where(table < 0, -1, at[table.clamp(min=0).long()]).to(torch.int32)
        s["refs"] = torch.bincount(s["table"][s["table"] >= 0].long(), minlength=case["pages"]).to(torch.int32)
        s["lengths"] = _ints(lengths)
        s["layers"] = _layers(gen, case, case["pages"])
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    return {"rope": _run_rope, "append": _run_append, "attn": _run_attn, "fork": _run_fork,
            "compact": _run_compact}[s["case"]["op"]](s)


def _package(s, make):
    """The package and its handle of a state's tensors, which a program keeps."""
    if "handle" not in s:
        import context_long_sequence_zigzag_gb300 as cpa

        s["package"], s["handle"] = cpa, make(cpa)
    return s["package"], s["handle"]


def _rotated(x, turn, first, pairing, inverse):
    """x [rows, heads, d] with the pairs of its channels from `first` on turned by turn [rows, pairs] (64 bits), in fp32."""
    m = turn.shape[-1]
    cos, sin = torch.cos(turn).float()[:, None], torch.sin(turn).float()[:, None]
    if inverse:
        sin = -sin
    part = x[..., first:first + 2 * m].float()
    a, b = (part[..., :m], part[..., m:]) if pairing == "halves" else (part[..., 0::2], part[..., 1::2])
    u, v = a * cos - b * sin, b * cos + a * sin
    part = torch.cat([u, v], -1) if pairing == "halves" else torch.stack([u, v], -1).flatten(-2)
    return torch.cat([x[..., :first], part.to(x.dtype), x[..., first + 2 * m:]], -1)


def _run_rope(s):
    """Queries and keys turned by their tokens' positions (or gradients turned back)."""
    case = s["case"]
    if own:
        cpa, rope = _package(s, lambda cpa: cpa.Rope(s["inv_freq"], axis=s["axis"], first=case["first"],
                                                     pairing=case["pairing"]))
        q, k = cpa.cp_rope(rope, s["positions"], s["q"], s["k"], inverse=case["inverse"])
        return {"q": q, "k": k}
    turn = s["positions"][:, s["axis"].cuda()].double() * s["inv_freq"].cuda()
    q = _rotated(s["q"], turn, case["first"], case["pairing"], case["inverse"])
    return {"q": q, "k": _rotated(s["k"], turn, case["first"], case["pairing"], case["inverse"])}


def _run_append(s):
    """New tokens into the pages, their keys turned by their positions."""
    case = s["case"]
    if own:
        cpa, (cache, rope) = _package(s, lambda cpa: (
            cpa.KvCache(s["k_pages"], s["v_pages"], s["table"], case["hkv"]),
            cpa.Rope(s["inv_freq"]) if case["dims"] else None))
        cpa.cp_kv_append(cache, s["k"], s["v"], s["cu"], s["start"], rows=s["rows"], rope=rope,
                         positions=s["positions"] if case["dims"] else None)
        return {"k": s["k_pages"], "v": s["v_pages"]}
    turn = s["positions"].double() * s["inv_freq"].cuda()
    rows, page = s["rows"].long(), s["table"][s["seq"], s["slot"] // case["page"]].long()
    k = _rotated(s["k"], turn, 0, "halves", False) if case["dims"] else s["k"]
    s["k_pages"][page, :, s["slot"] % case["page"]] = k[rows]
    s["v_pages"][page, :, s["slot"] % case["page"]] = s["v"][rows]
    return {"k": s["k_pages"], "v": s["v_pages"]}


def _run_attn(s):
    """One decoding step: the newest n_q queries of every sequence against the tokens it holds."""
    case = s["case"]
    if own:
        cpa, cache = _package(s, lambda cpa: cpa.KvCache(s["k_pages"], s["v_pages"], s["table"], case["hq"]))
        o, lse = cpa.cp_kv_attn(cache, s["q"], s["lengths"])
        return {"o": o, "lse": lse}
    hkv, n_q, b = case["hkv"], case["n_q"], case["batch"]
    g = case["hq"] // hkv
    table = s["table"].clamp(min=0).long()
    k = s["k_pages"][table].transpose(1, 2).flatten(2, 3).float()  # [B, hkv, slots, d]
    q = s["q"].float().unflatten(2, (hkv, g)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [B, hkv, n_q * g, d]
    x = (q * case["d_qk"] ** -0.5) @ k.transpose(-1, -2)
    del k
    at = torch.arange(x.shape[-1], device="cuda")
    behind = (n_q - 1 - torch.arange(n_q, device="cuda")).repeat_interleave(g)
    seen = (at < (s["lengths"][:, None, None] - behind[:, None]))[:, None]
    x = torch.where(seen, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    held = (at < s["lengths"][:, None])[:, None, :, None]
    v = s["v_pages"][table].transpose(1, 2).flatten(2, 3).float()
    o = p @ torch.where(held, v, torch.zeros_like(v))
    o = o.unflatten(2, (n_q, g)).permute(0, 2, 1, 3, 4).flatten(2, 3).to(_dtype(case))
    lse = (top + torch.log(total)).squeeze(-1).unflatten(2, (n_q, g)).permute(1, 3, 0, 2).reshape(case["hq"], b * n_q)
    return {"o": o, "lse": lse}


def _run_fork(s):
    """A step of a beam search: beams go on from their parents, with pages of their own to write and room for a token."""
    case = s["case"]
    page = case["page"]
    if own:
        cpa, (pool, refs) = _package(s, lambda cpa: (lambda r: (cpa.PagePool(r, s["layers"], page), r))(s["refs"].clone()))
        refs.copy_(s["refs"])
        table, lengths, counts = cpa.cp_pages_fork(pool, s["table"], s["lengths"], s["parents"])
        more = cpa.cp_pages_reserve(pool, table, lengths, s["extra"])
        return {"table": table, "lengths": lengths, "refs": refs, "counts": torch.stack([counts, more]),
                "layers": s["layers"]}
    pages = s["refs"].shape[0]
    from_row, alive = s["parents"].clamp(min=0).long(), s["parents"] >= 0
    lengths = torch.where(alive, s["lengths"][from_row], 0)
    at = torch.arange(s["table"].shape[1], device="cuda")
    table = torch.where(at < ((lengths + page - 1) // page)[:, None], s["table"][from_row], -1)
    # what the old sequences let go of, and the whole pages that the new ones hold
    count = lambda t: torch.zeros(pages, dtype=torch.int32, device="cuda").index_add_(  # noqa: E731
        0, t.clamp(min=0).flatten().long(), (t >= 0).flatten().to(torch.int32))
    refs = s["refs"] - count(s["table"]) + count(torch.where(at < (lengths // page)[:, None], table, -1))
    # the first to hold a page in part keeps it if nobody else does, the others take free ones
    last = (lengths // page).long()
    part = torch.where(lengths % page > 0, table.gather(1, last[:, None])[:, 0], -1)
    row = torch.arange(len(part), device="cuda")
    earlier = ((part[:, None] == part) & (row < row[:, None])).any(1)
    keep = (part >= 0) & ~earlier & (refs[part.clamp(min=0).long()] == 0)
    refs.index_add_(0, part.clamp(min=0).long(), keep.to(torch.int32))
    wants = (part >= 0) & ~keep
    took, unmet = _take(refs, wants)
    table[row, last] = torch.where(wants, took, table.gather(1, last[:, None])[:, 0])
    counts = torch.stack([(refs > 0).sum(), unmet]).to(torch.int32)
    src, dst = part[wants].long(), took[wants].long()
    _copied(s["layers"], src, dst)
    # room for what comes
    new = -(-(lengths + s["extra"]) // page)
    held = -(-lengths // page)
    wants = (at >= held[:, None]) & (at < new[:, None])
    took, unmet = _take(refs, wants.flatten())
    table = torch.where(wants, took.view(wants.shape), table)
    more = torch.stack([(refs > 0).sum(), unmet]).to(torch.int32)
    return {"table": table, "lengths": lengths, "refs": refs, "counts": torch.stack([counts, more]), "layers": s["layers"]}


def _take(refs, wants):
    """The lowest free pages for the wants in their order (-1: none left), counted in refs; how many got none."""
    free = torch.nonzero(refs == 0)[:, 0]
    rank = torch.cumsum(wants, 0) - 1
    got = wants & (rank < len(free))
    page = torch.nn.functional.pad(free, (0, 1), value=-1)[torch.where(got, rank, len(free))]
    refs.index_add_(0, page.clamp(min=0), got.to(torch.int32))
    return page.to(torch.int32), (wants & ~got).sum()


def _copied(layers, src, dst):
    for x in layers:
        x[dst] = x[src]


def _run_compact(s):
    """The held pages moved to the front of the pool."""
    case = s["case"]
    if own:
        cpa, (pool, refs) = _package(s, lambda cpa: (lambda r: (cpa.PagePool(r, s["layers"], case["page"]), r))(s["refs"].clone()))
        refs.copy_(s["refs"])
        table, moved, counts = cpa.cp_pages_compact(pool, s["table"], s["lengths"])
        return {"table": table, "moved": moved, "refs": refs, "counts": counts, "layers": s["layers"]}
    pages = case["pages"]
    used = s["refs"] > 0
    n = used.sum()
    at = torch.arange(pages, device="cuda")
    src, dst = torch.nonzero(used & (at >= n))[:, 0], torch.nonzero(~used & (at < n))[:, 0]
    moved = torch.where(used, at, -1)
    moved[src] = dst
    refs = torch.where(at < n, s["refs"], 0)
    refs[dst] = s["refs"][src]
    _copied(s["layers"], src, dst)
    held = torch.arange(s["table"].shape[1], device="cuda") < (-(-s["lengths"] // case["page"]))[:, None]
    table = torch.where(held, moved[s["table"].clamp(min=0).long()], -1).to(torch.int32)
    counts = torch.stack([n, torch.zeros_like(n)]).to(torch.int32)
    return {"table": table, "moved": moved.to(torch.int32), "refs": refs, "counts": counts, "layers": s["layers"]}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "rope":
        heads = case["hq"] + case["hkv"]
        return {"bytes": case["tokens"] * (2.0 * _elt(case) * heads * case["d"] + 4 * len(_sections(case))),
                "flops": 3.0 * case["tokens"] * heads * case["dims"]}
    if op == "append":
        tokens = sum(_append_rows(case)[1])
        return {"bytes": tokens * (2.0 * _elt(case) * case["hkv"] * (case["d_qk"] + case["d_v"]) + 8),
                "flops": 3.0 * tokens * case["hkv"] * case["dims"]}
    if op == "attn":
        tokens, wide = sum(_lengths(case)), case["d_qk"] + case["d_v"]
        rows = case["batch"] * case["n_q"] * case["hq"]
        return {"bytes": _elt(case) * (float(tokens) * case["hkv"] * wide + rows * wide) + 4.0 * rows,
                "flops": 2.0 * tokens * case["n_q"] * case["hq"] * wide}
    size = 4.0 * case["layers"] * case["hkv"] * case["page"] * case["d"]  # K and V of a page in all layers
    if op == "fork":
        lengths, _, parents = _beams(case)
        part = [p for p in parents if p >= 0 and lengths[p] % case["page"]]
        table = sum(-(-n // case["page"]) for n in lengths)
        return {"bytes": 2.0 * size * (len(part) - len(set(part))) + 8.0 * table, "flops": 0.0}
    used = sum(-(-n // case["page"]) for n in _spread(case))
    return {"bytes": 2.0 * size * used * (case["pages"] - used) / case["pages"] + 8.0 * case["pages"], "flops": 0.0}


# ---------------------------------------------------------------- from the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        sign = -1.0 if case["inverse"] else 1.0
        angle = sign * torch.stack([s["positions"][:, a].double() * f for a, f in zip(s["axis"].tolist(), s["inv_freq"].tolist())], 1)
        return {x: _turned_64(s[x], angle, case["first"], case["pairing"]) for x in ("q", "k")}
    if op == "append":
        return _exact_append(case, s)
    if op == "attn":
        return _exact_attn(case, s)
    return _exact_fork(case, s) if op == "fork" else _exact_compact(case, s)


def _turned_64(x, angle, first, pairing):
    """Every pair of channels as a complex number, times exp(i angle)."""
    m = angle.shape[1]
    out = x.double()
    i = torch.arange(m, device="cuda")
    re, im = (first + i, first + m + i) if pairing == "halves" else (first + 2 * i, first + 2 * i + 1)
    z = torch.complex(out[..., re], out[..., im]) * torch.polar(torch.ones_like(angle), angle)[:, None]
    out[..., re], out[..., im] = z.real, z.imag
    return out


def _exact_append(case, s):
    start, counts = _append_rows(case)
    page = case["page"]
    slot = np.concatenate([np.arange(a, a + n) for a, n in zip(start, counts)])
    seq = np.repeat(np.arange(len(counts)), counts)
    row = s["rows"].long()
    k = s["k"][row]
    if case["dims"]:
        k = _turned_64(k, torch.from_numpy(slot).cuda().double()[:, None] * s["inv_freq"].cuda(), 0, "halves")
    flat = torch.from_numpy(s["table"].cpu().numpy()[seq, slot // page].astype(np.int64)).cuda()
    at = torch.from_numpy(slot % page).cuda()
    kp, vp = s["k_pages"].double(), s["v_pages"].double()
    kp[flat, :, at], vp[flat, :, at] = k.double(), s["v"][row].double()
    return {"k": kp, "v": vp}


def _exact_attn(case, s):
    hq, hkv, n_q, page = case["hq"], case["hkv"], case["n_q"], case["page"]
    group = hq // hkv
    o = torch.zeros(case["batch"], n_q, hq, case["d_v"], dtype=torch.float64, device="cuda")
    lse = torch.full((hq, case["batch"], n_q), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lengths(case)):
        ids = s["table"][b, :-(-n // page)].long()
        for h in range(hkv):
            k, v = (s[x][ids, h].flatten(0, 1)[:n].double() for x in ("k_pages", "v_pages"))
            heads = slice(h * group, (h + 1) * group)
            for t in range(n_q):
                m = n - (n_q - 1 - t)
                if m > 0:
                    x = s["q"][b, t, heads].double() @ k[:m].t() / math.sqrt(case["d_qk"])
                    lse[heads, b, t] = torch.logsumexp(x, -1)
                    o[b, t, heads] = torch.exp(x - lse[heads, b, t][:, None]) @ v[:m]
    return {"o": o, "lse": lse.flatten(1)}


def _lists(s, page):
    """Pages of every sequence, and every page's count without this batch."""
    lengths, table, refs = s["lengths"].tolist(), s["table"].tolist(), s["refs"].tolist()
    return lengths, [table[b][:-(-n // page)] for b, n in enumerate(lengths)], refs


def _rows(lists, columns):
    return _ints([x + [-1] * (columns - len(x)) for x in lists]).view(len(lists), columns)


def _exact_fork(case, s):
    page = case["page"]
    held, lists, refs = _lists(s, page)
    parents, extra = s["parents"].tolist(), s["extra"].tolist()
    for x in lists:
        for p in x:
            refs[p] -= 1
    new = [list(lists[p]) if p >= 0 else [] for p in parents]
    lengths = [held[p] if p >= 0 else 0 for p in parents]
    for b, x in enumerate(new):
        for p in x[:lengths[b] // page]:
            refs[p] += 1
    kept = set()
    for b, x in enumerate(new):  # (those that keep theirs first, so that no page in use counts as free)
        if lengths[b] % page and refs[x[-1]] == 0:
            kept.add(b)
            refs[x[-1]] = 1
    layers = [x.clone() for x in s["layers"]]
    counts, unmet = [], 0
    for b, x in enumerate(new):
        if lengths[b] % page and b not in kept:
            p = refs.index(0) if 0 in refs else -1
            unmet += p < 0
            if p >= 0:
                refs[p] = 1
                for y in layers:
                    y[p] = y[x[-1]]
            x[-1] = p
    counts.append([sum(r > 0 for r in refs), unmet])
    unmet = 0
    for b, x in enumerate(new):
        for _ in range(-(-lengths[b] // page), -(-(lengths[b] + extra[b]) // page)):
            p = refs.index(0) if 0 in refs else -1
            unmet += p < 0
            if p >= 0:
                refs[p] = 1
            x.append(p)
    counts.append([sum(r > 0 for r in refs), unmet])
    return {"table": _rows(new, s["table"].shape[1]), "lengths": _ints(lengths), "refs": _ints(refs),
            "counts": _ints(counts), "layers": [y.double() for y in layers]}


def _exact_compact(case, s):
    _, lists, refs = _lists(s, case["page"])
    used = sum(r > 0 for r in refs)
    goes = {p: p for p in range(used) if refs[p]}
    layers = [x.clone() for x in s["layers"]]
    holes = iter([p for p in range(used) if not refs[p]])
    for p in range(used, case["pages"]):
        if refs[p]:
            goes[p] = next(holes)
            refs[goes[p]], refs[p] = refs[p], 0
            for y in layers:
                y[goes[p]] = y[p]
    return {"table": _rows([[goes[p] for p in x] for x in lists], s["table"].shape[1]),
            "moved": _ints([goes.get(p, -1) for p in range(case["pages"])]), "refs": _ints(refs),
            "counts": _ints([used, 0]), "layers": [y.double() for y in layers]}
