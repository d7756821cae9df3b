"""The 4-bit key/value cache: its format, attention over it, eviction by
accumulated attention weight, and a prompt's key weights (oracle; test
infrastructure; the format is the one ``include/cp_attn.h`` describes).

The source pages stop at training; decoding over a cache takes the
conventions of their attention: a query's softmax runs over the slots it
sees, o = 0 and lse = -inf where it sees none.
"""

from __future__ import annotations

import math

import numpy as np

PAGE, SUB, GROUP = 64, 32, 64


def bf16_bits(x):
    """Nearest-even bf16 bit patterns of float32 values."""
    u = np.asarray(x, np.float32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def bf16_values(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def bf16_floor(x):
    """Largest bf16 not above x (finite, in bf16's range)."""
    x = np.asarray(x, np.float64)
    near = bf16_bits(x)
    v = bf16_values(near)
    down = np.where(v > 0, near - 1, np.where((near & 0x7FFF) == 0, 0x8001, near + 1)).astype(np.uint16)
    return bf16_values(np.where(v > x, down, near))


def kv4_codes(x, low, scale):
    """Codes of x [..., d] for the given lows and scales [..., d / 64] (float64)."""
    g = np.asarray(x, np.float64).reshape(x.shape[:-1] + (-1, GROUP))
    s = np.where(scale > 0, scale, 1.0)[..., None]
    n = np.clip(np.rint((g - low[..., None]) / s), 0, 15)
    return np.where(scale[..., None] > 0, n, 0).reshape(x.shape).astype(np.uint8)


def kv4_quantise(x):
    """(codes [..., d], lows, scales [..., d / 64]) of x [..., d]."""
    g = np.asarray(x, np.float64).reshape(x.shape[:-1] + (-1, GROUP))
    low = bf16_floor(g.min(-1))
    scale = bf16_values(bf16_bits((g.max(-1) - low) / 15.0))
    return kv4_codes(x, low, scale), low, scale


def kv4_values(codes, low, scale):
    g = codes.reshape(low.shape + (GROUP,)).astype(np.float64)
    return (g * scale[..., None] + low[..., None]).reshape(codes.shape)


def _word_position(w, lanes, d):
    return (w % lanes) * (d // (8 * lanes)) + w // lanes


def _offsets(d_qk, d_v):
    nk, nv = d_qk // GROUP, d_v // GROUP
    at = np.cumsum([0, SUB * d_qk // 2, SUB * d_v // 2, SUB * nk * 4, SUB * nv * 2, SUB * nv * 2])
    return [int(a) for a in at]


def kv4_block_bytes(d_qk, d_v):
    return 2 * _offsets(d_qk, d_v)[-1]


def kv4_pack(k, v):
    """Block bytes [..., bytes] of pages' heads from (codes [..., 64, d], lows, scales [..., 64, d / 64]) of k and of v."""
    (kc, kl, ks), (vc, vl, vs) = k, v
    d_qk, d_v = kc.shape[-1], vc.shape[-1]
    o = _offsets(d_qk, d_v)
    lead = kc.shape[:-2]
    out = np.zeros(lead + (2, o[-1]), np.uint8)

    def rows(codes, d, lanes):
        b = np.zeros(lead + (2, SUB, d // 8, 4), np.uint8)
        pairs = codes.reshape(lead + (2, SUB, d // 8, 4, 2)).astype(np.uint8)
        for w in range(d // 8):
            b[..., _word_position(w, lanes, d), :] = pairs[..., w, :, 0] | (pairs[..., w, :, 1] << 4)
        return b.reshape(lead + (2, -1))

    def halves(x):  # x [..., 2, n]
        return np.ascontiguousarray(bf16_bits(x.astype(np.float32))).view(np.uint8)

    split = lambda x: x.reshape(lead + (2, SUB, -1))  # noqa: E731
    out[..., o[0]:o[1]] = rows(kc, d_qk, 4)
    out[..., o[1]:o[2]] = rows(vc, d_v, 8)
    out[..., o[2]:o[3]] = halves(np.stack([split(ks), split(kl)], -2).reshape(lead + (2, -1)))
    out[..., o[3]:o[4]] = halves(split(vs).reshape(lead + (2, -1)))
    out[..., o[4]:o[5]] = halves(np.swapaxes(split(vl), -1, -2).reshape(lead + (2, -1)))
    return out.reshape(lead + (-1,))


def kv4_unpack(block, d_qk, d_v):
    """((codes, lows, scales) of k, the same of v) of a page's head block, 64 rows each."""
    o = _offsets(d_qk, d_v)
    subs = np.asarray(block, np.uint8).reshape(2, o[-1])
    got = []
    for off, d, lanes in ((o[0], d_qk, 4), (o[1], d_v, 8)):
        b = subs[:, off:off + SUB * d // 2].reshape(2 * SUB, d // 8, 4)
        b = b[:, [_word_position(w, lanes, d) for w in range(d // 8)]]
        codes = np.stack([b & 15, b >> 4], -1).reshape(2 * SUB, d)
        if lanes == 4:
            p = subs[:, o[2]:o[3]].copy().view(np.uint16).reshape(2 * SUB, 2, d // GROUP)
            scale, low = bf16_values(p[:, 0]), bf16_values(p[:, 1])
        else:
            scale = bf16_values(subs[:, o[3]:o[4]].copy().view(np.uint16).reshape(2 * SUB, d // GROUP))
            low = bf16_values(subs[:, o[4]:o[5]].copy().view(np.uint16).reshape(2, d // GROUP, SUB).transpose(0, 2, 1)
                              .reshape(2 * SUB, d // GROUP))
        got.append((codes, low, scale))
    return got


def kv4_attention(q, k, v, n, scale, kv_of):
    """One sequence: q [n_q, hq, d], k [slots, hkv, d_qk], v [slots, hkv, d_v], n slots held, the queries' own the last.

    Returns o [n_q, hq, d_v], lse [hq, n_q] and the slots' weights [slots, hkv]."""
    n_q, hq, _ = q.shape
    o, lse = np.zeros((n_q, hq, v.shape[2])), np.full((hq, n_q), -np.inf)
    w = np.zeros(k.shape[:2])
    for t in range(n_q):
        m = n - (n_q - 1 - t)
        if m <= 0:
            continue
        for h in range(hq):
            c = kv_of(h)
            s = scale * (k[:m, c] @ q[t, h])
            top = s.max()
            e = np.exp(s - top)
            lse[h, t] = top + math.log(e.sum())
            p = e / e.sum()
            o[t, h] = p @ v[:m, c]
            w[:m, c] += p
    return o, lse, w


def kv4_keep(w, n, budget, recent):
    """Slots kept of n with weights w [n]: the last `recent`, and of the others the heaviest (ties: the lowest slot)."""
    if n <= budget:
        return list(range(n))
    old = n - recent
    order = sorted(range(old), key=lambda j: (0 if math.isnan(w[j]) else 1, 0.0 if math.isnan(w[j]) else -w[j], j))
    return sorted(order[:budget - recent]) + list(range(old, n))


def attn_key_weights(q, k, lse, cu_seqlens, scale, causal=True, last=None, gqa_interleaved=False):
    """w [hkv, T]: attention probabilities summed over queries and heads; global order, from the given lse [hq, T]."""
    T, hq, _ = q.shape
    hkv = k.shape[1]
    w = np.zeros((hkv, T))
    for s in range(len(cu_seqlens) - 1):
        a, b = int(cu_seqlens[s]), int(cu_seqlens[s + 1])
        first = a if last is None else max(a, b - last)
        for h in range(hq):
            c = h % hkv if gqa_interleaved else h // (hq // hkv)
            x = np.exp(scale * (q[first:b, h] @ k[a:b, c].T) - lse[h, first:b, None])
            if causal:
                x[np.arange(first, b)[:, None] < np.arange(a, b)] = 0.0
            w[c, a:b] += x.sum(0)
    return w
