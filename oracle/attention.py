"""Float64 definitions of the attention operators next to the indexer.

Plain loops and full sorts on the CPU, sharing no code with the GPU path:
causal attention of packed sequences, the 4-bit (microscaling FP4) cache
format, attention over cached keys, accumulated weights, eviction.
"""
from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


# ----------------------------------------------------------------------------
# attention
# ----------------------------------------------------------------------------
def attend(q, k, v, scale, visible):
    """One query head: q [d], k, v [n, d], visible [n] bool (or counts).  Returns the output, lse, the
    weights [n], sum_j w_j |v_j| and the largest scale * sum_e |q_e k_je| (what error bounds need)."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    w = np.zeros(k.shape[0])
    count = np.asarray(visible, np.float64)
    on = count > 0
    if not on.any():
        return np.zeros(v.shape[1]), -np.inf, w, np.zeros(v.shape[1]), 0.0
    s = (k[on] @ q) * scale
    top = s.max()
    e = np.exp(s - top) * count[on]
    w[on] = e / e.sum()
    size = float((np.abs(k[on]) @ np.abs(q)).max() * scale)
    return w @ v, top + np.log(e.sum()), w, w @ np.abs(v), size


def prompt(q, k, v, q_lens, kv_lens, scale):
    """Causal attention of packed sequences; (out, lse, abs_out, size) per query row and head."""
    nq, H, d = q.shape
    g = H // k.shape[1]
    out, ab = np.zeros((nq, H, d)), np.zeros((nq, H, d))
    lse, size = np.full((nq, H), -np.inf), np.zeros((nq, H))
    q0 = k0 = 0
    for ql, kl in zip(q_lens, kv_lens):
        for i in range(ql):
            see = np.arange(kl) <= kl - ql + i
            for h in range(H):
                o, l, _, a, z = attend(q[q0 + i, h], k[k0:k0 + kl, h // g], v[k0:k0 + kl, h // g], scale, see)
                out[q0 + i, h], lse[q0 + i, h], ab[q0 + i, h], size[q0 + i, h] = o, l, a, z
        q0 += ql
        k0 += kl
    return out, lse, ab, size


# ----------------------------------------------------------------------------
# 4-bit rows
# ----------------------------------------------------------------------------
def mx_encode(x):
    """Rows [..., d] (d a multiple of 32) -> (codes [..., d/2], scales [..., d/32]) uint8."""
    x = np.asarray(x, np.float64)
    y = x.reshape(*x.shape[:-1], -1, 32)
    amax = np.abs(y).max(-1)
    e = np.full(amax.shape, 1)
    for cand in range(254, 0, -1):          # smallest e in 1..254 with amax < 7 * 2^(e-127)
        e = np.where(amax < np.ldexp(7.0, cand - 127), cand, e)
    e = np.where(amax >= np.ldexp(7.0, 254 - 127), 254, e)
    a = np.abs(y) / np.ldexp(1.0, e - 127)[..., None]
    dist = np.abs(a[..., None] - GRID)
    best = dist.min(-1, keepdims=True)
    near = dist == best
    # nearest code; of two equally near ones the even
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(near.sum(-1) > 1, even.argmax(-1), near.argmax(-1)).astype(np.uint8)
    code = code | (np.signbit(y).astype(np.uint8) << 3)
    code = code.reshape(*x.shape[:-1], -1, 2)
    return code[..., 0] | (code[..., 1] << 4), e.astype(np.uint8)


def mx_decode(codes, scales):
    """(codes [..., d/2], scales [..., d/32]) -> rows [..., d]."""
    nib = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1)
    val = np.where(nib & 8, -GRID[nib & 7], GRID[nib & 7])
    return val * np.repeat(np.ldexp(1.0, scales.astype(np.int64) - 127), 32, -1)


# ----------------------------------------------------------------------------
# the paged cache
# ----------------------------------------------------------------------------
def slots(table, b, n, page, num_pages):
    """Pool slot of positions 0..n-1 of sequence b, -1 where the table names no page."""
    p = np.arange(n)
    pg = table[b][p // page].astype(np.int64)
    return np.where((pg >= 0) & (pg < num_pages), pg * page + p % page, -1)


def cached_rows(codes, scales, at):
    """Rows [n, Hkv, d] of pool slots (zeros for -1)."""
    c = codes.reshape(-1, *codes.shape[2:])[np.maximum(at, 0)]
    s = scales.reshape(-1, *scales.shape[2:])[np.maximum(at, 0)]
    s = np.where((at < 0)[:, None, None], 1, s).astype(np.uint8)
    return mx_decode(np.where((at < 0)[:, None, None], 0, c).astype(np.uint8), s)


def cache_attention(q, cache, q_lens, kv_lens, scale, idx=None):
    """cache: dict k_codes, k_scales, v_codes, v_scales, table.  (out, lse, abs_out, size, weights):
    weights is a list of [kv, H, q_len] per sequence."""
    nq, H, d = q.shape
    pages, page, hk, _ = cache["k_codes"].shape
    g = H // hk
    out, ab = np.zeros((nq, H, d)), np.zeros((nq, H, d))
    lse, size = np.full((nq, H), -np.inf), np.zeros((nq, H))
    weights, row = [], 0
    for b, (ql, kl) in enumerate(zip(q_lens, kv_lens)):
        at = slots(cache["table"], b, kl, page, pages)
        k = cached_rows(cache["k_codes"], cache["k_scales"], at)
        v = cached_rows(cache["v_codes"], cache["v_scales"], at)
        W = np.zeros((kl, H, ql))
        for i in range(ql):
            see = ((np.arange(kl) <= kl - ql + i) & (at >= 0)).astype(np.float64)
            if idx is not None:
                times = np.zeros(kl)
                for p in idx[row + i]:
                    if 0 <= p < kl:
                        times[p] += 1
                see = see * times
            for h in range(H):
                o, l, w, a, z = attend(q[row + i, h], k[:, h // g], v[:, h // g], scale, see)
                out[row + i, h], lse[row + i, h], ab[row + i, h], size[row + i, h] = o, l, a, z
                W[:, h, i] = w
        weights.append(W)
        row += ql
    return out, lse, ab, size, weights


def accumulate(cache, weights, q_lens, kv_lens, acc, acc_out):
    """acc_out (a copy is returned) after adding every key's weights."""
    pages, page = cache["k_codes"].shape[:2]
    res = np.array(acc_out, np.float64).reshape(-1)
    old = None if acc is None else np.asarray(acc, np.float64).reshape(-1)
    for b, (ql, kl) in enumerate(zip(q_lens, kv_lens)):
        if ql == 0:
            continue
        at = slots(cache["table"], b, kl, page, pages)
        for j in range(kl):
            if at[j] >= 0:
                res[at[j]] = (old[at[j]] if old is not None and j < kl - ql else 0.0) + weights[b][j].sum()
    return res.reshape(pages, page)


# ----------------------------------------------------------------------------
# eviction
# ----------------------------------------------------------------------------
def evict(acc, kv_len, new_len, prefix, window, pos=None, seen=None, there=None):
    """Source index of each kept key 0..new_len-1.  acc, pos: values by key index; there: whether the key
    has a page (None: all have).  An index in front of the new end without a page stays as it is, so that
    no key moves to it; such keys behind it go first."""
    place = np.arange(kv_len) if pos is None else np.asarray(pos[:kv_len])
    seen = kv_len if seen is None else seen
    there = np.ones(kv_len, bool) if there is None else np.asarray(there)
    safe = np.where(there, (place < prefix) | (place >= seen - window), np.arange(kv_len) < new_len)
    order = sorted(range(kv_len), key=lambda j: (0 if safe[j] else 1 if there[j] else 2,
                                                 -float(acc[j]) if there[j] and not safe[j] else 0.0, j))
    kept = set(order[:new_len])
    movers = [j for j in range(new_len, kv_len) if j in kept]
    src, nth = [], 0
    for j in range(new_len):
        if j in kept:
            src.append(j)
        else:
            src.append(movers[nth])
            nth += 1
    return np.array(src, np.int64)
