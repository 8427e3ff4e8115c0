"""Float64 definitions of the operators on paged keys and values.

Plain loops on the CPU, sharing no code with the GPU path: page tables and slot
maps, 8-bit block summaries, the choice of blocks, attention over pages and over
listed blocks.
"""
from __future__ import annotations

import math

import numpy as np

from .attention import attend, slots


def assign(table, free, count, q_lens, kv_lens, page, num_pages):
    """(table after the call, slots, positions, pages left)."""
    table, left, s, p = np.array(table), count, [], []
    for b, (q, n) in enumerate(zip(q_lens, kv_lens)):
        for i in range(-(-(n - q) // page), -(-n // page)):
            left -= 1
            table[b, i] = free[left]
        for pos in range(n - q, n):
            pg = int(table[b, pos // page])
            s.append(pg * page + pos % page if 0 <= pg < num_pages else -1)
            p.append(pos)
    return table, np.array(s, np.int64), np.array(p, np.int64), left


def release(table, free, count, new_lens, kv_lens, page):
    """(table, free list, pages free) after the call."""
    table, free = np.array(table), np.array(free)
    back = []
    for b, (new, n) in enumerate(zip(new_lens, kv_lens)):
        for i in range(-(-new // page), -(-n // page)):
            back.append(table[b, i])
            table[b, i] = -1
    for x in reversed(back):
        free[count] = x
        count += 1
    return table, free, count


def to_grid(x):
    """Row [d] -> whole numbers -127..127 and the exponent of their unit."""
    most = float(np.finfo(np.float32).max)
    x = np.nan_to_num(np.asarray(x, np.float64), nan=0.0, posinf=most, neginf=-most)
    top = float(np.abs(x).max())
    e = -126
    while e < 127 and top >= 127.5 * 2.0 ** e:
        e += 1
    return np.rint(x / 2.0 ** e).astype(np.int64), e


def _sum(x):
    with np.errstate(invalid="ignore"):
        return math.fsum(x) if np.isfinite(x).all() else float(np.sum(x))


def summaries(k_pages, table, q_lens, kv_lens, block, codes, scales):
    """codes, scales (copies are returned) after the blocks that the newest tokens complete."""
    pages, page = k_pages.shape[:2]
    codes, scales = np.array(codes), np.array(scales)
    for b, (q, n) in enumerate(zip(q_lens, kv_lens)):
        at = slots(table, b, n, page, pages)
        for j in range((n - q) // block, n // block):
            if (j + 1) * block <= n - q or at[j * block] < 0:
                continue
            rows = k_pages.reshape(-1, *k_pages.shape[2:])[at[j * block:(j + 1) * block]].astype(np.float64)
            for h in range(k_pages.shape[2]):
                mean = np.array([_sum(rows[:, h, c]) / block for c in range(rows.shape[2])])
                row, e = to_grid(mean)
                pg, blk = divmod(int(at[j * block]) // block, page // block)
                codes[pg, blk, h], scales[pg, blk, h] = row, e + 127
    return codes, scales


def select(q, codes, scales, table, q_lens, kv_lens, block, page, topn, sinks, local):
    """idx [total_q, Hkv, topn]."""
    pages, per, hk, _ = codes.shape
    g = q.shape[1] // hk
    idx = np.full((q.shape[0], hk, topn), -1, np.int64)
    row = 0
    for b, (ql, n) in enumerate(zip(q_lens, kv_lens)):
        for i in range(ql):
            own = (n - ql + i) // block
            must = [j for j in range(own + 1) if j < sinks or j > own - local or own < topn]
            others = [j for j in range(own + 1) if j not in set(must)]
            pgs = np.array([table[b][j * block // page] for j in others], np.int64)
            there = (pgs >= 0) & (pgs < pages)
            for h in range(hk):
                at = [(int(p) if t else 0, j % per) for p, t, j in zip(pgs, there, others)]
                rows = [to_grid(q[row + i, h * g + x]) for x in range(g)]
                top = max(e for _, e in rows)
                score = np.full(len(others), -np.inf, np.float32)
                if others:
                    pg, blk = np.array(at).T
                    c, s = codes[pg, blk, h].astype(np.int64), scales[pg, blk, h].astype(np.int64)
                    best = np.max([(c @ a) * 2.0 ** max(e - top, -100) for a, e in rows], 0)
                    score = np.where(there, np.ldexp(best, s - 142).astype(np.float32), np.float32(-np.inf))
                order = sorted(range(len(others)), key=lambda x: (-float(score[x]), others[x]))
                take = sorted(must + [others[x] for x in order[:topn - len(must)]])
                idx[row + i, h, :len(take)] = take
        row += ql
    return idx


def pages_attention(q, k_pages, v_pages, table, q_lens, kv_lens, scale, idx=None, block=0):
    """(out, lse, abs_out, size) per query row and head; idx, block: over the listed blocks."""
    nq, H, d = q.shape
    pages, page, hk, _ = k_pages.shape
    g = H // hk
    out, ab = np.zeros((nq, H, d)), np.zeros((nq, H, d))
    lse, size = np.full((nq, H), -np.inf), np.zeros((nq, H))
    row = 0
    for b, (ql, kl) in enumerate(zip(q_lens, kv_lens)):
        at = slots(table, b, kl, page, pages)
        ok = (at >= 0)[:, None, None]
        k = np.where(ok, k_pages.reshape(-1, hk, d)[np.maximum(at, 0)], 0.0)
        v = np.where(ok, v_pages.reshape(-1, hk, d)[np.maximum(at, 0)], 0.0)
        for i in range(ql):
            see = ((np.arange(kl) <= kl - ql + i) & (at >= 0)).astype(np.float64)
            for h in range(H):
                times = see
                if idx is not None:
                    times = np.zeros(kl)
                    for j in map(int, idx[row + i, h // g]):
                        if 0 <= j * block < kl:
                            times[j * block:(j + 1) * block] += 1
                    times = times * see
                o, l, _, a, z = attend(q[row + i, h], k[:, h // g], v[:, h // g], scale, times)
                out[row + i, h], lse[row + i, h], ab[row + i, h], size[row + i, h] = o, l, a, z
        row += ql
    return out, lse, ab, size
