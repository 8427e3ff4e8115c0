"""Paged keys and values in 16 or 32 bits: what is measured, and the plain forms.

Five operators of one serving path.  The page tables and slot maps of a step,
built from the requests' lengths; the write of new keys and values into the
pages, with a summary of every block that it completes; attention of the new
tokens (chunks of prompts and single tokens) over the pages; the choice of a
few blocks per query by a cheap score on the summaries; and attention over the
chosen blocks.

A block's summary is the mean of its keys in 8 bits: a row of integers in
-127..127 times one scale 2^(e-127), e the smallest byte in 1..254 for which
every element lies below 127.5 scales, rounded to the nearest, ties to even.
Queries are rounded the same way, so a score is an integer times a power of
two, and which blocks are chosen does not depend on how sums are ordered.

Lengths come from this package's workloads: decode with one or two query tokens
per sequence over pages of 64 permuted keys, prompts of up to 32768 tokens,
chunks of a long one.
"""
import math

import torch

own = False

DEV = "cuda"
_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def _join(v):
    return ",".join(str(int(x)) for x in v)


def listed():
    return [
        # one decode step of 128 sequences: a token each, some of which open a page
        dict(name="assign_step", op="assign", page=64, q_lens=_join([1] * 128),
             kv_lens=_join(1000 + 37 * i for i in range(128))),
        # admission of 300 prompts, 1.2M tokens
        dict(name="assign_prompts", op="assign", page=64, q_lens=_join(512 + 7919 * i % 7001 for i in range(300)),
             kv_lens=_join(512 + 7919 * i % 7001 for i in range(300))),
        # the same decode step's rows, two tokens per sequence; a few blocks become complete
        dict(name="append_step", op="append", dtype="bf16", kv_heads=8, d=128, page=64, block=64,
             q_lens=_join([2] * 64), kv_lens=_join(4099 + 61 * i for i in range(64))),
        # prompts and a chunk, 31K tokens
        dict(name="append_prompts", op="append", dtype="bf16", kv_heads=8, d=128, page=128, block=64,
             q_lens="16384,8001,5111,1515", kv_lens="16384,8001,9303,1515"),
        # one sequence, one token: the smallest step (fp32, odd length, small pages)
        dict(name="attend_single_f32", op="attend", dtype="f32", heads=16, kv_heads=2, d=64, page=16,
             q_lens="1", kv_lens="5003"),
        # batched decode over all keys
        dict(name="attend_decode", op="attend", dtype="bf16", heads=64, kv_heads=8, d=128, page=64,
             q_lens=_join([1] * 48), kv_lens=_join(4096 + 613 * i for i in range(48))),
        # a scheduler's step: two chunks of prompts between decoding sequences
        dict(name="attend_mixed", op="attend", dtype="bf16", heads=32, kv_heads=8, d=128, page=64,
             q_lens=_join([1] * 12 + [1024, 700] + [1] * 12),
             kv_lens=_join([2000 + 700 * i for i in range(12)] + [9216, 700] + [777 + 501 * i for i in range(12)])),
        # a chunk of a long prompt
        dict(name="attend_chunk", op="attend", dtype="bf16", heads=32, kv_heads=8, d=128, page=64,
             q_lens="4096", kv_lens="65536"),
        # decode with two tokens per sequence: 32 of up to 1600 blocks for each
        dict(name="select_step", op="select", dtype="bf16", heads=64, kv_heads=8, d=128, page=64, block=64, topn=32,
             sinks=1, local=2, q_lens=_join([2] * 32), kv_lens=_join(3001 + 3203 * i for i in range(32))),
        # a chunk of a long prompt: 16 blocks for each of 4096 queries
        dict(name="select_chunk", op="select", dtype="bf16", heads=32, kv_heads=8, d=128, page=128, block=64, topn=16,
             sinks=1, local=2, q_lens="4096", kv_lens="65536"),
        # the same decode step's attention over its blocks
        dict(name="sparse_step", op="sparse", dtype="bf16", heads=64, kv_heads=8, d=128, page=64, block=64, topn=32,
             sinks=1, local=2, q_lens=_join([2] * 32), kv_lens=_join(3001 + 3203 * i for i in range(32))),
        # chunks of two prompts over their blocks
        dict(name="sparse_chunk", op="sparse", dtype="bf16", heads=64, kv_heads=8, d=128, page=64, block=64, topn=16,
             sinks=1, local=2, q_lens="4096,1500", kv_lens="32768,9001"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["assign", "append", "attend", "attend", "select", "sparse"])
    kv = rng.choice([1, 2, 3, 4, 8])
    heads = kv * rng.choice([1, 2, 4, 5, 8, 16])
    c = dict(op=op)
    if op == "assign":
        c["page"] = rng.choice([16, 48, 64, 128, 256])
        n = _log(rng, 1, 400)
        ql = [_log(rng, 1, 4000) if rng.random() < 0.5 else rng.choice([0, 1, 2, 4]) for _ in range(n)]
        ql[0] = max(1, ql[0])
        kl = [max(1, q + (_log(rng, 1, 20000) if rng.random() < 0.6 else 0)) for q in ql]
        return dict(c, q_lens=_join(ql), kv_lens=_join(kl))
    c.update(dtype=rng.choice(["bf16", "bf16", "f32"]), kv_heads=kv, d=rng.choice([64, 128]))
    if op != "attend":
        c["block"] = rng.choice([16, 32, 64, 64, 128])
        c["page"] = c["block"] * rng.choice([1, 2, 3, 4])
    else:
        c["page"] = rng.choice([16, 48, 64, 128, 256])
    if op == "append":
        ql = [_log(rng, 1, 8192) for _ in range(rng.randint(1, 40))]
        ql = ql if sum(ql) < 30000 else ql[:3]
        kl = [q + (_log(rng, 1, 5000) if rng.random() < 0.5 else 0) for q in ql]
        return dict(c, q_lens=_join(ql), kv_lens=_join(kl))
    c["heads"] = heads
    if op == "attend":
        n = _log(rng, 1, 48)
        kl = [_log(rng, 64, 30000) for _ in range(n)]
        ql = [min(k, rng.choice([1, 1, 1, 2, 4])) for k in kl]
        if rng.random() < 0.6:      # chunks between them
            for i in range(rng.randint(1, min(3, n))):
                ql[i] = min(kl[i], _log(rng, 8, 4096 if c["dtype"] == "bf16" else 400))
        return dict(c, q_lens=_join(ql), kv_lens=_join(kl))
    c["topn"] = rng.choice([4, 8, 16, 16, 32, 63])
    c["sinks"], c["local"] = rng.choice([0, 1, 1, 2]), rng.choice([1, 2, 2])
    if rng.random() < 0.5:
        kl = [_log(rng, 64, 60000) for _ in range(_log(rng, 1, 32))]
        kl[0] = max(kl[0], c["block"] * (c["topn"] + 9) - 5)      # one at least with blocks to choose from
        ql = [min(k, rng.choice([1, 2, 3])) for k in kl]
    else:
        kl = [_log(rng, 200, 30000) for _ in range(rng.randint(1, 3))]
        kl[0] = max(kl[0], c["block"] * (c["topn"] + 9) - 5)
        ql = [min(k, _log(rng, 4, 1300 if c["dtype"] == "bf16" else 300)) for k in kl]
    return dict(c, q_lens=_join(ql), kv_lens=_join(kl))


def _lens(text):
    return [int(x) for x in text.split(",")]


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _rows(gen, n, h, d, dtype, loud=False):
    """Activations: normal values; keys and values have a few channels several times as large."""
    x = torch.randn(n, h, d, generator=gen, device=DEV)
    if loud:
        x[..., ::29] *= 4.0
    return x.to(_TYPES[dtype])


def _pool(gen, pages, page, h, d, dtype):
    """Rows in every slot of a pool, made a slab at a time."""
    out = torch.empty(pages, page, h, d, dtype=_TYPES[dtype], device=DEV)
    step = max(1, (1 << 26) // (page * h * d))
    for a in range(0, pages, step):
        b = min(pages, a + step)
        out[a:b] = _rows(gen, (b - a) * page, h, d, dtype, loud=True).view(b - a, page, h, d)
    return out


def _drift(gen, n, every, *shape):
    """[n, *shape]: neighbours are alike, as the queries of neighbouring tokens are; unit variance."""
    a = torch.randn(-(-n // every) + 1, *shape, generator=gen, device=DEV)
    t = torch.arange(n, device=DEV)
    w = ((t % every).float() / every).view(-1, *([1] * len(shape)))
    x = a[t // every] * (1 - w) + a[t // every + 1] * w + 0.5 * torch.randn(n, *shape, generator=gen, device=DEV)
    return x / ((1 - w) ** 2 + w ** 2 + 0.25).sqrt()


def _tables(gen, lens, page):
    """A permuted page table [batch, max_pages] (-1 behind a sequence's pages), the pages that are left over, and
    the number of pages."""
    per = [-(-k // page) for k in lens]
    total = sum(per) + 3
    perm = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((len(lens), max(max(per), 1)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, perm[at:], total


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed * 1000003 + 29)
    s = dict(case)
    ql, kl = _lens(s["q_lens"]), _lens(s["kv_lens"])
    s["q_lens"], s["kv_lens"] = ql, kl
    op, page = s["op"], s["page"]
    nq = sum(ql)
    if own:
        import exact_top_token_amd as E

        s["E"] = E
    if op == "assign":
        # the pages of the tokens before the step are given out, a permutation of the rest is free
        old = [k - q for q, k in zip(ql, kl)]
        need = sum(-(-k // page) + (-o // page) for k, o in zip(kl, old))
        held, rest, total = _tables(gen, old, page)
        cap = max(-(-k // page) for k in kl)
        s["table"] = torch.full((len(kl), cap), -1, dtype=torch.int32, device=DEV)
        s["table"][:, :held.shape[1]] = held[:, :cap]
        fresh = torch.randperm(need + 5, generator=gen, device=DEV).to(torch.int32) + total
        s["free"] = torch.full((total + need + 5,), -1, dtype=torch.int32, device=DEV)
        s["count"] = rest.numel() + fresh.numel()
        s["free"][:s["count"]] = torch.cat((rest, fresh))
        s["slots"] = torch.zeros(nq, dtype=torch.int32, device=DEV)
        s["positions"] = torch.zeros(nq, dtype=torch.int32, device=DEV)
        return s
    table, _, pages = _tables(gen, kl, page)
    s["table"] = table
    hk, d = s["kv_heads"], s["d"]
    if op in ("append", "select"):
        shape = (pages, page // s["block"], hk)
        s["codes"] = torch.zeros(*shape, d, dtype=torch.int8, device=DEV)
        s["scales"] = torch.ones(*shape, dtype=torch.uint8, device=DEV)
        s["steps"] = _pow2(torch.arange(256, device=DEV) - 127).float()
        if op == "select":
            # the means of normal keys with loud channels, larger for some blocks than for others
            m = _rows(gen, shape[0] * shape[1], hk, d, "f32", loud=True) / math.sqrt(s["block"])
            m *= (0.5 * torch.randn(m.shape[0], hk, 1, generator=gen, device=DEV)).exp()
            codes, e = _encode(m.double())
            s["codes"].view(-1, hk, d)[:] = codes
            s["scales"].view(-1, hk)[:] = e
        if own:
            s["blocks"] = E.Blocks(s["codes"], s["scales"], page)
    if op == "select":
        s["q"] = _drift(gen, nq, 32, s["heads"], d).to(_TYPES[s["dtype"]])
        s["idx"] = torch.full((nq, hk, s["topn"]), -1, dtype=torch.int32, device=DEV)
        return s
    s["k_pages"], s["v_pages"] = (_pool(gen, pages, page, hk, d, s["dtype"]) for _ in range(2))
    if own:
        s["pages"] = E.Pages(s["k_pages"], s["v_pages"], table)
    if op == "append":
        s["k"], s["v"] = (_rows(gen, nq, hk, d, s["dtype"], loud=True) for _ in range(2))
        return s
    s["scale"] = 1.0 / math.sqrt(d)
    s["q"] = _rows(gen, nq, s["heads"], d, s["dtype"])
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(nq, s["heads"], device=DEV)
    if op == "sparse":
        # blocks as a choice leaves them: sinks, the latest, and others that neighbouring queries share
        s["idx"] = torch.empty(nq, hk, s["topn"], dtype=torch.int32, device=DEV)
        row = 0
        for q, k in zip(ql, kl):
            for a in range(0, q, 2048):
                b = min(q, a + 2048)
                pos = torch.arange(k - q + a, k - q + b, device=DEV)
                score = _drift(gen, b - a, 32, hk, -(-k // s["block"]))
                s["idx"][row + a:row + b] = _choose(score, pos, s["block"], s["topn"], s["sinks"], s["local"])
            row += q
    if own:
        n = (E.block_workspace_size(ql, kl, s["heads"], hk, d, s["dtype"], s["block"], s["topn"]) if op == "sparse"
             else E.pages_workspace_size(ql, kl, s["heads"], hk, d, s["dtype"]))
        s["ws"] = torch.empty(n, dtype=torch.uint8, device=DEV)
    return s


# ----------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------
def _slots(table, b, n, page):
    """Pool slots of positions 0..n-1 of sequence b."""
    p = torch.arange(n, device=table.device)
    return table[b].long()[p // page] * page + p % page


def _plain_assign(s):
    ql, kl = (torch.tensor(s[n], device=DEV) for n in ("q_lens", "kv_lens"))
    page = s["page"]
    old = kl - ql
    first = (old + page - 1) // page
    need = (kl + page - 1) // page - first
    seqs = torch.arange(len(s["q_lens"]), device=DEV)
    new = sum(-(-k // page) - -(-(k - q) // page) for q, k in zip(s["q_lens"], s["kv_lens"]))
    nth = torch.arange(new, device=DEV)
    b = torch.repeat_interleave(seqs, need, output_size=new)
    s["table"][b, nth - (need.cumsum(0) - need)[b] + first[b]] = s["free"][s["count"] - 1 - nth]
    t = torch.arange(sum(s["q_lens"]), device=DEV)
    b = torch.repeat_interleave(seqs, ql, output_size=t.numel())
    pos = t - (ql.cumsum(0) - ql)[b] + old[b]
    s["slots"].copy_(s["table"][b, pos // page].long() * page + pos % page)
    s["positions"].copy_(pos)
    return s["table"], s["slots"], s["positions"], s["count"] - new


def _pow2(e):
    """2^e in 64 bits, by its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _encode(x):
    """64-bit rows [..., d] -> codes int8 [..., d], scale bytes [...]."""
    amax = x.abs().amax(-1)
    m, t = torch.frexp(amax)                 # amax = m 2^t, m in [.5, 1)
    e = torch.where(m < 127.5 / 128, t - 7, t - 6)
    e = torch.where(amax > 0, e, torch.full_like(e, -126)).clamp(-126, 127)
    return torch.round(x * _pow2(-e)[..., None]).to(torch.int8), (e + 127).to(torch.uint8)


def _plain_append(s):
    rows = torch.cat([_slots(s["table"], b, kl, s["page"])[kl - ql:]
                      for b, (ql, kl) in enumerate(zip(s["q_lens"], s["kv_lens"]))])
    for x in "kv":
        s[x + "_pages"].flatten(0, 1)[rows] = s[x]
    # blocks that the call completes
    at = torch.cat([_slots(s["table"], b, kl, s["page"])[(kl - ql) // s["block"] * s["block"]:kl // s["block"] * s["block"]]
                    for b, (ql, kl) in enumerate(zip(s["q_lens"], s["kv_lens"]))]).view(-1, s["block"])
    mean = s["k_pages"].flatten(0, 1)[at].double().sum(1) / s["block"]
    codes, scales = _encode(mean)
    s["codes"].flatten(0, 1)[at[:, 0] // s["block"]] = codes
    s["scales"].flatten(0, 1)[at[:, 0] // s["block"]] = scales
    return s["k_pages"], s["v_pages"], _summaries(s)


def _summaries(s):
    """The values that the summaries stand for."""
    return s["codes"] * s["steps"][s["scales"].long()][..., None]


def _softmax_rows(q, k, v, scale, hide):
    """q [g, n, d], k/v [m, d], hide [n, m] true where masked: output [g, n, d], lse [g, n]."""
    sc = torch.matmul(q, k.t()) * scale
    sc = sc.masked_fill(hide, float("-inf"))
    top = sc.amax(-1, keepdim=True)
    p = (sc - top).exp()
    tot = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / tot, (top + tot.log())[..., 0]


def _plain_attend(s):
    out, lse = s["out"], s["lse"]
    g, hk = s["heads"] // s["kv_heads"], s["kv_heads"]
    row = 0
    for b, (ql, kl) in enumerate(zip(s["q_lens"], s["kv_lens"])):
        slots = _slots(s["table"], b, kl, s["page"])
        k, v = s["k_pages"].flatten(0, 1)[slots], s["v_pages"].flatten(0, 1)[slots]
        for h in range(hk):
            kh, vh = k[:, h].float(), v[:, h].float()
            for a in range(0, ql, 1024):
                e = min(ql, a + 1024)
                seen = kl - ql + e
                q = s["q"][row + a:row + e, h * g:(h + 1) * g].float().transpose(0, 1).contiguous()
                hide = torch.arange(seen, device=q.device)[None] > torch.arange(kl - ql + a, seen, device=q.device)[:, None]
                o, l = _softmax_rows(q, kh[:seen], vh[:seen], s["scale"], hide)
                out[row + a:row + e, h * g:(h + 1) * g] = o.transpose(0, 1).to(out.dtype)
                lse[row + a:row + e, h * g:(h + 1) * g] = l.transpose(0, 1)
        row += ql
    return out, lse


def _choose(score, pos, block, topn, sinks, local):
    """score [n, h, blocks], pos [n]: the blocks of each row, ascending, -1 behind."""
    j = torch.arange(score.shape[-1], device=score.device)
    mine = (pos // block)[:, None]
    rank = score.masked_fill(((j < sinks) | (j > mine - local))[:, None], float("inf"))
    rank = rank.masked_fill((j > mine)[:, None], float("-inf"))
    best = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :topn]
    best = torch.where(best <= mine[..., None], best, torch.full_like(best, 1 << 30)).sort(-1).values
    out = torch.full((*score.shape[:2], topn), -1, dtype=torch.int32, device=score.device)
    out[..., :best.shape[-1]] = torch.where(best < 1 << 30, best, torch.full_like(best, -1)).to(torch.int32)
    return out


def _plain_select(s):
    hk, g, block = s["kv_heads"], s["heads"] // s["kv_heads"], s["block"]
    row = 0
    for b, (ql, kl) in enumerate(zip(s["q_lens"], s["kv_lens"])):
        n = -(-kl // block)
        at = _slots(s["table"], b, kl, s["page"])[::block] // block
        codes = s["codes"].flatten(0, 1)[at].float()
        scales = s["scales"].flatten(0, 1)[at].int()
        for a in range(0, ql, 1024):
            e = min(ql, a + 1024)
            pos = torch.arange(kl - ql + a, kl - ql + e, device=DEV)
            qc, qe = _encode(s["q"][row + a:row + e].double().view(e - a, hk, g, -1))
            qe = qe.int()
            rel = (qe - qe.amax(-1, keepdim=True)).clamp(min=-100)
            score = torch.empty(e - a, hk, n, device=DEV)
            for h in range(hk):
                # sums of at most 128 products of 7 bits: exact
                dot = torch.matmul(qc[:, h].float().view(-1, s["d"]), codes[:, h].t().contiguous()).view(e - a, g, n)
                best = (dot.double() * _pow2(rel[:, h])[..., None]).amax(1)
                score[:, h] = (best * _pow2(scales[:, h] - 142)).float()
            s["idx"][row + a:row + e] = _choose(score, pos, block, s["topn"], s["sinks"], s["local"])
        row += ql
    return s["idx"]


def _plain_sparse(s):
    out, lse = s["out"], s["lse"]
    g, hk, block, d = s["heads"] // s["kv_heads"], s["kv_heads"], s["block"], s["d"]
    row = 0
    for b, (ql, kl) in enumerate(zip(s["q_lens"], s["kv_lens"])):
        slots = _slots(s["table"], b, -(-kl // block) * block, s["page"])
        for h in range(hk):
            k, v = s["k_pages"][:, :, h].flatten(0, 1), s["v_pages"][:, :, h].flatten(0, 1)
            step = max(1, (1 << 27) // (s["topn"] * block * d))
            for a in range(0, ql, step):
                e = min(ql, a + step)
                idx = s["idx"][row + a:row + e, h].long()
                key = (idx[..., None] * block + torch.arange(block, device=DEV)).flatten(1)
                pos = torch.arange(kl - ql + a, kl - ql + e, device=DEV)
                hide = (key < 0) | (key > pos[:, None])
                at = slots[key.clamp(0, slots.numel() - 1)]
                q = s["q"][row + a:row + e, h * g:(h + 1) * g].float()
                sc = torch.matmul(q, k[at].float().transpose(1, 2).contiguous()) * s["scale"]
                sc = sc.masked_fill(hide[:, None], float("-inf"))
                top = sc.amax(-1, keepdim=True)
                p = (sc - top).exp()
                tot = p.sum(-1, keepdim=True)
                out[row + a:row + e, h * g:(h + 1) * g] = (torch.matmul(p, v[at].float()) / tot).to(out.dtype)
                lse[row + a:row + e, h * g:(h + 1) * g] = (top + tot.log())[..., 0]
        row += ql
    return out, lse


def run(s):
    op = s["op"]
    if not own:
        return {"assign": _plain_assign, "append": _plain_append, "attend": _plain_attend, "select": _plain_select,
                "sparse": _plain_sparse}[op](s)
    E = s["E"]
    if op == "assign":
        left = E.dsa_pages_assign(s["table"], s["page"], s["free"], s["count"], s["q_lens"], s["kv_lens"],
                                  slots=s["slots"], positions=s["positions"])
        return s["table"], s["slots"], s["positions"], left
    if op == "append":
        E.dsa_pages_append(s["pages"], s["k"], s["v"], s["q_lens"], s["kv_lens"], blocks=s["blocks"])
        return s["k_pages"], s["v_pages"], _summaries(s)
    if op == "attend":
        E.dsa_pages_attention(s["pages"], s["q"], s["q_lens"], s["kv_lens"], s["out"], s["lse"], scale=s["scale"],
                              workspace=s["ws"])
        return s["out"], s["lse"]
    if op == "select":
        E.dsa_block_select(s["blocks"], s["table"], s["q"], s["q_lens"], s["kv_lens"], s["idx"], sinks=s["sinks"],
                           local=s["local"])
        return s["idx"]
    E.dsa_block_attention(s["pages"], s["q"], s["q_lens"], s["kv_lens"], s["idx"], s["block"], s["out"], s["lse"],
                          scale=s["scale"], workspace=s["ws"])
    return s["out"], s["lse"]


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    ql, kl = _lens(case["q_lens"]), _lens(case["kv_lens"])
    page = case["page"]
    if case["op"] == "assign":
        new = sum(-(-k // page) - -(-(k - q) // page) for q, k in zip(ql, kl))
        # every new page read from the list and written to the table, a slot and a position a token
        return {"bytes": 8 * new + 8 * sum(ql) + 4 * len(ql), "flops": 2 * sum(ql)}
    d, hk = case["d"], case["kv_heads"]
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "append":
        blk = case["block"]
        done = sum(k // blk - (k - q) // blk for q, k in zip(ql, kl))
        before = sum((k - q) % blk for q, k in zip(ql, kl) if k // blk > (k - q) // blk)
        return {"bytes": hk * (4 * sum(ql) * d * size + before * d * size + done * (d + 1)), "flops": done * blk * hk * d}
    h = case["heads"]
    if case["op"] == "attend":
        pairs = sum(q * (k - q) + q * (q + 1) // 2 for q, k in zip(ql, kl))
        return {"bytes": sum(ql) * h * (2 * d * size + 4) + sum(kl) * hk * d * 2 * size, "flops": 4 * pairs * h * d}
    blk = case["block"]
    if case["op"] == "select":
        seen = sum(-(-k // blk) for k in kl)
        pairs = sum((k - q + i) // blk + 1 for q, k in zip(ql, kl) for i in range(q))
        return {"bytes": sum(ql) * (h * d * size + 4 * hk * case["topn"]) + seen * hk * (d + 1), "flops": 2 * pairs * h * d}
    keys = rows = 0
    for q, k in zip(ql, kl):
        mine = sum(min(case["topn"] * blk, k - q + i + 1) for i in range(q))
        keys += mine
        rows += min(mine, k)
    return {"bytes": sum(ql) * (h * (2 * d * size + 4) + 4 * hk * case["topn"]) + rows * hk * d * 2 * size,
            "flops": 4 * keys * h * d}


# ----------------------------------------------------------------------------
# the definition in 64 bits
# ----------------------------------------------------------------------------
_TWO = [2.0 ** i for i in range(-400, 401)]


def _two(e):
    return torch.tensor(_TWO, dtype=torch.float64, device=DEV)[e.long() + 400]


def _grid(x):
    """64-bit rows [..., d] -> whole numbers in -127..127 and the power of two they count."""
    x = x.double()
    amax = x.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(amax.clamp(min=2.0 ** -140) / 127.5)) - 1.0
    for _ in range(3):
        e = torch.where(amax >= 127.5 * _two(e), e + 1.0, e)
    e = e.clamp(-126.0, 127.0)
    return torch.round(x / _two(e)), e


def _where(s, b, n):
    """Pool slots of the first n positions, page by page."""
    page = s["page"]
    return torch.cat([torch.arange(page, device=DEV) + int(p) * page for p in s["table"][b, :-(-n // page)].tolist()])[:n]


def exact(case, seed):
    s = prepare(case, seed)
    op, ql, kl, page = s["op"], s["q_lens"], s["kv_lens"], s["page"]
    if op == "assign":
        stack = s["free"][:s["count"]].tolist()
        table, slots, positions = s["table"].tolist(), [], []
        for b, (q, k) in enumerate(zip(ql, kl)):
            for p in range(-(-(k - q) // page), -(-k // page)):
                table[b][p] = stack.pop()
            pos = torch.arange(k - q, k)
            slots.append(torch.tensor(table[b])[pos // page] * page + pos % page)
            positions.append(pos)
        whole = lambda x: torch.as_tensor(x, dtype=torch.int32, device=DEV)
        return whole(table), whole(torch.cat(slots)), whole(torch.cat(positions)), len(stack)
    hk, d = s["kv_heads"], s["d"]
    if op == "append":
        blk = s["block"]
        k, v = s["k_pages"].clone().flatten(0, 1), s["v_pages"].clone().flatten(0, 1)
        mean = torch.zeros(s["scales"].shape + (d,), dtype=torch.float64, device=DEV).flatten(0, 1)
        row = 0
        for b, (q, n) in enumerate(zip(ql, kl)):
            at = _where(s, b, n)
            k[at[n - q:]], v[at[n - q:]] = s["k"][row:row + q], s["v"][row:row + q]
            for j in range((n - q) // blk, n // blk):
                mean[at[j * blk] // blk] = k[at[j * blk:(j + 1) * blk]].double().mean(0)
            row += q
        c, e = _grid(mean)
        return k.double().view(s["k_pages"].shape), v.double().view(s["v_pages"].shape), \
            (c * _two(e)).view(s["codes"].shape)
    g, row = s["heads"] // hk, 0
    if op == "select":
        blk = s["block"]
        idx = torch.full_like(s["idx"], -1)
        for b, (q, n) in enumerate(zip(ql, kl)):
            at = _where(s, b, n)[::blk] // blk
            key = s["codes"].view(-1, hk, d)[at].double() * _two(s["scales"].view(-1, hk)[at].int() - 142)[..., None]
            for h in range(hk):
                c, e = _grid(s["q"][row:row + q, h * g:(h + 1) * g])
                top = e.amax(1, keepdim=True)
                c = c * _two(torch.clamp(e - top, min=-100.0))
                for i in range(0, q, 512):
                    best = torch.full((min(512, q - i), at.numel()), float("-inf"), dtype=torch.float64, device=DEV)
                    for x in range(g):
                        best = torch.maximum(best, c[i:i + 512, x] @ key[:, h].T.contiguous())
                    mine = (torch.arange(i, i + best.shape[0], device=DEV) + n - q) // blk
                    j = torch.arange(at.numel(), device=DEV).expand_as(best)
                    must = (j < s["sinks"]) | (j > (mine - s["local"])[:, None])
                    late = j > mine[:, None]
                    best = torch.where(must, torch.full_like(best, 1e300), best)
                    best = torch.where(late, torch.full_like(best, -1e300), best)
                    order = torch.argsort(-best, dim=1, stable=True)
                    place = torch.empty_like(order).scatter_(1, order, j)        # rank of each block
                    take = (place < s["topn"]) & ~late
                    count = take.sum(1)
                    r, col = torch.nonzero(take, as_tuple=True)
                    to = torch.arange(r.numel(), device=DEV) - (count.cumsum(0) - count)[r]
                    idx[row + i + r, h, to] = col.int()
            row += q
        return idx
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    for b, (q, n) in enumerate(zip(ql, kl)):
        at = _where(s, b, n)
        pos = torch.arange(n - q, n, device=DEV)
        for h in range(hk):
            k, v = s["k_pages"].view(-1, hk, d)[at, h].double(), s["v_pages"].view(-1, hk, d)[at, h].double()
            kt = k.T.contiguous()
            step = max(16, (1 << 25) // n)
            for i in range(0, q, step):
                p = pos[i:i + step]
                see = torch.arange(n, device=DEV)[None] <= p[:, None]
                if op == "sparse":
                    listed_ = torch.zeros(p.numel(), -(-n // s["block"]) + 1, dtype=torch.bool, device=DEV)
                    pick = s["idx"][row + i:row + i + p.numel(), h].long()
                    listed_.scatter_(1, torch.where(pick < 0, listed_.shape[1] - 1, pick), True)
                    see &= listed_[:, :-1].repeat_interleave(s["block"], 1)[:, :n]
                for x in range(h * g, (h + 1) * g):
                    logit = (s["q"][row + i:row + i + p.numel(), x].double() @ kt) * s["scale"]
                    logit = torch.where(see, logit, torch.full_like(logit, float("-inf")))
                    l = torch.logsumexp(logit, 1)
                    lse[row + i:row + i + p.numel(), x] = l
                    out[row + i:row + i + p.numel(), x] = torch.exp(logit - l[:, None]) @ v
        row += q
    return out, lse
