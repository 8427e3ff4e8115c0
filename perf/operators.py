"""The attention operators next to the Top-K indexer: what is measured, and their plain forms.

Five operators of one serving path.  A prompt's causal attention over packed
sequences with grouped heads; the write of new keys and values into a paged
cache of 4-bit codes; attention over that cache, over every visible key or
over the keys the indexer selected; the attention weight each cached key
received, accumulated; and the eviction of the keys that received least.

The 4-bit format: blocks of 32 consecutive elements of a key or value row share
one scale 2^(e-127) (a byte e, 1..254, the smallest for which every element of
the block lies below 7 scales in magnitude), and an element is one of
0, .5, 1, 1.5, 2, 3, 4, 6 scales with a sign (a nibble, low nibble first),
rounded to the nearest, ties to the even code.

Lengths come from this package's workloads: tiny prefill (L = 2048, d = 64,
fp32), prefill of 32768 tokens, decode with two query tokens per sequence over
pages of 64 permuted keys, Top-K 2048.
"""
import math

import torch

own = False

DEV = "cuda"
_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def listed():
    return [
        # a handful of short fp32 prompts at the tiny prefill's head size: latency
        dict(name="prompt_short_f32", op="prompt", dtype="f32", heads=8, kv_heads=2, d=64,
             q_lens="1,7,33,64,129,250", kv_lens="1,7,33,64,200,250"),
        # a packed batch of prompts and one later chunk of a long one, as a scheduler packs them
        dict(name="prompt_packed_bf16", op="prompt", dtype="bf16", heads=32, kv_heads=8, d=128,
             q_lens="4096,2777,1501,1024,333,64,1", kv_lens="4096,2777,1501,8192,333,64,777"),
        # one long prompt, the 32K prefill's length
        dict(name="prompt_long_bf16", op="prompt", dtype="bf16", heads=32, kv_heads=8, d=128,
             q_lens="32768", kv_lens="32768"),
        # one decode step of 64 sequences, two tokens each: the write is launch-bound
        dict(name="append_decode", op="append", dtype="bf16", kv_heads=8, d=128, page=64,
             q_lens=",".join(["2"] * 64), kv_lens=",".join(str(4099 + 61 * i) for i in range(64))),
        # the keys and values of packed prompts, 42K tokens
        dict(name="append_prompt", op="append", dtype="bf16", kv_heads=8, d=128, page=64,
             q_lens="32768,8001,1111,515", kv_lens="32768,8001,9303,515"),
        # one sequence, one token: the smallest decode step (fp32 queries, odd length, small pages)
        dict(name="attend_single_f32", op="attend", dtype="f32", heads=16, kv_heads=2, d=64, page=16, topk=0,
             q_lens="1", kv_lens="4133"),
        # batched decode with two query tokens per sequence over every cached key
        dict(name="attend_decode", op="attend", dtype="bf16", heads=64, kv_heads=8, d=128, page=64, topk=0,
             q_lens=",".join(["2"] * 64), kv_lens=",".join(str(8192 + 907 * i) for i in range(64))),
        # the same step over the 2048 keys the indexer selected for each query
        dict(name="attend_selected", op="attend", dtype="bf16", heads=64, kv_heads=8, d=128, page=64, topk=2048,
             q_lens=",".join(["2"] * 32), kv_lens=",".join(str(1500 + 1009 * i) for i in range(32))),
        # weight each cached key received in a decode step of 16 sequences
        dict(name="weights_decode", op="weights", dtype="bf16", heads=32, kv_heads=8, d=128, page=64,
             q_lens=",".join(["1"] * 16), kv_lens=",".join(str(3001 + 2003 * i) for i in range(16))),
        # weight the keys of two prompts received from all their queries
        dict(name="weights_prompt", op="weights", dtype="bf16", heads=32, kv_heads=8, d=128, page=64,
             q_lens="8192,1031", kv_lens="8192,3000"),
        # the periodic eviction of a decode batch: 64 keys over a budget of 4096, four sinks and
        # the latest 256 tokens stay, earlier evictions have moved keys out of order
        dict(name="evict_steady", op="evict", kv_heads=8, d=128, page=64, moved=True, prefix=4, window=256,
             kv_lens=",".join(["4160"] * 16), new_lens=",".join(["4096"] * 16)),
        # the first eviction after long prompts: most keys go
        dict(name="evict_prompt", op="evict", kv_heads=8, d=128, page=64, moved=False, prefix=4, window=512,
             kv_lens="32768,20011,65536,9999", new_lens="4096,4096,8192,2047"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _join(v):
    return ",".join(str(int(x)) for x in v)


def _heads(rng):
    kv = rng.choice([1, 2, 3, 4, 8])
    return kv * rng.choice([1, 2, 4, 5, 8]), kv


def draw(rng):
    op = rng.choice(["prompt", "prompt", "append", "attend", "attend", "weights", "evict"])
    heads, kv = _heads(rng)
    d = rng.choice([64, 128])
    page = rng.choice([16, 48, 64, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "prompt":
        top = 8192 if dtype == "bf16" else 2500
        ql = [_log(rng, 1, top) for _ in range(rng.randint(1, 6))]
        kl = [q + (_log(rng, 1, 4096) if rng.random() < 0.4 else 0) for q in ql]
        return dict(op=op, dtype=dtype, heads=heads, kv_heads=kv, d=d, q_lens=_join(ql), kv_lens=_join(kl))
    if op == "append":
        ql = [_log(rng, 1, 8192) for _ in range(rng.randint(1, 40))]
        ql = ql if sum(ql) < 40000 else ql[:4]
        kl = [q + (_log(rng, 1, 5000) if rng.random() < 0.5 else 0) for q in ql]
        return dict(op=op, dtype=dtype, kv_heads=kv, d=d, page=page, q_lens=_join(ql), kv_lens=_join(kl))
    if op == "attend":
        n = _log(rng, 1, 64)
        kl = [_log(rng, 64, 60000) for _ in range(n)]
        ql = [min(k, rng.choice([1, 1, 2, 4])) for k in kl]
        topk = rng.choice([0, 0, _log(rng, 16, 2048)])
        return dict(op=op, dtype=dtype, heads=heads, kv_heads=kv, d=d, page=page, topk=topk, q_lens=_join(ql),
                    kv_lens=_join(kl))
    if op == "weights":
        if rng.random() < 0.5:
            kl = [_log(rng, 64, 30000) for _ in range(_log(rng, 1, 32))]
            ql = [min(k, rng.choice([1, 2, 3])) for k in kl]
        else:
            ql = [_log(rng, 16, 4096) for _ in range(rng.randint(1, 3))]
            kl = [q + rng.choice([0, 0, _log(rng, 1, 3000)]) for q in ql]
        return dict(op=op, dtype=dtype, heads=heads, kv_heads=kv, d=d, page=page, q_lens=_join(ql), kv_lens=_join(kl))
    kl = [_log(rng, 300, 40000) for _ in range(rng.randint(1, 6))]
    nl = [max(100, int(k * rng.choice([0.1, 0.25, 0.5, 0.98]))) for k in kl]
    return dict(op=op, kv_heads=kv, d=d, page=page, moved=rng.random() < 0.5, prefix=rng.choice([0, 4]),
                window=rng.choice([0, 32, 96]), kv_lens=_join(kl), new_lens=_join(nl))


def _lens(text):
    return [int(x) for x in text.split(",")]


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _rows(gen, n, h, d, dtype, loud=False):
    """Activations: normal values; keys and values have a few channels several times as large."""
    x = torch.randn(n, h, d, generator=gen, device=DEV)
    if loud:
        gain = torch.ones(h, d, device=DEV)
        gain[:, ::29] = 4.0
        x = x * gain
    return x.to(_TYPES[dtype])


def _tables(gen, kv_lens, page):
    """A permuted page table [batch, max_pages] and the number of pages; unused entries are page 0."""
    per = [-(-k // page) for k in kv_lens]
    total = sum(per) + 3
    perm = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    table = torch.zeros(len(kv_lens), max(max(per), 1), dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, total


def _cache_buffers(num_pages, page, kv_heads, d):
    return {n: torch.zeros(num_pages, page, kv_heads, w, dtype=torch.uint8, device=DEV)
            for n, w in (("k_codes", d // 2), ("k_scales", d // 32), ("v_codes", d // 2), ("v_scales", d // 32))}


def _fill_cache(gen, bufs):
    """Every slot of the pool quantised from normal rows with loud channels, a block of slots at a time."""
    pages, page, h, half = bufs["k_codes"].shape
    step = max(1, (1 << 26) // (page * h * half * 2))
    for which in ("k", "v"):
        for a in range(0, pages, step):
            b = min(pages, a + step)
            x = _rows(gen, (b - a) * page, h, half * 2, "bf16", loud=True)
            codes, scales = _encode(x.float())
            bufs[which + "_codes"][a:b] = codes.view(b - a, page, h, half)
            bufs[which + "_scales"][a:b] = scales.view(b - a, page, h, -1)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed * 1000003 + 17)
    s = dict(case)
    for key in ("q_lens", "kv_lens", "new_lens"):
        if key in s:
            s[key] = _lens(s[key])
    op = s["op"]
    if own:
        import exact_top_token_amd as E

        s["E"] = E
    if op == "prompt":
        s["scale"] = 1.0 / math.sqrt(s["d"])
        nq, nk = sum(s["q_lens"]), sum(s["kv_lens"])
        s["q"] = _rows(gen, nq, s["heads"], s["d"], s["dtype"])
        s["k"] = _rows(gen, nk, s["kv_heads"], s["d"], s["dtype"])
        s["v"] = _rows(gen, nk, s["kv_heads"], s["d"], s["dtype"])
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(nq, s["heads"], device=DEV)
        if own:
            n = E.prompt_workspace_size(s["q_lens"], s["kv_lens"], s["heads"], s["kv_heads"], s["d"], s["dtype"])
            s["ws"] = torch.empty(n, dtype=torch.uint8, device=DEV)
        return s
    table, pages = _tables(gen, s["kv_lens"], s["page"])
    s["table"] = table
    if op == "evict":
        # a cache of bf16 rows, the accumulated weights (a long tail, and keys that never received
        # any) and each key's position in the text
        h, d, page = s["kv_heads"], s["d"], s["page"]
        s["k"] = torch.randn(pages, page, h, d, generator=gen, device=DEV).to(torch.bfloat16)
        s["v"] = torch.randn(pages, page, h, d, generator=gen, device=DEV).to(torch.bfloat16)
        u = torch.rand(pages, page, generator=gen, device=DEV)
        s["acc"] = torch.where(u < 0.1, torch.zeros_like(u), (u * 6.0).exp() * 1e-3)
        s["acc_out"] = torch.zeros_like(s["acc"])
        s["seen"] = list(s["kv_lens"])
        s["pos"] = torch.zeros(pages, page, dtype=torch.int32, device=DEV)
        s["pos_out"] = torch.zeros_like(s["pos"])
        for b, n in enumerate(s["kv_lens"]):
            p = torch.arange(n, device=DEV)
            if s["moved"]:      # keys of a longer text, out of order
                s["seen"][b] = 3 * n
                p = torch.randperm(3 * n, generator=gen, device=DEV)[:n]
            rows = _slots(table, b, n, page)
            s["pos"].view(-1)[rows] = p.to(torch.int32)
        s["out_src"] = torch.full((len(s["kv_lens"]), max(s["new_lens"])), -1, dtype=torch.int32, device=DEV)
        if own:
            s["ws"] = torch.empty(E.evict_workspace_size(s["kv_lens"], s["new_lens"]), dtype=torch.uint8, device=DEV)
        return s
    s.update(_cache_buffers(pages, s["page"], s["kv_heads"], s["d"]))
    nq = sum(s["q_lens"])
    if op == "append":
        s["k"] = _rows(gen, nq, s["kv_heads"], s["d"], s["dtype"], loud=True)
        s["v"] = _rows(gen, nq, s["kv_heads"], s["d"], s["dtype"], loud=True)
        s["k_back"] = torch.empty(nq, s["kv_heads"], s["d"], device=DEV)
        s["v_back"] = torch.empty(nq, s["kv_heads"], s["d"], device=DEV)
    else:
        s["scale"] = 1.0 / math.sqrt(s["d"])
        _fill_cache(gen, s)
        s["q"] = _rows(gen, nq, s["heads"], s["d"], s["dtype"])
        if op == "attend":
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(nq, s["heads"], device=DEV)
            s["idx"] = None
            if s["topk"]:
                # distinct visible positions in no order, -1 behind the last
                s["idx"] = torch.full((nq, s["topk"]), -1, dtype=torch.int32, device=DEV)
                row = 0
                for ql, kl in zip(s["q_lens"], s["kv_lens"]):
                    for i in range(ql):
                        seen = kl - ql + i + 1
                        n = min(seen, s["topk"])
                        s["idx"][row, :n] = torch.randperm(seen, generator=gen, device=DEV)[:n].to(torch.int32)
                        row += 1
        else:
            # what some sixteen earlier steps left
            part = 32.0 * s["heads"] * len(s["kv_lens"]) / sum(s["kv_lens"])
            s["acc"] = torch.rand(pages, s["page"], generator=gen, device=DEV) * part
            s["acc_out"] = torch.zeros_like(s["acc"])
            # the normaliser an attention call returned for these queries
            s["lse"] = _cache_lse(s)
    if own:
        s["cache"] = E.Cache(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], s["table"])
        if op != "append":
            shape = (s["q_lens"], s["kv_lens"], s["heads"], s["kv_heads"], s["d"])
            n = E.cache_workspace_size(*shape, s["topk"]) if op == "attend" else E.weights_workspace_size(*shape)
            s["ws"] = torch.empty(n, dtype=torch.uint8, device=DEV)
    return s


# ----------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------
def _slots(table, b, n, page):
    """Pool slots of positions 0..n-1 of sequence b."""
    p = torch.arange(n, device=table.device)
    return table[b].long()[p // page] * page + p % page


def _encode(x):
    """fp32 [n, h, d] -> codes [n, h, d/2], scales [n, h, d/32]."""
    n, h, d = x.shape
    y = x.view(n, h, d // 32, 32)
    amax = y.abs().amax(-1)
    # smallest e with amax < 7 * 2^e: frexp gives amax = m 2^t with m in [.5, 1)
    m, t = torch.frexp(amax)
    e = torch.where(m < 0.875, t - 3, t - 2)
    e = torch.where(amax > 0, e, torch.full_like(e, -126)).clamp(-126, 127)
    a = torch.ldexp(y, -e[..., None])
    mag = a.abs()
    code = torch.zeros_like(mag, dtype=torch.uint8)
    # a border between two codes belongs to the even one
    for i, edge in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        code += (mag > edge) if i % 2 == 0 else (mag >= edge)
    code = code | ((y < 0) & (code > 0)).to(torch.uint8) * 8
    code = code.view(n, h, d // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), (e + 127).to(torch.uint8)


def _decode(codes, scales):
    """codes [n, h, d/2], scales [n, h, d/32] -> fp32 [n, h, d]."""
    n, h, half = codes.shape
    one = torch.tensor([*_GRID, *(-g for g in _GRID)], device=codes.device)
    byte = torch.arange(256, device=codes.device)
    pair = torch.stack((one[byte & 15], one[byte >> 4]), -1)
    val = pair[codes.int()].view(n, h, scales.shape[-1], 32)
    return torch.ldexp(val, scales.int()[..., None] - 127).view(n, h, 2 * half)


def _softmax_rows(q, k, v, scale, hide):
    """q [g, n, d], k/v [m, d], hide [n, m] true where masked: output [g, n, d], lse [g, n]."""
    sc = torch.matmul(q, k.t()) * scale
    sc = sc.masked_fill(hide, float("-inf"))
    top = sc.amax(-1, keepdim=True)
    p = (sc - top).exp()
    tot = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / tot, (top + tot.log())[..., 0]


def _plain_prompt(s):
    out, lse = torch.empty_like(s["q"]), torch.empty_like(s["lse"])
    g = s["heads"] // s["kv_heads"]
    q0 = k0 = 0
    for ql, kl in zip(s["q_lens"], s["kv_lens"]):
        for h in range(s["kv_heads"]):
            k, v = s["k"][k0:k0 + kl, h].float(), s["v"][k0:k0 + kl, h].float()
            for a in range(0, ql, 2048):
                b = min(ql, a + 2048)
                seen = kl - ql + b
                q = s["q"][q0 + a:q0 + b, h * g:(h + 1) * g].float().transpose(0, 1).contiguous()
                at = torch.arange(kl - ql + a, seen, device=q.device)
                hide = torch.arange(seen, device=q.device)[None] > at[:, None]
                o, l = _softmax_rows(q, k[:seen], v[:seen], s["scale"], hide)
                out[q0 + a:q0 + b, h * g:(h + 1) * g] = o.transpose(0, 1).to(out.dtype)
                lse[q0 + a:q0 + b, h * g:(h + 1) * g] = l.transpose(0, 1)
        q0 += ql
        k0 += kl
    return out, lse


def _plain_append(s):
    rows = torch.cat([_slots(s["table"], b, kl, s["page"])[kl - ql:]
                      for b, (ql, kl) in enumerate(zip(s["q_lens"], s["kv_lens"]))])
    back = []
    for which in ("k", "v"):
        codes, scales = _encode(s[which].float())
        s[which + "_codes"].flatten(0, 1)[rows] = codes
        s[which + "_scales"].flatten(0, 1)[rows] = scales
        back.append(_decode(s[which + "_codes"].flatten(0, 1)[rows], s[which + "_scales"].flatten(0, 1)[rows]))
    return tuple(back)


def _cached(s, which, rows):
    return _decode(s[which + "_codes"].flatten(0, 1)[rows], s[which + "_scales"].flatten(0, 1)[rows])


def _plain_attend(s):
    out, lse = torch.empty_like(s["q"]), torch.empty_like(s["lse"])
    g, hk, d = s["heads"] // s["kv_heads"], s["kv_heads"], s["d"]
    row = 0
    for b, (ql, kl) in enumerate(zip(s["q_lens"], s["kv_lens"])):
        slots = _slots(s["table"], b, kl, s["page"])
        parts = [(0, ql, slots)] if s["idx"] is None else [(i, i + 1, None) for i in range(ql)]
        for a, e, rows in parts:
            if rows is None:
                sel = s["idx"][row + a].long()
                rows = slots[sel.clamp(min=0)]
                hide = (sel < 0)[None]
            else:
                hide = torch.arange(kl, device=slots.device)[None] > torch.arange(kl - ql, kl, device=slots.device)[:, None]
            k, v = _cached(s, "k", rows), _cached(s, "v", rows)
            q = s["q"][row + a:row + e].float().view(e - a, hk, g, d)
            for h in range(hk):
                o, l = _softmax_rows(q[:, h].transpose(0, 1).contiguous(), k[:, h].contiguous(), v[:, h].contiguous(),
                                     s["scale"], hide)
                out[row + a:row + e, h * g:(h + 1) * g] = o.transpose(0, 1).to(out.dtype)
                lse[row + a:row + e, h * g:(h + 1) * g] = l.transpose(0, 1)
        row += ql
    return out, lse


def _score_blocks(s, b, row, ql, kl, step=512):
    """Scaled scores of sequence b by head and block of queries: (first query, last, head, scores
    [g, n, kl] with -inf where masked)."""
    g, hk = s["heads"] // s["kv_heads"], s["kv_heads"]
    k = _cached(s, "k", _slots(s["table"], b, kl, s["page"]))
    for h in range(hk):
        kh = k[:, h].contiguous()
        for a in range(0, ql, step):
            e = min(ql, a + step)
            q = s["q"][row + a:row + e, h * g:(h + 1) * g].float().transpose(0, 1).contiguous()
            sc = torch.matmul(q, kh.t()) * s["scale"]
            hide = torch.arange(kl, device=q.device)[None] > torch.arange(kl - ql + a, kl - ql + e, device=q.device)[:, None]
            yield a, e, h, sc.masked_fill(hide, float("-inf"))


def _cache_lse(s):
    lse = torch.empty(sum(s["q_lens"]), s["heads"], device=DEV)
    g, row = s["heads"] // s["kv_heads"], 0
    for b, (ql, kl) in enumerate(zip(s["q_lens"], s["kv_lens"])):
        for a, e, h, sc in _score_blocks(s, b, row, ql, kl):
            lse[row + a:row + e, h * g:(h + 1) * g] = sc.logsumexp(-1).transpose(0, 1)
        row += ql
    return lse


def _plain_weights(s):
    out = s["acc_out"]
    g, row = s["heads"] // s["kv_heads"], 0
    for b, (ql, kl) in enumerate(zip(s["q_lens"], s["kv_lens"])):
        tot = torch.zeros(kl, device=DEV)
        for a, e, h, sc in _score_blocks(s, b, row, ql, kl):
            l = s["lse"][row + a:row + e, h * g:(h + 1) * g].transpose(0, 1)
            tot += (sc - l[..., None]).exp().sum((0, 1))
        rows = _slots(s["table"], b, kl, s["page"])
        old = s["acc"].view(-1)[rows]
        old[kl - ql:] = 0.0          # the step's own keys had none before
        out.view(-1)[rows] = old + tot
        row += ql
    return out


def _plain_evict(s):
    for b, (kl, nl) in enumerate(zip(s["kv_lens"], s["new_lens"])):
        rows = _slots(s["table"], b, kl, s["page"])
        acc, pos = s["acc"].view(-1)[rows], s["pos"].view(-1)[rows]
        safe = (pos < s["prefix"]) | (pos >= s["seen"][b] - s["window"])
        rank = torch.where(safe, torch.full_like(acc, float("inf")), acc)
        best = torch.sort(rank, descending=True, stable=True).indices[:nl]
        kept = torch.zeros(kl, dtype=torch.bool, device=DEV)
        kept[best] = True
        at = torch.arange(kl, device=DEV)
        # the n-th kept key behind the new end moves into the n-th hole before it
        movers = torch.sort(torch.where(kept & (at >= nl), at, torch.full_like(at, kl))).values[:nl]
        hole = ~kept[:nl]
        nth = hole.long().cumsum(0) - 1
        src = torch.where(hole, movers[nth.clamp(min=0)], at[:nl])
        s["out_src"][b, :nl] = src.to(torch.int32)
        to, frm = rows[:nl], rows[src]
        for name in ("k", "v"):
            flat = s[name].flatten(0, 1)
            flat[to] = flat[frm]
        s["acc_out"].view(-1)[to] = s["acc"].view(-1)[frm]
        s["pos_out"].view(-1)[to] = s["pos"].view(-1)[frm]
    return s["out_src"], s["k"], s["v"], s["acc_out"], s["pos_out"]


def run(s):
    op = s["op"]
    if not own:
        return {"prompt": _plain_prompt, "append": _plain_append, "attend": _plain_attend,
                "weights": _plain_weights, "evict": _plain_evict}[op](s)
    E = s["E"]
    if op == "prompt":
        E.dsa_prompt_attention(s["q"], s["k"], s["v"], s["q_lens"], s["kv_lens"], s["out"], s["lse"],
                               scale=s["scale"], workspace=s["ws"])
        return s["out"], s["lse"]
    if op == "append":
        E.dsa_cache_append(s["cache"], s["k"], s["v"], s["q_lens"], s["kv_lens"])
        E.dsa_cache_read(s["cache"], s["k_back"], s["v_back"], s["q_lens"], s["kv_lens"])
        return s["k_back"], s["v_back"]
    if op == "attend":
        E.dsa_cache_attention(s["cache"], s["q"], s["q_lens"], s["kv_lens"], s["out"], s["lse"], idx=s["idx"],
                              scale=s["scale"], workspace=s["ws"])
        return s["out"], s["lse"]
    if op == "weights":
        E.dsa_cache_weights(s["cache"], s["q"], s["lse"], s["q_lens"], s["kv_lens"], s["acc"], s["acc_out"],
                            scale=s["scale"], workspace=s["ws"])
        return s["acc_out"]
    E.dsa_cache_evict(s["acc"], s["table"], s["kv_lens"], s["new_lens"],
                      [(s["k"], s["k"]), (s["v"], s["v"]), (s["acc"], s["acc_out"]), (s["pos"], s["pos_out"])],
                      s["out_src"], pos=s["pos"], seen_lens=s["seen"], prefix=s["prefix"], window=s["window"],
                      workspace=s["ws"])
    return s["out_src"], s["k"], s["v"], s["acc_out"], s["pos_out"]


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    kl = _lens(case["kv_lens"])
    if case["op"] == "evict":
        # every accumulated weight and position read once to choose, the kept ones written; the
        # keys that change place are at least those a random choice leaves behind the new end
        nl = _lens(case["new_lens"])
        row = case["kv_heads"] * case["d"] * 4
        moved = sum(n * (k - n) / k for k, n in zip(kl, nl))
        return {"bytes": int(8 * sum(kl) + 12 * sum(nl) + 2 * row * moved), "flops": 2 * sum(kl)}
    ql = _lens(case["q_lens"])
    d, hk = case["d"], case["kv_heads"]
    size = 4 if case.get("dtype") == "f32" else 2
    packed = d // 2 + d // 32
    if case["op"] == "append":
        # read in the input's type, written in 4 bits, read back, returned in fp32
        return {"bytes": sum(ql) * hk * 2 * (d * size + 2 * packed + 4 * d), "flops": sum(ql) * hk * 2 * d * 4}
    h = case["heads"]
    pairs = sum(q * (k - q) + q * (q + 1) // 2 for q, k in zip(ql, kl))
    if case["op"] == "prompt":
        return {"bytes": sum(ql) * h * (2 * d * size + 4) + sum(kl) * hk * d * 2 * size, "flops": 4 * pairs * h * d}
    if case["op"] == "weights":
        return {"bytes": sum(ql) * h * (d * size + 4) + sum(kl) * (hk * packed + 8), "flops": 2 * pairs * h * d}
    keys = sum(kl)
    if case["topk"]:
        pairs = keys = sum(min(case["topk"], k - q + i + 1) for q, k in zip(ql, kl) for i in range(q))
    return {"bytes": sum(ql) * h * (2 * d * size + 4) + keys * hk * 2 * packed + (4 * keys if case["topk"] else 0),
            "flops": 4 * pairs * h * d}


# ----------------------------------------------------------------------------
# the definition in 64 bits
# ----------------------------------------------------------------------------
def _values(codes, scales):
    """The 64-bit values of stored 4-bit rows, from the bits: sign, exponent, one mantissa bit."""
    nib = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    e, m = (nib >> 1) & 3, (nib & 1).double()
    mag = torch.where(e == 0, m * 0.5, (1.0 + 0.5 * m) * torch.pow(2.0, (e - 1).double()))
    mag = torch.where(nib >= 8, -mag, mag)
    return mag * torch.pow(2.0, scales.double() - 127.0).repeat_interleave(32, -1)


def _nearest(x):
    """64-bit values of rows after the 4-bit rounding: the nearest multiple within each binade."""
    y = x.double().unflatten(-1, (-1, 32))
    amax = y.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(amax.clamp(min=2.0 ** -126) / 7.0)) - 1.0
    for _ in range(3):
        e = torch.where(amax >= 7.0 * torch.pow(2.0, e), e + 1.0, e)
    e = e.clamp(-126.0, 127.0)
    a = y / torch.pow(2.0, e)
    step = torch.where(a.abs() < 2.0, 0.5, torch.where(a.abs() < 4.0, 1.0, 2.0)).double()
    r = (torch.round(a / step) * step).clamp(-6.0, 6.0)     # round: ties to even multiples
    return (r * torch.pow(2.0, e)).flatten(-2)


def _attention64(q, k, v, scale, first):
    """q [n, h, d] at positions first.., k/v [m, hk, d] in 64 bits: output [n, h, d] and lse [n, h]."""
    n, h, d = q.shape
    hk = k.shape[1]
    out, lse = torch.empty(n, h, d, dtype=torch.float64, device=q.device), torch.empty(n, h, dtype=torch.float64, device=q.device)
    for i in range(h):
        kk, vv = k[:, i * hk // h].double(), v[:, i * hk // h].double()
        for a in range(0, n, 2048):
            e = min(n, a + 2048)
            m = min(kk.shape[0], first + e)
            logit = (q[a:e, i].double() @ kk[:m].T.contiguous()) * scale
            late = torch.arange(m, device=q.device) > first + torch.arange(a, e, device=q.device).unsqueeze(1)
            logit[late] = float("-inf")
            l = torch.logsumexp(logit, 1)
            lse[a:e, i] = l
            out[a:e, i] = torch.exp(logit - l.unsqueeze(1)) @ vv[:m]
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    ql, kl = s.get("q_lens"), s["kv_lens"]
    if op == "append":
        return _nearest(s["k"]), _nearest(s["v"])
    if op == "prompt":
        outs, at = [], 0
        for q, b, n in zip(s["q"].split(ql), range(len(kl)), kl):
            outs.append(_attention64(q, s["k"][at:at + n], s["v"][at:at + n], s["scale"], n - ql[b]))
            at += n
        return torch.cat([o for o, _ in outs]), torch.cat([l for _, l in outs])
    page = s["page"]
    where = [torch.cat([torch.arange(page, device=DEV) + int(p) * page for p in s["table"][b, :-(-n // page)].tolist()])[:n]
             for b, n in enumerate(kl)]
    if op == "attend":
        outs, row = [], 0
        for b, n in enumerate(kl):
            def pool(which, at):
                return _values(s[which + "_codes"].view(-1, s["kv_heads"], s["d"] // 2)[at],
                               s[which + "_scales"].view(-1, s["kv_heads"], s["d"] // 32)[at])
            if s["idx"] is None:
                outs.append(_attention64(s["q"][row:row + ql[b]], pool("k", where[b]), pool("v", where[b]), s["scale"], n - ql[b]))
            else:
                for i in range(row, row + ql[b]):
                    pick = s["idx"][i]
                    pick = where[b][pick[pick >= 0].long()]
                    outs.append(_attention64(s["q"][i:i + 1], pool("k", pick), pool("v", pick), s["scale"], pick.numel()))
            row += ql[b]
        return torch.cat([o for o, _ in outs]), torch.cat([l for _, l in outs])
    if op == "weights":
        out = torch.zeros(s["acc_out"].shape, dtype=torch.float64, device=DEV)
        row = 0
        for b, n in enumerate(kl):
            k = _values(s["k_codes"].view(-1, s["kv_heads"], s["d"] // 2)[where[b]],
                        s["k_scales"].view(-1, s["kv_heads"], s["d"] // 32)[where[b]])
            got = s["acc"].view(-1)[where[b]].double()
            got[n - ql[b]:] = 0
            for i in range(s["heads"]):
                kk = k[:, i * s["kv_heads"] // s["heads"]].T.contiguous()
                for a in range(row, row + ql[b], 1024):
                    e = min(row + ql[b], a + 1024)
                    w = torch.exp((s["q"][a:e, i].double() @ kk) * s["scale"] - s["lse"][a:e, i].double().unsqueeze(1))
                    seen = torch.arange(a - row, e - row, device=DEV).unsqueeze(1) + (n - ql[b])
                    got += torch.where(torch.arange(n, device=DEV) <= seen, w, torch.zeros_like(w)).sum(0)
            out.view(-1)[where[b]] = got
            row += ql[b]
        return out
    src = torch.full_like(s["out_src"], -1)
    k, v = s["k"].clone().flatten(0, 1), s["v"].clone().flatten(0, 1)
    acc, pos = torch.zeros_like(s["acc"]).view(-1), torch.zeros_like(s["pos"]).view(-1)
    for b, (n, keep) in enumerate(zip(kl, s["new_lens"])):
        w = s["acc"].view(-1)[where[b]].double().tolist()
        p = s["pos"].view(-1)[where[b]].tolist()
        big = [x < s["prefix"] or x >= s["seen"][b] - s["window"] for x in p]
        order = sorted(range(n), key=lambda i: (not big[i], 0.0 if big[i] else -w[i], i))[:keep]
        stay = set(order)
        late = iter(sorted(i for i in order if i >= keep))
        take = torch.tensor([i if i in stay else next(late) for i in range(keep)], device=DEV)
        src[b, :keep] = take.int()
        k[where[b][:keep]] = k[where[b][take]]
        v[where[b][:keep]] = v[where[b][take]]
        acc[where[b][:keep]] = s["acc"].view(-1)[where[b][take]]
        pos[where[b][:keep]] = s["pos"].view(-1)[where[b][take]]
    return src, k.view_as(s["k"]), v.view_as(s["v"]), acc.view_as(s["acc_out"]), pos.view_as(s["pos_out"])
