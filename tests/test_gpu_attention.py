"""The attention entry points on the GPU against their float64 definitions."""
import numpy as np
import pytest
import torch

import exact_top_token_amd as E
from attention_helpers import U, check_attention, filled_cache, rows, table, weight_err
from oracle import attention as A

pytestmark = pytest.mark.gpu


def say(*a):
    print("[gpu]", *a, flush=True)


def host(t):
    return t.float().cpu().numpy()


def space(n):
    """A workspace of exactly n bytes, full of NaN bytes."""
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")


# ----------------------------------------------------------------------------
# prompt attention
# ----------------------------------------------------------------------------
def run_prompt(q, k, v, ql, kl, scale=None, want_lse=True):
    out = torch.full((q.shape[0], q.shape[1], q.shape[2]), float("nan"), dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], float("nan"), device="cuda") if want_lse else None
    ws = space(E.prompt_workspace_size(ql, kl, q.shape[1], k.shape[1], q.shape[2], q.dtype))
    E.dsa_prompt_attention(q, k, v, ql, kl, out, lse, scale=scale, workspace=ws)
    torch.cuda.synchronize()
    return out, lse


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hk,ql,kl", [
    (1, 1, [1], [1]),
    (4, 2, [0, 3, 0], [0, 3, 5]),
    (8, 8, [15, 16, 17], [15, 16, 17]),
    (6, 2, [33, 1, 64, 65], [33, 40, 64, 130]),
    (16, 1, [2, 1, 5], [129, 63, 300]),
    (5, 5, [128, 127], [128, 255]),
    (12, 3, [1, 1, 1, 1], [1, 64, 65, 500]),
])
def test_prompt(dtype, d, hq, hk, ql, kl):
    say("prompt", dtype, d, hq, hk, ql, kl)
    rng = np.random.default_rng(hq * 100 + d)
    q, k, v = (rows(rng, n, h, d, dtype) for n, h in ((sum(ql), hq), (sum(kl), hk), (sum(kl), hk)))
    out, lse = run_prompt(q.cuda(), k.cuda(), v.cuda(), ql, kl)
    ref = A.prompt(host(q), host(k), host(v), ql, kl, d ** -0.5)
    check_attention(out, lse, ref, d, max(kl), dtype == "bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompt_long_chunks(dtype):
    """Few rows over many keys (ranges joined) next to many rows over few."""
    rng = np.random.default_rng(5)
    ql, kl = [2, 130, 1], [9000, 200, 4097]
    q, k, v = (rows(rng, n, h, 128, dtype) for n, h in ((sum(ql), 4), (sum(kl), 2), (sum(kl), 2)))
    say("prompt chunks", dtype)
    out, lse = run_prompt(q.cuda(), k.cuda(), v.cuda(), ql, kl, scale=0.3)
    check_attention(out, lse, A.prompt(host(q), host(k), host(v), ql, kl, 0.3), 128, max(kl), dtype == "bf16")


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_chunks_with_joined_ranges(d):
    """Chunks of more than 16 rows over long keys: the tiled kernel's key ranges joined, row tiles that end
    inside it, key counts off its tiles, next to sequences of the other kernel."""
    rng = np.random.default_rng(50 + d)
    ql, kl = [20, 100, 3, 9], [3001, 4999, 700, 520]
    q, k, v = (rows(rng, n, h, d, "bf16") for n, h in ((sum(ql), 6), (sum(kl), 2), (sum(kl), 2)))
    say("prompt joined ranges", d)
    out, lse = run_prompt(q.cuda(), k.cuda(), v.cuda(), ql, kl)
    check_attention(out, lse, A.prompt(host(q), host(k), host(v), ql, kl, d ** -0.5), d, max(kl), True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_strided_operands(dtype, d):
    """q, k, v as slices of one fused projection; outputs next to guards."""
    rng = np.random.default_rng(6)
    hq, hk, ql = 6, 2, [70, 9, 150]
    n = sum(ql)
    fused = rows(rng, n, hq + 2 * hk + 1, d, dtype).cuda()
    q, k, v = fused[:, :hq], fused[:, hq:hq + hk], fused[:, hq + hk:hq + 2 * hk]
    say("prompt strided", dtype, d)
    guard = torch.full((n + 2, hq, d), 7.0, dtype=q.dtype, device="cuda")
    ws = space(E.prompt_workspace_size(ql, ql, hq, hk, d, q.dtype))
    E.dsa_prompt_attention(q, k, v, ql, ql, guard[1:-1], None, workspace=ws)
    torch.cuda.synchronize()
    assert torch.all(guard[0] == 7) and torch.all(guard[-1] == 7)
    check_attention(guard[1:-1], None, A.prompt(host(q), host(k), host(v), ql, ql, d ** -0.5), d, max(ql), dtype == "bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompt_large_scores(dtype):
    """Scores in the hundreds and equal maxima: the running maximum moves, weights underflow."""
    rng = np.random.default_rng(7)
    ql = [200, 96]
    q, k, v = (rows(rng, sum(ql), h, 64, dtype) * f for h, f in ((4, 8), (2, 8), (2, 1)))
    k[100:] = k[100]
    k[:50] *= -1
    say("prompt large scores", dtype)
    out, lse = run_prompt(q.cuda(), k.cuda(), v.cuda(), ql, ql, scale=1.0)
    check_attention(out, lse, A.prompt(host(q), host(k), host(v), ql, ql, 1.0), 64, 200, dtype == "bf16")


def test_prompt_many_sequences():
    """More sequences than one launch takes, some of them empty."""
    rng = np.random.default_rng(8)
    kl = [int(x) for x in rng.integers(0, 40, 150)]
    ql = [int(rng.integers(0, k + 1)) for k in kl]
    for dtype in ("f32", "bf16"):
        q, k, v = (rows(rng, n, h, 64, dtype) for n, h in ((sum(ql), 4), (sum(kl), 2), (sum(kl), 2)))
        say("prompt many", dtype)
        out, lse = run_prompt(q.cuda(), k.cuda(), v.cuda(), ql, kl)
        check_attention(out, lse, A.prompt(host(q), host(k), host(v), ql, kl, 0.125), 64, 40, dtype == "bf16")


# ----------------------------------------------------------------------------
# cache write and read-back
# ----------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hk,page,ql,kl", [
    (1, 16, [1], [1]),
    (2, 64, [2, 0, 33], [2, 9, 100]),
    (3, 48, [17, 50], [40, 50]),
    (8, 128, [129, 1], [300, 7]),
    (40, 16, [5], [20]),
])
def test_append_and_read(dtype, d, hk, page, ql, kl):
    rng = np.random.default_rng(hk)
    t, pages = table(rng, kl, page)
    n = sum(ql)
    x = {w: rows(rng, n, hk + 1, d, dtype, loud=True) * torch.exp(4 * torch.from_numpy(rng.normal(size=(n, 1, 1)))).to(torch.float32)
         for w in "kv"}
    x = {w: y.to(torch.bfloat16 if dtype == "bf16" else torch.float32) for w, y in x.items()}
    x["k"][0, 0] = 0
    c = E.Cache.empty(pages, page, hk, d, torch.from_numpy(t).cuda())
    for b in (c.k_codes, c.k_scales, c.v_codes, c.v_scales):
        b.fill_(0xA5)
    pos = torch.full((pages, page), -9, dtype=torch.int32, device="cuda")
    seen = [k + 1000 * (i + 1) for i, k in enumerate(kl)]
    say("append", dtype, d, hk, page, ql, kl)
    g = {w: y.cuda()[:, :hk] for w, y in x.items()}      # strided rows
    E.dsa_cache_append(c, g["k"], g["v"], ql, kl, pos=pos, seen_lens=seen)
    back = {w: torch.empty(n, hk, d, dtype=x[w].dtype, device="cuda") for w in "kv"}
    E.dsa_cache_read(c, back["k"], back["v"], ql, kl)
    wide = {w: torch.full((n, hk + 2, d), 5.0, device="cuda") for w in "kv"}
    E.dsa_cache_read(c, wide["k"][:, 1:-1], wide["v"][:, 1:-1], ql, kl)
    torch.cuda.synchronize()
    at = np.concatenate([A.slots(t, b, kl[b], page, pages)[kl[b] - ql[b]:] for b in range(len(kl))])
    for w in "kv":
        codes, scales = A.mx_encode(host(x[w])[:, :hk])
        want_c = np.full((pages * page, hk, d // 2), 0xA5, np.uint8)
        want_s = np.full((pages * page, hk, d // 32), 0xA5, np.uint8)
        want_c[at], want_s[at] = codes, scales
        assert np.array_equal(getattr(c, w + "_codes").cpu().numpy().reshape(want_c.shape), want_c)
        assert np.array_equal(getattr(c, w + "_scales").cpu().numpy().reshape(want_s.shape), want_s)
        val = A.mx_decode(codes, scales)
        assert np.array_equal(host(back[w]), val)
        assert np.array_equal(host(wide[w])[:, 1:-1], val)
        assert torch.all(wide[w][:, 0] == 5) and torch.all(wide[w][:, -1] == 5)
    p = np.full(pages * page, -9)
    p[at] = np.concatenate([np.arange(s - q, s) for s, q in zip(seen, ql)])
    assert np.array_equal(pos.cpu().numpy().reshape(-1), p)


def test_append_borders():
    """Every border between two codes and its neighbours, at scales over the whole range."""
    edges = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 0.0], np.float32)
    v = np.concatenate([edges, np.nextafter(edges, np.float32(9)), np.nextafter(edges, np.float32(-9))])
    v = np.concatenate([v, -v])
    blocks = []
    for e in (-126, -120, -60, -1, 0, 5, 60, 120):
        for i in range(0, len(v), 31):
            blk = np.zeros(32, np.float32)
            part = v[i:i + 31]
            blk[:len(part)] = part
            blk[31] = 4.0            # fixes the scale at 2^e
            blocks.append(np.ldexp(blk, e).astype(np.float32))
    for top in (7.0, np.nextafter(np.float32(7), np.float32(0)), 3.5, np.nextafter(np.float32(3.5), np.float32(0)), 1e-44, 1e-40):
        blocks.append(np.array([top] + [0.0] * 31, np.float32))
    while len(blocks) % 2:
        blocks.append(np.zeros(32, np.float32))
    x = np.stack(blocks).reshape(-1, 1, 64)
    n = len(x)
    t = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    c = E.Cache.empty(1, -(-n // 16) * 16, 1, 64, t)
    g = torch.from_numpy(x).cuda()
    say("append borders")
    E.dsa_cache_append(c, g, -g, [n], [n])
    torch.cuda.synchronize()
    for w, y in (("k", x), ("v", -x)):
        codes, scales = A.mx_encode(y)
        assert np.array_equal(getattr(c, w + "_scales").cpu().numpy().reshape(-1, 1, 2)[:n], scales)
        got = getattr(c, w + "_codes").cpu().numpy().reshape(-1, 1, 32)[:n]
        assert np.array_equal(A.mx_decode(got, scales), A.mx_decode(codes, scales))


def test_append_pages_that_do_not_exist():
    kl, ql, page = [70, 40], [70, 40], 16
    rng = np.random.default_rng(3)
    t, pages = table(rng, kl, page)
    t[0, 2], t[1, 0] = -1, pages
    c = E.Cache.empty(pages, page, 2, 64, torch.from_numpy(t).cuda())
    for b in (c.k_codes, c.k_scales, c.v_codes, c.v_scales):
        b.fill_(0x11)
    x = rows(rng, 110, 2, 64, "bf16").cuda()
    pos = torch.full((pages, page), -9, dtype=torch.int32, device="cuda")
    say("append bad pages")
    E.dsa_cache_append(c, x, x, ql, kl, pos=pos)
    k, v = torch.full_like(x, 9.0), torch.full_like(x, 9.0)
    E.dsa_cache_read(c, k, v, ql, kl)
    torch.cuda.synchronize()
    gone = np.concatenate([A.slots(t, b, kl[b], page, pages) < 0 for b in range(2)])
    want = A.mx_decode(*A.mx_encode(host(x)))
    want[gone] = 0
    assert np.array_equal(host(k), want) and np.array_equal(host(v), want)
    assert int((pos == -9).sum()) == pages * page - int((~gone).sum())


# ----------------------------------------------------------------------------
# attention over the cache
# ----------------------------------------------------------------------------
def run_cache(c, q, ql, kl, idx=None, scale=None):
    out = torch.full(tuple(q.shape), float("nan"), dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], float("nan"), device="cuda")
    ws = space(E.cache_workspace_size(ql, kl, q.shape[1], c.Hkv, c.d, 0 if idx is None else idx.shape[1]))
    E.dsa_cache_attention(c, q, ql, kl, out, lse, idx=idx, scale=scale, workspace=ws)
    torch.cuda.synchronize()
    return out, lse


CACHE_SHAPES = [
    (1, 1, 16, [1], [1]),
    (4, 2, 64, [1, 0, 2], [63, 5, 65]),
    (16, 2, 64, [2, 2, 1], [130, 64, 700]),
    (6, 3, 48, [3, 1], [200, 47]),
    (40, 8, 128, [1, 4], [129, 256]),
    (64, 1, 256, [1, 2], [300, 10]),
    (8, 4, 16, [17, 40], [50, 40]),
    (15, 5, 64, [9], [500]),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hk,page,ql,kl", CACHE_SHAPES)
def test_cache_attention(dtype, d, hq, hk, page, ql, kl):
    rng = np.random.default_rng(hq + page)
    c, h = filled_cache(rng, kl, page, hk, d)
    q = rows(rng, sum(ql), hq, d, dtype)
    say("cache attention", dtype, d, hq, hk, page, ql, kl)
    out, lse = run_cache(c, q.cuda(), ql, kl)
    check_attention(out, lse, A.cache_attention(host(q), h, ql, kl, d ** -0.5), d, max(kl), dtype == "bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("page", [64, 80])
def test_cache_attention_long(dtype, page):
    """Long caches: many joined key ranges."""
    rng = np.random.default_rng(2)
    ql, kl = [1, 2], [20011, 4097]
    c, h = filled_cache(rng, kl, page, 2, 128)
    q = rows(rng, 3, 6, 128, dtype)
    say("cache attention long", dtype, page)
    out, lse = run_cache(c, q.cuda(), ql, kl)
    check_attention(out, lse, A.cache_attention(host(q), h, ql, kl, 128 ** -0.5), 128, max(kl), dtype == "bf16")


@pytest.mark.parametrize("page", [16, 64])
def test_cache_attention_pages_that_do_not_exist(page):
    """Keys of a bad table entry are not seen; a row all of whose keys are gone is empty."""
    rng = np.random.default_rng(4)
    ql, kl = [2, 1, 3], [300, 60, 129]
    c, h = filled_cache(rng, kl, page, 2, 64)
    t = h["table"].copy()
    t[0, 1], t[0, -1], t[1, :], t[2, 0] = -1, -5, 1 << 20, c.num_pages
    h["table"] = t
    c = E.Cache(c.k_codes, c.k_scales, c.v_codes, c.v_scales, torch.from_numpy(t).cuda())
    for dtype in ("f32", "bf16"):
        q = rows(rng, 6, 4, 64, dtype)
        say("cache attention bad pages", page, dtype)
        out, lse = run_cache(c, q.cuda(), ql, kl)
        ref = A.cache_attention(host(q), h, ql, kl, 0.125)
        assert np.all(~np.isfinite(ref[1][2])) and np.all(np.isfinite(ref[1][0]))
        check_attention(out, lse, ref, 64, 300, dtype == "bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hk,page,topk,ql,kl", [
    (4, 2, 64, 1, [1, 2], [30, 5]),
    (16, 2, 64, 37, [2, 0, 3], [100, 9, 30]),
    (8, 8, 16, 64, [1, 1], [65, 64]),
    (40, 1, 48, 130, [2], [400]),
    (6, 2, 64, 900, [3, 1], [1200, 40]),
])
def test_cache_attention_selected(dtype, d, hq, hk, page, topk, ql, kl):
    rng = np.random.default_rng(topk)
    c, h = filled_cache(rng, kl, page, hk, d)
    q = rows(rng, sum(ql), hq, d, dtype)
    idx = np.full((sum(ql), topk), -1, np.int32)
    r = 0
    for b in range(len(ql)):
        for i in range(ql[b]):
            see = kl[b] - ql[b] + i + 1
            n = min(see, topk)
            idx[r, :n] = rng.permutation(see)[:n]
            idx[r] = idx[r][rng.permutation(topk)]        # -1 anywhere
            r += 1
    say("cache attention selected", dtype, d, hq, hk, page, topk, ql, kl)
    out, lse = run_cache(c, q.cuda(), ql, kl, torch.from_numpy(idx).cuda())
    check_attention(out, lse, A.cache_attention(host(q), h, ql, kl, d ** -0.5, idx), d, topk, dtype == "bf16")


def test_cache_attention_selected_oddities():
    """Entries past the query, far outside, repeated, and rows of nothing."""
    rng = np.random.default_rng(9)
    ql, kl = [3, 2], [90, 20]
    c, h = filled_cache(rng, kl, 16, 2, 64)
    h["table"][1, 1] = -3
    c = E.Cache(c.k_codes, c.k_scales, c.v_codes, c.v_scales, torch.from_numpy(h["table"]).cuda())
    idx = rng.integers(-5, 200, (5, 100)).astype(np.int32)
    idx[0] = -1
    idx[1, ::2], idx[1, 1::2] = 2 ** 31 - 1, -2 ** 31
    idx[2] = 7
    idx[3] = 17        # in the page that does not exist
    for dtype in ("f32", "bf16"):
        q = rows(rng, 5, 4, 64, dtype)
        say("cache attention selected oddities", dtype)
        out, lse = run_cache(c, q.cuda(), ql, kl, torch.from_numpy(idx).cuda())
        ref = A.cache_attention(host(q), h, ql, kl, 0.125, idx)
        assert np.all(~np.isfinite(ref[1][[0, 1, 3]]))
        check_attention(out, lse, ref, 64, 100, dtype == "bf16")


def test_cache_attention_many_sequences():
    rng = np.random.default_rng(10)
    kl = [int(x) for x in rng.integers(1, 90, 140)]
    ql = [int(rng.integers(0, min(k, 3) + 1)) for k in kl]
    c, h = filled_cache(rng, kl, 16, 2, 64)
    q = rows(rng, sum(ql), 4, 64, "bf16")
    say("cache attention many")
    out, lse = run_cache(c, q.cuda(), ql, kl)
    check_attention(out, lse, A.cache_attention(host(q), h, ql, kl, 0.125), 64, 90, True)


# ----------------------------------------------------------------------------
# accumulated weights
# ----------------------------------------------------------------------------
def check_weights(c, h, q, ql, kl, dtype, acc_mode):
    rng = np.random.default_rng(1)
    d, H = q.shape[2], q.shape[1]
    ref = A.cache_attention(host(q), h, ql, kl, d ** -0.5)
    lse = torch.from_numpy(ref[1].astype(np.float32)).cuda()
    shape = (c.num_pages, c.page_size)
    acc = None if acc_mode == "none" else torch.from_numpy(rng.random(shape).astype(np.float32)).cuda()
    out = acc if acc_mode == "in place" else torch.full(shape, 3.0, device="cuda")
    first = out.cpu().numpy().copy()
    old = None if acc is None else acc.cpu().numpy().copy()
    ws = space(E.weights_workspace_size(ql, kl, H, c.Hkv, d))
    E.dsa_cache_weights(c, q.cuda(), lse, ql, kl, acc, out, workspace=ws)
    torch.cuda.synchronize()
    want = A.accumulate(h, ref[4], ql, kl, old, first)
    # each weight off by its own error and lse's rounding; up to q_len * H of them summed
    e = float((weight_err(ref[3], ref[1], d, 0) + 2 * U * np.abs(np.where(np.isfinite(ref[1]), ref[1], 0))).max())
    n = max(ql) * H
    got = out.cpu().numpy().astype(np.float64)
    tol = (np.abs(want) + 1e-30) * (e + (n + 4) * U)
    assert np.all(np.abs(got - want) <= tol), float((np.abs(got - want) - tol).max())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hk,page,ql,kl", CACHE_SHAPES)
def test_weights(dtype, d, hq, hk, page, ql, kl):
    rng = np.random.default_rng(hq + page)
    c, h = filled_cache(rng, kl, page, hk, d)
    q = rows(rng, sum(ql), hq, d, dtype)
    say("weights", dtype, d, hq, hk, page, ql, kl)
    check_weights(c, h, q, ql, kl, dtype, {0: "none", 1: "in place", 2: "other"}[(hq + d // 64) % 3])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_weights_prompt(dtype):
    """Whole prompts: many row tiles shared by several workgroups."""
    rng = np.random.default_rng(11)
    ql, kl = [300, 77], [300, 200]
    c, h = filled_cache(rng, kl, 64, 2, 64)
    q = rows(rng, sum(ql), 8, 64, dtype)
    say("weights prompt", dtype)
    check_weights(c, h, q, ql, kl, dtype, "other")


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 64)])
def test_weights_prompt_chunks(dtype, d):
    """Several 512-key chunks, row shares that a chunk's first rows leave empty, odd groups."""
    rng = np.random.default_rng(60 + d)
    ql, kl = [600, 40], [1300, 520]
    c, h = filled_cache(rng, kl, 48 if d == 64 else 64, 2, d)
    q = rows(rng, sum(ql), 6, d, dtype)
    say("weights prompt chunks", dtype, d)
    check_weights(c, h, q, ql, kl, dtype, "in place")


def test_weights_bad_pages_and_empty_rows():
    rng = np.random.default_rng(12)
    ql, kl = [2, 1], [150, 30]
    c, h = filled_cache(rng, kl, 64, 2, 64)
    h["table"][0, 0], h["table"][1, 0] = -1, c.num_pages + 3
    c = E.Cache(c.k_codes, c.k_scales, c.v_codes, c.v_scales, torch.from_numpy(h["table"]).cuda())
    say("weights bad pages")
    check_weights(c, h, rows(rng, 3, 4, 64, "bf16"), ql, kl, "bf16", "other")


def test_weights_many_sequences():
    rng = np.random.default_rng(13)
    kl = [int(x) for x in rng.integers(1, 90, 140)]
    ql = [int(rng.integers(0, min(k, 3) + 1)) for k in kl]
    c, h = filled_cache(rng, kl, 16, 2, 64)
    say("weights many")
    check_weights(c, h, rows(rng, sum(ql), 4, 64, "bf16"), ql, kl, "bf16", "in place")


# ----------------------------------------------------------------------------
# eviction
# ----------------------------------------------------------------------------
def check_evict(kl, nl, page, prefix=0, window=0, moved=False, values="distinct", seed=0, stride=None):
    rng = np.random.default_rng(seed)
    t, pages = table(rng, kl, page)
    acc = np.full((pages, page), 1e9, np.float32)
    pos = np.zeros((pages, page), np.int32)
    seen = [k + (50 * k if moved else 0) for k in kl]
    at = [A.slots(t, b, n, page, pages) for b, n in enumerate(kl)]
    for b, n in enumerate(kl):
        a = {"distinct": rng.random(n), "ties": rng.integers(0, 3, n) / 4, "same": np.zeros(n),
             "signs": rng.choice([0.0, -0.0, -1.5, 2.0, np.inf, -np.inf, 1e-42], n)}[values]
        acc.reshape(-1)[at[b]] = a
        pos.reshape(-1)[at[b]] = rng.permutation(seen[b])[:n] if moved else np.arange(n)
    codes = rng.integers(0, 256, (pages, page, 3, 32)).astype(np.uint8)          # 96-byte rows
    odd = rng.integers(0, 256, (pages, page, 7)).astype(np.uint8)
    g = [torch.from_numpy(x.copy()).cuda() for x in (acc, pos, codes, odd)]
    acc_o, odd_o = torch.full_like(g[0], -2.0), torch.full_like(g[3], 9)
    width = max(nl, default=0) + (3 if stride is None else stride)
    out = torch.full((len(kl), width), 77, dtype=torch.int32, device="cuda")
    ws = space(E.evict_workspace_size(kl, nl))
    say("evict", kl[:4], nl[:4], page, prefix, window, moved, values)
    E.dsa_cache_evict(g[0], torch.from_numpy(t).cuda(), kl, nl,
                      [(g[0], acc_o), (g[1], g[1]), (g[2], g[2]), (g[3], odd_o)], out,
                      pos=g[1] if moved else None, seen_lens=seen if moved else None, prefix=prefix, window=window,
                      workspace=ws)
    torch.cuda.synchronize()
    want_out = np.full((len(kl), width), -1)
    acc_w, odd_w, pos_w, codes_w = np.full_like(acc, -2).reshape(-1), np.full_like(odd, 9).reshape(-1, 7), pos.copy().reshape(-1), codes.copy().reshape(-1, 3, 32)
    for b, (n, k) in enumerate(zip(kl, nl)):
        src = A.evict(acc.reshape(-1)[at[b]], n, k, prefix, window, pos.reshape(-1)[at[b]] if moved else None, seen[b])
        want_out[b, :k] = src
        to, frm = at[b][:k], at[b][src]
        acc_w[to], odd_w[to] = acc.reshape(-1)[frm], odd.reshape(-1, 7)[frm]
        pos_w[to], codes_w[to] = pos.reshape(-1)[frm], codes.reshape(-1, 3, 32)[frm]
    assert np.array_equal(out.cpu().numpy(), want_out)
    assert np.array_equal(acc_o.cpu().numpy().reshape(-1), acc_w)
    assert np.array_equal(odd_o.cpu().numpy().reshape(-1, 7), odd_w)
    assert np.array_equal(g[1].cpu().numpy().reshape(-1), pos_w)
    assert np.array_equal(g[2].cpu().numpy().reshape(-1, 3, 32), codes_w)
    assert np.array_equal(g[0].cpu().numpy(), acc)


@pytest.mark.parametrize("kl,nl,page,kw", [
    ([1], [0], 16, {}),
    ([1], [1], 16, {}),
    ([0, 5, 5], [0, 5, 0], 16, {}),
    ([100], [60], 16, dict(prefix=4, window=16)),
    ([1000, 1025, 64], [999, 513, 1], 64, {}),
    ([3000, 70], [300, 69], 48, dict(prefix=4, window=20, moved=True)),
    ([2048], [1024], 64, dict(values="ties")),
    ([1500], [700], 64, dict(values="same")),
    ([900], [450], 64, dict(values="signs")),
    ([900], [450], 64, dict(values="signs", prefix=3, window=9, moved=True)),
    ([9000], [4500], 64, dict(values="ties", prefix=1, window=100, moved=True)),
    ([70000], [4096], 128, dict(prefix=4, window=64)),
    ([66000], [65990], 128, dict(values="ties")),
    ([40], [30], 16, dict(prefix=30, window=0)),
    ([20, 40], [20, 30], 16, dict(prefix=15, window=15)),
])
def test_evict(kl, nl, page, kw):
    check_evict(kl, nl, page, **kw)


def test_evict_many_sequences():
    rng = np.random.default_rng(14)
    kl = [int(x) for x in rng.integers(0, 300, 150)]
    nl = [int(rng.integers(0, k + 1)) for k in kl]
    check_evict(kl, nl, 16)


def test_evict_very_long():
    check_evict([300000, 5], [123457, 5], 64, prefix=4, window=1000)


# ----------------------------------------------------------------------------
# shapes the kernels divide differently
# ----------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hq,hk,page,ql,kl", [
    (48, 24, 64, [1, 2], [200, 70]),       # more head pairs than wavefronts
    (22, 11, 16, [2], [150]),              # an odd number of kv heads, more than wavefronts
    (8, 2, 64, [150, 1], [400, 65]),       # a chunk of a prompt over the cache
    (24, 1, 48, [3], [210]),               # all heads on one, rows beyond one tile
])
def test_cache_attention_and_weights_of_other_shapes(dtype, hq, hk, page, ql, kl):
    rng = np.random.default_rng(hq * hk)
    for d in (64, 128):
        c, h = filled_cache(rng, kl, page, hk, d)
        q = rows(rng, sum(ql), hq, d, dtype)
        say("other shapes", dtype, d, hq, hk, page, ql, kl)
        out, lse = run_cache(c, q.cuda(), ql, kl)
        check_attention(out, lse, A.cache_attention(host(q), h, ql, kl, d ** -0.5), d, max(kl), dtype == "bf16")
        idx = rng.integers(-1, min(kl), (sum(ql), 70)).astype(np.int32)
        out, lse = run_cache(c, q.cuda(), ql, kl, torch.from_numpy(idx).cuda())
        check_attention(out, lse, A.cache_attention(host(q), h, ql, kl, d ** -0.5, idx), d, 70, dtype == "bf16")
        check_weights(c, h, q, ql, kl, dtype, "other")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_cache_calls_with_strided_queries_on_another_stream(dtype):
    """Queries as a slice of a fused projection, calls on the stream that is current."""
    rng = np.random.default_rng(70)
    ql, kl, hq, hk, d = [2, 40], [300, 100], 4, 2, 64
    c, h = filled_cache(rng, kl, 64, hk, d)
    q = rows(rng, sum(ql), hq + 3, d, dtype).cuda()[:, 1:1 + hq]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    say("strided queries", dtype)
    with torch.cuda.stream(s):
        out, lse = run_cache(c, q, ql, kl)
        ref = A.cache_attention(host(q), h, ql, kl, d ** -0.5)
        check_attention(out, lse, ref, d, max(kl), dtype == "bf16")
        acc = torch.zeros(c.num_pages, c.page_size, device="cuda")
        E.dsa_cache_weights(c, q, lse, ql, kl, None, acc, workspace=space(E.weights_workspace_size(ql, kl, hq, hk, d)))
    s.synchronize()
    want = A.accumulate(h, ref[4], ql, kl, None, np.zeros((c.num_pages, c.page_size)))
    e = float(weight_err(ref[3], ref[1], d, max(kl)).max()) * 3
    assert np.all(np.abs(acc.cpu().numpy() - want) <= (np.abs(want) + 1e-30) * (e + max(ql) * hq * U * 2))


def test_append_many_sequences():
    rng = np.random.default_rng(71)
    kl = [int(x) for x in rng.integers(0, 60, 150)]
    ql = [int(rng.integers(0, k + 1)) for k in kl]
    t, pages = table(rng, kl, 16)
    c = E.Cache.empty(pages, 16, 2, 64, torch.from_numpy(t).cuda())
    x = rows(rng, sum(ql), 2, 64, "bf16", True).cuda()
    say("append many")
    E.dsa_cache_append(c, x, x, ql, kl)
    k, v = torch.empty_like(x), torch.empty_like(x)
    E.dsa_cache_read(c, k, v, ql, kl)
    torch.cuda.synchronize()
    want = A.mx_decode(*A.mx_encode(host(x)))
    assert np.array_equal(host(k), want) and np.array_equal(host(v), want)


# ----------------------------------------------------------------------------
# offsets beyond 32 bits
# ----------------------------------------------------------------------------
@pytest.mark.parametrize("page", [64, 48])
def test_cache_slots_beyond_4_gib(page):
    """A pool of more than 4 GiB a buffer, the sequences' pages at its far end (and one at its start)."""
    rng = np.random.default_rng(30)
    hq, hk, d, kl, ql = 8, 8, 128, [200, 90], [3, 1]
    pages = (9 << 20) // page                       # 9M slots of 512 bytes
    t = np.full((2, 8), -1, np.int32)
    per = [-(-k // page) for k in kl]
    t[0, :per[0]] = pages - 1 - np.arange(per[0])
    t[1, :per[1]] = pages - 20 - np.arange(per[1])
    t[1, 0] = 0
    c = E.Cache.empty(pages, page, hk, d, torch.from_numpy(t).cuda())
    assert c.k_codes.numel() > 1 << 32
    k, v = rows(rng, sum(kl), hk, d, "bf16", True), rows(rng, sum(kl), hk, d, "bf16")
    say("4 GiB cache", page)
    E.dsa_cache_append(c, k.cuda(), v.cuda(), kl, kl)
    kb, vb = torch.empty_like(k, device="cuda"), torch.empty_like(v, device="cuda")
    E.dsa_cache_read(c, kb, vb, kl, kl)
    torch.cuda.synchronize()
    val = {n: A.mx_decode(*A.mx_encode(host(x))) for n, x in (("k", k), ("v", v))}
    assert np.array_equal(host(kb), val["k"]) and np.array_equal(host(vb), val["v"])
    # the oracle on a small pool with the same rows
    h = {}
    for n, x in (("k", k), ("v", v)):
        h[n + "_codes"], h[n + "_scales"] = (y[None] for y in A.mx_encode(host(x)))
    h["table"] = np.zeros((2, 1), np.int32)
    small = {n: np.concatenate([h[n][0][:200], np.zeros((100,) + h[n].shape[2:], np.uint8), h[n][0][200:],
                                np.zeros((210,) + h[n].shape[2:], np.uint8)]).reshape(2, 300, *h[n].shape[2:])
             for n in h if n != "table"}
    small["table"] = np.array([[0], [1]], np.int32)
    q = rows(rng, sum(ql), hq, d, "bf16")
    out, lse = run_cache(c, q.cuda(), ql, kl)
    ref = A.cache_attention(host(q), small, ql, kl, d ** -0.5)
    check_attention(out, lse, ref, d, 200, True)
    idx = torch.from_numpy(rng.integers(0, 80, (4, 64)).astype(np.int32))
    out, lse = run_cache(c, q.cuda(), ql, kl, idx.cuda())
    check_attention(out, lse, A.cache_attention(host(q), small, ql, kl, d ** -0.5, idx.numpy()), d, 64, True)
    acc = torch.zeros(pages, page, device="cuda")
    _, lse = run_cache(c, q.cuda(), ql, kl)
    E.dsa_cache_weights(c, q.cuda(), lse, ql, kl, None, acc, workspace=space(E.weights_workspace_size(ql, kl, hq, hk, d)))
    qp = rows(rng, 200, hq, d, "bf16").cuda()       # the prompts' kernel
    _, lp = run_cache(c, qp, [200, 0], kl)
    accp = torch.zeros(pages, page, device="cuda")
    E.dsa_cache_weights(c, qp, lp, [200, 0], kl, None, accp, workspace=space(E.weights_workspace_size([200, 0], kl, hq, hk, d)))
    torch.cuda.synchronize()
    for got, r, b in ((acc, ref, 0), (acc, ref, 1), (accp, A.cache_attention(host(qp), small, [200, 0], kl, d ** -0.5), 0)):
        at = A.slots(t, b, kl[b], page, pages)
        x = got.view(-1)[torch.from_numpy(at).cuda()].cpu().numpy()
        want = r[4][b].sum((1, 2))
        e = float(weight_err(r[3], r[1], d, 200).max()) + 4 * U * float(np.abs(r[1]).max())
        assert np.all(np.abs(x - want) <= want * (e + 200 * hq * U) + 1e-30)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompt_rows_beyond_2_31_elements(dtype):
    """Token strides of 2^23 elements: the last rows lie past 2^31 elements."""
    rng = np.random.default_rng(31)
    stride, n, hq, hk, d = 1 << 23, 290, 4, 2, 64
    x = torch.empty(stride * (n - 1) + (hq + 2 * hk) * d, dtype=torch.float32 if dtype == "f32" else torch.bfloat16, device="cuda")
    cut = lambda at, h: x[at:].as_strided((n, h, d), (stride, d, 1))
    q, k, v = cut(0, hq), cut(hq * d, hk), cut((hq + hk) * d, hk)
    a, b, c = rows(rng, n, hq, d, dtype), rows(rng, n, hk, d, dtype), rows(rng, n, hk, d, dtype)
    q.copy_(a), k.copy_(b), v.copy_(c)
    ql = [30, 260]
    say("far rows", dtype)
    out, lse = run_prompt(q, k, v, ql, ql)
    check_attention(out, lse, A.prompt(host(a), host(b), host(c), ql, ql, d ** -0.5), d, 260, dtype == "bf16")


# ----------------------------------------------------------------------------
# together, as a server uses them
# ----------------------------------------------------------------------------
def test_serving_run():
    """Prompt attention and the prompt's weights, decode steps over the growing cache, the indexer's
    selection read by the attention, eviction, and decoding on over the smaller cache."""
    from exact_top_token_amd.runner import Runner, to_device
    import synth

    rng = np.random.default_rng(20)
    hq, hk, d, page, kl = 8, 2, 64, 16, [150, 83]
    per = [-(-(k + 40) // page) for k in kl]
    t = np.full((2, max(per)), -1, np.int32)
    perm = rng.permutation(sum(per))
    t[0, :per[0]], t[1, :per[1]] = perm[:per[0]], perm[per[0]:]
    c = E.Cache.empty(sum(per), page, hk, d, torch.from_numpy(t).cuda())
    shape = (c.num_pages, page)
    acc, pos = torch.zeros(shape, device="cuda"), torch.zeros(shape, dtype=torch.int32, device="cuda")
    copy = lambda: dict(k_codes=c.k_codes.cpu().numpy(), k_scales=c.k_scales.cpu().numpy(),
                        v_codes=c.v_codes.cpu().numpy(), v_scales=c.v_scales.cpu().numpy(), table=t)

    def step(ql, kl, seen, idx=None):
        nq = sum(ql)
        q, k, v = rows(rng, nq, hq, d, "bf16").cuda(), rows(rng, nq, hk, d, "bf16", True).cuda(), rows(rng, nq, hk, d, "bf16").cuda()
        E.dsa_cache_append(c, k, v, ql, kl, pos=pos, seen_lens=seen)
        out, lse = run_cache(c, q, ql, kl)
        ref = A.cache_attention(host(q), copy(), ql, kl, d ** -0.5)
        check_attention(out, lse, ref, d, max(kl), True)
        before = acc.cpu().numpy()
        ws = space(E.weights_workspace_size(ql, kl, hq, hk, d))
        E.dsa_cache_weights(c, q, lse, ql, kl, acc, acc, workspace=ws)
        want = A.accumulate(copy(), ref[4], ql, kl, before, before)
        e = float(weight_err(ref[3], ref[1], d, max(kl)).max()) * 3
        assert np.all(np.abs(acc.cpu().numpy() - want) <= (np.abs(want) + 1e-30) * (e + max(ql) * hq * U * 2))
        return q, k, v

    say("serving: prompt")
    q, k, v = step(kl, kl, kl)
    out, lse = run_prompt(q, k, v, kl, kl)
    check_attention(out, lse, A.prompt(host(q), host(k), host(v), kl, kl, d ** -0.5), d, max(kl), True)
    seen = list(kl)
    for i in range(3):
        say("serving: decode", i)
        kl, seen = [k + 2 for k in kl], [s + 2 for s in seen]
        step([2, 2], kl, seen)
    # the indexer's choice, read by the attention
    wl = synth.custom(0, [(2, kl[0]), (2, kl[1])], H=8, d=64, topk=32, q_dtype="bf16", k_dtype="bf16")
    idx, _ = Runner(to_device(wl), "dosa")()
    q = rows(rng, 4, hq, d, "bf16").cuda()
    say("serving: selected")
    out, lse = run_cache(c, q, [2, 2], kl, idx)
    check_attention(out, lse, A.cache_attention(host(q), copy(), [2, 2], kl, d ** -0.5, idx.cpu().numpy()), d, 32, True)
    for new in ([96, 64], [80, 50]):
        say("serving: evict", new)
        src = torch.empty(2, 96, dtype=torch.int32, device="cuda")
        old, oldp, was = acc.cpu().numpy().reshape(-1), pos.cpu().numpy().reshape(-1), copy()
        E.dsa_cache_evict(acc, c.page_table, kl, new, c.arrays() + [(acc, acc), (pos, pos)], src, pos=pos, seen_lens=seen,
                          prefix=4, window=16, workspace=space(E.evict_workspace_size(kl, new)))
        torch.cuda.synchronize()
        for b in range(2):
            at = A.slots(t, b, kl[b], page, c.num_pages)
            want = A.evict(old[at], kl[b], new[b], 4, 16, oldp[at], seen[b])
            assert np.array_equal(src.cpu().numpy()[b, :new[b]], want)
            for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
                now = getattr(c, name).cpu().numpy()
                assert np.array_equal(now.reshape(-1, *now.shape[2:])[at[:new[b]]],
                                      was[name].reshape(-1, *now.shape[2:])[at[want]])
            assert np.array_equal(acc.cpu().numpy().reshape(-1)[at[:new[b]]], old[at[want]])
            assert np.array_equal(pos.cpu().numpy().reshape(-1)[at[:new[b]]], oldp[at[want]])
        kl = list(new)
        kl, seen = [k + 1 for k in kl], [s + 1 for s in seen]
        step([1, 1], kl, seen)


def test_captured_and_replayed():
    """A decode step captured into a graph and replayed, with eager work on other workspaces between the
    replays; a second graph shares the workspace."""
    rng = np.random.default_rng(21)
    ql, kl, hq, hk, d = [1, 2], [5000, 300], 8, 2, 128
    c, h = filled_cache(rng, kl, 64, hk, d)
    shape = (c.num_pages, c.page_size)
    need = max(E.cache_workspace_size(ql, kl, hq, hk, d), E.weights_workspace_size(ql, kl, hq, hk, d),
               E.evict_workspace_size(kl, [4000, 200]))
    ws = space(need)
    graphs = []
    say("capture")
    for _ in range(2):
        b = dict(q=torch.zeros(3, hq, d, dtype=torch.bfloat16, device="cuda"), k=torch.zeros(3, hk, d, dtype=torch.bfloat16, device="cuda"),
                 out=torch.zeros(3, hq, d, dtype=torch.bfloat16, device="cuda"), lse=torch.zeros(3, hq, device="cuda"),
                 acc=torch.zeros(shape, device="cuda"), acc2=torch.zeros(shape, device="cuda"),
                 src=torch.zeros(2, 4000, dtype=torch.int32, device="cuda"))
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            E.dsa_cache_append(c, b["k"], b["k"], ql, kl)
            E.dsa_cache_attention(c, b["q"], ql, kl, b["out"], b["lse"], workspace=ws)
            E.dsa_cache_weights(c, b["q"], b["lse"], ql, kl, b["acc"], b["acc"], workspace=ws)
            E.dsa_cache_evict(b["acc"], c.page_table, kl, [4000, 200], [(b["acc"], b["acc2"])], b["src"], prefix=4, window=8, workspace=ws)
        graphs.append((g, b))
    ws2 = space(need)
    for rep in range(3):
        for g, b in graphs:
            say("replay", rep)
            b["q"].copy_(rows(rng, 3, hq, d, "bf16"))
            b["k"].copy_(rows(rng, 3, hk, d, "bf16"))
            acc0 = b["acc"].clone()
            g.replay()
            torch.cuda.synchronize()
            got = {n: b[n].clone() for n in ("out", "lse", "acc", "acc2", "src")}
            e = {n: torch.zeros_like(x) for n, x in got.items()}
            E.dsa_cache_append(c, b["k"], b["k"], ql, kl)
            E.dsa_cache_attention(c, b["q"], ql, kl, e["out"], e["lse"], workspace=ws2)
            e["acc"].copy_(acc0)
            E.dsa_cache_weights(c, b["q"], e["lse"], ql, kl, e["acc"], e["acc"], workspace=ws2)
            E.dsa_cache_evict(e["acc"], c.page_table, kl, [4000, 200], [(e["acc"], e["acc2"])], e["src"], prefix=4, window=8, workspace=ws2)
            torch.cuda.synchronize()
            for n in ("out", "lse", "acc", "src"):
                assert torch.equal(got[n], e[n]), n
            at = torch.from_numpy(np.concatenate([A.slots(h["table"], i, n, 64, c.num_pages) for i, n in enumerate([4000, 200])])).cuda()
            assert torch.equal(got["acc2"].view(-1)[at], e["acc2"].view(-1)[at])


def test_captured_prompt():
    rng = np.random.default_rng(22)
    ql, kl = [200, 3], [200, 2000]
    for dtype in ("bf16", "f32"):
        q, k, v = (rows(rng, n, h, 64, dtype).cuda() for n, h in ((203, 4), (2200, 2), (2200, 2)))
        out, lse = torch.zeros_like(q), torch.zeros(203, 4, device="cuda")
        ws = space(E.prompt_workspace_size(ql, kl, 4, 2, 64, q.dtype))
        say("capture prompt", dtype)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            E.dsa_prompt_attention(q, k, v, ql, kl, out, lse, workspace=ws)
        for _ in range(3):
            q.copy_(rows(rng, 203, 4, 64, dtype))
            g.replay()
            torch.cuda.synchronize()
            o2, l2 = run_prompt(q, k, v, ql, kl)
            assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_two_streams_at_once():
    """Two calls in flight on two streams with a workspace each."""
    rng = np.random.default_rng(23)
    ql, kl = [1, 1], [9000, 7000]
    c, h = filled_cache(rng, kl, 64, 2, 128)
    streams = [torch.cuda.Stream() for _ in range(2)]
    qs = [rows(rng, 2, 8, 128, "bf16").cuda() for _ in range(2)]
    want = [run_cache(c, q, ql, kl) for q in qs]
    got = [(torch.zeros_like(q), torch.zeros(2, 8, device="cuda")) for q in qs]
    wss = [space(E.cache_workspace_size(ql, kl, 8, 2, 128)) for _ in qs]
    torch.cuda.synchronize()
    say("two streams")
    for _ in range(20):
        for s, q, (o, l), ws in zip(streams, qs, got, wss):
            E.dsa_cache_attention(c, q, ql, kl, o, l, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for (o, l), (o2, l2) in zip(got, want):
        assert torch.equal(o, o2) and torch.equal(l, l2)


def test_repeated_calls_agree():
    rng = np.random.default_rng(24)
    ql, kl = [1, 3], [3000, 900]
    c, h = filled_cache(rng, kl, 64, 4, 64)
    q = rows(rng, 4, 8, 64, "bf16").cuda()
    first = run_cache(c, q, ql, kl)
    acc = torch.zeros(c.num_pages, c.page_size, device="cuda")
    ws = space(E.weights_workspace_size(ql, kl, 8, 4, 64))
    E.dsa_cache_weights(c, q, first[1], ql, kl, None, acc, workspace=ws)
    say("repeat")
    for _ in range(5):
        again = run_cache(c, q, ql, kl)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
        acc2 = torch.zeros_like(acc)
        E.dsa_cache_weights(c, q, first[1], ql, kl, None, acc2, workspace=ws)
        assert torch.equal(acc, acc2)


def test_pass_times_are_reported():
    """The per-pass profile names the new passes."""
    rng = np.random.default_rng(25)
    ql, kl = [1], [3000]
    c, h = filled_cache(rng, kl, 64, 2, 64)
    q = rows(rng, 1, 4, 64, "bf16").cuda()
    run_cache(c, q, ql, kl)
    E.profile_begin()
    run_cache(c, q, ql, kl)
    t = E.profile_end()
    assert t["cache_attention"][0] == 1 and t["attention_join"][0] == 1


# ----------------------------------------------------------------------------
# table entries without a page, and a first page that holds nothing
# ----------------------------------------------------------------------------
def without_first_page(c, h):
    """The cache with its first page in no table row and full of 0xFF: its rows move to a spare page."""
    t = h["table"].copy()
    used = set(t[(t >= 0) & (t < c.num_pages)].tolist())
    spare = max(set(range(c.num_pages)) - used)
    assert spare > 0
    t[t == 0] = spare
    for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
        if 0 in used:
            h[n][spare] = h[n][0]
        h[n][0] = 0xFF
        getattr(c, n).copy_(torch.from_numpy(h[n]))
    h["table"] = t


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hk,page,ql,kl", [
    (4, 2, 16, [2, 1, 3], [300, 60, 129]),
    (4, 2, 64, [2, 1, 3], [300, 60, 129]),
    (3, 3, 64, [2, 1, 3], [300, 60, 129]),
    (4, 2, 128, [2, 1, 3], [300, 60, 129]),
    (16, 8, 64, [1] * 60, [600, 60] * 30),       # ranges longer than a page: head pairs,
    (9, 9, 64, [1] * 60, [600, 60] * 30),        # single heads,
    (16, 8, 64, [1] * 7 + [80], [600, 60] * 3 + [130, 2400]),      # two row tiles
    (9, 9, 128, [80, 1], [2400, 100]),
])
def test_cache_attention_missing_pages_next_to_an_unused_one(dtype, d, hq, hk, page, ql, kl):
    """Nothing of a page that no table entry names reaches a result, whatever its bytes: neither the rows of
    a query that sees other keys nor those of one that sees none."""
    rng = np.random.default_rng(80 + hk)
    c, h = filled_cache(rng, kl, page, hk, d)
    without_first_page(c, h)
    t = h["table"]
    for b, n in enumerate(kl):
        last = (n - 1) // page
        if b % 3 == 1:
            t[b] = -1 - b                                # every page gone
        elif last > 0:
            t[b, last // 2] = (-1, c.num_pages)[b & 1]   # one inside
            if b % 3 == 2:
                t[b, 0] = 1 << 20                        # and the first
    c = E.Cache(c.k_codes, c.k_scales, c.v_codes, c.v_scales, torch.from_numpy(t).cuda())
    q = rows(rng, sum(ql), hq, d, dtype)
    say("missing pages", dtype, d, hq, hk, page, ql[-1], kl[-1])
    out, lse = run_cache(c, q.cuda(), ql, kl)
    ref = A.cache_attention(host(q), h, ql, kl, d ** -0.5)
    assert np.any(~np.isfinite(ref[1])) and np.any(np.isfinite(ref[1]))
    check_attention(out, lse, ref, d, max(kl), dtype == "bf16")
    check_weights(c, h, q, ql, kl, dtype, "other")


@pytest.mark.parametrize("kl,nl,page,kw", [
    ([100], [60], 16, {}),
    ([200, 64, 30], [130, 40, 16], 16, dict(prefix=4, window=9)),
    ([3000, 500], [700, 480], 64, dict(prefix=4, window=40)),
    ([9000], [5000], 48, dict(prefix=1, window=100)),
    ([70000], [20000], 128, dict(prefix=4, window=64)),
])
def test_evict_without_some_pages(kl, nl, page, kw):
    """Keys move only to indices that have a page: those of largest acc are all still there afterwards."""
    rng = np.random.default_rng(sum(kl))
    t, pages = table(rng, kl, page)
    for b, n in enumerate(kl):
        for p in range(-(-n // page)):
            if p % 3 == 1:
                t[b, p] = (-1, pages)[p & 1]
    at = [A.slots(t, b, n, page, pages) for b, n in enumerate(kl)]
    acc = rng.random((pages, page)).astype(np.float32)
    rows_ = rng.integers(0, 256, (pages, page, 48)).astype(np.uint8)
    a, r = torch.from_numpy(acc.copy()).cuda(), torch.from_numpy(rows_.copy()).cuda()
    away = torch.zeros_like(r)
    out = torch.full((len(kl), max(nl)), 77, dtype=torch.int32, device="cuda")
    say("evict missing pages", kl, nl, page)
    E.dsa_cache_evict(a, torch.from_numpy(t).cuda(), kl, nl, [(r, r), (r.clone(), away), (a, a)], out,
                      workspace=space(E.evict_workspace_size(kl, nl)), **kw)
    torch.cuda.synchronize()
    pre, win = kw.get("prefix", 0), kw.get("window", 0)
    for b, (n, k) in enumerate(zip(kl, nl)):
        there = at[b] >= 0
        src = A.evict(acc.reshape(-1)[at[b]], n, k, pre, win, there=there)
        got = out.cpu().numpy()[b]
        assert np.array_equal(got[:k], src) and np.all(got[k:] == -1)
        to, frm = at[b][:k], at[b][src]
        assert np.array_equal(to < 0, frm < 0)                 # no row goes where none can be
        to, frm = to[to >= 0], frm[frm >= 0]
        assert np.array_equal(r.cpu().numpy().reshape(-1, 48)[to], rows_.reshape(-1, 48)[frm])
        assert np.array_equal(away.cpu().numpy().reshape(-1, 48)[to], rows_.reshape(-1, 48)[frm])
        # the weights that stay are the largest that the remaining places hold, protected keys first
        place = np.arange(n)
        safe = there & ((place < pre) | (place >= n - win))
        want = np.sort(np.concatenate([acc.reshape(-1)[at[b][safe]],
                                       -np.sort(-acc.reshape(-1)[at[b][there & ~safe]])[:max(len(to) - safe.sum(), 0)]]))
        if safe.sum() <= len(to):
            assert np.array_equal(np.sort(a.cpu().numpy().reshape(-1)[to]), want)


# ----------------------------------------------------------------------------
# ends of the number ranges
# ----------------------------------------------------------------------------
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ql,kl", [([2, 1], [100, 20]), ([70], [150])])
def test_cache_calls_with_the_largest_fp32_queries(d, ql, kl):
    """Queries up to the largest fp32 number over keys so small that the scores are ordinary."""
    rng = np.random.default_rng(90 + d)
    c, h = filled_cache(rng, kl, 64, 2, d)
    vis = h["k_scales"] != 0xFF
    h["k_scales"][vis] -= 64
    c.k_scales.copy_(torch.from_numpy(h["k_scales"]))
    q = rows(rng, sum(ql), 4, d, "f32") * 2.0 ** 100
    top = float(np.finfo(np.float32).max)
    q[:, :, 3], q[:, 1::2, 5] = top, -top
    scale = 2.0 ** -67
    say("largest queries", d, ql, kl)
    out, lse = run_cache(c, q.cuda(), ql, kl, scale=scale)
    ref = A.cache_attention(host(q), h, ql, kl, scale)
    assert ref[3].max() < 500
    check_attention(out, lse, ref, d, max(kl), False)
    acc = torch.zeros(c.num_pages, c.page_size, device="cuda")
    E.dsa_cache_weights(c, q.cuda(), torch.from_numpy(ref[1].astype(np.float32)).cuda(), ql, kl, None, acc, scale=scale,
                        workspace=space(E.weights_workspace_size(ql, kl, 4, 2, d)))
    torch.cuda.synchronize()
    want = A.accumulate(h, ref[4], ql, kl, None, np.zeros((c.num_pages, c.page_size)))
    e = float((weight_err(ref[3], ref[1], d, 0) + 2 * U * np.abs(ref[1])).max())
    assert np.all(np.abs(acc.cpu().numpy() - want) <= (np.abs(want) + 1e-30) * (e + (max(ql) * 4 + 4) * U))


def test_read_of_every_code_and_scale():
    """A cache that other code wrote: every scale byte in 0..254 with every code whose value is finite."""
    n, d = 256, 64
    codes = np.tile(np.arange(16, dtype=np.uint8), 4)
    scales = np.zeros((n, 1, 2), np.uint8)
    scales[:255, 0, :] = np.arange(255, dtype=np.uint8)[:, None]
    x = np.repeat(codes[None], n, 0)
    big = A.GRID[x & 7] * np.ldexp(1.0, scales[:, 0, :1].astype(int) - 127) >= 2.0 ** 128
    x[big] &= 8
    packed = (x[:, ::2] | (x[:, 1::2] << 4)).astype(np.uint8)[:, None, :]
    t = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    c = E.Cache.empty(1, n, 1, d, t)
    for w in "kv":
        getattr(c, w + "_codes").copy_(torch.from_numpy(packed[None]))
        getattr(c, w + "_scales").copy_(torch.from_numpy(scales[None]))
    want = A.mx_decode(packed, scales)
    for dtype in (torch.float32, torch.bfloat16):
        say("every code", dtype)
        k, v = (torch.empty(n, 1, d, dtype=dtype, device="cuda") for _ in "kv")
        E.dsa_cache_read(c, k, v, [n], [n])
        torch.cuda.synchronize()
        for y in (k, v):
            bad = np.argwhere(y.double().cpu().numpy() != want)
            assert len(bad) == 0, bad[:4].tolist()


def far_scores(rng, n, h, d, dtype):
    """Small whole numbers: products, their sums and 4-bit codes are exact, and equal scores occur."""
    return torch.from_numpy(rng.integers(-3, 4, (n, h, d)).astype(np.float32)).to(torch.bfloat16 if dtype == "bf16" else torch.float32)


def check_far(out, lse, ref, bf16):
    """Scores so far apart that only a row's largest count, each with the same weight: the mean of their
    values, n * U for its sum, the division and, with bf16, the rounding of the result (weights of 1 are
    exact); lse the largest score."""
    o, l, ab = ref[0], ref[1], ref[2]
    got = out.double().cpu().numpy()
    tol = (1000 * U + (1.01 * 2.0 ** -8 if bf16 else 0)) * ab
    assert np.all(np.abs(got - o) <= tol), float((np.abs(got - o) - tol).max())
    assert np.all(np.abs(lse.double().cpu().numpy() - l) <= 4 * U * np.abs(l))


@pytest.mark.parametrize("scale", [2.0 ** 20, 2.0 ** 34, 2.0 ** 100])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_of_scores_far_beyond_the_exponential(dtype, d, scale):
    """|scale q.k| up to 2^110: the largest score's weight is 1 however large it is."""
    rng = np.random.default_rng(95 + d)
    hq, hk = 4, 2
    for ql, kl in (([70, 3], [150, 600]), ([1, 2], [900, 64])):
        say("far scores", dtype, d, scale, ql)
        q, k, v = (far_scores(rng, n, h, d, dtype) for n, h in ((sum(ql), hq), (sum(kl), hk), (sum(kl), hk)))
        out, lse = run_prompt(q.cuda(), k.cuda(), v.cuda(), ql, kl, scale=scale)
        check_far(out, lse, A.prompt(host(q), host(k), host(v), ql, kl, scale), dtype == "bf16")
        for page in (64, 48):
            t, pages = table(rng, kl, page)
            c = E.Cache.empty(pages, page, hk, d, torch.from_numpy(t).cuda())
            for x in (c.k_codes, c.k_scales, c.v_codes, c.v_scales):
                x.fill_(0xFF)
            E.dsa_cache_append(c, k.cuda(), v.cuda(), kl, kl)
            h = {n: getattr(c, n).cpu().numpy() for n in ("k_codes", "k_scales", "v_codes", "v_scales")}
            h["table"] = t
            out, lse = run_cache(c, q.cuda(), ql, kl, scale=scale)
            ref = A.cache_attention(host(q), h, ql, kl, scale)
            check_far(out, lse, ref, dtype == "bf16")
            idx = rng.integers(0, min(kl), (sum(ql), 90)).astype(np.int32)
            o2, l2 = run_cache(c, q.cuda(), ql, kl, torch.from_numpy(idx).cuda(), scale=scale)
            check_far(o2, l2, A.cache_attention(host(q), h, ql, kl, scale, idx), dtype == "bf16")


@pytest.mark.parametrize("scale", [2.0 ** 20, 2.0 ** 34, 2.0 ** 100])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_weights_of_scores_far_beyond_the_exponential(dtype, d, scale):
    """With such scores a key's weight is the number of rows whose largest score is its own, since a
    normaliser of that size is the largest score itself in fp32."""
    rng = np.random.default_rng(97 + d)
    hq, hk, page = 4, 2, 64
    for ql, kl in (([70, 3], [150, 600]), ([1, 2], [900, 64])):
        say("far weights", dtype, d, scale, ql)
        q, k = far_scores(rng, sum(ql), hq, d, dtype), far_scores(rng, sum(kl), hk, d, dtype)
        t, pages = table(rng, kl, page)
        c = E.Cache.empty(pages, page, hk, d, torch.from_numpy(t).cuda())
        E.dsa_cache_append(c, k.cuda(), k.cuda(), kl, kl)
        lse, want = np.zeros((sum(ql), hq), np.float32), np.zeros((pages * page))
        r = k0 = 0
        for b in range(len(ql)):
            at = A.slots(t, b, kl[b], page, pages)
            for i in range(ql[b]):
                for h in range(hq):
                    s = host(k)[k0:k0 + kl[b] - ql[b] + i + 1, h // 2].astype(np.float64) @ host(q)[r, h].astype(np.float64)
                    lse[r, h] = s.max() * scale
                    np.add.at(want, at[:len(s)][s == s.max()], 1.0)
                r += 1
            k0 += kl[b]
        assert np.abs(lse).min() > 1e6
        acc = torch.zeros(pages, page, device="cuda")
        E.dsa_cache_weights(c, q.cuda(), torch.from_numpy(lse).cuda(), ql, kl, None, acc, scale=scale,
                            workspace=space(E.weights_workspace_size(ql, kl, hq, hk, d)))
        torch.cuda.synchronize()
        assert np.array_equal(acc.cpu().numpy().reshape(-1), want)
