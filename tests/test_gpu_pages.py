"""The entry points on paged keys and values on the GPU against their float64 definitions."""
import numpy as np
import pytest
import torch

import exact_top_token_amd as E
from attention_helpers import B, U, check_attention, rows, table, weight_err
from oracle import attention as A
from oracle import pages as P

pytestmark = pytest.mark.gpu


def say(*a):
    print("[gpu]", *a, flush=True)


def host(t):
    return t.float().cpu().numpy()


def space(n):
    """A workspace of exactly n bytes, full of NaN bytes."""
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")


def ints(x):
    return torch.tensor(np.asarray(x, np.int32), dtype=torch.int32, device="cuda")


# ----------------------------------------------------------------------------
# page tables
# ----------------------------------------------------------------------------
ASSIGN = [
    ([1], [1], 16),
    ([0, 3, 0], [0, 3, 50], 16),
    ([16, 17, 1, 1], [16, 33, 17, 48], 16),
    ([1000, 1, 64, 2], [1000, 129, 64, 5000], 64),
    ([300, 48, 49], [301, 96, 97], 48),
    ([7, 0, 260], [4096 + 7, 9, 260], 256),
]


def grow(rng, ql, kl, page, spare=2, wide=1):
    """Table before the call (the pages of the tokens before it), free list, number free, pages of the pool."""
    old = [k - q for q, k in zip(ql, kl)]
    t, used = table(rng, old, page, spare=0, extra=0)
    need = sum(-(-k // page) + (-o // page) for k, o in zip(kl, old))
    pool = used + need + spare
    full = np.full((len(kl), max(-(-k // page) for k in kl) + wide), -7, np.int32)
    full[:, :t.shape[1]] = np.where(t < used, t, -7)[:, :full.shape[1]]
    free = np.full(pool, -9, np.int32)
    free[:need + spare] = rng.permutation(need + spare) + used
    return full, free, need + spare, pool


@pytest.mark.parametrize("ql,kl,page", ASSIGN)
def test_assign_and_release(ql, kl, page):
    say("assign", ql, kl, page)
    rng = np.random.default_rng(page + len(ql))
    t, free, count, pool = grow(rng, ql, kl, page)
    want = P.assign(t, free, count, ql, kl, page, pool)
    gt, gf = ints(t), ints(free)
    n = sum(ql)
    slots, pos = ints(np.full(n + 3, -5)), ints(np.full(n + 3, -5))
    left = E.dsa_pages_assign(gt, page, gf, count, ql, kl, slots=slots[:n], positions=pos[:n])
    torch.cuda.synchronize()
    assert left == want[3]
    assert np.array_equal(gt.cpu().numpy(), want[0])
    assert np.array_equal(slots.cpu().numpy(), [*want[1], -5, -5, -5])
    assert np.array_equal(pos.cpu().numpy(), [*want[2], -5, -5, -5])
    assert np.array_equal(gf.cpu().numpy(), free)
    # again, without the maps: the same
    gt2 = ints(t)
    assert E.dsa_pages_assign(gt2, page, gf, count, ql, kl) == left
    assert torch.equal(gt, gt2)
    # and back: to the lengths before, then to nothing
    old = [k - q for q, k in zip(ql, kl)]
    for new, at in ((old, kl), ([0] * len(kl), old)):
        wt, wf, wn = P.release(gt.cpu().numpy(), gf.cpu().numpy(), left, new, at, page)
        left = E.dsa_pages_release(gt, page, gf, left, new, at)
        assert left == wn and np.array_equal(gt.cpu().numpy(), wt) and np.array_equal(gf.cpu().numpy(), wf)
    assert left == pool and sorted(gf.cpu().tolist()) == list(range(pool))


def test_assign_many_sequences():
    """More sequences than one launch takes, many without new tokens, on another stream."""
    rng = np.random.default_rng(3)
    ql = [int(x) for x in rng.integers(0, 40, 700) * rng.integers(0, 2, 700)]
    kl = [q + int(x) for q, x in zip(ql, rng.integers(0, 100, 700))]
    say("assign many")
    t, free, count, pool = grow(rng, ql, kl, 16)
    want = P.assign(t, free, count, ql, kl, 16, pool)
    gt, gf, slots, pos = ints(t), ints(free), ints(np.zeros(sum(ql))), ints(np.zeros(sum(ql)))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    left = E.dsa_pages_assign(gt, 16, gf, count, ql, kl, slots=slots, positions=pos, stream=st)
    back = E.dsa_pages_release(gt, 16, gf, left, [k - q for q, k in zip(ql, kl)], kl, stream=st)
    st.synchronize()
    assert left == want[3] and back == count
    assert np.array_equal(slots.cpu().numpy(), want[1]) and np.array_equal(pos.cpu().numpy(), want[2])
    assert np.array_equal(gf.cpu().numpy(), free)
    assert np.array_equal(gt.cpu().numpy(), np.where(t == -7, np.where(want[0] == -7, -7, -1), t))


def test_assign_of_entries_that_name_no_page():
    """A free list and a table row with entries outside the pool: kept as they are, their tokens have no slot."""
    t = np.array([[1, 99, -7, -7]], np.int32)
    free = np.array([0, -3, 50, 2], np.int32)
    say("assign bad entries")
    gt, s = ints(t), ints(np.zeros(40))
    assert E.dsa_pages_assign(gt, 16, ints(free), 4, [40], [63], slots=s) == 2
    want = P.assign(t, free, 4, [40], [63], 16, 4)
    assert np.array_equal(gt.cpu().numpy(), want[0]) and np.array_equal(s.cpu().numpy(), want[1])
    assert (s.cpu().numpy() < 0).sum() == 9 + 15


# ----------------------------------------------------------------------------
# pages
# ----------------------------------------------------------------------------
def filled(rng, kl, page, hk, d, dtype, gone=()):
    """Pages on the GPU whose visible slots hold rows and whose other slots hold NaN, and host copies; gone:
    (sequence, page) table entries that name no page."""
    t, n = table(rng, kl, page)
    for i, (b, j) in enumerate(gone):
        t[b, j] = (-1, n, 1 << 30)[i % 3]
    kv = []
    for which in "kv":
        x = torch.full((n, page, hk, d), float("nan"), dtype=torch.bfloat16 if dtype == "bf16" else torch.float32)
        for b, m in enumerate(kl):
            at = A.slots(t, b, m, page, n)
            r = rows(rng, m, hk, d, dtype, loud=True)
            x.view(-1, hk, d)[at[at >= 0]] = r[torch.from_numpy(at >= 0)]
        kv.append(x)
    return E.Pages(kv[0].cuda(), kv[1].cuda(), torch.from_numpy(t).cuda()), host(kv[0]), host(kv[1]), t


def run_pages(p, q, ql, kl, scale=None, idx=None, block=0, stream=None, want_lse=True):
    out = torch.full(tuple(q.shape), float("nan"), dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], float("nan"), device="cuda") if want_lse else None
    if idx is None:
        ws = space(E.pages_workspace_size(ql, kl, q.shape[1], p.Hkv, p.d, q.dtype))
        E.dsa_pages_attention(p, q, ql, kl, out, lse, scale=scale, workspace=ws, stream=stream)
    else:
        ws = space(E.block_workspace_size(ql, kl, q.shape[1], p.Hkv, p.d, q.dtype, block, idx.shape[2]))
        E.dsa_block_attention(p, q, ql, kl, idx, block, out, lse, scale=scale, workspace=ws, stream=stream)
    torch.cuda.synchronize()
    return out, lse


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hk,page,block,ql,kl", [
    (1, 16, 16, [1], [1]),
    (2, 32, 16, [16, 15, 17, 0, 1], [16, 15, 33, 40, 32]),
    (3, 64, 64, [64, 1, 130], [64, 128, 200]),
    (8, 128, 32, [33, 2, 1], [97, 64, 65]),
    (5, 384, 128, [127, 129, 1], [127, 400, 512]),
    (9, 48, 0, [50, 3, 16], [50, 19, 64]),
    (1, 16, 0, [1, 31], [17, 31]),
])
def test_append(dtype, d, hk, page, block, ql, kl):
    say("append", dtype, d, hk, page, block, ql, kl)
    rng = np.random.default_rng(hk * 10 + d)
    n = sum(ql)
    fused = rows(rng, n, 2 * hk + 1, d, dtype, loud=True).cuda()          # keys and values of a fused projection
    k, v = fused[:, :hk], fused[:, hk:2 * hk]
    old = [a - b for a, b in zip(kl, ql)]
    p, hkp, hvp, t = filled(rng, kl, page, hk, d, dtype)
    for b, m in enumerate(kl):                                            # the call's own slots are not written yet
        at = torch.from_numpy(A.slots(t, b, m, page, p.num_pages)[old[b]:]).cuda()
        p.k.view(-1, hk, d)[at] = p.v.view(-1, hk, d)[at] = 7.0
    wk, wv = p.k.clone(), p.v.clone()
    row = 0
    for b, (q, m) in enumerate(zip(ql, kl)):
        at = torch.from_numpy(A.slots(t, b, m, page, p.num_pages)[old[b]:]).cuda()
        wk.view(-1, hk, d)[at], wv.view(-1, hk, d)[at] = k[row:row + q], v[row:row + q]
        row += q
    blocks = E.Blocks.empty(p, block) if block else None
    if block:
        blocks.codes.fill_(101)
        blocks.scales.fill_(77)
    E.dsa_pages_append(p, k, v, ql, kl, blocks=blocks)
    torch.cuda.synchronize()
    bits = lambda x: x.view(torch.int16 if dtype == "bf16" else torch.int32)
    assert torch.equal(bits(p.k), bits(wk)) and torch.equal(bits(p.v), bits(wv))
    if block:
        want = P.summaries(host(wk), t, ql, kl, block, np.full(blocks.codes.shape, 101), np.full(blocks.scales.shape, 77))
        assert np.array_equal(blocks.codes.cpu().numpy(), want[0])
        assert np.array_equal(blocks.scales.cpu().numpy(), want[1])


def test_append_summaries_at_borders():
    """Means at and next to 127.5 units and at ties, zeros, the smallest and largest numbers."""
    d, block, page = 64, 16, 16
    cases = []
    for scale in (1.0, 2.0 ** -140, 2.0 ** -126, 2.0 ** -7, 2.0 ** 90, 2.0 ** 120):
        for top in (127.5, 127.25, 127.0, 63.75, 64.0, 1.0):
            r = np.zeros((block, d), np.float32)
            r[:] = np.float32(top * scale) * (np.arange(d) == 0)
            r[:, 1:40] = (np.arange(39) - 19.5) * scale          # ties between codes
            r[:, 40:50] = np.float32(0.25 * scale)
            cases.append(r)
    cases.append(np.zeros((block, d), np.float32))
    r = np.zeros((block, d), np.float32)
    r[:8, 3], r[8:, 3], r[:, 4] = 3e38, -3e38, 1e-3              # sums that cancel
    cases.append(r)
    n = len(cases)
    x = np.stack(cases).reshape(n * block, 1, d)
    say("append borders")
    for dtype in ("f32", "bf16"):
        k = torch.from_numpy(x).to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
        p = E.Pages.empty(n, page, 1, d, ints(np.arange(n)[None]), dtype)
        b = E.Blocks.empty(p, block)
        E.dsa_pages_append(p, k, k, [n * block], [n * block], blocks=b)
        want = P.summaries(host(k).reshape(n, page, 1, d), np.arange(n)[None], [n * block], [n * block], block,
                           np.zeros(b.codes.shape), np.zeros(b.scales.shape))
        assert np.array_equal(b.codes.cpu().numpy(), want[0]) and np.array_equal(b.scales.cpu().numpy(), want[1])


def test_append_many_sequences_and_missing_pages():
    rng = np.random.default_rng(11)
    kl = [int(x) for x in rng.integers(1, 90, 150)]
    ql = [int(rng.integers(0, k + 1)) for k in kl]
    say("append many")
    t, n = table(rng, kl, 32)
    t[3, 0], t[7, 0] = -1, n
    k = rows(rng, sum(ql), 2, 64, "bf16").cuda()
    p = E.Pages(torch.full((n, 32, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda"),
                torch.full((n, 32, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda"), torch.from_numpy(t).cuda())
    b = E.Blocks(torch.full((n, 2, 2, 64), 5, dtype=torch.int8, device="cuda"),
                 torch.full((n, 2, 2), 5, dtype=torch.uint8, device="cuda"), 32)
    E.dsa_pages_append(p, k, k, ql, kl, blocks=b)
    want, row = np.full((n * 32, 2, 64), 3.0, np.float32), 0
    for i, (q, m) in enumerate(zip(ql, kl)):
        at = A.slots(t, i, m, 32, n)[m - q:]
        want[at[at >= 0]] = host(k[row:row + q])[at >= 0]
        row += q
    assert np.array_equal(host(p.k).reshape(want.shape), want) and torch.equal(p.k, p.v)
    codes, scales = P.summaries(want.reshape(n, 32, 2, 64), t, ql, kl, 16, np.full(b.codes.shape, 5), np.full(b.scales.shape, 5))
    assert np.array_equal(b.codes.cpu().numpy(), codes) and np.array_equal(b.scales.cpu().numpy(), scales)


# ----------------------------------------------------------------------------
# attention over pages
# ----------------------------------------------------------------------------
PAGED = [
    (1, 1, 16, [1], [1]),
    (4, 2, 64, [0, 3, 0], [0, 3, 5]),
    (8, 8, 16, [15, 16, 17], [15, 16, 17]),
    (6, 2, 48, [33, 1, 64, 65], [33, 40, 64, 130]),
    (16, 1, 64, [2, 1, 5, 3], [129, 63, 300, 64]),
    (5, 5, 128, [128, 127], [128, 255]),
    (12, 3, 80, [1, 1, 1, 40], [1, 64, 65, 500]),
    (20, 1, 64, [1, 2, 100], [200, 65, 101]),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hk,page,ql,kl", PAGED)
def test_pages_attention(dtype, d, hq, hk, page, ql, kl):
    say("pages attention", dtype, d, hq, hk, page, ql, kl)
    rng = np.random.default_rng(hq * 100 + d)
    p, kp, vp, t = filled(rng, kl, page, hk, d, dtype)
    q = rows(rng, sum(ql), hq, d, dtype).cuda()
    out, lse = run_pages(p, q, ql, kl)
    ref = P.pages_attention(host(q), kp, vp, t, ql, kl, d ** -0.5)
    check_attention(out, lse, ref, d, max(kl), dtype == "bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("page", [16, 64, 112])
def test_pages_attention_joined_ranges(dtype, page):
    """Few rows over many keys, chunks whose key ranges are joined, and single tokens in one call."""
    rng = np.random.default_rng(page)
    ql, kl = [2, 20, 100, 1, 9], [9000, 3001, 4999, 4097, 520]
    say("pages joined", dtype, page)
    p, kp, vp, t = filled(rng, kl, page, 2, 128, dtype)
    q = rows(rng, sum(ql), 4, 128, dtype).cuda()
    out, lse = run_pages(p, q, ql, kl, scale=0.2)
    check_attention(out, lse, P.pages_attention(host(q), kp, vp, t, ql, kl, 0.2), 128, max(kl), dtype == "bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 48, 64])
def test_pages_attention_missing_pages(dtype, d, page):
    """Pages that the table does not name, the first of a sequence (rows that see nothing), the last, all of
    them; page 0 and every unused slot hold NaN."""
    rng = np.random.default_rng(page + d)
    ql, kl = [90, 1, 3, 150, 2, 70], [200, 150, 66, 150, 40, 300]
    last = lambda n: (n - 1) // page
    gone = [(0, 1), (0, last(200)), (1, 0), (2, last(66)), (3, 0), (5, 0), (5, 1), (5, 2)] + [(4, i) for i in range(last(40) + 1)]
    say("pages missing", dtype, d, page)
    p, kp, vp, t = filled(rng, kl, page, 2, d, dtype, gone)
    q = rows(rng, sum(ql), 6, d, dtype).cuda()
    out, lse = run_pages(p, q, ql, kl)
    ref = P.pages_attention(host(q), kp, vp, t, ql, kl, d ** -0.5)
    assert np.isinf(ref[1]).any()
    check_attention(out, lse, ref, d, max(kl), dtype == "bf16")
    assert torch.all(out[torch.from_numpy(np.isinf(ref[1])).cuda()] == 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_pages_attention_strided_on_another_stream(dtype, d):
    """Queries as a slice of a fused projection, on another stream, outputs next to guards, no normaliser."""
    rng = np.random.default_rng(d)
    hq, hk, page, ql, kl = 6, 2, 64, [70, 1, 150], [70, 300, 151]
    p, kp, vp, t = filled(rng, kl, page, hk, d, dtype)
    n = sum(ql)
    q = rows(rng, n, hq + 3, d, dtype).cuda()[:, 1:hq + 1]
    guard = torch.full((n + 2, hq, d), 7.0, dtype=q.dtype, device="cuda")
    ws = space(E.pages_workspace_size(ql, kl, hq, hk, d, dtype))
    say("pages strided", dtype, d)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    E.dsa_pages_attention(p, q, ql, kl, guard[1:-1], None, workspace=ws, stream=st)
    st.synchronize()
    assert torch.all(guard[0] == 7) and torch.all(guard[-1] == 7)
    check_attention(guard[1:-1], None, P.pages_attention(host(q), kp, vp, t, ql, kl, d ** -0.5), d, max(kl), dtype == "bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_pages_attention_many_sequences(dtype):
    rng = np.random.default_rng(8)
    kl = [int(x) for x in rng.integers(1, 60, 150)]
    ql = [int(rng.integers(0, k + 1)) for k in kl]
    say("pages many", dtype)
    p, kp, vp, t = filled(rng, kl, 16, 2, 64, dtype)
    q = rows(rng, sum(ql), 4, 64, dtype).cuda()
    out, lse = run_pages(p, q, ql, kl)
    check_attention(out, lse, P.pages_attention(host(q), kp, vp, t, ql, kl, 64 ** -0.5), 64, max(kl), dtype == "bf16")


@pytest.mark.parametrize("scale", [1.0, 2.0 ** 20, 2.0 ** 100])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_pages_attention_large_scores(dtype, scale):
    """Scores far beyond the exponential's range, and equal maxima: a row's largest keys share its weight.
    Products of small whole numbers, so that scores are exact."""
    rng = np.random.default_rng(9)
    ql, kl, d, page = [3, 60], [70, 130], 64, 16
    p, _, _, t = filled(rng, kl, page, 2, d, dtype)
    p.k.copy_(torch.from_numpy(rng.integers(-2, 3, p.k.shape)).to(p.k.dtype))
    q = torch.from_numpy(rng.integers(-2, 3, (sum(ql), 4, d))).to(p.k.dtype).cuda()
    say("pages large scores", dtype, scale)
    out, lse = run_pages(p, q, ql, kl, scale=scale)
    ref = P.pages_attention(host(q), host(p.k), host(p.v), t, ql, kl, scale)
    if scale == 1.0:
        check_attention(out, lse, ref, d, max(kl), dtype == "bf16")
        return
    # scores are exact and a row's differ by nothing or far beyond the exponential: its weights are 1 before
    # they are divided by their number.  n sums, a reciprocal and a product; bf16: the result's rounding
    o, l, ab, _ = ref
    tol = (max(kl) + 4) * U * ab + (B if dtype == "bf16" else 2 * U) * np.abs(o)
    assert np.all(np.abs(host(out) - o) <= tol)
    assert np.all(np.abs(lse.cpu().numpy() - l) <= 2 * U * np.abs(l) + 2.0 ** -20)


@pytest.mark.parametrize("page", [64, 48])
@pytest.mark.parametrize("ql", [[1], [40]])
def test_pages_beyond_4_gib(page, ql):
    """A pool of more than 2^32 bytes: the sequence's pages lie at its end."""
    hk, d, kl = 8, 128, [333]
    n = (1 << 32) // (page * hk * d * 2) + 40
    say("pages beyond 4 GiB", page, ql)
    rng = np.random.default_rng(page)
    per = -(-kl[0] // page)
    t = (n - 1 - rng.permutation(30)[:per]).astype(np.int32)[None]
    k, v = (torch.empty(n, page, hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    p = E.Pages(k, v, ints(t))
    x = [rows(rng, kl[0], hk, d, "bf16").cuda() for _ in range(2)]
    b = E.Blocks(torch.zeros(n, page // 16, hk, d, dtype=torch.int8, device="cuda"),
                 torch.zeros(n, page // 16, hk, dtype=torch.uint8, device="cuda"), page)
    E.dsa_pages_append(p, x[0], x[1], kl, kl, blocks=b)
    q = rows(rng, ql[0], 16, d, "bf16").cuda()
    out, lse = run_pages(p, q, ql, kl)
    ref = A.prompt(host(q), host(x[0]), host(x[1]), ql, kl, d ** -0.5)
    check_attention(out, lse, ref, d, kl[0], True)
    idx = torch.full((ql[0], hk, 21), -1, dtype=torch.int32, device="cuda")
    E.dsa_block_select(b, p.page_table, q, ql, kl, idx)
    out, lse = run_pages(p, q, ql, kl, idx=idx, block=16)
    check_attention(out, lse, ref, d, kl[0], True)               # all 21 blocks


# ----------------------------------------------------------------------------
# choice of blocks
# ----------------------------------------------------------------------------
def summarised(rng, kl, page, block, hk, d):
    """Random summaries (integers, scales in a narrow range), with equal rows among them."""
    t, n = table(rng, kl, page)
    c = rng.integers(-127, 128, (n, page // block, hk, d)).astype(np.int8)
    c[rng.random(c.shape[:3]) < 0.2] = c[0, 0, 0]
    s = rng.integers(118, 124, c.shape[:3]).astype(np.uint8)
    return E.Blocks(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda(), page), c, s, t


def run_select(b, t, q, ql, kl, topn, sinks, local, stream=None):
    idx = torch.full((sum(ql) + 2, b.Hkv, topn), -5, dtype=torch.int32, device="cuda")
    E.dsa_block_select(b, ints(t), q, ql, kl, idx[1:-1], sinks=sinks, local=local, stream=stream)
    torch.cuda.synchronize()
    assert torch.all(idx[0] == -5) and torch.all(idx[-1] == -5)
    return idx[1:-1].cpu().numpy()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hk,page,block,topn,sinks,local,ql,kl", [
    (1, 1, 16, 16, 3, 0, 1, [1], [1]),
    (1, 1, 16, 16, 3, 0, 1, [40], [300]),
    (4, 2, 32, 16, 4, 1, 2, [1, 3, 0, 20], [400, 33, 50, 200]),
    (6, 2, 64, 64, 5, 1, 1, [17, 2], [1500, 4000]),
    (5, 1, 96, 32, 8, 2, 2, [33, 1], [999, 2500]),
    (16, 2, 128, 64, 16, 0, 2, [9, 65], [5000, 2100]),
    (16, 1, 64, 32, 4, 1, 3, [3, 5], [700, 1000]),       # nothing to choose: sinks and the latest fill the row
    (20, 1, 128, 128, 3, 0, 1, [5], [1800]),
    (40, 1, 48, 16, 7, 3, 2, [2, 6], [650, 300]),
    (6, 3, 64, 16, 63, 20, 33, [4], [3000]),
])
def test_select(dtype, d, hq, hk, page, block, topn, sinks, local, ql, kl):
    say("select", dtype, d, hq, hk, page, block, topn, ql, kl)
    rng = np.random.default_rng(hq * 7 + d)
    b, c, s, t = summarised(rng, kl, page, block, hk, d)
    q = rows(rng, sum(ql), hq, d, dtype)
    got = run_select(b, t, q.cuda(), ql, kl, topn, sinks, local)
    assert np.array_equal(got, P.select(host(q), c, s, t, ql, kl, block, page, topn, sinks, local))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_select_many_blocks(dtype):
    """More blocks than a wavefront keeps in registers, and more than several tokens' scores fit for."""
    rng = np.random.default_rng(12)
    for hq, kl, topn in ((4, 16 * 1030, 40), (2, 16 * 5000, 4), (8, 16 * 20011, 9), (1, 16 * 32768, 4096)):
        say("select many blocks", dtype, hq, kl)
        b, c, s, t = summarised(rng, [kl], 64, 16, 1, 64)
        q = rows(rng, 3, hq, 64, dtype)
        got = run_select(b, t, q.cuda(), [3], [kl], topn, 1, 2)
        assert np.array_equal(got, P.select(host(q), c, s, t, [3], [kl], 16, 64, topn, 1, 2))


def test_select_ties_missing_pages_and_extreme_scales():
    rng = np.random.default_rng(13)
    hq, hk, d, page, block, ql, kl = 4, 2, 64, 32, 16, [3, 2, 1], [900, 500, 700]
    say("select oddities")
    b, c, s, t = summarised(rng, kl, page, block, hk, d)
    q = rows(rng, 6, hq, d, "f32")
    q[0], q[1, 0] = 0, 0                                  # every score 0; one head of zeros
    q[2, 1] *= 2.0 ** -110                                # next to a head far larger
    q[3] *= 2.0 ** 120
    q[4] *= 2.0 ** -140                                   # subnormal queries
    for scales in (s, np.where(rng.random(s.shape) < 0.5, 1, 254).astype(np.uint8), rng.integers(1, 25, s.shape).astype(np.uint8),
                   np.full(s.shape, 127, np.uint8)):
        b.scales.copy_(torch.from_numpy(scales))
        got = run_select(b, t, q.cuda(), ql, kl, 6, 1, 2)
        assert np.array_equal(got, P.select(host(q), c, scales, t, ql, kl, block, page, 6, 1, 2))
    c[:] = c[0, 0, 0]                                     # all scores of a row equal: the lowest blocks
    b.codes.copy_(torch.from_numpy(c))
    got = run_select(b, t, q.cuda(), ql, kl, 6, 1, 2)
    assert np.array_equal(got, P.select(host(q), c, scales, t, ql, kl, block, page, 6, 1, 2))
    assert got[5, 0].tolist() == [0, 1, 2, 3, 42, 43]
    t[0, 5:20], t[1, :], t[2, 1:] = -1, 1 << 30, -2       # pages that the table does not name come last
    got = run_select(b, t, q.cuda(), ql, kl, 6, 1, 2)
    assert np.array_equal(got, P.select(host(q), c, scales, t, ql, kl, block, page, 6, 1, 2))


@pytest.mark.parametrize("hq", [1, 4, 20])
def test_select_many_of_many(hq):
    """Choices of 60 and more among hundreds, and hundreds of equal scores."""
    rng = np.random.default_rng(30 + hq)
    ql, kl, d, block, page = [9, 2], [16 * 700 + 3, 16 * 400], 64, 16, 64
    say("select many of many", hq)
    b, c, s, t = summarised(rng, kl, page, block, 1, d)
    q = rows(rng, 11, hq, d, "bf16")
    for rounds in range(2):
        for topn in (17, 62, 67, 130, 390):
            got = run_select(b, t, q.cuda(), ql, kl, topn, 1, 2)
            assert np.array_equal(got, P.select(host(q), c, s, t, ql, kl, block, page, topn, 1, 2))
        c[rng.random(c.shape[:3]) < 0.9] = c[0, 0, 0]         # most scores equal, some above and some below
        b.codes.copy_(torch.from_numpy(c))
        s[:] = 120
        b.scales.copy_(torch.from_numpy(s))


def test_select_many_sequences():
    rng = np.random.default_rng(14)
    kl = [int(x) for x in rng.integers(1, 500, 150)]
    ql = [int(min(k, rng.integers(0, 6))) for k in kl]
    say("select many")
    b, c, s, t = summarised(rng, kl, 16, 16, 2, 64)
    q = rows(rng, sum(ql), 6, 64, "bf16")
    got = run_select(b, t, q.cuda(), ql, kl, 5, 1, 1)
    assert np.array_equal(got, P.select(host(q), c, s, t, ql, kl, 16, 16, 5, 1, 1))


# ----------------------------------------------------------------------------
# attention over listed blocks
# ----------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hk,page,block,topn,ql,kl", [
    (1, 1, 16, 16, 1, [1], [1]),
    (4, 2, 32, 16, 3, [0, 3, 20], [9, 40, 100]),
    (8, 1, 64, 64, 4, [5, 1], [400, 333]),
    (8, 2, 64, 64, 4, [40, 1, 300], [1400, 333, 310]),
    (5, 1, 32, 16, 6, [100, 37], [700, 60]),
    (3, 3, 64, 32, 3, [200], [500]),
    (32, 1, 256, 128, 3, [70], [900]),
    (48, 1, 16, 16, 5, [33, 8], [300, 8]),
    (6, 3, 96, 32, 5, [3, 2], [300, 500]),
    (20, 1, 128, 128, 2, [4], [700]),
    (40, 2, 64, 16, 7, [2, 1], [200, 33]),
    (4, 4, 64, 64, 33, [2], [4000]),
])
def test_block_attention(dtype, d, hq, hk, page, block, topn, ql, kl):
    say("block attention", dtype, d, hq, hk, page, block, topn, ql, kl)
    rng = np.random.default_rng(hq + d)
    p, kp, vp, t = filled(rng, kl, page, hk, d, dtype)
    q = rows(rng, sum(ql), hq, d, dtype).cuda()
    idx = np.full((sum(ql), hk, topn), -1, np.int32)
    row = 0
    for a, n in zip(ql, kl):
        for i in range(a):
            own = (n - a + i) // block
            for h in range(hk):
                pick = rng.permutation(own + 1)[:topn]
                idx[row + i, h, :len(pick)] = pick
        row += a
    out, lse = run_pages(p, q, ql, kl, idx=ints(idx), block=block)
    check_attention(out, lse, P.pages_attention(host(q), kp, vp, t, ql, kl, d ** -0.5, idx, block), d,
                    min(topn * block, max(kl)), dtype == "bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_block_attention_oddities(dtype):
    """Lists with blocks behind the query, twice the same, garbage, nothing; pages that are not there."""
    rng = np.random.default_rng(15)
    hq, hk, d, page, block, ql, kl = 4, 2, 64, 32, 16, [4, 3], [100, 70]
    idx = np.array([[5, 0, 6, 1 << 30], [2, 2, 2, -1], [-1, -1, -1, -1], [6, 1, -(1 << 31), 0x7fffffff],
                    [4, 3, 2, 1], [0, 5, 0, 4], [7, 9, 100, -3]], np.int32)
    idx = np.stack([idx, idx[::-1]], 1)
    say("block oddities", dtype)
    for gone in ((), ((0, 0), (0, 3), (1, 1))):
        p, kp, vp, t = filled(rng, kl, page, hk, d, dtype, gone)
        q = rows(rng, 7, hq, d, dtype).cuda()
        out, lse = run_pages(p, q, ql, kl, idx=ints(idx), block=block)
        ref = P.pages_attention(host(q), kp, vp, t, ql, kl, d ** -0.5, idx, block)
        check_attention(out, lse, ref, d, 70, dtype == "bf16")
        assert torch.all(out[torch.from_numpy(np.isinf(ref[1])).cuda()] == 0) and np.isinf(ref[1]).any()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hk,page,block", [(8, 1, 32, 16), (4, 2, 64, 64), (16, 1, 128, 128), (40, 1, 32, 32), (1, 1, 48, 16)])
def test_block_attention_oddities_of_many_rows(d, hq, hk, page, block):
    """The same for chunks of queries whose lists are merged: lists in any order, entries twice, garbage, rows that
    list nothing, long lists, pages that are not there; page 0 and every unused slot hold NaN."""
    rng = np.random.default_rng(hq + d)
    ql, kl = [130, 1, 75], [5 * page + 7, 40, 76]
    for topn, gone in ((3, ()), (5, ((0, 0), (0, 3), (2, 1))), (150, ((0, 1),))):
        say("block oddities, many rows", d, hq, page, block, topn)
        p, kp, vp, t = filled(rng, kl, page, hk, d, "bf16", gone)
        q = rows(rng, sum(ql), hq, d, "bf16").cuda()
        idx = rng.integers(-2, max(kl) // block + 3, (sum(ql), hk, topn)).astype(np.int32)
        idx[rng.random(sum(ql)) < 0.5] = np.sort(idx, -1)[0]
        idx[3:9] = -1
        idx[20, 0, 0], idx[21, 0, 1] = 0x7fffffff, -(1 << 31)
        out, lse = run_pages(p, q, ql, kl, idx=ints(idx), block=block)
        ref = P.pages_attention(host(q), kp, vp, t, ql, kl, d ** -0.5, idx, block)
        check_attention(out, lse, ref, d, min(topn * block, 3 * max(kl)), True)
        assert torch.all(out[torch.from_numpy(np.isinf(ref[1])).cuda()] == 0) and np.isinf(ref[1]).any()


def test_block_attention_many_rows_and_sequences():
    rng = np.random.default_rng(16)
    kl = [int(x) for x in rng.integers(1, 200, 100)]
    ql = [int(min(k, rng.integers(0, 9))) for k in kl]
    say("block many")
    for dtype in ("bf16", "f32"):
        p, kp, vp, t = filled(rng, kl, 16, 2, 64, dtype)
        q = rows(rng, sum(ql), 4, 64, dtype).cuda()
        idx = rng.integers(-1, 13, (sum(ql), 2, 3)).astype(np.int32)
        out, lse = run_pages(p, q, ql, kl, idx=ints(idx), block=16)
        check_attention(out, lse, P.pages_attention(host(q), kp, vp, t, ql, kl, 0.125, idx, 16), 64, 48, dtype == "bf16")


# ----------------------------------------------------------------------------
# together, as a server uses them
# ----------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_serving_run(dtype):
    """Prompts, decode steps and a chunk: pages assigned, rows and summaries written, dense and block attention,
    the indexer's keys written by the slot map and selected from, a sequence released and its pages used again."""
    rng = np.random.default_rng(20)
    hq, hk, d, page, block, topn, batch = 8, 2, 64, 32, 16, 5, 3
    pool = 40
    tab, free, left = ints(np.full((batch, 12), -1)), ints(rng.permutation(pool)), pool
    p = E.Pages.empty(pool, page, hk, d, tab, dtype)
    p.k.fill_(float("nan"))
    p.v.fill_(float("nan"))
    b = E.Blocks.empty(p, block)
    ikeys = torch.zeros(pool * page, d, dtype=torch.bfloat16, device="cuda")
    text = [np.zeros((0, hk, d), np.float32)] * batch, [np.zeros((0, hk, d), np.float32)] * batch
    itext = [np.zeros((0, d), np.float32)] * batch
    kl = [0] * batch

    def step(ql):
        nonlocal left, kl
        kl = [k + q for k, q in zip(kl, ql)]
        n = sum(ql)
        slots, pos = ints(np.zeros(n)), ints(np.zeros(n))
        left = E.dsa_pages_assign(tab, page, free, left, ql, kl, slots=slots, positions=pos)
        q, k, v = (rows(rng, n, h, d, dtype).cuda() for h in (hq, hk, hk))
        ik = rows(rng, n, 1, d, "bf16").cuda()[:, 0]
        E.dsa_pages_append(p, k, v, ql, kl, blocks=b)
        ikeys[slots.long()] = ik
        row = 0
        for i, m in enumerate(ql):
            for x, y in zip(text, (k, v)):
                x[i] = np.concatenate([x[i], host(y[row:row + m])])
            itext[i] = np.concatenate([itext[i], host(ik[row:row + m])])
            assert pos[row:row + m].tolist() == list(range(kl[i] - m, kl[i]))
            row += m
        say("serving", dtype, ql, kl)
        out, lse = run_pages(p, q, ql, kl)
        ref = A.prompt(host(q), *(np.concatenate(x) for x in text), ql, kl, d ** -0.5)
        check_attention(out, lse, ref, d, max(kl), dtype == "bf16")
        idx = torch.full((n, hk, topn), -5, dtype=torch.int32, device="cuda")
        E.dsa_block_select(b, tab, q, ql, kl, idx)
        want = P.select(host(q), b.codes.cpu().numpy(), b.scales.cpu().numpy(), tab.cpu().numpy(), ql, kl, block, page, topn, 1, 2)
        assert np.array_equal(idx.cpu().numpy(), want)
        out, lse = run_pages(p, q, ql, kl, idx=idx, block=block)
        ref = P.pages_attention(host(q), np.nan_to_num(host(p.k)), np.nan_to_num(host(p.v)), tab.cpu().numpy(), ql, kl,
                                d ** -0.5, want, block)
        check_attention(out, lse, ref, d, topn * block, dtype == "bf16")
        # the indexer over its own keys, written by the slot map
        iq, w = rows(rng, n, 8, d, "bf16").cuda(), torch.from_numpy(rng.normal(size=(n, 8)).astype(np.float32)).cuda()
        oi = torch.empty(n, 16, dtype=torch.int32, device="cuda")
        osc = torch.empty(n, 16, device="cuda")
        ws = space(E.workspace_size(ql, kl, 8, d, 16, "bf16", "bf16", True, True))
        E.dsa_indexer_topk(iq, "bf16", None, w, ikeys, "bf16", None, ql, kl, tab, page, 8, d, 16, oi, osc, ws)
        row = 0
        for i, m in enumerate(ql):
            for x in range(m):
                seen = kl[i] - m + x + 1
                sc = (np.maximum(host(iq[row + x]) @ itext[i][:seen].T, 0) * host(w[row + x])[:, None]).sum(0)
                best = np.sort(sc)[::-1][:16]
                got = oi[row + x].cpu().numpy()
                assert np.allclose(np.sort(sc[got[got >= 0]])[::-1], best, rtol=1e-3, atol=1e-2)
            row += m

    step([150, 83, 7])
    for _ in range(3):
        step([2, 1, 2])
    step([1, 60, 0])
    before = left
    left = E.dsa_pages_release(tab, page, free, left, [kl[0], 0, kl[2]], kl)
    assert left == before + -(-kl[1] // page) and torch.all(tab[1] == -1)
    kl[1] = 0
    for x in (*text, itext):
        x[1] = x[1][:0]
    step([1, 100, 1])
    left = E.dsa_pages_release(tab, page, free, left, [0] * 3, kl)
    assert left == pool and sorted(free.tolist()) == list(range(pool))


def test_summaries_alone():
    """Summaries of keys that are in the pages already: after an eviction, of all blocks; of the newest only."""
    rng = np.random.default_rng(25)
    hk, d, page, kl, new = 2, 64, 32, [100, 70], [64, 48]
    p, kp, vp, t = filled(rng, kl, page, hk, d, "bf16")
    acc = torch.rand(p.num_pages, page, device="cuda")
    src = torch.empty(2, 64, dtype=torch.int32, device="cuda")
    E.dsa_cache_evict(acc, p.page_table, kl, new, [(p.k, p.k), (p.v, p.v)], src, workspace=space(E.evict_workspace_size(kl, new)))
    for ql in (new, [20, 1], [0, 16]):
        say("summaries alone", ql)
        b = E.Blocks.empty(p, 16)
        b.codes.fill_(3)
        b.scales.fill_(9)
        k, v = p.k.clone(), p.v.clone()
        E.dsa_pages_append(p, None, None, ql, new, blocks=b)
        codes, scales = P.summaries(np.nan_to_num(host(p.k)), t, ql, new, 16, np.full(b.codes.shape, 3), np.full(b.scales.shape, 9))
        assert np.array_equal(b.codes.cpu().numpy(), codes) and np.array_equal(b.scales.cpu().numpy(), scales)
        bits = lambda x: x.view(torch.int16)
        assert torch.equal(bits(k), bits(p.k)) and torch.equal(bits(v), bits(p.v))


def test_evicted_pages_and_attention():
    """Eviction moves rows of these pages as of any per-slot array; attention over the smaller cache."""
    rng = np.random.default_rng(22)
    hq, hk, d, page, kl, new = 4, 2, 64, 16, [100, 70], [48, 40]
    p, kp, vp, t = filled(rng, kl, page, hk, d, "bf16")
    acc = torch.rand(p.num_pages, page, device="cuda")
    src = torch.empty(2, 48, dtype=torch.int32, device="cuda")
    say("evict")
    E.dsa_cache_evict(acc, p.page_table, kl, new, [(p.k, p.k), (p.v, p.v)], src, prefix=2, window=8,
                      workspace=space(E.evict_workspace_size(kl, new)))
    q = rows(rng, 2, hq, d, "bf16").cuda()
    out, lse = run_pages(p, q, [1, 1], new)
    ks, vs = [], []
    for b, n in enumerate(kl):
        at = A.slots(t, b, n, page, p.num_pages)[src[b, :new[b]].cpu().numpy()]
        ks.append(kp.reshape(-1, hk, d)[at])
        vs.append(vp.reshape(-1, hk, d)[at])
    check_attention(out, lse, A.prompt(host(q), np.concatenate(ks), np.concatenate(vs), [1, 1], new, 0.125), d, 48, True)


def test_captured_and_replayed():
    """A whole step captured into a graph and replayed, with eager work on other workspaces between the replays;
    a second graph shares the workspace."""
    rng = np.random.default_rng(21)
    ql, kl, hq, hk, d, page, block, topn = [1, 2, 40], [5000, 300, 400], 8, 2, 128, 64, 64, 4
    t, free, count, pool = grow(rng, ql, kl, page)
    old = [k - q for q, k in zip(ql, kl)]
    tab, gf = ints(t), ints(free)
    p = E.Pages(torch.randn(pool, page, hk, d, device="cuda").bfloat16(), torch.randn(pool, page, hk, d, device="cuda").bfloat16(), tab)
    b = E.Blocks.empty(p, block)
    b.codes.random_(-127, 128)
    b.scales.fill_(120)
    n = sum(ql)
    q, k, v = (rows(rng, n, h, d, "bf16").cuda() for h in (hq, hk, hk))
    ws = space(max(E.pages_workspace_size(ql, kl, hq, hk, d, "bf16"), E.block_workspace_size(ql, kl, hq, hk, d, "bf16", block, topn)))
    mk = lambda *s, **kw: torch.zeros(*s, device="cuda", **kw)
    slots, idx = mk(n, dtype=torch.int32), mk(n, hk, topn, dtype=torch.int32)
    outs = [mk(n, hq, d, dtype=torch.bfloat16) for _ in range(2)]
    lses = [mk(n, hq) for _ in range(2)]

    def first():
        E.dsa_pages_assign(tab, page, gf, count, ql, kl, slots=slots)
        E.dsa_pages_append(p, k, v, ql, kl, blocks=b)
        E.dsa_pages_attention(p, q, ql, kl, outs[0], lses[0], workspace=ws)

    def second():
        E.dsa_block_select(b, tab, q, ql, kl, idx)
        E.dsa_block_attention(p, q, ql, kl, idx, block, outs[1], lses[1], workspace=ws)

    say("captured: eager")
    first()
    second()
    torch.cuda.synchronize()
    want = [x.clone() for x in (tab, slots, p.k, p.v, b.codes, b.scales, idx, *outs, *lses)]
    st = torch.cuda.Stream()
    graphs = []
    for fn in (first, second):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            fn()
        graphs.append(g)
    for i in range(3):
        say("captured: replay", i)
        tab.copy_(ints(t))
        for x in (slots, idx, *outs, *lses):
            x.fill_(9)
        other = torch.randn(1 << 20, device="cuda").sum()
        for g in graphs:
            g.replay()
        run_pages(p, q, ql, kl)
        torch.cuda.synchronize()
        for x, y in zip((tab, slots, p.k, p.v, b.codes, b.scales, idx, *outs, *lses), want):
            assert torch.equal(x, y)
    for g in graphs:
        g.reset()


def test_two_streams_and_repeated_calls_agree():
    rng = np.random.default_rng(23)
    ql, kl, page = [1, 70, 2], [3000, 600, 900], 64
    p, _, _, t = filled(rng, kl, page, 2, 128, "bf16")
    b, c, s, _ = summarised(rng, kl, page, 64, 2, 128)
    q = rows(rng, sum(ql), 8, 128, "bf16").cuda()
    idx = torch.empty(sum(ql), 2, 4, dtype=torch.int32, device="cuda")
    E.dsa_block_select(b, p.page_table, q, ql, kl, idx)
    dense, sparse = run_pages(p, q, ql, kl), run_pages(p, q, ql, kl, idx=idx, block=64)
    say("two streams")
    res = []
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    n1, n2 = E.pages_workspace_size(ql, kl, 8, 2, 128, "bf16"), E.block_workspace_size(ql, kl, 8, 2, 128, "bf16", 64, 4)
    wss = [(space(n1), space(n2)) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(3):
        for st, (w1, w2) in zip(streams, wss):
            o = [torch.empty_like(q) for _ in range(2)]
            l = [torch.empty(q.shape[:2], device="cuda") for _ in range(2)]
            i2 = torch.empty_like(idx)
            st.wait_stream(torch.cuda.current_stream())
            E.dsa_pages_attention(p, q, ql, kl, o[0], l[0], workspace=w1, stream=st)
            E.dsa_block_select(b, p.page_table, q, ql, kl, i2, stream=st)
            E.dsa_block_attention(p, q, ql, kl, i2, 64, o[1], l[1], workspace=w2, stream=st)
            res.append((o, l, i2))
    torch.cuda.synchronize()
    for o, l, i2 in res:
        assert torch.equal(i2, idx) and torch.equal(o[0], dense[0]) and torch.equal(l[0], dense[1])
        assert torch.equal(o[1], sparse[0]) and torch.equal(l[1], sparse[1])


def test_pass_times_are_reported():
    rng = np.random.default_rng(24)
    ql, kl, page = [1, 40], [3000, 100], 64
    p, _, _, t = filled(rng, kl, page, 2, 64, "bf16")
    b, _, _, _ = summarised(rng, kl, page, 64, 2, 64)
    q, k = rows(rng, 41, 4, 64, "bf16").cuda(), rows(rng, 41, 2, 64, "bf16").cuda()
    idx = torch.empty(41, 2, 4, dtype=torch.int32, device="cuda")
    say("pass times")
    E.profile_begin()
    left = E.dsa_pages_assign(ints(np.full((1, 4), -1)), page, ints(np.arange(9)), 9, [100], [100])
    E.dsa_pages_release(ints(np.arange(4)[None]), page, ints(np.arange(9)), left - 2, [0], [100])
    E.dsa_pages_append(p, k, k, ql, kl, blocks=b)
    E.dsa_block_select(b, p.page_table, q, ql, kl, idx)
    run_pages(p, q, ql, kl)
    run_pages(p, q, ql, kl, idx=idx, block=64)
    t = E.profile_end()
    assert {"pages_assign", "pages_release", "pages_append", "pages_attention", "block_select", "block_attention"} <= set(t)
    assert all(n >= 1 and ms > 0 for n, ms in t.values())


# ----------------------------------------------------------------------------
# what a sequence gets does not depend on its neighbours
# ----------------------------------------------------------------------------
def check_two_terms(out, ref, d, n):
    """out (bf16, of softmax weights in two bf16 terms) against oracle (out, lse, abs_out, size).  The first term is
    off by B of the weight at most, the second by B of that: B^2 of each product; then the result's rounding."""
    o, l, ab, size = ref
    e = weight_err(size, l, d, n)[..., None]
    tol = (ab * (2 * e + n * U + B * B) + 4 * U * np.abs(o)) * (1 + B) + B * np.abs(o)
    bad = np.abs(host(out) - o) - tol
    assert np.all(bad <= 1e-30), (float(bad.max()), np.argwhere(bad > 0)[:4].tolist())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group,few,more", [(8, [1, 2, 2, 1], [3, 4]), (1, [16, 1, 5, 16], [17, 32]), (5, [3, 1, 2, 3], [6, 60])])
def test_few_rows_keep_two_terms_next_to_more_rows(d, group, few, more):
    """Sequences of up to 16 rows between sequences of 17 to 32, and of a chunk's."""
    rng = np.random.default_rng(group + d)
    hk, page = 2, 64
    ql, kl = [few[0], more[0], few[1], more[1], few[2], few[3]], [60, 1500, 2900, 700, 63, 333]
    say("few rows next to more", d, group)
    p, kp, vp, t = filled(rng, kl, page, hk, d, "bf16")
    q = rows(rng, sum(ql), group * hk, d, "bf16").cuda()
    out, lse = run_pages(p, q, ql, kl)
    ref = P.pages_attention(host(q), kp, vp, t, ql, kl, d ** -0.5)
    check_attention(out, lse, ref, d, max(kl), True)
    at = np.cumsum([0] + ql)
    for i in (0, 2, 4, 5):
        r = slice(at[i], at[i + 1])
        check_two_terms(out[r], [x[r] for x in ref], d, kl[i])
    # one range of keys, alone and in company: the same bits
    for i in (0, 4):
        alone = E.Pages(p.k, p.v, p.page_table[i:i + 1])
        r = slice(at[i], at[i + 1])
        o, l = run_pages(alone, q[r], ql[i:i + 1], kl[i:i + 1])
        assert torch.equal(o, out[r]) and torch.equal(l, lse[r])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group,ql", [(8, [8, 1, 40]), (16, [4, 2, 30]), (1, [64, 7, 100])])
def test_block_attention_of_few_rows_in_two_terms(d, group, ql):
    """Sequences of up to 64 rows next to one of more."""
    rng = np.random.default_rng(group + d)
    hk, page, block, topn, kl = 2, 64, 32, 6, [900, 1300, 800]
    say("block attention, few rows", d, group)
    p, kp, vp, t = filled(rng, kl, page, hk, d, "bf16")
    q = rows(rng, sum(ql), group * hk, d, "bf16").cuda()
    idx = np.sort(rng.integers(0, 24, (sum(ql), hk, topn)), -1).astype(np.int32)
    out, lse = run_pages(p, q, ql, kl, idx=ints(idx), block=block)
    ref = P.pages_attention(host(q), kp, vp, t, ql, kl, d ** -0.5, idx, block)
    check_attention(out, lse, ref, d, topn * block, True)
    n = ql[0] + ql[1]
    check_two_terms(out[:n], [x[:n] for x in ref], d, topn * block)


@pytest.mark.parametrize("group,ql", [(48, [30, 9]), (72, [25]), (128, [10, 3]), (160, [9]), (5, [70, 20])])
def test_block_attention_stays_in_its_workspace(group, ql):
    """Groups whose heads take several row tiles, units that begin within a query; long lists in any order, and
    guards on both sides of the workspace."""
    rng = np.random.default_rng(group)
    hk, d, page, block, topn, kl = 1, 64, 64, 32, 40, [2000, 1700][:len(ql)]
    say("block attention workspace", group, ql)
    p, kp, vp, t = filled(rng, kl, page, hk, d, "bf16")
    q = rows(rng, sum(ql), group, d, "bf16").cuda()
    idx = np.stack([rng.permutation(60)[:topn] for _ in range(sum(ql))])[:, None].astype(np.int32)
    n = E.block_workspace_size(ql, kl, group, hk, d, "bf16", block, topn)
    ws = torch.full((n + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    E.dsa_block_attention(p, q, ql, kl, ints(idx), block, out, lse, workspace=ws[4096:4096 + n])
    torch.cuda.synchronize()
    assert torch.all(ws[:4096] == 0xA5) and torch.all(ws[4096 + n:] == 0xA5)
    check_attention(out, lse, P.pages_attention(host(q), kp, vp, t, ql, kl, d ** -0.5, idx, block), d, topn * block, True)


def test_select_lengths_in_two_threads_and_a_graph():
    """The scores of 3 tokens, of 30000 blocks and of few, in turn from two host threads on their own streams: the
    kernel's limit of LDS is one for all of them.  Then the largest captured and replayed."""
    import threading

    rng = np.random.default_rng(31)
    hk, d, page, block = 1, 64, 64, 16
    lens = [16 * 30001, 16 * 9000, 16 * 700]
    b, c, s, t = summarised(rng, [max(lens)], page, block, hk, d)
    tab, q = ints(t), rows(rng, 3, 16, d, "bf16").cuda()
    want = {n: torch.from_numpy(run_select(b, t, q, [3], [n], 9, 1, 2)) for n in lens}
    for n in lens[1:]:
        ref = P.select(host(q), c, s, t, [3], [n], block, page, 9, 1, 2)
        assert np.array_equal(want[n].numpy(), ref)
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        st = torch.cuda.Stream()
        for r in range(30):
            n = lens[(r + i) % 3]
            idx = torch.empty(3, hk, 9, dtype=torch.int32, device="cuda")
            st.wait_stream(torch.cuda.current_stream())
            E.dsa_block_select(b, tab, q, [3], [n], idx, stream=st)
            got[i].append((n, idx))
        st.synchronize()

    say("select from two threads")
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    torch.cuda.synchronize()
    assert [len(x) for x in got] == [30, 30]
    for n, idx in got[0] + got[1]:
        assert torch.equal(idx.cpu(), want[n])
    idx = torch.empty(3, hk, 9, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        E.dsa_block_select(b, tab, q, [3], [lens[0]], idx)
    for r in range(3):
        idx.fill_(-9)
        E.dsa_block_select(b, tab, q, [3], [lens[2]], torch.empty_like(idx))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(idx.cpu(), want[lens[0]])
    g.reset()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_summaries_of_keys_that_are_not_finite(dtype, d):
    """Infinite and undefined means: the largest number of their sign, and 0; other heads and blocks as ever."""
    rng = np.random.default_rng(40 + d)
    hk, page, block, kl = 3, 32, 16, [96]
    say("summaries, not finite", dtype, d)
    k = rows(rng, 96, hk, d, dtype)
    k[3, 0, 5], k[7, 0, 5] = float("inf"), 1.0
    k[20, 1, 0], k[21, 1, 0], k[22, 1, 7] = float("inf"), float("-inf"), float("-inf")
    k[40, 2, 63], k[41, 2, 8] = float("nan"), 3e38
    k[50, :, :] = float("nan")
    k[70, 0, :], k[80, 1, ::2] = float("-inf"), float("inf")
    p = E.Pages.empty(3, page, hk, d, ints([[2, 0, 1]]), dtype)
    b = E.Blocks.empty(p, block)
    E.dsa_pages_append(p, k.cuda(), k.cuda(), kl, kl, blocks=b)
    codes, scales = P.summaries(host(p.k), np.array([[2, 0, 1]]), kl, kl, block, np.zeros(b.codes.shape), np.zeros(b.scales.shape))
    assert np.array_equal(b.codes.cpu().numpy(), codes) and np.array_equal(b.scales.cpu().numpy(), scales)
    assert codes.reshape(6, hk, d)[[4, 0, 2], [0, 0, 2], [5, 5, 63]].tolist()[0] == 64


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hq", [1, 4, 20])
def test_select_with_queries_that_are_not_finite(dtype, hq):
    rng = np.random.default_rng(41 + hq)
    ql, kl, d, page, block = [12], [900], 64, 32, 16
    say("select, not finite", dtype, hq)
    b, c, s, t = summarised(rng, kl, page, block, 1, d)
    q = rows(rng, 12, hq, d, dtype)
    q[0, 0, 3], q[1, 0, 5], q[2, 0, 7] = float("inf"), float("-inf"), float("nan")
    q[3], q[4], q[5] = float("nan"), float("inf"), float("-inf")
    q[6, hq - 1] = float("nan")
    q[7, hq - 1, ::2], q[8, hq - 1, 1::3] = float("-inf"), float("inf")
    q[9, 0, 0], q[9, 0, 1] = float("inf"), float("-inf")
    got = run_select(b, t, q.cuda(), ql, kl, 6, 1, 2)
    assert np.array_equal(got, P.select(host(q), c, s, t, ql, kl, block, page, 6, 1, 2))


@pytest.mark.parametrize("group,q,topn,window", [(1, 130, 40, 32), (4, 70, 150, 64), (8, 40, 300, 128)])
@pytest.mark.parametrize("order", ["any", "ascending"])
def test_block_attention_of_lists_longer_than_the_merge_holds(group, q, topn, window, order):
    """The merge of a unit's lists keeps `window` entries of each at a time: so many units that every list is one
    range, lists a few times as long, with entries twice, entries to skip and lists that end early."""
    rng = np.random.default_rng(group)
    hk, d, page, block, kl = 128, 64, 32, 16, 700
    say("block lists of several windows", group, order)
    tok = min(8, 16 // group)
    units = -(-(-(-q // tok)) // 8) * hk
    n = E.block_workspace_size([q], [kl], group * hk, hk, d, "bf16", block, topn)
    assert topn > window and 0 <= n - units * (8 * tok * topn + 8) * 16 < 512        # one range
    p, kp, vp, t = filled(rng, [kl], page, hk, d, "bf16")
    x = rows(rng, q, group * hk, d, "bf16").cuda()
    idx = rng.integers(-3, kl // block + 4, (q, hk, topn)).astype(np.int32)
    if order == "ascending":
        idx = np.sort(np.where(idx < 0, 1 << 20, idx), -1).astype(np.int32)
        idx[idx == 1 << 20] = -1
    idx[3, :, 5:], idx[7] = -1, -1
    out, lse = run_pages(p, x, [q], [kl], idx=ints(idx), block=block)
    for h in (0, 57, 127):
        g, one = slice(h * group, (h + 1) * group), slice(h, h + 1)
        ref = P.pages_attention(host(x[:, g]), kp[:, :, one], vp[:, :, one], t, [q], [kl], d ** -0.5, idx[:, one], block)
        check_attention(out[:, g], lse[:, g], ref, d, topn * block, True)
