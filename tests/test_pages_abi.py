"""Refusals of the entry points on paged keys and values: every bad call becomes an error on the host, before
anything touches a GPU.  The tensors are CPU tensors; the binding's own refusal of those is lifted, so that a
call gets to the library's checks."""
import contextlib
import ctypes

import pytest
import torch

import exact_top_token_amd as E
from exact_top_token_amd import attention as AT

STREAM = 0


@pytest.fixture(autouse=True)
def _cpu_tensors(request, monkeypatch):
    if "cpu_tensors_refused" not in request.node.name:
        monkeypatch.setattr(AT, "_on", lambda device, stream: contextlib.nullcontext(stream))


def i32(*s, fill=0):
    return torch.full(s, fill, dtype=torch.int32)


def pages(n=4, page=32, hk=2, d=64, batch=2, per=2, dtype=torch.bfloat16):
    return E.Pages.empty(n, page, hk, d, i32(batch, per), dtype)


def space(n=1 << 20):
    return torch.empty(n, dtype=torch.uint8)


def refused(call, status=-1):
    with pytest.raises(E.DosaError) as ei:
        call()
    assert ei.value.status == status and str(ei.value)


def test_struct_layout_matches_header():
    assert ctypes.sizeof(E.DsaPages) == 48 and E.DsaPages.dtype.offset == 24
    assert ctypes.sizeof(E.DsaBlocks) == 40 and E.DsaBlocks.num_pages.offset == 16


def test_cpu_tensors_refused():
    p = pages()
    b = E.Blocks.empty(p, 16)
    q, k = torch.zeros(1, 4, 64, dtype=torch.bfloat16), torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    for stream in (None, 0):
        for call in (lambda: E.dsa_pages_assign(p.page_table, 32, i32(4), 4, [1], [1], stream=stream),
                     lambda: E.dsa_pages_release(p.page_table, 32, i32(4), 0, [0], [1], stream=stream),
                     lambda: E.dsa_pages_append(p, k, k, [1], [1], blocks=b, stream=stream),
                     lambda: E.dsa_pages_attention(p, q, [1], [1], torch.empty_like(q), workspace=space(), stream=stream),
                     lambda: E.dsa_block_select(b, p.page_table, q, [1], [1], i32(1, 2, 4), stream=stream),
                     lambda: E.dsa_block_attention(p, q, [1], [1], i32(1, 2, 4), 16, torch.empty_like(q),
                                                   workspace=space(), stream=stream)):
            with pytest.raises(E.DosaError) as ei:
                call()
            assert ei.value.status == -1 and "GPU" in str(ei.value)


@pytest.mark.parametrize("over,status", [
    (dict(count=2), -1),                       # three pages needed
    (dict(count=-1), -1),
    (dict(count=9), -1),                       # more than there are
    (dict(count=2 ** 32 + 8), -1),
    (dict(ql=[41, 1]), -1),
    (dict(ql=[-1, 1]), -1),
    (dict(kl=[70, 1]), -1),                    # the table row ends before the tokens
    (dict(page=20), -1),
    (dict(page=0), -1),
    (dict(page=1 << 30), -2),
    (dict(ql=[1, 1, 1], kl=[1, 1, 1]), -1),
    (dict(ql=[1], kl=[1, 1]), -1),
    (dict(ql=[2 ** 31, 1]), -1),
    (dict(slots=i32(41)), -1),
    (dict(slots=torch.zeros(42)), -1),
    (dict(positions=i32(42, 2)[:, 0]), -1),
    (dict(free=torch.zeros(8, dtype=torch.int64)), -1),
    (dict(free=i32(2, 4)), -1),
    (dict(table=i32(2, 2).long()), -1),
    (dict(table=i32(4)), -1),
])
def test_assign_refusals(over, status):
    a = dict(ql=[40, 2], kl=[40, 2], page=32, count=8, free=i32(8), table=i32(2, 2), slots=None, positions=None)
    a.update(over)
    before = a["table"].clone()
    refused(lambda: E.dsa_pages_assign(a["table"], a["page"], a["free"], a["count"], a["ql"], a["kl"], slots=a["slots"],
                                       positions=a["positions"], stream=STREAM), status)
    assert torch.equal(before, a["table"])


def test_release_refusals():
    t, f = i32(2, 2), i32(8)
    call = lambda new, kl, count=0, page=32: E.dsa_pages_release(t, page, f, count, new, kl, stream=STREAM)
    refused(lambda: call([2, 0], [1, 1]))
    refused(lambda: call([-1, 0], [1, 1]))
    refused(lambda: call([0, 0], [65, 1]))
    refused(lambda: call([0, 0], [64, 64], count=5))          # nine pages of eight
    refused(lambda: call([0], [1, 1]))
    refused(lambda: call([0, 0], [1, 1], page=24))


def test_free_count_is_left_alone_by_a_refusal():
    n = ctypes.c_int32(1)
    t, f = i32(1, 4), i32(4)
    ql = (ctypes.c_int32 * 1)(64)
    assert E.lib().dsa_pages_assign(t.data_ptr(), 4, 32, 4, f.data_ptr(), ctypes.byref(n), ql, ql, 1, None, None, None) == -1
    assert n.value == 1 and "2 pages needed, 1 free" in E.status_string(-1)
    assert E.lib().dsa_pages_assign(t.data_ptr(), 4, 32, 4, f.data_ptr(), None, ql, ql, 1, None, None, None) == -1
    n.value = 4
    assert E.lib().dsa_pages_assign(t.data_ptr(), 4, 32, 4, None, ctypes.byref(n), ql, ql, 1, None, None, None) == -1
    assert E.lib().dsa_pages_assign(None, 4, 32, 4, f.data_ptr(), ctypes.byref(n), ql, ql, 1, None, None, None) == -1
    assert n.value == 4


def test_pages_and_blocks_object_refusals():
    t = i32(1, 2)
    k = torch.zeros(4, 32, 2, 64)
    E.Pages(k, k.clone(), t)
    for bad in ((k[0], k, t), (k, k.bfloat16(), t), (k, k[..., ::2], t), (k.half(), k.half(), t), (k, k, t.long()),
                (k, k, t[0]), (k.double(), k.double(), t)):
        refused(lambda: E.Pages(*bad))
    c, s = torch.zeros(4, 2, 2, 64, dtype=torch.int8), torch.zeros(4, 2, 2, dtype=torch.uint8)
    assert E.Blocks(c, s, 32).block == 16
    for bad in ((c[0], s, 32), (c, s[:3], 32), (c.to(torch.uint8), s, 32), (c, s.to(torch.int8), 32), (c, s, 33),
                (c.transpose(0, 1), s, 32)):
        refused(lambda: E.Blocks(*bad))
    refused(lambda: E.Blocks.empty(pages(), 24))


@pytest.mark.parametrize("fn", ["append", "attend", "sparse"])
@pytest.mark.parametrize("over,status", [
    (dict(page=24), -1),
    (dict(d=96), -2),
    (dict(hk=129, hq=129), -2),
    (dict(kl=[20, 80]), -1),                   # the table row ends before the keys
    (dict(ql=[21, 1]), -1),
    (dict(ql=[1, 1, 1], kl=[1, 1, 1]), -1),    # more sequences than table rows
    (dict(x=torch.float32), -1),               # not the pages' type
])
def test_paged_refusals(fn, over, status):
    a = dict(page=32, d=64, hk=2, hq=4, ql=[1, 2], kl=[20, 64], x=torch.bfloat16)
    a.update(over)
    p = pages(page=a["page"], d=a["d"], hk=a["hk"])
    nq = sum(a["ql"])
    x, q = torch.zeros(nq, a["hk"], a["d"], dtype=a["x"]), torch.zeros(nq, a["hq"], a["d"], dtype=a["x"])
    call = {"append": lambda: E.dsa_pages_append(p, x, x, a["ql"], a["kl"], stream=STREAM),
            "attend": lambda: E.dsa_pages_attention(p, q, a["ql"], a["kl"], torch.empty_like(q), workspace=space(),
                                                    stream=STREAM),
            "sparse": lambda: E.dsa_block_attention(p, q, a["ql"], a["kl"], i32(nq, a["hk"], 4), 16, torch.empty_like(q),
                                                    workspace=space(), stream=STREAM)}[fn]
    if fn == "sparse" and a["page"] == 24:
        status = -1
    refused(call, status)


def test_attention_refusals():
    p = pages()
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    call = lambda **o: E.dsa_pages_attention(**{**dict(pages=p, q=q, q_lens=[1, 2], kv_lens=[20, 64],
                                                       out=torch.empty_like(q), workspace=space(), stream=STREAM), **o})
    for o in (dict(scale=0.0), dict(scale=float("nan")), dict(scale=1e-40), dict(scale=3e38), dict(q=q[:2]),
              dict(q=q.transpose(1, 2)), dict(out=q.float()), dict(lse=torch.zeros(3, 4).double()), dict(lse=torch.zeros(4, 4)),
              dict(q=torch.zeros(3, 5, 64, dtype=torch.bfloat16), out=torch.zeros(3, 5, 64, dtype=torch.bfloat16))):
        refused(lambda: call(**o))
    for ws in (None, space(16)):
        refused(lambda: call(workspace=ws), -3)


def test_append_refusals():
    p = pages()
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    call = lambda **o: E.dsa_pages_append(**{**dict(pages=p, k=k, v=k, q_lens=[1, 2], kv_lens=[20, 64], stream=STREAM), **o})
    for o in (dict(k=k[:2]), dict(v=k.float()), dict(k=torch.zeros(3, 2, 128, dtype=torch.bfloat16)[..., :64]),
              dict(k=torch.zeros(1, 2, 64, dtype=torch.bfloat16).expand(3, 2, 64)),
              dict(blocks=E.Blocks.empty(pages(n=5), 16)), dict(blocks=E.Blocks.empty(pages(page=64), 16)),
              dict(k=None), dict(v=None), dict(k=None, v=None), dict(blocks=E.Blocks.empty(pages(hk=1), 16)), dict(blocks=E.Blocks.empty(pages(d=128), 16))):
        refused(lambda: call(**o))
    refused(lambda: call(pages=pages(page=48), blocks=E.Blocks.empty(pages(page=48), 48)), -2)


@pytest.mark.parametrize("over,status", [
    (dict(sinks=-1), -1),
    (dict(local=0), -1),
    (dict(sinks=3, local=2), -1),              # more than topn
    (dict(ql=[3, 2], kl=[2, 64]), -1),
    (dict(kl=[20, 65]), -1),
    (dict(hq=5), -1),
    (dict(topn=4097), -2),
    (dict(block=8), -2),
])
def test_select_refusals(over, status):
    a = dict(sinks=1, local=2, topn=4, ql=[1, 2], kl=[20, 64], hq=4, block=16)
    a.update(over)
    p = pages()
    q = torch.zeros(sum(a["ql"]), a["hq"], 64)
    refused(lambda: E.dsa_block_select(E.Blocks.empty(p, a["block"]), p.page_table, q, a["ql"], a["kl"],
                                       i32(sum(a["ql"]), 2, a["topn"]), sinks=a["sinks"], local=a["local"],
                                       stream=STREAM), status)


def test_select_layout_refusals():
    p = pages()
    b = E.Blocks.empty(p, 16)
    q = torch.zeros(3, 4, 64)
    call = lambda **o: E.dsa_block_select(**{**dict(blocks=b, page_table=p.page_table, q=q, q_lens=[1, 2], kv_lens=[20, 64],
                                                    idx=i32(3, 2, 4), stream=STREAM), **o})
    for o in (dict(idx=i32(3, 2, 4).long()), dict(idx=i32(3, 1, 4)), dict(idx=i32(3, 2, 0)), dict(idx=i32(3, 8)),
              dict(idx=i32(3, 2, 8)[..., :4]), dict(q=q.half()), dict(q=q[..., :32]), dict(page_table=i32(1, 2)),
              dict(page_table=i32(2, 2).long()), dict(q_lens=[3])):
        refused(lambda: call(**o))
    # more blocks than a workgroup's LDS holds the scores of
    big = E.Pages.empty(1, 1 << 20, 1, 64, i32(1, 1), torch.bfloat16)
    bb = E.Blocks.empty(big, 16)
    refused(lambda: E.dsa_block_select(bb, big.page_table, torch.zeros(1, 1, 64), [1], [32768 * 16 + 1], i32(1, 1, 4),
                                       stream=STREAM), -2)


def test_block_attention_refusals():
    p = pages()
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    call = lambda **o: E.dsa_block_attention(**{**dict(pages=p, q=q, q_lens=[1, 2], kv_lens=[20, 64], idx=i32(3, 2, 4),
                                                       block=16, out=torch.empty_like(q), workspace=space(),
                                                       stream=STREAM), **o})
    for o in (dict(idx=i32(3, 2, 4).long()), dict(idx=i32(3, 4, 4)), dict(idx=i32(3, 2, 0)), dict(block=64), dict(scale=-1.0)):
        refused(lambda: call(**o))
    refused(lambda: call(block=8), -2)
    refused(lambda: call(idx=i32(3, 2, (1 << 16) + 1)), -2)
    refused(lambda: call(workspace=space(16)), -3)


def test_workspace_sizes():
    ok = E.pages_workspace_size([1, 2], [20, 64], 4, 2, 64, "bf16")
    assert ok > 0 and E.block_workspace_size([1, 2], [20, 64], 4, 2, 64, "f32", 16, 4) > 0
    for args in (([2], [1], 4, 2, 64, "bf16"), ([1], [1], 3, 2, 64, "bf16"), ([1], [1], 4, 2, 80, "bf16")):
        refused(lambda: E.pages_workspace_size(*args), -2)
    for block, topn in ((8, 4), (16, 0), (128, 8193)):
        refused(lambda: E.block_workspace_size([1], [1], 4, 2, 64, "bf16", block, topn), -2)


def test_empty_calls():
    """No sequences, or none with new tokens: nothing is enqueued and nothing is needed."""
    p = pages()
    q, k = torch.zeros(0, 4, 64, dtype=torch.bfloat16), torch.zeros(0, 2, 64, dtype=torch.bfloat16)
    for lens in (([], []), ([0, 0], [0, 33])):
        assert E.dsa_pages_assign(p.page_table, 32, i32(4), 3, *lens, stream=STREAM) == 3
        assert E.dsa_pages_release(p.page_table, 32, i32(4), 3, lens[1], lens[1], stream=STREAM) == 3
        E.dsa_pages_append(p, k, k, *lens, blocks=E.Blocks.empty(p, 16), stream=STREAM)
        E.dsa_pages_attention(p, q, *lens, torch.empty_like(q), workspace=space(256), stream=STREAM)
        E.dsa_block_select(E.Blocks.empty(p, 16), p.page_table, q, *lens, i32(0, 2, 4), stream=STREAM)
        E.dsa_block_attention(p, q, *lens, i32(0, 2, 4), 16, torch.empty_like(q), workspace=space(256), stream=STREAM)


@pytest.mark.parametrize("group", [1, 2, 3, 5, 8, 16, 17, 20, 24, 32, 40, 64, 128, 200, 256])
def test_block_workspace_holds_the_lists_of_a_units_queries(group):
    """More than 512 units and so one range of keys, no partial results: units of eight row tiles, each with the lists of its queries and
    eight records behind them.  The most queries of a unit by counting them."""
    q, block, topn = 4096, 64, 300
    tile_q, per_query = max(1, min(16 // group, 8)), -(-group // 16)      # queries of a tile, tiles of a query
    first = [t // per_query if group > 16 else t * tile_q for t in range(0, 8 * 1000)]
    most = max(len({first[t + x] for x in range(8)}) * tile_q for t in range(0, len(first), 8))
    units = -(-(-(-q // tile_q) * per_query) // 8)
    for hk in (1, 4, 8, 16):
        if group * hk > 1024 or units * hk <= 512:
            continue
        got = E.block_workspace_size([q], [q * 20], group * hk, hk, 128, "bf16", block, topn)
        assert 0 <= got - units * hk * (most * topn + 8) * 16 < 512


def test_block_workspace_of_large_groups():
    """16 bytes an entry, not 128, where a query's heads fill a unit."""
    entries = 4096 * 2048
    for hq in (64, 128):
        got = E.block_workspace_size([4096], [1 << 20], hq, 1, 128, "bf16", 64, 2048)
        assert got <= 16 * entries + 128 * 4096 + 512


def test_block_workspace_of_lists_that_fill_no_whole_step():
    """150 blocks of 16, ranges in steps of 64 keys: room for 150 entries of a list, not 152."""
    got = E.block_workspace_size([70], [700], 512, 128, 64, "bf16", 16, 150)
    assert 0 <= got - 3 * 128 * (32 * 150 + 8) * 16 < 512
