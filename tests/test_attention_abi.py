"""Refusals of the attention entry points: every bad call is turned into an error on the host, before
anything touches a GPU.  The tensors are CPU tensors; the binding's own refusal of those is lifted, so
that a call gets to the library's checks."""
import contextlib
import ctypes
from types import SimpleNamespace

import pytest
import torch

import exact_top_token_amd as E
from exact_top_token_amd import attention as AT

STREAM = 0


@pytest.fixture(autouse=True)
def _cpu_tensors(request, monkeypatch):
    if "cpu_tensors_refused" not in request.node.name:
        monkeypatch.setattr(AT, "_on", lambda device, stream: contextlib.nullcontext(stream))


def test_cpu_tensors_refused():
    q = torch.zeros(1, 2, 64)
    c = _cache()
    acc = torch.zeros(4, 16)
    for stream in (None, 0):
        for call in (lambda: E.dsa_prompt_attention(q, q, q, [1], [1], torch.empty_like(q), workspace=_space(1 << 20), stream=stream),
                     lambda: E.dsa_cache_append(c, q, q, [1], [1], stream=stream),
                     lambda: E.dsa_cache_attention(c, q, [1], [1], torch.empty_like(q), workspace=_space(1 << 20), stream=stream),
                     lambda: E.dsa_cache_evict(acc, c.page_table, [1], [1], [], torch.zeros(1, 1, dtype=torch.int32),
                                               workspace=_space(1024), stream=stream)):
            with pytest.raises(E.DosaError) as ei:
                call()
            assert ei.value.status == -1 and "GPU" in str(ei.value)


def _space(n):
    return torch.empty(n, dtype=torch.uint8)


def _prompt(**over):
    a = dict(hq=4, hk=2, d=64, ql=[3, 2], kl=[3, 5], dtype=torch.bfloat16, scale=0.1, ws=None)
    a.update(over)
    nq, nk = sum(a["ql"]), sum(a["kl"])
    q = torch.zeros(nq, a["hq"], a["d"], dtype=a["dtype"])
    k = torch.zeros(nk, a["hk"], a["d"], dtype=a["dtype"])
    n = 1 << 20
    E.dsa_prompt_attention(q, k, k.clone(), a["ql"], a["kl"], torch.empty_like(q), None, scale=a["scale"],
                           workspace=_space(n) if a["ws"] is None else a["ws"], stream=STREAM)


@pytest.mark.parametrize("over,status", [
    (dict(ql=[4, 2], kl=[3, 5]), -1),
    (dict(ql=[-1, 2], kl=[3, 5]), -1),
    (dict(hq=5), -1),
    (dict(d=96), -2),
    (dict(d=32), -2),
    (dict(hq=2048, hk=1), -2),
    (dict(hq=129, hk=129), -2),
    (dict(dtype=torch.float16), -1),
    (dict(scale=0.0), -1),
    (dict(scale=-1.0), -1),
    (dict(scale=float("nan")), -1),
    (dict(scale=float("inf")), -1),
    (dict(scale=1e-40), -1),
    (dict(ws=_space(16)), -3),
])
def test_prompt_refusals(over, status):
    with pytest.raises(E.DosaError) as ei:
        _prompt(**over)
    assert ei.value.status == status and str(ei.value)


def test_prompt_layout_refusals():
    q = torch.zeros(4, 4, 64)
    k = torch.zeros(4, 2, 64)
    out, ws = torch.empty_like(q), _space(1 << 20)
    call = lambda **o: E.dsa_prompt_attention(**{**dict(q=q, k=k, v=k, q_lens=[4], kv_lens=[4], out=out, lse=None,
                                                        scale=0.1, workspace=ws, stream=STREAM), **o})
    bad = [
        dict(q=q.transpose(1, 2)),                                  # heads of a token not together
        dict(q=torch.zeros(4, 4, 128)[..., :64]),                   # gaps between heads
        dict(k=k.bfloat16()),
        dict(k=torch.zeros(5, 2, 64)),
        dict(v=torch.zeros(4, 1, 64)),
        dict(out=torch.zeros(4, 8, 64)[:, :4]),                     # strided output
        dict(out=out.bfloat16()),
        dict(lse=torch.zeros(4, 4, dtype=torch.float64)),
        dict(lse=torch.zeros(4, 5)),
        dict(lse=torch.zeros(4, 8)[:, :4]),
        dict(k=torch.zeros(4 * 130).as_strided((4, 2, 64), (130, 64, 1))),   # token stride not a multiple of 16 bytes
        dict(q=torch.zeros(4 * 256 + 1)[1:].view(4, 4, 64)),        # first row off 16 bytes
        dict(k=torch.zeros(1, 2, 64).expand(4, 2, 64)),             # tokens overlap
    ]
    for o in bad:
        with pytest.raises(E.DosaError) as ei:
            call(**o)
        assert ei.value.status == -1, o
    with pytest.raises(E.DosaError):
        call(q_lens=[4, 0])


def _cache(pages=4, page=16, hk=2, d=64, batch=2, per=2):
    return E.Cache.empty(pages, page, hk, d, torch.zeros(batch, per, dtype=torch.int32))


def test_cache_object_refusals():
    t = torch.zeros(1, 2, dtype=torch.int32)
    u = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    ok = (u(4, 16, 2, 32), u(4, 16, 2, 2), u(4, 16, 2, 32), u(4, 16, 2, 2))
    E.Cache(*ok, t)
    for i, x in ((0, u(4, 16, 2)), (1, u(4, 16, 2, 4)), (2, u(4, 16, 2, 64)[..., ::2]), (3, u(4, 16, 1, 2)),
                 (0, torch.zeros(4, 16, 2, 32))):
        bad = list(ok)
        bad[i] = x
        with pytest.raises(E.DosaError):
            E.Cache(*bad, t)
    with pytest.raises(E.DosaError):
        E.Cache(*ok, t.long())
    with pytest.raises(E.DosaError):
        E.Cache(*ok, t[0])


@pytest.mark.parametrize("fn", ["append", "read", "attend", "weights"])
@pytest.mark.parametrize("over,status", [
    (dict(page=20), -1),                       # not a multiple of 16
    (dict(d=96), -2),
    (dict(kl=[20, 40]), -1),                   # the table row ends before the keys
    (dict(ql=[21, 1]), -1),
    (dict(ql=[1, 1, 1], kl=[1, 1, 1]), -1),    # more sequences than table rows
])
def test_cache_refusals(fn, over, status):
    a = dict(page=16, d=64, ql=[1, 2], kl=[20, 32])
    a.update(over)
    c = _cache(page=a["page"], d=a["d"])
    nq = sum(a["ql"])
    x = torch.zeros(nq, 2, a["d"])
    q = torch.zeros(nq, 4, a["d"])
    acc = torch.zeros(4, a["page"])
    with pytest.raises(E.DosaError) as ei:
        if fn == "append":
            E.dsa_cache_append(c, x, x, a["ql"], a["kl"], stream=STREAM)
        elif fn == "read":
            E.dsa_cache_read(c, x, x.clone(), a["ql"], a["kl"], stream=STREAM)
        elif fn == "attend":
            E.dsa_cache_attention(c, q, a["ql"], a["kl"], torch.empty_like(q), workspace=_space(1 << 20), stream=STREAM)
        else:
            E.dsa_cache_weights(c, q, torch.zeros(nq, 4), a["ql"], a["kl"], acc, acc, workspace=_space(1 << 20),
                                stream=STREAM)
    assert ei.value.status == status, ei.value


def test_cache_attention_own_refusals():
    c = _cache()
    q = torch.zeros(3, 4, 64)
    call = lambda **o: E.dsa_cache_attention(**{**dict(cache=c, q=q, q_lens=[1, 2], kv_lens=[20, 32],
                                                       out=torch.empty_like(q), workspace=_space(1 << 20),
                                                       scale=0.1, stream=STREAM), **o})
    for o, status in ((dict(idx=torch.zeros(3, 0, dtype=torch.int32)), -1), (dict(idx=torch.zeros(2, 8, dtype=torch.int32)), -1),
                      (dict(idx=torch.zeros(3, 8, dtype=torch.int64)), -1), (dict(idx=torch.zeros(3, dtype=torch.int32)), -1),
                      (dict(workspace=None), -3), (dict(workspace=_space(8)), -3), (dict(q=torch.zeros(3, 3, 64)), -1),
                      (dict(scale=-0.5), -1)):
        if "q" in o:
            o = dict(o, out=torch.empty_like(o["q"]))
        with pytest.raises(E.DosaError) as ei:
            call(**o)
        assert ei.value.status == status, (o, ei.value)


def test_weights_and_append_own_refusals():
    c = _cache()
    q, lse, acc = torch.zeros(3, 4, 64), torch.zeros(3, 4), torch.zeros(4, 16)
    w = lambda **o: E.dsa_cache_weights(**{**dict(cache=c, q=q, lse=lse, q_lens=[1, 2], kv_lens=[20, 32], acc=acc,
                                                  acc_out=acc, workspace=_space(1 << 20), scale=0.1, stream=STREAM), **o})
    for o, status in ((dict(lse=None), -1), (dict(acc_out=None), -1), (dict(acc=acc.double()), -1),
                      (dict(acc_out=torch.zeros(4, 17)), -1), (dict(workspace=_space(8)), -3), (dict(scale=0.0), -1)):
        with pytest.raises(E.DosaError) as ei:
            w(**o)
        assert ei.value.status == status, o
    x = torch.zeros(3, 2, 64)
    for o in (dict(pos=torch.zeros(4, 16)), dict(pos=torch.zeros(4, 15, dtype=torch.int32)), dict(seen_lens=[19, 32]),
              dict(seen_lens=[20])):
        with pytest.raises(E.DosaError) as ei:
            E.dsa_cache_append(c, x, x, [1, 2], [20, 32], stream=STREAM, **o)
        assert ei.value.status == -1, o


def test_evict_refusals():
    acc = torch.zeros(4, 16)
    base = dict(acc=acc, page_table=torch.zeros(2, 2, dtype=torch.int32), kv_lens=[20, 32], new_lens=[10, 32],
                arrays=[], out_src=torch.zeros(2, 32, dtype=torch.int32), workspace=_space(4096), stream=STREAM)
    pos, other = torch.zeros(4, 16, dtype=torch.int32), torch.zeros(4, 16)
    for o, status in (
            (dict(new_lens=[21, 32]), -1), (dict(new_lens=[-1, 32]), -1), (dict(kv_lens=[20, 33]), -1),
            (dict(prefix=-1), -1), (dict(window=-2), -1), (dict(prefix=4, window=7), -1),
            (dict(out_src=torch.zeros(2, 31, dtype=torch.int32)), -1), (dict(out_src=torch.zeros(1, 32, dtype=torch.int32)), -1),
            (dict(out_src=torch.zeros(2, 32)), -1), (dict(acc=acc.double()), -1), (dict(pos=pos[:3]), -1),
            (dict(seen_lens=[20, 32]), -1), (dict(pos=pos, seen_lens=[19, 32]), -1), (dict(workspace=None), -3),
            (dict(workspace=_space(64)), -3), (dict(arrays=[(acc, acc)] * 2), -1), (dict(arrays=[(other, acc)]), -1),
            (dict(arrays=[(acc, other), (other, other)]), -1), (dict(arrays=[(acc, pos)]), -1),
            (dict(arrays=[(acc[:3], acc[:3])]), -1), (dict(pos=pos, arrays=[(other.int(), pos)]), -1),
            (dict(arrays=[(acc, torch.zeros(4, 16)) for _ in range(17)]), -1)):
        with pytest.raises(E.DosaError) as ei:
            E.dsa_cache_evict(**{**base, **o})
        assert ei.value.status == status, (o, ei.value)


def test_null_pointers_and_reserved_at_the_c_interface():
    L = E.lib()
    one, two = AT._lens([1]), AT._lens([20])
    assert L.dsa_cache_append(None, 1 << 12, 128, 1 << 12, 128, 0, one, two, 1, None, None, None) == -1
    s = AT.DsaCache(1 << 12, 1 << 12, 1 << 12, 1 << 12, 1 << 12, 4, 16, 2, 2, 64, 0)
    call = lambda st, k=1 << 12: L.dsa_cache_append(ctypes.byref(st), k, 128, 1 << 12, 128, 0, one, two, 1, None, None, None)
    assert call(s, None) == -1
    for field, value in (("k_codes", None), ("v_scales", None), ("page_table", None), ("k_codes", (1 << 12) + 8),
                         ("k_scales", (1 << 12) + 2), ("num_pages", 0), ("page_size", 0), ("page_size", 8),
                         ("max_pages", 1), ("reserved", 1), ("Hkv", 0), ("d", 0)):
        t = AT.DsaCache.from_buffer_copy(s)
        setattr(t, field, value)
        assert call(t) == -1, field
    t = AT.DsaCache.from_buffer_copy(s)
    t.num_pages, t.page_size = 1 << 20, 1 << 12
    assert call(t) == -2
    assert L.dsa_prompt_attention(None, 64, 1 << 12, 64, 1 << 12, 64, 1, one, two, 1, 1, 1, 64, 0.1, 1 << 12, None,
                                  1 << 12, 1 << 20, None) == -1
    assert L.dsa_prompt_attention(1 << 12, 64, 1 << 12, 64, 1 << 12, 64, 2, one, two, 1, 1, 1, 64, 0.1, 1 << 12, None,
                                  1 << 12, 1 << 20, None) == -2            # fp8 is not a type of these calls
    assert L.dsa_prompt_attention(1 << 12, 64, 1 << 12, (1 << 23) + 8, 1 << 12, 64, 1, one, two, 1, 1, 1, 64, 0.1, 1 << 12,
                                  None, 1 << 12, 1 << 20, None) == -2      # token stride
    assert L.dsa_prompt_attention(1 << 12, 64, 1 << 12, 64, 1 << 12, 64, 1, None, two, 1, 1, 1, 64, 0.1, 1 << 12, None,
                                  1 << 12, 1 << 20, None) == -1
    assert L.dsa_prompt_attention(1 << 12, 64, 1 << 12, 64, 1 << 12, 64, 1, one, two, -1, 1, 1, 64, 0.1, 1 << 12, None,
                                  1 << 12, 1 << 20, None) == -1


def test_limits_of_32_bit_counts():
    L = E.lib()
    big = (1 << 31) - (1 << 16)
    one = AT._lens([1])
    # tokens of a batch, slots of a cache, rows of a sequence
    assert L.dsa_cache_workspace_size(1, one, AT._lens([big]), 8, 8, 64, 0) > 0
    assert L.dsa_cache_workspace_size(1, one, AT._lens([big + 1]), 8, 8, 64, 0) == 0
    assert L.dsa_cache_workspace_size(2, AT._lens([1, 1]), AT._lens([big - 5, 6]), 8, 8, 64, 0) == 0
    n = 1 << 25
    assert L.dsa_weights_workspace_size(1, AT._lens([n]), AT._lens([n]), 32, 1, 64) > 0
    assert L.dsa_weights_workspace_size(1, AT._lens([n + 1]), AT._lens([n + 1]), 32, 1, 64) == 0
    assert L.dsa_prompt_workspace_size(1, AT._lens([n + 1]), AT._lens([n + 1]), 32, 1, 64, 1) == 0
    s = AT.DsaCache(1 << 12, 1 << 12, 1 << 12, 1 << 12, 1 << 12, (1 << 27) - (1 << 12) + 1, 16, 2, 2, 64, 0)
    assert L.dsa_cache_append(ctypes.byref(s), 1 << 12, 128, 1 << 12, 128, 0, one, AT._lens([20]), 1, None, None, None) == -2
    acc = torch.zeros(4, 16)
    wide = torch.zeros(4, 16, (1 << 20) + 1, dtype=torch.uint8)
    with pytest.raises(E.DosaError) as ei:
        E.dsa_cache_evict(acc, torch.zeros(1, 2, dtype=torch.int32), [20], [10], [(wide, wide)],
                          torch.zeros(1, 10, dtype=torch.int32), workspace=_space(4096), stream=STREAM)
    assert ei.value.status == -2


def test_workspace_sizes():
    n = E.cache_workspace_size([1], [100000], 32, 8, 128)
    # partial outputs and statistics of at most a few thousand row tiles
    assert 8 * 16 * 128 * 4 < n < 128 << 20
    assert E.prompt_workspace_size([4096], [4096], 32, 8, 128, torch.bfloat16) > 0
    assert E.prompt_workspace_size([], [], 32, 8, 128, "f32") > 0
    assert E.weights_workspace_size([8192], [8192], 32, 8, 128) > 0
    assert E.evict_workspace_size([100], [50]) >= 200
    for bad in (lambda: E.cache_workspace_size([5], [4], 8, 8, 128), lambda: E.cache_workspace_size([1], [4], 8, 3, 128),
                lambda: E.cache_workspace_size([1], [4], 8, 8, 80), lambda: E.cache_workspace_size([1], [4], 8, 8, 64, -1),
                lambda: E.cache_workspace_size([1], [4], 8, 8, 64, (1 << 20) + 1),
                lambda: E.prompt_workspace_size([1], [4], 8, 8, 64, torch.float16),
                lambda: E.weights_workspace_size([1], [0], 8, 8, 64), lambda: E.evict_workspace_size([4], [5])):
        with pytest.raises(E.DosaError):
            bad()


def test_empty_calls_do_nothing():
    """No sequences or no queries: accepted, nothing is launched (there is no GPU here)."""
    e = torch.empty(0, 4, 64)
    E.dsa_prompt_attention(e, torch.empty(0, 2, 64), torch.empty(0, 2, 64), [], [], e, workspace=_space(256), scale=0.1,
                           stream=STREAM)
    E.dsa_prompt_attention(e, torch.empty(7, 2, 64), torch.empty(7, 2, 64), [0, 0], [0, 7], e, workspace=_space(256),
                           scale=0.1, stream=STREAM)
    c = _cache()
    x = torch.empty(0, 2, 64)
    E.dsa_cache_append(c, x, x, [0, 0], [5, 9], stream=STREAM)
    E.dsa_cache_read(c, x, x, [0, 0], [5, 9], stream=STREAM)
    E.dsa_cache_attention(c, e, [0, 0], [5, 9], e, workspace=_space(256), scale=0.1, stream=STREAM)
    E.dsa_cache_attention(c, e, [0, 0], [5, 9], e, idx=torch.empty(0, 8, dtype=torch.int32), workspace=_space(256), scale=0.1,
                          stream=STREAM)
    E.dsa_cache_weights(c, e, torch.empty(0, 4), [0, 0], [5, 9], None, torch.zeros(4, 16), workspace=_space(256), scale=0.1,
                        stream=STREAM)
    E.dsa_cache_evict(torch.zeros(4, 16), c.page_table, [], [], [], torch.empty(0, 0, dtype=torch.int32),
                      workspace=_space(256), stream=STREAM)


@pytest.mark.parametrize("scale", [2.4e38, 3.4e38])
def test_scales_whose_base_2_form_overflows_are_refused(scale):
    """scale * log2(e), which the kernels multiply by, must be finite in fp32."""
    q, c = torch.zeros(1, 2, 64), _cache()
    acc = torch.zeros(4, 16)
    for call in (lambda s: E.dsa_prompt_attention(q, q, q.clone(), [1], [1], torch.empty_like(q), scale=s,
                                                  workspace=_space(1 << 20), stream=STREAM),
                 lambda s: E.dsa_cache_attention(c, q, [1], [1], torch.empty_like(q), scale=s, workspace=_space(1 << 20),
                                                 stream=STREAM),
                 lambda s: E.dsa_cache_weights(c, q, torch.zeros(1, 2), [1], [1], acc, acc, scale=s,
                                               workspace=_space(1 << 20), stream=STREAM)):
        with pytest.raises(E.DosaError) as ei:
            call(scale)
        assert ei.value.status == -1 and "scale" in str(ei.value)


def test_workspace_size_of_zero_if_either_query_type_is_refused():
    """2^30 rows a head on 32 heads: 2^31 row tiles of 16 for fp32 queries, one more than a call may have, half
    as many for bf16 ones."""
    n = [1 << 30]
    with pytest.raises(E.DosaError) as ei:
        E.cache_workspace_size(n, n, 32, 32, 64)
    assert ei.value.status == -2
    assert E.cache_workspace_size(n, n, 31, 31, 64) > 0


def test_launches_of_2_32_threads_are_refused():
    """Calls whose lengths pass but whose launch would have too many threads; nothing is read of the pointers."""
    L, p, big = E.lib(), 1 << 12, 1 << 40
    n = lambda x: AT._lens([x])
    cache = lambda hk: ctypes.byref(AT.DsaCache(p, p, p, p, p, 4, 1 << 14, 1 << 16, hk, 64, 0))
    m = 1 << 20        # selected keys: a tile for each query and head
    assert L.dsa_cache_attention(cache(64), p, 64 * 64, 0, n(m), n(m), 1, 64, p, 2048, 0.1, p, None, p, big, None) == -2
    m = 1 << 27        # 2^30 rows a head
    assert L.dsa_prompt_attention(p, 64 * 64, p, 8 * 64, p, 8 * 64, 1, n(m), n(m), 1, 64, 8, 64, 0.1, p, None, p, big, None) == -2
    m = 1 << 30        # 2^24 tiles of 64 keys
    assert L.dsa_cache_weights(cache(1), p, 64, 0, p, n(40), n(m), 1, 1, 0.1, None, p, p, big, None) == -2
    m = 1 << 28
    for fn, tail in ((L.dsa_cache_append, (None, None, None)), (L.dsa_cache_read, (None,))):
        assert fn(cache(1), p, 64, p, 64, 1, n(m), n(m), 1, *tail) == -2
    assert L.dsa_cache_evict(p, None, p, 1 << 14, 1 << 16, 4, n(1 << 29), n(1 << 28), None, 1, 0, 0, None, 0, p, 1 << 28, p, big,
                             None) == -2
    assert "2^32" in E.status_string(-2)


def test_cpu_tensors_refused_and_streams_of_another_device():
    """A stream belongs to the tensors' device (the binding's own check, before it touches a GPU)."""
    other = SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=1 << 12)
    with pytest.raises(E.DosaError) as ei:
        with AT._On(torch.device("cuda", 0), other):
            pass
    assert ei.value.status == -1 and "stream" in str(ei.value)
