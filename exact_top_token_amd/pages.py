"""Python binding of paged keys and values in 16 or 32 bits.

Argument marshalling and the checks that need a tensor, as in attention.py;
arguments and results are those of include/dosa_indexer.h:

    dsa_pages_assign/release   page tables and slot maps from lengths
    Pages                      pages of keys and values, with their page table
    Blocks                     8-bit summaries of blocks of keys
    dsa_pages_append           write tokens (and summaries of completed blocks)
    dsa_pages_attention        attention of chunks and single tokens over the pages
    dsa_block_select           a few blocks per query and kv head
    dsa_block_attention        attention over listed blocks
"""
from __future__ import annotations

import ctypes
from typing import Optional

from . import attention as AT
from .attention import _bad, _check, _code, _lens, _lib, _rows, _size, _space, _tensor

_I32, _I64, _F32, _VP, _SZ = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t


class DsaPages(ctypes.Structure):
    _fields_ = [("k", _VP), ("v", _VP), ("page_table", _VP), ("dtype", _I32), ("num_pages", _I32), ("page_size", _I32),
                ("max_pages", _I32), ("Hkv", _I32), ("d", _I32)]


class DsaBlocks(ctypes.Structure):
    _fields_ = [("codes", _VP), ("scales", _VP), ("num_pages", _I32), ("page_size", _I32), ("block", _I32),
                ("Hkv", _I32), ("d", _I32), ("reserved", _I32)]


def declare(L) -> None:
    """Argument types of these entry points of a loaded library."""
    pp, pb, pi = ctypes.POINTER(DsaPages), ctypes.POINTER(DsaBlocks), ctypes.POINTER(_I32)
    for name, args, res in (
        ("dsa_pages_assign", [_VP, _I32, _I32, _I32, _VP, pi, _VP, _VP, _I32, _VP, _VP, _VP], ctypes.c_int),
        ("dsa_pages_release", [_VP, _I32, _I32, _I32, _VP, pi, _VP, _VP, _I32, _VP], ctypes.c_int),
        ("dsa_pages_append", [pp, pb, _VP, _I64, _VP, _I64, _VP, _VP, _I32, _VP], ctypes.c_int),
        ("dsa_pages_workspace_size", [_I32, _VP, _VP, _I32, _I32, _I32, _I32], _SZ),
        ("dsa_pages_attention", [pp, _VP, _I64, _VP, _VP, _I32, _I32, _F32, _VP, _VP, _VP, _SZ, _VP], ctypes.c_int),
        ("dsa_block_select", [pb, _VP, _I32, _VP, _I64, _I32, _VP, _VP, _I32, _I32, _I32, _I32, _VP, _I32, _VP],
         ctypes.c_int),
        ("dsa_block_workspace_size", [_I32, _VP, _VP, _I32, _I32, _I32, _I32, _I32, _I32], _SZ),
        ("dsa_block_attention", [pp, _VP, _I64, _VP, _VP, _I32, _I32, _VP, _I32, _I32, _F32, _VP, _VP, _VP, _SZ, _VP],
         ctypes.c_int),
    ):
        fn = getattr(L, name)
        fn.argtypes, fn.restype = args, res


def _torch():
    import torch

    return torch


def _table(page_table, device, batch: int):
    torch = _torch()
    if page_table.dim() != 2 or page_table.shape[0] < batch:
        _bad(f"page_table must be int32 [at least {batch}, max_pages]")
    return _tensor(page_table, "page_table", torch.int32, page_table.shape, device)


def _pair(a, b, an: str, bn: str) -> int:
    if len(a) != len(b):
        _bad(f"{an} and {bn} differ in length")
    return len(a)


class Pages:
    """Pages of keys and values: k, v fp32 or bf16 [num_pages, page_size, Hkv, d], page_table int32 [batch,
    max_pages], all contiguous on one device.  :meth:`empty` allocates the two."""

    def __init__(self, k, v, page_table):
        torch = _torch()
        if k.dim() != 4:
            _bad("k must be [num_pages, page_size, Hkv, d]")
        code = _code(k.dtype, "k")
        self.k, self.v, self.page_table, self.device, self.dtype = k, v, page_table, k.device, k.dtype
        self.num_pages, self.page_size, self.Hkv, self.d = k.shape
        for name in "kv":
            _tensor(getattr(self, name), name, k.dtype, k.shape, k.device)
        if page_table.dim() != 2:
            _bad("page_table must be int32 [batch, max_pages]")
        _tensor(page_table, "page_table", torch.int32, page_table.shape, k.device)
        self.batch, self.max_pages = page_table.shape
        self.struct = DsaPages(k.data_ptr(), v.data_ptr(), page_table.data_ptr(), code, self.num_pages, self.page_size,
                               self.max_pages, self.Hkv, self.d)

    @classmethod
    def empty(cls, num_pages: int, page_size: int, Hkv: int, d: int, page_table, dtype):
        torch = _torch()
        dtype = {"f32": torch.float32, "bf16": torch.bfloat16}.get(dtype, dtype)
        mk = lambda: torch.empty(num_pages, page_size, Hkv, d, dtype=dtype, device=page_table.device)
        return cls(mk(), mk(), page_table)

    def _batch(self, q_lens, kv_lens) -> int:
        if not (len(q_lens) == len(kv_lens) <= self.batch):
            _bad(f"{len(q_lens)} q_lens, {len(kv_lens)} kv_lens for a page table of {self.batch} rows")
        return len(q_lens)


class Blocks:
    """Summaries of the blocks of pages of ``page_size`` positions: codes int8 [num_pages, page_size / block,
    Hkv, d], scales uint8 [num_pages, page_size / block, Hkv], contiguous on one device."""

    def __init__(self, codes, scales, page_size: int):
        torch = _torch()
        if codes.dim() != 4 or codes.shape[1] == 0 or page_size % codes.shape[1] != 0:
            _bad("codes must be [num_pages, page_size / block, Hkv, d]")
        self.num_pages, per, self.Hkv, self.d = codes.shape
        self.codes, self.scales, self.device = codes, scales, codes.device
        self.page_size, self.block = int(page_size), int(page_size) // per
        _tensor(codes, "codes", torch.int8, codes.shape, codes.device)
        _tensor(scales, "scales", torch.uint8, codes.shape[:3], codes.device)
        self.struct = DsaBlocks(codes.data_ptr(), scales.data_ptr(), self.num_pages, self.page_size, self.block, self.Hkv,
                                self.d, 0)

    @classmethod
    def empty(cls, pages: Pages, block: int):
        torch = _torch()
        if block <= 0 or pages.page_size % block != 0:
            _bad("the block must divide page_size")
        shape = (pages.num_pages, pages.page_size // block, pages.Hkv)
        return cls(torch.empty(*shape, pages.d, dtype=torch.int8, device=pages.device),
                   torch.empty(*shape, dtype=torch.uint8, device=pages.device), pages.page_size)


def _free(page_table, free_pages, free_count):
    torch = _torch()
    if free_pages.dim() != 1:
        _bad("free_pages must be int32 [num_pages]")
    if not 0 <= free_count <= free_pages.shape[0]:
        _bad(f"free_count must be in 0..{free_pages.shape[0]}, is {free_count}")
    return _tensor(free_pages, "free_pages", torch.int32, free_pages.shape, page_table.device)


def dsa_pages_assign(page_table, page_size: int, free_pages, free_count: int, q_lens, kv_lens, slots=None,
                     positions=None, stream=None) -> int:
    """Give the sequences that grow by q_lens[b] tokens to kv_lens[b] the pages they need from the end of the
    free list (int32 [num_pages], free_count of them free); returns the number of pages left.  slots,
    positions int32 [total_q] or None: pool slot and position of each new token."""
    L, torch = _lib(), _torch()
    n = _pair(q_lens, kv_lens, "q_lens", "kv_lens")
    dev = page_table.device
    ptab, pfree = _table(page_table, dev, n), _free(page_table, free_pages, free_count)
    nq = sum(q_lens)
    ps, pp = _tensor(slots, "slots", torch.int32, (nq,), dev), _tensor(positions, "positions", torch.int32, (nq,), dev)
    left = _I32(int(free_count))
    with AT._on(dev, stream) as st:
        _check(L.dsa_pages_assign(ptab, page_table.shape[1], page_size, free_pages.shape[0], pfree, ctypes.byref(left),
                                  _lens(q_lens), _lens(kv_lens), n, ps, pp, st))
    return left.value


def dsa_pages_release(page_table, page_size: int, free_pages, free_count: int, new_lens, kv_lens, stream=None) -> int:
    """Give back the pages behind the first new_lens[b] tokens of each sequence; returns the number of free
    pages."""
    L = _lib()
    n = _pair(new_lens, kv_lens, "new_lens", "kv_lens")
    dev = page_table.device
    ptab, pfree = _table(page_table, dev, n), _free(page_table, free_pages, free_count)
    left = _I32(int(free_count))
    with AT._on(dev, stream) as st:
        _check(L.dsa_pages_release(ptab, page_table.shape[1], page_size, free_pages.shape[0], pfree, ctypes.byref(left),
                                   _lens(new_lens), _lens(kv_lens), n, st))
    return left.value


def dsa_pages_append(pages: Pages, k, v, q_lens, kv_lens, blocks: Optional[Blocks] = None, stream=None):
    """Write the newest q_lens[b] tokens of each sequence, k, v [total_q, Hkv, d] of the pages' type, and the
    summaries of the blocks that they complete.  k = v = None: the summaries alone, from the pages."""
    L = _lib()
    n = pages._batch(q_lens, kv_lens)
    nq = sum(q_lens)
    if blocks is not None and blocks.device != pages.device:
        _bad(f"blocks must be on {pages.device}")
    if (k is None) != (v is None) or (k is None and blocks is None):
        _bad("k and v go together, and without them blocks are needed")
    rows = (None, 0, None, 0)
    if k is not None:
        if k.device != pages.device or k.dtype != pages.dtype:
            _bad(f"k must be {pages.dtype} on {pages.device}")
        rows = (k.data_ptr(), _rows(k, "k", pages.Hkv, pages.d, nq, k), v.data_ptr(), _rows(v, "v", pages.Hkv, pages.d, nq, k))
    with AT._on(pages.device, stream) as st:
        _check(L.dsa_pages_append(ctypes.byref(pages.struct), None if blocks is None else ctypes.byref(blocks.struct), *rows,
                                  _lens(q_lens), _lens(kv_lens), n, st))


def pages_workspace_size(q_lens, kv_lens, Hq: int, Hkv: int, d: int, dtype) -> int:
    n = _pair(q_lens, kv_lens, "q_lens", "kv_lens")
    return _size(_lib().dsa_pages_workspace_size(n, _lens(q_lens), _lens(kv_lens), Hq, Hkv, d, _code(dtype, "dtype")),
                 "attention over pages")


def _queries(pages, q, q_lens, kv_lens, out, lse):
    """Checked operands of an attention call: (batch, tokens, heads, token stride, lse address)."""
    n = pages._batch(q_lens, kv_lens)
    nq = sum(q_lens)
    if q.dim() != 3 or q.device != pages.device or q.dtype != pages.dtype:
        _bad(f"q must be {pages.dtype} [tokens, heads, d] on {pages.device}")
    hq = q.shape[1]
    sq = _rows(q, "q", hq, pages.d, nq, q)
    _rows(out, "out", hq, pages.d, nq, q, True)
    return n, nq, hq, sq, _tensor(lse, "lse", _torch().float32, (nq, hq), q.device)


def dsa_pages_attention(pages: Pages, q, q_lens, kv_lens, out, lse=None, scale: Optional[float] = None, workspace=None,
                        stream=None):
    """Attention of the newest q_lens[b] tokens over the pages: q, out [total_q, Hq, d] of the pages' type, lse
    fp32 [total_q, Hq] or None; scale defaults to d ** -0.5."""
    L = _lib()
    n, _, hq, sq, plse = _queries(pages, q, q_lens, kv_lens, out, lse)
    ws, nb = _space(workspace, q.device)
    with AT._on(q.device, stream) as st:
        _check(L.dsa_pages_attention(ctypes.byref(pages.struct), q.data_ptr(), sq, _lens(q_lens), _lens(kv_lens), n, hq,
                                     pages.d ** -0.5 if scale is None else scale, out.data_ptr(), plse, ws, nb, st))


def _listed(idx, nq: int, hk: int, device) -> int:
    if idx.dim() != 3 or idx.shape[2] == 0:
        _bad("idx must be int32 [total_q, Hkv, topn], topn at least 1")
    return _tensor(idx, "idx", _torch().int32, (nq, hk, idx.shape[2]), device)


def dsa_block_select(blocks: Blocks, page_table, q, q_lens, kv_lens, idx, sinks: int = 1, local: int = 2, stream=None):
    """Choose idx.shape[2] blocks for each query and kv head: q [total_q, Hq, d], idx int32 [total_q, Hkv, topn]."""
    L = _lib()
    n = _pair(q_lens, kv_lens, "q_lens", "kv_lens")
    nq = sum(q_lens)
    ptab = _table(page_table, blocks.device, n)
    if q.dim() != 3 or q.device != blocks.device:
        _bad(f"q must be [tokens, heads, d] on {blocks.device}")
    hq = q.shape[1]
    sq = _rows(q, "q", hq, blocks.d, nq, q)
    pidx = _listed(idx, nq, blocks.Hkv, blocks.device)
    with AT._on(blocks.device, stream) as st:
        _check(L.dsa_block_select(ctypes.byref(blocks.struct), ptab, page_table.shape[1], q.data_ptr(), sq,
                                  _code(q.dtype, "q"), _lens(q_lens), _lens(kv_lens), n, hq, sinks, local, pidx,
                                  idx.shape[2], st))


def block_workspace_size(q_lens, kv_lens, Hq: int, Hkv: int, d: int, dtype, block: int, topn: int) -> int:
    n = _pair(q_lens, kv_lens, "q_lens", "kv_lens")
    return _size(_lib().dsa_block_workspace_size(n, _lens(q_lens), _lens(kv_lens), Hq, Hkv, d, _code(dtype, "dtype"), block,
                                                 topn), "block attention")


def dsa_block_attention(pages: Pages, q, q_lens, kv_lens, idx, block: int, out, lse=None, scale: Optional[float] = None,
                        workspace=None, stream=None):
    """Attention of each query and kv head over the keys of its blocks idx [total_q, Hkv, topn]; otherwise as
    :func:`dsa_pages_attention`."""
    L = _lib()
    n, nq, hq, sq, plse = _queries(pages, q, q_lens, kv_lens, out, lse)
    pidx = _listed(idx, nq, pages.Hkv, pages.device)
    ws, nb = _space(workspace, q.device)
    with AT._on(q.device, stream) as st:
        _check(L.dsa_block_attention(ctypes.byref(pages.struct), q.data_ptr(), sq, _lens(q_lens), _lens(kv_lens), n, hq,
                                     pidx, idx.shape[2], block, pages.d ** -0.5 if scale is None else scale,
                                     out.data_ptr(), plse, ws, nb, st))
