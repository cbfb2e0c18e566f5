"""A cache of keys and values in 8 bits for generation frame by frame or token by token:
the tables and slots of a step (cache_extend), the write of its new keys and values
(cache_write) and attention over the cache (attn_cache_fwd). Calls mirror the C ABI in
include/sparsp.h; argument marshalling only.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import BF16, CACHE_CAUSAL, F32, _buffer, _check, _I32, _new, _refuse, _space, _stream, _want, lib

CODE = torch.float8_e4m3fn


class CacheShape(ctypes.Structure):
    """blocks of bt tokens (64 or 128) with `heads` key/value heads of d columns (64 or 128)."""
    _fields_ = [(n, _I32) for n in ("blocks", "heads", "d", "bt")]


@dataclass
class CachePool:
    """Codes float8_e4m3fn [blocks, heads, bt, d] and scales float32 [blocks, heads] of K and
    V: a value is code * scale."""
    shape: CacheShape
    k: torch.Tensor
    k_scale: torch.Tensor
    v: torch.Tensor
    v_scale: torch.Tensor

    def addresses(self, dev: int) -> tuple:
        s = self.shape
        codes, scales = (s.blocks, s.heads, s.bt, s.d), (s.blocks, s.heads)
        return (_want("pool.k", self.k, codes, CODE, dev), _want("pool.k_scale", self.k_scale, scales, torch.float32, dev),
                _want("pool.v", self.v, codes, CODE, dev), _want("pool.v_scale", self.v_scale, scales, torch.float32, dev))


def block_pool(blocks: int, heads: int, d: int, bt: int, device="cuda") -> CachePool:
    """An empty pool."""
    codes, scales = (blocks, heads, bt, d), (blocks, heads)
    k, v = (torch.zeros(codes, dtype=torch.uint8, device=device).view(CODE) for _ in range(2))
    ks, vs = (torch.ones(scales, dtype=torch.float32, device=device) for _ in range(2))
    return CachePool(CacheShape(blocks, heads, d, bt), k, ks, v, vs)


def _table_dims(table, requests: int) -> tuple:
    if not isinstance(table, torch.Tensor) or table.dim() != 2 or table.shape[0] != requests or table.shape[1] < 1:
        _refuse("table", table, f"a contiguous [{requests}, blocks per request] int32 tensor")
    return tuple(table.shape)


def cache_extend(shape: CacheShape, length, add, free, table, tokens: int, used=None, len_out=None, start=None,
                 slots=None, used_out=None, status=None, stream=None):
    """The tables and slots of a step: request b holds length[b] tokens and gets add[b] more
    (int32 [B]); the blocks it needs come from free[used ...] (int32), request by request,
    and are entered into table (int32 [B, blocks per request], in place). tokens: the packed
    new tokens there is room for. Returns (len_out [B], start [B+1], slots [tokens],
    used_out [1]); len_out may be length and used_out used. Requests that find too few
    blocks or slots wait (CAPACITY in status): their length stays and their slots are -1. Their
    tokens keep their place in start, so attn_cache_fwd's rows there mean nothing: drop rows whose
    slot is -1 and bring those tokens again."""
    dev, i32 = torch.cuda.current_device(), torch.int32
    if not isinstance(length, torch.Tensor) or length.dim() != 1:
        _refuse("length", length, "a contiguous int32 [B] tensor")
    B = length.shape[0]
    dims = _table_dims(table, B)
    if len_out is None:
        len_out = _new(stream, (B,), i32, length.device)
    if start is None:
        start = _new(stream, (B + 1,), i32, length.device)
    if slots is None:
        slots = _new(stream, (tokens,), i32, length.device)
    if used_out is None:
        used_out = _new(stream, (1,), i32, length.device)
    _check("sparsp_cache_extend", lib().sparsp_cache_extend(
        ctypes.byref(shape), B, dims[1], _want("length", length, (B,), i32, dev), _want("add", add, (B,), i32, dev),
        _buffer("free", free, i32, dev), free.numel(), _want("used", used, (1,), i32, dev, True),
        _want("table", table, dims, i32, dev), _want("len_out", len_out, (B,), i32, dev),
        _want("start", start, (B + 1,), i32, dev), _want("slots", slots, (tokens,), i32, dev), tokens,
        _want("used_out", used_out, (1,), i32, dev), _buffer("status", status, i32, dev, True), _stream(stream)))
    return len_out, start, slots, used_out


def _rows(name: str, t, heads: int, d: int, dev: int, n: int | None = None) -> tuple:
    """(address, elements between tokens, between heads) of rows [tokens, heads, d] whose
    columns are contiguous."""
    if not isinstance(t, torch.Tensor) or t.dim() != 3 or t.get_device() != dev:
        _refuse(name, t, f"a [tokens, {heads}, {d}] tensor")
    shape, st = t.shape, t.stride()
    if shape[1] != heads or shape[2] != d or n is not None and shape[0] != n or shape[0] and st[2] != 1:
        _refuse(name, t, f"a [tokens, {heads}, {d}] tensor with contiguous columns")
    if shape[0] > 1 and st[0] == 0 or shape[0] and heads > 1 and st[1] == 0:   # the call takes 0 for packed rows
        _refuse(name, t, f"a [tokens, {heads}, {d}] tensor of its own, not a broadcast view,")
    # a stride over a single token or head says nothing
    return t.data_ptr(), st[0] if shape[0] > 1 else 0, st[1] if heads > 1 else 0


def cache_write(pool: CachePool, k, v, slots, status=None, stream=None) -> None:
    """Rounds new keys and values [tokens, heads, d] (float32 or bfloat16; any strides
    between tokens and heads, e.g. slices of a fused projection, or tile order
    transposed; no broadcast views) into the pool's blocks at `slots` (of cache_extend; negative: left out),
    with one power-of-two scale per block and head."""
    s, dev = pool.shape, torch.cuda.current_device()
    if not isinstance(slots, torch.Tensor) or slots.dim() != 1:
        _refuse("slots", slots, "a contiguous int32 [tokens] tensor")
    n = slots.shape[0]
    pk, pv = _rows("k", k, s.heads, s.d, dev, n), _rows("v", v, s.heads, s.d, dev, n)
    if k.dtype is not v.dtype or k.dtype not in (torch.float32, torch.bfloat16):
        _refuse("k and v", v, "float32 or bfloat16 of one kind")
    _check("sparsp_cache_write", lib().sparsp_cache_write(
        ctypes.byref(s), F32 if k.dtype is torch.float32 else BF16, *pk, *pv, _want("slots", slots, (n,), torch.int32, dev),
        n, *pool.addresses(dev), _buffer("status", status, torch.int32, dev, True), _stream(stream)))


def attn_cache_workspace_size(shape: CacheShape, requests: int, heads: int, tokens: int, max_add: int,
                              max_blocks: int) -> int:
    """Bytes of workspace of attn_cache_fwd with `heads` query heads, packed `tokens`, at most
    max_add of one request, and tables of max_blocks blocks."""
    return lib().sparsp_attn_cache_workspace_size(ctypes.byref(shape), requests, heads, tokens, max_add, max_blocks)


def attn_cache_fwd(pool: CachePool, q, start, length, table, max_add: int, scale: float = 0.0, causal: bool = True,
                   row_ptr=None, col_idx=None, o=None, lse=None, ws=None, status=None, stream=None):
    """Attention of packed new tokens q [tokens, H, d] (bfloat16, may be a slice of a fused
    projection) over the cache: request b has rows start[b] .. start[b+1]-1 (at most
    max_add), the last of its length[b] tokens, in the blocks table[b]. H is a multiple of
    the pool's heads. causal: a row sees the tokens up to its own, else all of its
    request. row_ptr, col_idx: the blocks seen, per request and key head (CSR). Rows of a
    request that waits in cache_extend (slots of -1) mean nothing. Returns
    (O [tokens, H, d], LSE [tokens, H]); a row that sees nothing has O = 0, LSE = -inf."""
    s, dev, i32 = pool.shape, torch.cuda.current_device(), torch.int32
    if not isinstance(length, torch.Tensor) or length.dim() != 1:
        _refuse("length", length, "a contiguous int32 [B] tensor")
    B = length.shape[0]
    dims = _table_dims(table, B)
    if not isinstance(q, torch.Tensor) or q.dim() != 3 or q.dtype is not torch.bfloat16:
        _refuse("q", q, "a bfloat16 [tokens, H, d] tensor")
    n, H = q.shape[:2]
    pq, qs, qh = _rows("q", q, H, s.d, dev)
    if qh not in (0, s.d):
        _refuse("q", q, "rows with contiguous heads")
    if o is None:
        o = _new(stream, (n, H, s.d), torch.bfloat16, q.device)
    if lse is None:
        lse = _new(stream, (n, H), torch.float32, q.device)
    if ws is None:
        ws = _new(stream, max(attn_cache_workspace_size(s, B, H, n, max_add, dims[1]), 16), torch.uint8, q.device)
    _check("sparsp_attn_cache_fwd", lib().sparsp_attn_cache_fwd(
        ctypes.byref(s), B, H, pq, qs, _want("start", start, (B + 1,), i32, dev), n, max_add,
        _want("length", length, (B,), i32, dev), _want("table", table, dims, i32, dev), dims[1], *pool.addresses(dev),
        _want("row_ptr", row_ptr, (B * s.heads + 1,), i32, dev, True), _buffer("col_idx", col_idx, i32, dev, True),
        0 if col_idx is None else col_idx.numel(), scale, CACHE_CAUSAL if causal else 0,
        _want("o", o, (n, H, s.d), torch.bfloat16, dev), _want("lse", lse, (n, H), torch.float32, dev), *_space(ws, dev),
        _buffer("status", status, i32, dev, True), _stream(stream)))
    return o, lse
