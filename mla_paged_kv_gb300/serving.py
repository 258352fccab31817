"""Operators around the decode: filling a paged cache, sharing and moving its
pages, and attention over the prompts that fill it (see include/mla_serving.h).

Functions named ``mla_*`` mirror the C entry points: they check torch tensors
and marshal them into pointers, sizes and a CUDA stream.  The helpers
(``cache_append``, ``cache_grow``, ``cache_fork``, ``cache_free``,
``cache_compact``, ``cache_copy_pages``, ``plan_prompt``, ``prompt_attention``,
``plan_shared_prefix``, ``shared_prefix_decode``) allocate outputs.  A helper without ``status`` reads the device status after
its call (which waits for the GPU) and raises ``MlaError``; with ``status`` (an
int32 tensor the caller zeroed) it does not wait, and the caller looks at the
word when it wants to.

Every tensor of a call lives on one device, which must be the current one;
tensors used on a stream other than the one they were made on follow torch's
usual rules (``record_stream``, events).
"""

from __future__ import annotations

import ctypes
import math

import torch

from . import (DTYPE_FP8_RECORD, _DTYPE_CODE, _F, _I, _P, _SZ, _check, _ptr, _stream, check_status, load_library,
               mla_num_parts)

_LL = ctypes.c_longlong

SERVING_SIGS = {
    "mla_cache_append": (_I, [_P, _LL, _P, _LL, _I, _I, _P, _P, _I, _P, _I, _P, _I, _I, _P, _F, _P, _I, _I, _P, _P,
                              _P]),
    "mla_cache_grow": (_I, [_P, _I, _P, _I, _I, _P, _P, _P, _I, _P, _P]),
    "mla_cache_fork": (_I, [_P, _I, _P, _I, _I, _P, _P, _P, _I, _P, _P, _P]),
    "mla_cache_free": (_I, [_P, _I, _P, _I, _I, _P, _P, _I, _P, _P]),
    "mla_cache_compact_workspace_bytes": (_SZ, [_I]),
    "mla_cache_compact": (_I, [_P, _I, _P, _I, _I, _P, _P, _P, _P, _SZ, _P, _P]),
    "mla_cache_copy_pages": (_I, [_P, _I, _LL, _I, _LL, _P, _P, _I, _P, _P]),
    "mla_prompt_plan_bytes": (_SZ, [_I, _I]),
    "mla_prompt_get_plan": (_I, [_P, _P, _I, _I, _I, _I, _P, _SZ, _P, _P]),
    "mla_prompt_attention_fwd": (_I, [_P, _LL, _LL, _P, _LL, _LL, _P, _LL, _LL, _I, _I, _I, _I, _I, _I, _I, _F, _P,
                                      _SZ, _P, _P, _P, _P]),
    "mla_shared_prefix_plan_bytes": (_SZ, [_I, _I, _I, _I]),
    "mla_shared_prefix_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "mla_shared_prefix_get_plan": (_I, [_P, _I, _P, _I, _I, _I, _I, _I, _P, _SZ, _P]),
    "mla_shared_prefix_decode_fwd": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P, _SZ, _I, _P, _SZ, _P, _I, _P,
                                          _P, _P]),
}
SERVING_SYMBOLS = tuple(SERVING_SIGS)

__all__ = [n for n in SERVING_SYMBOLS] + [
    "SERVING_SYMBOLS", "cache_append", "cache_grow", "cache_fork", "cache_free", "cache_compact", "cache_copy_pages",
    "PromptPlan", "plan_prompt", "prompt_attention", "SharedPrefixPlan", "plan_shared_prefix", "shared_prefix_decode",
]


def _same_device(first, *rest):
    """Checks that every tensor is on `first`'s CUDA device and that it is current."""
    dev = first.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    for t in rest:
        if t is not None and t.device != dev:
            raise ValueError(f"tensors on different devices: {dev} and {t.device}")
    if dev.index != torch.cuda.current_device():
        raise ValueError(f"tensors are on {dev}, the current device is cuda:{torch.cuda.current_device()}")


def _plain(t, dtype, name, dims):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != dims or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with {dims} dims, got {tuple(t.shape)}")


def _rows16(t, dtype, width, name):
    """A [n, width] tensor of 16-bit values with contiguous rows; its row stride."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2 or t.shape[1] != width or t.stride(1) != 1:
        raise ValueError(f"{name} must be [tokens, {width}] with contiguous rows")
    return t.stride(0) if t.shape[0] > 1 else width


def _status(status, like):
    if status is None:
        return torch.zeros(1, dtype=torch.int32, device=like.device)
    _plain(status, torch.int32, "status", 1)
    return status


# ------------------------------------------------------------------ append


def mla_cache_append(c, r, cache, block_table, cache_seqlens, status, cu_seqlens=None, norm_weight=None,
                     norm_eps=1e-6, cos_sin=None, rope_interleaved=False, refcount=None, stream=None):
    """New tokens' latent rows c [tokens, 512] and RoPE rows r [tokens, 64]
    (bf16 or fp16, row strides free) into a paged cache: 16-bit
    [pages, 64, 576] of the same type, or FP8 records uint8 [pages, 64, 656]."""
    if c.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError("c must be bf16 or fp16")
    cs, rs = _rows16(c, c.dtype, 512, "c"), _rows16(r, c.dtype, 64, "r")
    if r.shape[0] != c.shape[0]:
        raise ValueError("c and r must have the same number of tokens")
    if cs % 8 or rs % 8:
        raise ValueError("row strides of c and r must be multiples of 8 elements")
    fp8 = cache.dtype == torch.uint8
    _plain(cache, torch.uint8 if fp8 else c.dtype, "cache", 3)
    if cache.shape[1] != 64 or cache.shape[2] != (656 if fp8 else 576):
        raise ValueError("cache must be [pages, 64, 576] (16-bit) or [pages, 64, 656] (uint8 records)")
    _plain(block_table, torch.int32, "block_table", 2)
    _plain(cache_seqlens, torch.int32, "cache_seqlens", 1)
    batch = block_table.shape[0]
    if cache_seqlens.shape[0] != batch:
        raise ValueError("block_table / cache_seqlens batch mismatch")
    if cu_seqlens is not None:
        _plain(cu_seqlens, torch.int32, "cu_seqlens", 1)
        if cu_seqlens.shape[0] != batch + 1:
            raise ValueError("cu_seqlens must have batch + 1 entries")
    elif batch == 0 or c.shape[0] % batch:
        raise ValueError("without cu_seqlens every request has tokens / batch tokens")
    if norm_weight is not None:
        _plain(norm_weight, c.dtype, "norm_weight", 1)
        if norm_weight.shape[0] != 512:
            raise ValueError("norm_weight must have 512 entries")
    if cos_sin is not None:
        _plain(cos_sin, torch.float32, "cos_sin", 2)
        if cos_sin.shape[1] != 64:
            raise ValueError("cos_sin must be [positions, 64]: 32 cosines, 32 sines")
    if refcount is not None:
        _plain(refcount, torch.int32, "refcount", 1)
        if refcount.shape[0] != cache.shape[0]:
            raise ValueError("refcount must have one entry a page")
    _plain(status, torch.int32, "status", 1)
    _same_device(c, r, cache, block_table, cache_seqlens, cu_seqlens, norm_weight, cos_sin, refcount, status)
    _check(load_library().mla_cache_append(
        c.data_ptr(), cs, r.data_ptr(), rs, _DTYPE_CODE[c.dtype], c.shape[0], _ptr(cu_seqlens),
        cache_seqlens.data_ptr(), batch, block_table.data_ptr(), block_table.shape[1], cache.data_ptr(),
        DTYPE_FP8_RECORD if fp8 else _DTYPE_CODE[c.dtype], cache.shape[0], _ptr(norm_weight), norm_eps,
        _ptr(cos_sin), 0 if cos_sin is None else cos_sin.shape[0], 1 if rope_interleaved else 0, _ptr(refcount),
        status.data_ptr(), _stream(stream)), "mla_cache_append")


def cache_append(c, r, cache, block_table, cache_seqlens, cu_seqlens=None, norm_weight=None, norm_eps=1e-6,
                 cos_sin=None, rope_interleaved=False, refcount=None, status=None):
    """Append new tokens to the cache in place (see mla_cache_append)."""
    st = _status(status, c)
    mla_cache_append(c, r, cache, block_table, cache_seqlens, st, cu_seqlens, norm_weight, norm_eps, cos_sin,
                     rope_interleaved, refcount)
    if status is None:
        check_status(st, "mla_cache_append")


# ------------------------------------------------------------------ pages


def _pages(refcount, block_table, seqlens, status, *lists):
    _plain(refcount, torch.int32, "refcount", 1)
    _plain(block_table, torch.int32, "block_table", 2)
    _plain(seqlens, torch.int32, "seqlens", 1)
    if seqlens.shape[0] != block_table.shape[0]:
        raise ValueError("block_table / seqlens row mismatch")
    for t in lists:
        _plain(t, torch.int32, "list", 1)
        if t.shape[0] != lists[0].shape[0]:
            raise ValueError("lists of different lengths")
    _plain(status, torch.int32, "status", 1)
    _same_device(refcount, block_table, seqlens, status, *lists)
    return (refcount.data_ptr(), refcount.shape[0], block_table.data_ptr(), block_table.shape[0],
            block_table.shape[1], seqlens.data_ptr())


def mla_cache_grow(refcount, block_table, seqlens, rows, new_tokens, status, stream=None):
    args = _pages(refcount, block_table, seqlens, status, rows, new_tokens)
    _check(load_library().mla_cache_grow(*args, rows.data_ptr(), new_tokens.data_ptr(), rows.shape[0],
                                         status.data_ptr(), _stream(stream)), "mla_cache_grow")


def mla_cache_fork(refcount, block_table, seqlens, parents, children, pairs, status, stream=None):
    args = _pages(refcount, block_table, seqlens, status, parents, children)
    _plain(pairs, torch.int32, "pairs", 2)
    if tuple(pairs.shape) != (parents.shape[0], 2):
        raise ValueError("pairs must be [n, 2]")
    _same_device(refcount, pairs)
    _check(load_library().mla_cache_fork(*args, parents.data_ptr(), children.data_ptr(), parents.shape[0],
                                         pairs.data_ptr(), status.data_ptr(), _stream(stream)), "mla_cache_fork")


def mla_cache_free(refcount, block_table, seqlens, rows, status, stream=None):
    args = _pages(refcount, block_table, seqlens, status, rows)
    _check(load_library().mla_cache_free(*args, rows.data_ptr(), rows.shape[0], status.data_ptr(), _stream(stream)),
           "mla_cache_free")


def mla_cache_compact_workspace_bytes(num_pages: int) -> int:
    return int(load_library().mla_cache_compact_workspace_bytes(int(num_pages)))


def mla_cache_compact(refcount, block_table, seqlens, pairs, count, workspace, status, stream=None):
    args = _pages(refcount, block_table, seqlens, status)
    _plain(pairs, torch.int32, "pairs", 2)
    _plain(count, torch.int32, "count", 1)
    _plain(workspace, torch.uint8, "workspace", 1)
    if pairs.shape[0] < refcount.shape[0] // 2 or pairs.shape[1] != 2 or count.shape[0] < 1:
        raise ValueError("pairs must be [num_pages // 2, 2] and count have one entry")
    _same_device(refcount, pairs, count, workspace)
    _check(load_library().mla_cache_compact(*args, pairs.data_ptr(), count.data_ptr(), workspace.data_ptr(),
                                            workspace.numel(), status.data_ptr(), _stream(stream)),
           "mla_cache_compact")


def mla_cache_copy_pages(pool, pairs, status, count=None, layered=False, stream=None):
    """pool: [pages, ...], or with layered [layers, pages, ...]; any type, pages
    contiguous and one after another; layers may be any distance apart."""
    lead = 2 if layered else 1
    if pool.dim() < lead + 1:
        raise ValueError("pool must be [pages, ...] or, layered, [layers, pages, ...]")
    first = pool[0] if layered else pool
    if not first.is_contiguous():
        raise ValueError("the pages of a layer must be contiguous")
    _plain(pairs, torch.int32, "pairs", 2)
    if pairs.shape[1] != 2:
        raise ValueError("pairs must be [n, 2]")
    if count is not None:
        _plain(count, torch.int32, "count", 1)
    _plain(status, torch.int32, "status", 1)
    _same_device(pool, pairs, count, status)
    size = pool.element_size()
    layers = pool.shape[0] if layered else 1
    page_bytes = first.stride(0) * size if first.shape[0] > 1 else first[0].numel() * size
    if page_bytes % 16 or (layers > 1 and pool.stride(0) * size % 16):
        raise ValueError("pages and layers must be multiples of 16 bytes")
    _check(load_library().mla_cache_copy_pages(
        pool.data_ptr(), layers, pool.stride(0) * size if layers > 1 else 0, first.shape[0], page_bytes,
        pairs.data_ptr(), _ptr(count), pairs.shape[0], status.data_ptr(), _stream(stream)), "mla_cache_copy_pages")


def cache_grow(refcount, block_table, seqlens, rows, new_tokens, status=None):
    """Lengthen rows of the block table in place, taking free pages."""
    st = _status(status, refcount)
    mla_cache_grow(refcount, block_table, seqlens, rows, new_tokens, st)
    if status is None:
        check_status(st, "mla_cache_grow")


def cache_fork(refcount, block_table, seqlens, parents, children, status=None):
    """Fork rows in place; returns the page pairs for cache_copy_pages."""
    st = _status(status, refcount)
    pairs = torch.empty(parents.shape[0], 2, dtype=torch.int32, device=refcount.device)
    mla_cache_fork(refcount, block_table, seqlens, parents, children, pairs, st)
    if status is None:
        check_status(st, "mla_cache_fork")
    return pairs


def cache_free(refcount, block_table, seqlens, rows, status=None):
    """Free rows in place."""
    st = _status(status, refcount)
    mla_cache_free(refcount, block_table, seqlens, rows, st)
    if status is None:
        check_status(st, "mla_cache_free")


def cache_compact(refcount, block_table, seqlens, status=None):
    """Move the pages in use to the front, bookkeeping only; returns the page
    pairs and their number (on the device) for cache_copy_pages."""
    st = _status(status, refcount)
    n = refcount.shape[0]
    pairs = torch.empty(n // 2, 2, dtype=torch.int32, device=refcount.device)
    count = torch.empty(1, dtype=torch.int32, device=refcount.device)
    ws = torch.empty(mla_cache_compact_workspace_bytes(n), dtype=torch.uint8, device=refcount.device)
    mla_cache_compact(refcount, block_table, seqlens, pairs, count, ws, st)
    if status is None:
        check_status(st, "mla_cache_compact")
    return pairs, count


def cache_copy_pages(pool, pairs, count=None, layered=False, status=None):
    """Copy pages inside the pool, for one layer or (layered) all of them."""
    st = _status(status, pairs)
    mla_cache_copy_pages(pool, pairs, st, count, layered)
    if status is None:
        check_status(st, "mla_cache_copy_pages")


# ------------------------------------------------------------------ prompt


class PromptPlan:
    """The tile list of a batch of prompts: reused by every layer."""

    def __init__(self, plan, batch, total_q, total_k, causal):
        self.plan = plan
        self.batch = batch
        self.total_q = total_q
        self.total_k = total_k
        self.causal = causal


def mla_prompt_plan_bytes(batch: int, total_q: int) -> int:
    return int(load_library().mla_prompt_plan_bytes(int(batch), int(total_q)))


def mla_prompt_get_plan(cu_seqlens_q, cu_seqlens_k, total_q, total_k, causal, plan, status, stream=None):
    _plain(cu_seqlens_q, torch.int32, "cu_seqlens_q", 1)
    if cu_seqlens_k is not None:
        _plain(cu_seqlens_k, torch.int32, "cu_seqlens_k", 1)
        if cu_seqlens_k.shape != cu_seqlens_q.shape:
            raise ValueError("cu_seqlens_q and cu_seqlens_k must have the same length")
    _plain(plan, torch.uint8, "plan", 1)
    _plain(status, torch.int32, "status", 1)
    _same_device(cu_seqlens_q, cu_seqlens_k, plan, status)
    _check(load_library().mla_prompt_get_plan(
        cu_seqlens_q.data_ptr(), _ptr(cu_seqlens_k), cu_seqlens_q.shape[0] - 1, int(total_q), int(total_k),
        1 if causal else 0, plan.data_ptr(), plan.numel(), status.data_ptr(), _stream(stream)),
        "mla_prompt_get_plan")


def mla_prompt_attention_fwd(q, k, v, pl, out, lse, status, softmax_scale=None, stream=None):
    """q [total_q, h_q, 192 or 128], k [total_k, h_kv, same], v [total_k, h_kv,
    128], bf16 or fp16, last dimension contiguous, other strides multiples of 8;
    pl a PromptPlan; out [total_q, h_q, 128] of q's type, lse fp32 [total_q, h_q]."""
    if q.dtype not in (torch.bfloat16, torch.float16) or k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k and v must be all bf16 or all fp16")
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k and v must be [tokens, heads, dim]")
    total_q, h_q, d = q.shape
    total_k, h_kv = k.shape[:2]
    if d not in (128, 192) or k.shape[2] != d or tuple(v.shape) != (total_k, h_kv, 128):
        raise ValueError("q and k must have 128 or 192 dims, v 128, k and v the same tokens and heads")
    if h_kv < 1 or h_q % h_kv:
        raise ValueError("the key heads must divide the query heads")
    if q.stride(2) != 1 or k.stride(2) != 1 or v.stride(2) != 1:
        raise ValueError("the last dimension of q, k and v must be contiguous")
    if pl.total_q != total_q or pl.total_k != total_k:
        raise ValueError("the plan was made for other token counts")
    _plain(out, q.dtype, "out", 3)
    _plain(lse, torch.float32, "lse", 2)
    if tuple(out.shape) != (total_q, h_q, 128) or tuple(lse.shape) != (total_q, h_q):
        raise ValueError("out must be [total_q, h_q, 128] and lse [total_q, h_q]")
    _plain(status, torch.int32, "status", 1)
    _same_device(q, k, v, pl.plan, out, lse, status)
    _check(load_library().mla_prompt_attention_fwd(
        q.data_ptr(), q.stride(0), q.stride(1), k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(), v.stride(0),
        v.stride(1), _DTYPE_CODE[q.dtype], total_q, total_k, pl.batch, h_q, h_kv, d,
        1.0 / math.sqrt(d) if softmax_scale is None else softmax_scale, pl.plan.data_ptr(), pl.plan.numel(),
        out.data_ptr(), lse.data_ptr(), status.data_ptr(), _stream(stream)), "mla_prompt_attention_fwd")


def plan_prompt(cu_seqlens_q, cu_seqlens_k=None, total_q=None, total_k=None, causal=True, status=None):
    """The plan of a batch of packed prompts.  total_q and total_k (the packed
    tensors' rows) default to the last offsets, which reads them from the GPU."""
    if total_q is None:
        total_q = int(cu_seqlens_q[-1])
    if total_k is None:
        total_k = total_q if cu_seqlens_k is None else int(cu_seqlens_k[-1])
    batch = cu_seqlens_q.shape[0] - 1
    if batch < 1:
        raise ValueError("cu_seqlens_q needs at least two entries")
    st = _status(status, cu_seqlens_q)
    plan = torch.empty(mla_prompt_plan_bytes(batch, total_q), dtype=torch.uint8, device=cu_seqlens_q.device)
    mla_prompt_get_plan(cu_seqlens_q, cu_seqlens_k, total_q, total_k, causal, plan, st)
    if status is None:
        check_status(st, "mla_prompt_get_plan")
    return PromptPlan(plan, batch, total_q, total_k, bool(causal))


def prompt_attention(q, k, v, cu_seqlens_q, cu_seqlens_k=None, causal=True, softmax_scale=None, pl=None,
                     status=None):
    """Attention over packed prompts; returns (out, lse)."""
    if pl is None:
        pl = plan_prompt(cu_seqlens_q, cu_seqlens_k, q.shape[0], k.shape[0], causal)
    elif pl.causal != bool(causal):
        raise ValueError("the plan was made with another causal setting")
    out = torch.empty(q.shape[0], q.shape[1], 128, dtype=q.dtype, device=q.device)
    lse = torch.empty(q.shape[0], q.shape[1], dtype=torch.float32, device=q.device)
    st = _status(status, q)
    mla_prompt_attention_fwd(q, k, v, pl, out, lse, st, softmax_scale)
    if status is None:
        check_status(st, "mla_prompt_attention_fwd")
    return out, lse


# ------------------------------------------------------------ shared prefix


class SharedPrefixPlan:
    """The units and split plan of a batch that shares a prefix, and its split
    workspace: reused by every layer of that batch, one call at a time."""

    def __init__(self, plan, batch, s_q, h_q, num_parts, causal, workspace):
        self.plan = plan
        self.batch = batch
        self.s_q = s_q
        self.h_q = h_q
        self.num_parts = num_parts
        self.causal = causal
        self.workspace = workspace


def mla_shared_prefix_plan_bytes(batch: int, s_q: int, h_q: int, num_parts: int) -> int:
    return int(load_library().mla_shared_prefix_plan_bytes(int(batch), int(s_q), int(h_q), int(num_parts)))


def mla_shared_prefix_workspace_bytes(batch: int, s_q: int, h_q: int, num_parts: int) -> int:
    return int(load_library().mla_shared_prefix_workspace_bytes(int(batch), int(s_q), int(h_q), int(num_parts)))


def mla_shared_prefix_get_plan(block_table, cache_seqlens, s_q, h_q, causal, num_parts, plan, stream=None):
    _plain(block_table, torch.int32, "block_table", 2)
    _plain(cache_seqlens, torch.int32, "cache_seqlens", 1)
    if cache_seqlens.shape[0] != block_table.shape[0]:
        raise ValueError("block_table / cache_seqlens batch mismatch")
    _plain(plan, torch.uint8, "plan", 1)
    _same_device(block_table, cache_seqlens, plan)
    _check(load_library().mla_shared_prefix_get_plan(
        block_table.data_ptr(), block_table.shape[1], cache_seqlens.data_ptr(), block_table.shape[0], int(s_q),
        int(h_q), 1 if causal else 0, int(num_parts), plan.data_ptr(), plan.numel(), _stream(stream)),
        "mla_shared_prefix_get_plan")


def mla_shared_prefix_decode_fwd(q, kv, block_table, pl, out, lse, status, softmax_scale=1.0 / 24.0, stream=None):
    """q [B, s_q, h_q, 576] and kv [pages, 64, 576], both bf16 or both fp16; pl a
    SharedPrefixPlan of this block table; out [B, s_q, h_q, 512] bf16, fp16 or
    fp32, lse fp32 [B, s_q, h_q]."""
    if q.dtype not in (torch.bfloat16, torch.float16) or kv.dtype != q.dtype:
        raise TypeError("q and kv must be both bf16 or both fp16")
    _plain(q, q.dtype, "q", 4)
    _plain(kv, q.dtype, "kv", 3)
    _plain(block_table, torch.int32, "block_table", 2)
    if out.dtype not in _DTYPE_CODE:
        raise TypeError("out must be bf16, fp16 or fp32")
    _plain(out, out.dtype, "out", 4)
    _plain(lse, torch.float32, "lse", 3)
    B, s_q, h_q, d = q.shape
    if d != 576 or tuple(kv.shape[1:]) != (64, 576):
        raise ValueError("q must be [B, s_q, h_q, 576] and kv [pages, 64, 576]")
    if tuple(out.shape) != (B, s_q, h_q, 512) or tuple(lse.shape) != (B, s_q, h_q):
        raise ValueError("out must be [B, s_q, h_q, 512] and lse [B, s_q, h_q]")
    if block_table.shape[0] != B or (pl.batch, pl.s_q, pl.h_q) != (B, s_q, h_q):
        raise ValueError("the plan or block table was made for another batch")
    _plain(status, torch.int32, "status", 1)
    _same_device(q, kv, block_table, pl.plan, pl.workspace, out, lse, status)
    _check(load_library().mla_shared_prefix_decode_fwd(
        q.data_ptr(), kv.data_ptr(), block_table.data_ptr(), block_table.shape[1], kv.shape[0], B, s_q, h_q,
        _DTYPE_CODE[q.dtype], softmax_scale, pl.plan.data_ptr(), pl.plan.numel(), pl.num_parts,
        pl.workspace.data_ptr(), pl.workspace.numel(), out.data_ptr(), _DTYPE_CODE[out.dtype], lse.data_ptr(),
        status.data_ptr(), _stream(stream)), "mla_shared_prefix_decode_fwd")


def plan_shared_prefix(block_table, cache_seqlens, s_q, h_q, causal=False, num_parts=None):
    """The plan of a batch: finds the pages that all requests start with."""
    B = block_table.shape[0]
    parts = mla_num_parts(128) if num_parts is None else int(num_parts)
    size = mla_shared_prefix_plan_bytes(B, s_q, h_q, parts)
    if size == 0:
        raise ValueError("batch, s_q, h_q or num_parts out of range")
    plan = torch.empty(size, dtype=torch.uint8, device=block_table.device)
    ws = torch.empty(mla_shared_prefix_workspace_bytes(B, s_q, h_q, parts), dtype=torch.uint8,
                     device=block_table.device)
    mla_shared_prefix_get_plan(block_table, cache_seqlens, s_q, h_q, causal, parts, plan)
    return SharedPrefixPlan(plan, B, s_q, h_q, parts, bool(causal), ws)


def shared_prefix_decode(q, kv, block_table, cache_seqlens, causal=False, softmax_scale=None, out_fp32=False,
                         pl=None, status=None):
    """Dense decode that attends the pages all requests share once; returns (out, lse)."""
    B, s_q, h_q, _ = q.shape
    if pl is None:
        pl = plan_shared_prefix(block_table, cache_seqlens, s_q, h_q, causal)
    elif pl.causal != bool(causal):
        raise ValueError("the plan was made with another causal setting")
    out = torch.empty(B, s_q, h_q, 512, dtype=torch.float32 if out_fp32 else q.dtype, device=q.device)
    lse = torch.empty(B, s_q, h_q, dtype=torch.float32, device=q.device)
    st = _status(status, q)
    mla_shared_prefix_decode_fwd(q, kv, block_table, pl, out, lse, st,
                                 1.0 / 24.0 if softmax_scale is None else softmax_scale)
    if status is None:
        check_status(st, "mla_shared_prefix_decode_fwd")
    return out, lse
