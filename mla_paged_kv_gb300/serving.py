"""Operators around the decode: filling a paged cache, sharing and moving its
pages, and attention over the prompts that fill it (see include/mla_serving.h).

Functions named ``mla_*`` mirror the C entry points: they check torch tensors
and marshal them into pointers, sizes and a CUDA stream.  The helpers
(``cache_append``, ``cache_grow``, ``cache_fork``, ``cache_free``,
``cache_compact``, ``cache_copy_pages``, ``plan_prompt``, ``prompt_attention``,
``plan_shared_prefix``, ``shared_prefix_decode``) allocate outputs.  A helper
without ``status`` reads the device status after its call (which waits for the
GPU) and raises ``MlaError``; with ``status`` (an int32 tensor the caller zeroed)
it does not wait, and the caller looks at the word when it wants to.

Softmax scales default to the width of the heads a call is given:
1 / sqrt(192 or 128) in prompt attention, 1 / sqrt(576) in the decodes.  A model
whose prompt heads are expanded from the latent rows that it decodes over has one
scale, that of its prompt heads: give it to both.

Every tensor of a call lives on one device, which must be the current one;
tensors used on a stream other than the one they were made on follow torch's
usual rules (``record_stream``, events).
"""

from __future__ import annotations

import ctypes
import math
from struct import Struct

import torch

from . import (DTYPE_FP8_RECORD, _DTYPE_CODE, _F, _I, _P, _SZ, _check, check_status, load_library, MlaError)

_LL, _D = ctypes.c_longlong, ctypes.c_double
_DTYPE_CODE16 = {d: _DTYPE_CODE[d] for d in (torch.bfloat16, torch.float16)}

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
    "mla_prompt_attention_checked_fwd": (_I, [_P, _LL, _LL, _P, _LL, _LL, _P, _LL, _LL, _I, _I, _I, _I, _I, _I, _I,
                                              _F, _P, _P, _P, _SZ, _P, _P, _P, _P]),
    "mla_shared_prefix_num_parts": (_I, [_I, _I, _I]),
    "mla_shared_prefix_plan_bytes": (_SZ, [_I, _I, _I, _I]),
    "mla_shared_prefix_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "mla_shared_prefix_get_plan": (_I, [_P, _I, _P, _I, _I, _I, _I, _I, _P, _SZ, _P]),
    "mla_shared_prefix_decode_fwd": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _P, _SZ, _I, _P, _SZ, _P, _I,
                                          _P, _P, _P]),
    "mla_shared_prefix_decode_checked_fwd": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P, _SZ, _I, _P, _SZ,
                                                  _P, _I, _P, _P, _P]),
    "mla_rope_frequencies": (_I, [_I, _D, _I, _D, _D, _D, _D, ctypes.POINTER(_D), ctypes.POINTER(_D)]),
    "mla_rope_table": (_I, [ctypes.POINTER(_D), _I, _D, _LL, _I, _P, _P]),
    "mla_rope_heads": (_I, [_P, _LL, _LL, _P, _LL, _LL, _I, _P, _P, _LL, _LL, _P, _LL, _LL, _I, _P, _I, _I, _I, _I, _I,
                            _I, _F, _P, _P, _P, _I, _P, _I, _P, _P]),
    "mla_cache_gather": (_I, [_P, _I, _I, _P, _I, _P, _P, _I, _I, _P, _LL, _P, _P]),
    "mla_chunk_num_parts": (_I, []),
    "mla_chunk_plan_bytes": (_SZ, [_I, _I, _I, _I]),
    "mla_chunk_workspace_bytes": (_SZ, [_I]),
    "mla_chunk_get_plan": (_I, [_P, _P, _I, _I, _I, _I, _I, _P, _SZ, _P, _P]),
    "mla_chunk_attention_fwd": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P, _SZ, _I, _P, _SZ, _P, _I, _P,
                                     _P, _P]),
    "mla_serving_call": (_I, [_I, ctypes.c_char_p, _SZ]),
}
for _hook, _of in (("mla_test_prompt_timeout", "mla_prompt_attention_fwd"),
                   ("mla_test_shared_prefix_timeout", "mla_shared_prefix_decode_fwd"),
                   ("mla_test_chunk_timeout", "mla_chunk_attention_fwd")):
    SERVING_SIGS[_hook] = SERVING_SIGS[_of]
SERVING_SYMBOLS = tuple(SERVING_SIGS)


def _refuse(t, dtype, dims, dev, name):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != dims or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with {dims} dims, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be on cuda:{dev}, is on {t.device}")


def _p(t, dtype, dims, dev, name):
    """Address of a contiguous tensor of that type and rank on that device.  (A
    launch-bound call spends most of its time in checks like this: few attribute
    reads, and the wording of a refusal apart.)"""
    if t.dtype is dtype and t.dim() == dims and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    _refuse(t, dtype, dims, dev, name)


def _q(stream, dev):
    """The stream's handle (the given one, or the current one) for tensors on
    CUDA device dev, which must be the current device."""
    if dev < 0:
        raise ValueError("tensors must be on a CUDA device")
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"tensors are on cuda:{dev}, the current device is cuda:{torch._C._cuda_getDevice()}")
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _status(status, like):
    return torch.zeros(1, dtype=torch.int32, device=like.device) if status is None else status


_INT32, _FP32, _UINT8 = torch.int32, torch.float32, torch.uint8

# The calls of mla_serving_call (mla_call_t): number, packing of the argument
# words, their bytes.
def _words(op, layout):
    s = Struct(layout)
    return op, s.pack, s.size


_APPEND, _GROW, _FORK, _FREE = _words(0, "15qd6q"), _words(1, "11q"), _words(2, "12q"), _words(3, "10q")
_COMPACT, _COPY_PAGES, _PROMPT = _words(4, "12q"), _words(5, "10q"), _words(6, "16qd6q")
_SHARED_PREFIX, _SHARED_PREFIX_CHECKED = _words(7, "10qd10q"), _words(8, "10qd11q")
_PROMPT_CHECKED = _words(9, "16qd8q")


def _call(op, name, *args):
    rc = load_library().mla_serving_call(op[0], op[1](*args), op[2])
    if rc:
        _check(rc, name)


def mla_serving_call(op, args):
    """The packed form of the calls (bytes of 8-byte words), as the functions below use it."""
    args = bytes(args)
    _check(load_library().mla_serving_call(int(op), args, len(args)), "mla_serving_call")


# ------------------------------------------------------------------ append


def _row_stride(t, dtype, width, dev, name):
    """Row stride of a [tokens, width] tensor with contiguous rows."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    stride = t.stride()
    if len(stride) != 2 or t.shape[1] != width or stride[1] != 1:
        raise ValueError(f"{name} must be [tokens, {width}] with contiguous rows")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, is on {t.device}")
    if stride[0] % 8 and t.shape[0] > 1:
        raise ValueError(f"the row stride of {name} must be a multiple of 8 elements")
    return stride[0] if t.shape[0] > 1 else width


def mla_cache_append(c, r, cache, block_table, cache_seqlens, status, cu_seqlens=None, norm_weight=None,
                     norm_eps=1e-6, cos_sin=None, rope_interleaved=False, refcount=None, stream=None):
    """New tokens' latent rows c [tokens, 512] and RoPE rows r [tokens, 64]
    (bf16 or fp16, row strides free) into a paged cache: 16-bit
    [pages, 64, 576] of the same type, or FP8 records uint8 [pages, 64, 656]."""
    dt = c.dtype
    code = _DTYPE_CODE16.get(dt)
    if code is None:
        raise TypeError("c must be bf16 or fp16")
    dev = c.get_device()
    cs, rs = _row_stride(c, dt, 512, dev, "c"), _row_stride(r, dt, 64, dev, "r")
    tokens = c.shape[0]
    if r.shape[0] != tokens:
        raise ValueError("c and r must have the same number of tokens")
    fp8 = cache.dtype is _UINT8
    cache_ptr = _p(cache, _UINT8 if fp8 else dt, 3, dev, "cache")
    pages, page, width = cache.shape
    if page != 64 or width != (656 if fp8 else 576):
        raise ValueError("cache must be [pages, 64, 576] (16-bit) or [pages, 64, 656] (uint8 records)")
    table_ptr, lens_ptr = _p(block_table, _INT32, 2, dev, "block_table"), _p(cache_seqlens, _INT32, 1, dev,
                                                                             "cache_seqlens")
    batch, max_pages = block_table.shape
    if cache_seqlens.shape[0] != batch:
        raise ValueError("block_table / cache_seqlens batch mismatch")
    cu_ptr = weight_ptr = cos_ptr = ref_ptr = max_pos = 0
    if cu_seqlens is not None:
        cu_ptr = _p(cu_seqlens, _INT32, 1, dev, "cu_seqlens")
        if cu_seqlens.shape[0] != batch + 1:
            raise ValueError("cu_seqlens must have batch + 1 entries")
    elif batch == 0 or tokens % batch:
        raise ValueError("without cu_seqlens every request has tokens / batch tokens")
    if norm_weight is not None:
        weight_ptr = _p(norm_weight, dt, 1, dev, "norm_weight")
        if norm_weight.shape[0] != 512:
            raise ValueError("norm_weight must have 512 entries")
    if cos_sin is not None:
        cos_ptr = _p(cos_sin, _FP32, 2, dev, "cos_sin")
        max_pos, width = cos_sin.shape
        if width != 64:
            raise ValueError("cos_sin must be [positions, 64]: 32 cosines, 32 sines")
    if refcount is not None:
        ref_ptr = _p(refcount, _INT32, 1, dev, "refcount")
        if refcount.shape[0] != pages:
            raise ValueError("refcount must have one entry a page")
    st_ptr = _p(status, _INT32, 1, dev, "status")
    _call(
        _APPEND, "mla_cache_append", c.data_ptr(), cs, r.data_ptr(), rs, code, tokens, cu_ptr, lens_ptr, batch,
        table_ptr, max_pages, cache_ptr,
        DTYPE_FP8_RECORD if fp8 else code, pages, weight_ptr, norm_eps, cos_ptr, max_pos,
        1 if rope_interleaved else 0, ref_ptr, st_ptr, _q(stream, dev))


def cache_append(c, r, cache, block_table, cache_seqlens, cu_seqlens=None, norm_weight=None, norm_eps=1e-6,
                 cos_sin=None, rope_interleaved=False, refcount=None, status=None):
    """Append new tokens to the cache in place (see mla_cache_append)."""
    st = _status(status, c)
    mla_cache_append(c, r, cache, block_table, cache_seqlens, st, cu_seqlens, norm_weight, norm_eps, cos_sin,
                     rope_interleaved, refcount)
    if status is None:
        check_status(st, "mla_cache_append")


# ------------------------------------------------------------------ pages


def _pages(refcount, block_table, seqlens, dev):
    args = (_p(refcount, _INT32, 1, dev, "refcount"), refcount.shape[0],
            _p(block_table, _INT32, 2, dev, "block_table"), *block_table.shape, _p(seqlens, _INT32, 1, dev, "seqlens"))
    if seqlens.shape[0] != args[3]:
        raise ValueError("block_table / seqlens row mismatch")
    return args


def mla_cache_grow(refcount, block_table, seqlens, rows, new_tokens, status, stream=None):
    dev = refcount.get_device()
    args = _pages(refcount, block_table, seqlens, dev)
    rows_ptr, new_ptr = _p(rows, _INT32, 1, dev, "rows"), _p(new_tokens, _INT32, 1, dev, "new_tokens")
    n = rows.shape[0]
    if new_tokens.shape[0] != n:
        raise ValueError("rows and new_tokens must have the same length")
    _call(_GROW, "mla_cache_grow", *args, rows_ptr, new_ptr, n, _p(status, _INT32, 1, dev, "status"),
          _q(stream, dev))


def mla_cache_fork(refcount, block_table, seqlens, parents, children, pairs, status, stream=None):
    dev = refcount.get_device()
    args = _pages(refcount, block_table, seqlens, dev)
    par_ptr, chi_ptr = _p(parents, _INT32, 1, dev, "parents"), _p(children, _INT32, 1, dev, "children")
    pairs_ptr = _p(pairs, _INT32, 2, dev, "pairs")
    n = parents.shape[0]
    if children.shape[0] != n or pairs.shape != (n, 2):
        raise ValueError("parents and children must have the same length n, and pairs be [n, 2]")
    _call(_FORK, "mla_cache_fork", *args, par_ptr, chi_ptr, n, pairs_ptr, _p(status, _INT32, 1, dev, "status"),
          _q(stream, dev))


def mla_cache_free(refcount, block_table, seqlens, rows, status, stream=None):
    dev = refcount.get_device()
    args = _pages(refcount, block_table, seqlens, dev)
    _call(_FREE, "mla_cache_free", *args, _p(rows, _INT32, 1, dev, "rows"), rows.shape[0],
          _p(status, _INT32, 1, dev, "status"), _q(stream, dev))


def mla_cache_compact_workspace_bytes(num_pages: int) -> int:
    return int(load_library().mla_cache_compact_workspace_bytes(int(num_pages)))


def mla_cache_compact(refcount, block_table, seqlens, pairs, count, workspace, status, stream=None):
    dev = refcount.get_device()
    args = _pages(refcount, block_table, seqlens, dev)
    pairs_ptr, count_ptr = _p(pairs, _INT32, 2, dev, "pairs"), _p(count, _INT32, 1, dev, "count")
    ws_ptr = _p(workspace, _UINT8, 1, dev, "workspace")
    if pairs.shape[0] < args[1] // 2 or pairs.shape[1] != 2 or count.shape[0] < 1:
        raise ValueError("pairs must be [num_pages // 2, 2] and count have one entry")
    _call(_COMPACT, "mla_cache_compact", *args, pairs_ptr, count_ptr, ws_ptr, workspace.shape[0],
          _p(status, _INT32, 1, dev, "status"), _q(stream, dev))


def mla_cache_copy_pages(pool, pairs, status, count=None, layered=False, stream=None):
    """pool: [pages, ...], or with layered [layers, pages, ...]; any type, pages
    contiguous and one after another; layers may be any distance apart."""
    dev = pool.get_device()
    shape, strides, size = pool.shape, pool.stride(), pool.element_size()
    lead = 2 if layered else 1
    if len(shape) < lead + 1:
        raise ValueError("pool must be [pages, ...] or, layered, [layers, pages, ...]")
    layers, layer_stride = (shape[0], strides[0] * size) if layered else (1, 0)
    page = 1
    for n, step in zip(reversed(shape[lead:]), reversed(strides[lead:])):
        if n != 1 and step != page:
            raise ValueError("the pages of a layer must be contiguous")
        page *= n
    if shape[lead - 1] > 1 and strides[lead - 1] != page:
        raise ValueError("the pages of a layer must be contiguous")
    page *= size
    if page % 16 or (layers > 1 and layer_stride % 16):
        raise ValueError("pages and layers must be multiples of 16 bytes")
    pairs_ptr = _p(pairs, _INT32, 2, dev, "pairs")
    if pairs.shape[1] != 2:
        raise ValueError("pairs must be [n, 2]")
    _call(
        _COPY_PAGES, "mla_cache_copy_pages", pool.data_ptr(), layers, layer_stride if layers > 1 else 0,
        shape[lead - 1], page, pairs_ptr,
        0 if count is None else _p(count, _INT32, 1, dev, "count"), pairs.shape[0],
        _p(status, _INT32, 1, dev, "status"), _q(stream, dev))


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
        self.bytes = plan.numel()
        self.batch = batch
        self.total_q = total_q
        self.total_k = total_k
        self.causal = causal


def mla_prompt_plan_bytes(batch: int, total_q: int) -> int:
    return int(load_library().mla_prompt_plan_bytes(int(batch), int(total_q)))


def mla_prompt_get_plan(cu_seqlens_q, cu_seqlens_k, total_q, total_k, causal, plan, status, stream=None):
    dev = cu_seqlens_q.get_device()
    cu_q, cu_k = _p(cu_seqlens_q, _INT32, 1, dev, "cu_seqlens_q"), None
    if cu_seqlens_k is not None:
        cu_k = _p(cu_seqlens_k, _INT32, 1, dev, "cu_seqlens_k")
        if cu_seqlens_k.shape != cu_seqlens_q.shape:
            raise ValueError("cu_seqlens_q and cu_seqlens_k must have the same length")
    _check(load_library().mla_prompt_get_plan(
        cu_q, cu_k, cu_seqlens_q.shape[0] - 1, int(total_q), int(total_k), 1 if causal else 0,
        _p(plan, _UINT8, 1, dev, "plan"), plan.shape[0], _p(status, _INT32, 1, dev, "status"), _q(stream, dev)),
        "mla_prompt_get_plan")


def _prompt(q, k, v, pl, softmax_scale, status, stream, out=None, lse=None, cu_seqlens_q=None, cu_seqlens_k=None,
            hook=False):
    """The checks and the call of mla_prompt_attention_fwd (with offsets, _checked_fwd; hook:
    mla_test_prompt_timeout); allocates out and lse if not given."""
    dt = q.dtype
    code = _DTYPE_CODE16.get(dt)
    if code is None or k.dtype is not dt or v.dtype is not dt:
        raise TypeError("q, k and v must be all bf16 or all fp16")
    qs, ks, vs = q.stride(), k.stride(), v.stride()
    if len(qs) != 3 or len(ks) != 3 or len(vs) != 3:
        raise ValueError("q, k and v must be [tokens, heads, dim]")
    total_q, h_q, d = q.shape
    total_k, h_kv, dk = k.shape
    if (d != 192 and d != 128) or dk != d or v.shape != (total_k, h_kv, 128):
        raise ValueError("q and k must have 128 or 192 dims, v 128, k and v the same tokens and heads")
    if h_kv < 1 or h_q % h_kv:
        raise ValueError("the key heads must divide the query heads")
    if qs[2] != 1 or ks[2] != 1 or vs[2] != 1:
        raise ValueError("the last dimension of q, k and v must be contiguous")
    if pl.total_q != total_q or pl.total_k != total_k:
        raise ValueError("the plan was made for other token counts")
    dev = q.get_device()
    if k.get_device() != dev or v.get_device() != dev:
        raise ValueError("q, k and v must be on one device")
    st = _p(status, _INT32, 1, dev, "status")
    plan = _p(pl.plan, _UINT8, 1, dev, "plan")
    queue = _q(stream, dev)
    if out is None:
        out = torch.empty((total_q, h_q, 128), dtype=dt, device=q.device)
        lse = torch.empty((total_q, h_q), dtype=_FP32, device=q.device)
        out_ptr, lse_ptr = out.data_ptr(), lse.data_ptr()
    else:
        out_ptr, lse_ptr = _p(out, dt, 3, dev, "out"), _p(lse, _FP32, 2, dev, "lse")
        if out.shape != (total_q, h_q, 128) or lse.shape != (total_q, h_q):
            raise ValueError("out must be [total_q, h_q, 128] and lse [total_q, h_q]")
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(d)
    if cu_seqlens_q is None:
        args = (q.data_ptr(), qs[0], qs[1], k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1], code, total_q,
                total_k, pl.batch, h_q, h_kv, d, softmax_scale, plan, pl.bytes, out_ptr, lse_ptr, st, queue)
        if hook:
            _check(load_library().mla_test_prompt_timeout(*args), "mla_test_prompt_timeout")
        else:
            _call(_PROMPT, "mla_prompt_attention_fwd", *args)
        return out, lse
    cu_q, cu_k = _p(cu_seqlens_q, _INT32, 1, dev, "cu_seqlens_q"), 0
    if cu_seqlens_k is not None:
        cu_k = _p(cu_seqlens_k, _INT32, 1, dev, "cu_seqlens_k")
    if cu_seqlens_q.shape[0] != pl.batch + 1 or (cu_k and cu_seqlens_k.shape[0] != pl.batch + 1):
        raise ValueError("the plan was made for another batch")
    _call(_PROMPT_CHECKED, "mla_prompt_attention_checked_fwd", q.data_ptr(), qs[0], qs[1], k.data_ptr(), ks[0], ks[1],
          v.data_ptr(), vs[0], vs[1], code, total_q, total_k, pl.batch, h_q, h_kv, d, softmax_scale, cu_q, cu_k, plan,
          pl.bytes, out_ptr, lse_ptr, st, queue)
    return out, lse


def mla_prompt_attention_fwd(q, k, v, pl, out, lse, status, softmax_scale=None, stream=None):
    """q [total_q, h_q, 192 or 128], k [total_k, h_kv, same], v [total_k, h_kv,
    128], bf16 or fp16, last dimension contiguous, other strides multiples of 8;
    pl a PromptPlan; out [total_q, h_q, 128] of q's type, lse fp32 [total_q, h_q]."""
    _prompt(q, k, v, pl, softmax_scale, status, stream, out, lse)


def mla_prompt_attention_checked_fwd(q, k, v, cu_seqlens_q, cu_seqlens_k, pl, out, lse, status, softmax_scale=None,
                                     stream=None):
    """mla_prompt_attention_fwd that also compares the offsets [batch + 1] (cu_seqlens_k None: the same) with the
    plan's on the device: others are MLA_ERR_STALE_PLAN in status."""
    _prompt(q, k, v, pl, softmax_scale, status, stream, out, lse, cu_seqlens_q, cu_seqlens_k)


def mla_test_prompt_timeout(q, k, v, pl, out, lse, status, softmax_scale=None, stream=None):
    """Test hook: mla_prompt_attention_fwd whose first key tile is never loaded (status: MLA_ERR_TIMEOUT)."""
    _prompt(q, k, v, pl, softmax_scale, status, stream, out, lse, hook=True)


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
    """Attention over packed prompts; returns (out, lse).  softmax_scale defaults to 1 / sqrt(dims of q).

    A plan holds the offsets it was made for.  With pl they are compared with cu_seqlens_q and cu_seqlens_k on the
    device, and a plan of others is MLA_ERR_STALE_PLAN."""
    st = _status(status, q)
    if pl is None:  # a plan made here is that of the offsets
        pl = plan_prompt(cu_seqlens_q, cu_seqlens_k, q.shape[0], k.shape[0], causal, st)
        cu_seqlens_q = cu_seqlens_k = None
    elif pl.causal != bool(causal):
        raise ValueError("the plan was made with another causal setting")
    out, lse = _prompt(q, k, v, pl, softmax_scale, st, None, cu_seqlens_q=cu_seqlens_q, cu_seqlens_k=cu_seqlens_k)
    if status is None:
        check_status(st, "mla_prompt_attention_fwd")
    return out, lse


# ------------------------------------------------------------ shared prefix


class SharedPrefixPlan:
    """The units and split plan of a batch that shares a prefix, and its split
    workspace: reused by every layer of that batch, one call at a time."""

    def __init__(self, plan, batch, max_pages, s_q, h_q, num_parts, causal, workspace):
        self.plan = plan
        self.batch = batch
        self.max_pages = max_pages
        self.s_q = s_q
        self.h_q = h_q
        self.num_parts = num_parts
        self.causal = causal
        self.workspace = workspace


def mla_shared_prefix_num_parts(batch: int, s_q: int, h_q: int) -> int:
    n = load_library().mla_shared_prefix_num_parts(int(batch), int(s_q), int(h_q))
    if n < 1:
        raise MlaError(-n, "mla_shared_prefix_num_parts")
    return n


def mla_shared_prefix_plan_bytes(batch: int, s_q: int, h_q: int, num_parts: int) -> int:
    return int(load_library().mla_shared_prefix_plan_bytes(int(batch), int(s_q), int(h_q), int(num_parts)))


def mla_shared_prefix_workspace_bytes(batch: int, s_q: int, h_q: int, num_parts: int) -> int:
    return int(load_library().mla_shared_prefix_workspace_bytes(int(batch), int(s_q), int(h_q), int(num_parts)))


def mla_shared_prefix_get_plan(block_table, cache_seqlens, s_q, h_q, causal, num_parts, plan, stream=None):
    dev = block_table.get_device()
    table_ptr = _p(block_table, _INT32, 2, dev, "block_table")
    lens_ptr = _p(cache_seqlens, _INT32, 1, dev, "cache_seqlens")
    batch, max_pages = block_table.shape
    if cache_seqlens.shape[0] != batch:
        raise ValueError("block_table / cache_seqlens batch mismatch")
    _check(load_library().mla_shared_prefix_get_plan(
        table_ptr, max_pages, lens_ptr, batch, int(s_q), int(h_q), 1 if causal else 0, int(num_parts),
        _p(plan, _UINT8, 1, dev, "plan"), plan.shape[0], _q(stream, dev)), "mla_shared_prefix_get_plan")


def _shared_prefix(q, kv, block_table, pl, softmax_scale, status, stream, out=None, lse=None, out_dtype=None,
                   cache_seqlens=None, hook=False):
    """The checks and the call of mla_shared_prefix_decode_fwd (with lengths, _checked_fwd; hook:
    mla_test_shared_prefix_timeout); allocates out and lse if not given."""
    dt = q.dtype
    code = _DTYPE_CODE16.get(dt)
    fp8 = kv.dtype is _UINT8
    if code is None or (kv.dtype is not dt and not (fp8 and dt is torch.bfloat16)):
        raise TypeError("q and kv must be both bf16 or both fp16, or a bf16 q over FP8 records")
    dev = q.get_device()
    q_ptr, kv_ptr = _p(q, dt, 4, dev, "q"), _p(kv, kv.dtype, 3, dev, "kv")
    table_ptr = _p(block_table, _INT32, 2, dev, "block_table")
    B, s_q, h_q, d = q.shape
    pages, page, width = kv.shape
    if d != 576 or page != 64 or width != (656 if fp8 else 576):
        raise ValueError("q must be [B, s_q, h_q, 576] and kv [pages, 64, 576] or records [pages, 64, 656]")
    batch, max_pages = block_table.shape
    if batch != B or pl.batch != B or pl.s_q != s_q or pl.h_q != h_q or pl.max_pages != max_pages:
        raise ValueError("the plan or block table was made for another batch")
    plan, ws, st = pl.plan, pl.workspace, _p(status, _INT32, 1, dev, "status")
    plan_ptr, ws_ptr = _p(plan, _UINT8, 1, dev, "plan"), _p(ws, _UINT8, 1, dev, "workspace")
    queue = _q(stream, dev)
    if out is None:
        out = torch.empty((B, s_q, h_q, 512), dtype=out_dtype, device=q.device)
        lse = torch.empty((B, s_q, h_q), dtype=_FP32, device=q.device)
        out_ptr, lse_ptr = out.data_ptr(), lse.data_ptr()
    else:
        out_dtype = out.dtype
        if out_dtype not in _DTYPE_CODE:
            raise TypeError("out must be bf16, fp16 or fp32")
        out_ptr, lse_ptr = _p(out, out_dtype, 4, dev, "out"), _p(lse, _FP32, 3, dev, "lse")
        if out.shape != (B, s_q, h_q, 512) or lse.shape != (B, s_q, h_q):
            raise ValueError("out must be [B, s_q, h_q, 512] and lse [B, s_q, h_q]")
    if cache_seqlens is None:
        args = (q_ptr, kv_ptr, table_ptr, max_pages, pages, B, s_q, h_q, DTYPE_FP8_RECORD if fp8 else code,
                1 if pl.causal else 0, softmax_scale, plan_ptr, plan.shape[0], pl.num_parts, ws_ptr, ws.shape[0],
                out_ptr, _DTYPE_CODE[out_dtype], lse_ptr, st, queue)
        if hook:
            _check(load_library().mla_test_shared_prefix_timeout(*args), "mla_test_shared_prefix_timeout")
        else:
            _call(_SHARED_PREFIX, "mla_shared_prefix_decode_fwd", *args)
        return out, lse
    lens_ptr = _p(cache_seqlens, _INT32, 1, dev, "cache_seqlens")
    if cache_seqlens.shape[0] != B:
        raise ValueError("block_table / cache_seqlens batch mismatch")
    _call(_SHARED_PREFIX_CHECKED, "mla_shared_prefix_decode_checked_fwd", q_ptr, kv_ptr, table_ptr, max_pages, pages,
          B, s_q, h_q, DTYPE_FP8_RECORD if fp8 else code, 1 if pl.causal else 0, softmax_scale, lens_ptr, plan_ptr,
          plan.shape[0], pl.num_parts, ws_ptr, ws.shape[0], out_ptr, _DTYPE_CODE[out_dtype], lse_ptr, st, queue)
    return out, lse


def mla_shared_prefix_decode_fwd(q, kv, block_table, pl, out, lse, status, softmax_scale=1.0 / 24.0, stream=None):
    """q [B, s_q, h_q, 576] and kv [pages, 64, 576], both bf16 or both fp16, or a
    bf16 q over FP8 records (uint8 [pages, 64, 656]); pl a SharedPrefixPlan of
    this block table; out [B, s_q, h_q, 512] bf16, fp16 or fp32, lse fp32
    [B, s_q, h_q]."""
    _shared_prefix(q, kv, block_table, pl, softmax_scale, status, stream, out, lse)


def mla_shared_prefix_decode_checked_fwd(q, kv, block_table, cache_seqlens, pl, out, lse, status,
                                         softmax_scale=1.0 / 24.0, stream=None):
    """mla_shared_prefix_decode_fwd that also compares the lengths [B] with the plan's on the device: another
    length, or a request that no longer ends its shared pages on the shared one, is MLA_ERR_STALE_PLAN in status."""
    _shared_prefix(q, kv, block_table, pl, softmax_scale, status, stream, out, lse, cache_seqlens=cache_seqlens)


def mla_test_shared_prefix_timeout(q, kv, block_table, pl, out, lse, status, softmax_scale=1.0 / 24.0, stream=None):
    """Test hook: mla_shared_prefix_decode_fwd whose first tile never comes (status: MLA_ERR_TIMEOUT)."""
    _shared_prefix(q, kv, block_table, pl, softmax_scale, status, stream, out, lse, hook=True)


def plan_shared_prefix(block_table, cache_seqlens, s_q, h_q, causal=False, num_parts=None):
    """The plan of a batch: finds the pages that all requests start with."""
    B, max_pages = block_table.shape
    parts = mla_shared_prefix_num_parts(B, s_q, h_q) if num_parts is None else int(num_parts)
    size = mla_shared_prefix_plan_bytes(B, s_q, h_q, parts)
    if size == 0:
        raise ValueError("batch, s_q, h_q or num_parts out of range")
    plan = torch.empty(size, dtype=torch.uint8, device=block_table.device)
    ws = torch.empty(mla_shared_prefix_workspace_bytes(B, s_q, h_q, parts), dtype=torch.uint8,
                     device=block_table.device)
    mla_shared_prefix_get_plan(block_table, cache_seqlens, s_q, h_q, causal, parts, plan)
    return SharedPrefixPlan(plan, B, max_pages, s_q, h_q, parts, bool(causal), ws)


def shared_prefix_decode(q, kv, block_table, cache_seqlens, causal=False, softmax_scale=None, out_fp32=False,
                         pl=None, status=None):
    """Dense decode that attends the pages all requests share once; returns (out, lse).  softmax_scale defaults to
    1 / sqrt(576), as decode's does: a model with prompt heads of 192 dims gives 192 ** -0.5.

    A plan holds the lengths it was made for.  With pl they are compared with cache_seqlens on the device, and a
    plan of other lengths (rows that have grown since, say) is MLA_ERR_STALE_PLAN."""
    lens = None  # a plan made here is that of the lengths
    if pl is None:
        pl = plan_shared_prefix(block_table, cache_seqlens, q.shape[1], q.shape[2], causal)
    elif pl.causal != bool(causal):
        raise ValueError("the plan was made with another causal setting")
    else:
        lens = cache_seqlens
    st = _status(status, q)
    out, lse = _shared_prefix(q, kv, block_table, pl, 1.0 / 24.0 if softmax_scale is None else softmax_scale, st, None,
                              out_dtype=_FP32 if out_fp32 else q.dtype, cache_seqlens=lens)
    if status is None:
        check_status(st, "mla_shared_prefix_decode_fwd")
    return out, lse


# (the entry points that chunks.py binds are its own)
__all__ = [n for n in SERVING_SYMBOLS if n in globals()] + [
    "SERVING_SYMBOLS", "cache_append", "cache_grow", "cache_fork", "cache_free", "cache_compact", "cache_copy_pages",
    "PromptPlan", "plan_prompt", "prompt_attention", "SharedPrefixPlan", "plan_shared_prefix", "shared_prefix_decode",
]
