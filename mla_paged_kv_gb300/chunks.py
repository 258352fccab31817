"""Operators that take chunks of new tokens through a paged latent cache (see
include/mla_serving.h): rotary tables, the rotation of query and key heads, rows
of the cache as packed rows, and the attention of ragged chunks over the cache.

The rules are those of ``serving``: functions named ``mla_*`` mirror the C entry
points, the helpers (``rope_frequencies``, ``rope_table``, ``rope_heads``,
``cache_gather``, ``plan_chunks``, ``chunk_attention``) allocate outputs and,
without ``status``, read the device status and raise ``MlaError``.

A step of a model that takes a chunk of every request:

    mla.rope_heads(q_proj[..., 128:], table, lens, cu_seqlens=cu, out=q[..., 512:])   # q[..., :512]: absorbed heads
    mla.cache_append(c, r, cache, block_table, lens, cu_seqlens=cu, norm_weight=w, cos_sin=table)
    out, lse = mla.chunk_attention(q, cache, block_table, lens, cu, softmax_scale=192 ** -0.5, pl=plan)

``cache_gather`` serves the other path, cheaper for chunks of some hundred tokens:
a cached context as rows, to be expanded into heads for ``prompt_attention``.
"""

from __future__ import annotations

import ctypes
import math

import torch

from . import DTYPE_FP8_RECORD, _DTYPE_CODE, _check, check_status, load_library, MlaError
from .serving import (_D, _DTYPE_CODE16, _FP32, _INT32, _UINT8, _call, _p, _q, _status, _words)

CHUNK_PAGE_BYTES = 64 * 512 * 2  # of a page whose values a call over FP8 records converts (MLA_CHUNK_PAGE_BYTES)
CHUNK_QUERY_BYTES = 1040  # of a query head in the workspace of such a call (MLA_CHUNK_QUERY_BYTES)
ROPE_SCALING = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "wavelength": 4}

__all__ = ["ROPE_SCALING", "CHUNK_PAGE_BYTES", "CHUNK_QUERY_BYTES", "rope_frequencies", "rope_table", "rope_heads",
           "cache_gather", "ChunkPlan", "plan_chunks", "chunk_workspace", "chunk_attention"]

_ROPE_HEADS, _GATHER, _CHUNK = _words(10, "22qd8q"), _words(11, "13q"), _words(12, "9qd12q")

# ------------------------------------------------------------------ rotary


def _frequencies(dim, base, scaling, factor, original, low, high):
    freq, size = (_D * max(dim // 2, 1))(), _D()
    rc = load_library().mla_rope_frequencies(dim, base, scaling, factor, original, low, high, freq, size)
    if rc:
        _check(rc, "mla_rope_frequencies")
    return freq, size.value


def _table(freq, dim, magnitude, first, positions, out, dev, stream):
    rc = load_library().mla_rope_table(freq, dim, magnitude, first, positions, out.data_ptr(), _q(stream, dev))
    if rc:
        _check(rc, "mla_rope_table")


def mla_rope_frequencies(dim, base, scaling, factor, original, low, high):
    """(frequencies, magnitude): dim / 2 floats, and what the table's values are multiplied by."""
    freq, size = _frequencies(int(dim), float(base), int(scaling), float(factor), float(original), float(low),
                              float(high))
    return list(freq), size


def mla_rope_table(freq, magnitude, first, cos_sin, stream=None):
    """The table of positions first .. first + cos_sin.shape[0] - 1 into cos_sin fp32 [positions, dim]."""
    dev = cos_sin.get_device()
    _p(cos_sin, _FP32, 2, dev, "cos_sin")
    positions, dim = cos_sin.shape
    if len(freq) * 2 != dim:
        raise ValueError("cos_sin must have two columns a frequency")
    _table((_D * len(freq))(*freq), dim, float(magnitude), int(first), positions, cos_sin, dev, stream)


def _scaling(scaling, high):
    code = ROPE_SCALING.get(scaling)
    if code is None:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALING)}")
    return code, (4.0 if scaling == "wavelength" else 32.0) if high is None else high


def rope_frequencies(dim=64, base=10000.0, scaling="none", factor=1.0, original=4096, low=1.0, high=None):
    """(frequencies, magnitude) of rotary positions whose context is stretched by factor: scaling "none", "linear",
    "ntk", "yarn" or "wavelength"; low and high are the turns over the original context (high defaults to 32 for
    "yarn", 4 for "wavelength")."""
    code, high = _scaling(scaling, high)
    return mla_rope_frequencies(dim, base, code, factor, original, low, high)


def rope_table(positions, dim=64, base=10000.0, scaling="none", factor=1.0, original=4096, low=1.0, high=None,
               magnitude=None, first=0, device="cuda"):
    """The fp32 table [positions, dim] that cache_append (dim 64) and rope_heads read: cosines, then sines, of the
    positions from first on.  magnitude (of the values) defaults to the scaling's own."""
    code, high = _scaling(scaling, high)
    freq, size = _frequencies(dim, base, code, factor, original, low, high)
    out = torch.empty((positions, dim), dtype=_FP32, device=device)
    _table(freq, dim, size if magnitude is None else magnitude, first, positions, out, out.get_device(), None)
    return out


def _heads(t, dtype, tokens, dim, dev, name):
    """Address, strides and heads of a [tokens, heads, dim] tensor with a contiguous last dimension, and the address
    behind it."""
    stride, shape = t.stride(), t.shape
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if len(shape) != 3 or shape[0] != tokens or shape[2] != dim or stride[2] != 1:
        raise ValueError(f"{name} must be [{tokens}, heads, {dim}] with a contiguous last dimension")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, is on {t.device}")
    ptr, heads = t.data_ptr(), shape[1]
    return ptr, stride[0], stride[1], heads, ptr + 2 * ((tokens - 1) * stride[0] + (heads - 1) * stride[1] + dim)


def _apart(a, b, tokens, dim):
    """Whether two such tensors share no element.  (Exact for equal strides; others have to lie one behind the other, or
    side by side in what their strides are multiples of.)"""
    if a[0] >= b[4] or b[0] >= a[4]:
        return True
    step, ts, hs = (b[0] - a[0]) // 2, a[1], a[2]
    # side by side in every token's rows, as the parts of a packed projection are
    if ts == b[1] > 0 and step % ts >= (a[3] - 1) * hs + dim and step % ts + (b[3] - 1) * b[2] + dim <= ts:
        return True
    # .. in what all strides repeat, as parts of the same heads are
    cell = math.gcd(ts, hs, b[1], b[2])
    if cell and dim <= step % cell <= cell - dim:
        return True
    if b[1:3] != (ts, hs) or ts <= 0 or hs <= 0:
        return False
    # .. or in rows that hold something else behind the heads (what follows would find it too: 0.3 ms for 128 heads)
    for by, n, m in ((step, a[3], b[3]), (-step, b[3], a[3])):
        head, place = divmod(by % ts, hs)
        if dim <= place <= hs - dim and max(n, head + m) * hs <= ts:
            return True
    # every distance between a token and head of a and one of b, step + i ts + n hs: the fewer of them one by one, the
    # two nearest of the others
    i, n = (ts, 1 - tokens, tokens - 1), (hs, 1 - a[3], b[3] - 1)
    few, many = (i, n) if 2 * tokens < a[3] + b[3] else (n, i)
    for k in range(few[1], few[2] + 1):
        at = step + k * few[0]
        j = min(max(-at // many[0], many[1]), many[2])
        if abs(at + j * many[0]) < dim or (j < many[2] and abs(at + (j + 1) * many[0]) < dim):
            return False
    return True


def _output(out, tokens, dim, others, same):
    """An output's elements share no memory among themselves, nor with other tensors of the call but `same`, which it
    may be as a whole (tensors as _heads gives them)."""
    ptr, ts, hs, heads, end = out
    if not ((heads == 1 or hs >= dim) and (tokens <= 1 or ts >= (heads - 1) * hs + dim)) and \
            not ((tokens <= 1 or ts >= dim) and (heads == 1 or hs >= (tokens - 1) * ts + dim)):
        raise ValueError("an output must not have elements that share memory")
    for t in others:
        if ptr < t[4] and t[0] < end and not (t is same and t[:4] == out[:4]) and not _apart(out, t, tokens, dim):
            raise ValueError("an output overlaps another tensor of the call")


def _fresh(t, tokens, dim):
    """A new tensor of the shape of t, which _heads has passed, and what that says of it."""
    heads = t.shape[1]
    out = torch.empty((tokens, heads, dim), dtype=t.dtype, device=t.device)
    ptr, row = out.data_ptr(), heads * dim
    return out, (ptr, row, dim, heads, ptr + 2 * tokens * row)


def mla_rope_heads(x, out, cos_sin, status, cache_seqlens=None, cu_seqlens=None, positions=None, k=None, k_out=None,
                   x_weight=None, k_weight=None, norm_eps=1e-6, offset=None, interleaved=False, stream=None):
    """x [tokens, heads, dim] (and k [tokens, k_heads, dim]), bf16 or fp16, into out (k_out), which may be x (k)
    itself; strides free, multiples of 8.  cos_sin fp32 [positions, rope_dim] turns dims offset .. offset + rope_dim
    (default: the last ones) of every head at positions [tokens], or at those of cache_append; None: norm only."""
    if out is None or (k is not None and k_out is None):
        raise ValueError("x needs out, and k needs k_out")
    _rope(x, out, cos_sin, status, cache_seqlens, cu_seqlens, positions, k, k_out, x_weight, k_weight, norm_eps, offset,
          interleaved, stream)


def _rope(x, out, cos_sin, status, cache_seqlens, cu_seqlens, positions, k, k_out, x_weight, k_weight, norm_eps, offset,
          interleaved, stream):
    """The checks and the call of mla_rope_heads; allocates out and k_out if not given, and returns them."""
    dt = x.dtype
    code = _DTYPE_CODE16.get(dt)
    if code is None:
        raise TypeError("x must be bf16 or fp16")
    if x.dim() != 3:
        raise ValueError("x must be [tokens, heads, dim]")
    dev = x.get_device()
    tokens, _, dim = x.shape
    src = _heads(x, dt, tokens, dim, dev, "x")
    heads = src[3]
    none = (0, 0, 0, 0, 0)
    k_src = k_dst = none
    if k is not None:
        k_src = _heads(k, dt, tokens, dim, dev, "k")
    elif k_out is not None or k_weight is not None:
        raise ValueError("k_out and k_weight need k")
    if out is None:
        out, dst = _fresh(x, tokens, dim)
    else:
        dst = _heads(out, dt, tokens, dim, dev, "out")
        if tokens:
            _output(dst, tokens, dim, (src, k_src), src)
    if heads == 0 or dst[3] != heads:
        raise ValueError("out must have the heads of x, at least one")
    if k is not None:
        if k_out is None:
            k_out, k_dst = _fresh(k, tokens, dim)
        else:
            k_dst = _heads(k_out, dt, tokens, dim, dev, "k_out")
            if tokens:
                _output(k_dst, tokens, dim, (src, k_src, dst), k_src)
        if k_src[3] == 0 or k_dst[3] != k_src[3]:
            raise ValueError("k_out must have the heads of k, at least one")
    w_ptr = kw_ptr = 0
    if x_weight is not None:
        w_ptr = _p(x_weight, dt, 1, dev, "x_weight")
        if x_weight.shape[0] != dim:
            raise ValueError("x_weight must have one entry a dim")
    if k_weight is not None:
        kw_ptr = _p(k_weight, dt, 1, dev, "k_weight")
        if k_weight.shape[0] != dim:
            raise ValueError("k_weight must have one entry a dim")
    cos_ptr = pos_ptr = cu_ptr = lens_ptr = rope = max_pos = 0
    batch = 0
    if cos_sin is not None:
        cos_ptr = _p(cos_sin, _FP32, 2, dev, "cos_sin")
        max_pos, rope = cos_sin.shape
        if (positions is None) == (cache_seqlens is None):
            raise ValueError("give positions, or cache_seqlens, not both")
    elif positions is not None or cache_seqlens is not None:
        raise ValueError("positions need cos_sin")
    if positions is not None:
        pos_ptr = _p(positions, _INT32, 1, dev, "positions")
        if positions.shape[0] != tokens or cu_seqlens is not None:
            raise ValueError("positions must have one entry a token, without cu_seqlens")
    elif cache_seqlens is not None:
        lens_ptr = _p(cache_seqlens, _INT32, 1, dev, "cache_seqlens")
        batch = cache_seqlens.shape[0]
        if cu_seqlens is not None:
            cu_ptr = _p(cu_seqlens, _INT32, 1, dev, "cu_seqlens")
            if cu_seqlens.shape[0] != batch + 1:
                raise ValueError("cu_seqlens must have batch + 1 entries")
        elif batch == 0 or tokens % batch:
            raise ValueError("without cu_seqlens every request has tokens / batch tokens")
    elif cu_seqlens is not None:
        raise ValueError("cu_seqlens need cache_seqlens")
    if offset is None:
        offset = dim - rope
    _call(_ROPE_HEADS, "mla_rope_heads", *src[:3], *dst[:3], heads, w_ptr, *k_src[:3], *k_dst[:3], k_src[3], kw_ptr,
          dim, code, tokens, rope, offset, 1 if interleaved else 0, norm_eps, pos_ptr, cu_ptr,
          lens_ptr, batch, cos_ptr, max_pos, _p(status, _INT32, 1, dev, "status"), _q(stream, dev))
    return out, k_out


def rope_heads(x, cos_sin, cache_seqlens=None, cu_seqlens=None, positions=None, out=None, k=None, k_out=None,
               norm_weight=None, k_norm_weight=None, norm_eps=1e-6, offset=None, interleaved=False, status=None):
    """Rotate part of each head of x (and of k), each optionally RMS-normalised first; returns out, with k (out,
    k_out).  out and k_out default to new tensors; x and k themselves turn them in place."""
    st = _status(status, x)
    out, k_out = _rope(x, out, cos_sin, st, cache_seqlens, cu_seqlens, positions, k, k_out, norm_weight, k_norm_weight,
                       norm_eps, offset, interleaved, None)
    if status is None:
        check_status(st, "mla_rope_heads")
    return out if k is None else (out, k_out)


# ------------------------------------------------------------------ gather


def _cache(cache, dev, name):
    """Address, C type code and pages of a cache: 16-bit [pages, 64, 576] or records uint8 [pages, 64, 656]."""
    dt = cache.dtype
    code = DTYPE_FP8_RECORD if dt is _UINT8 else _DTYPE_CODE16.get(dt)
    if code is None:
        raise TypeError(f"{name} must be bf16, fp16 or FP8 records (uint8)")
    ptr = _p(cache, dt, 3, dev, name)
    pages, page, width = cache.shape
    if page != 64 or width != (656 if dt is _UINT8 else 576):
        raise ValueError(f"{name} must be [pages, 64, 576] or records [pages, 64, 656]")
    return ptr, code, pages


def mla_cache_gather(cache, block_table, cu_seqlens, out, status, starts=None, stream=None):
    """Rows of the cache into out [total, 576] (the cache's type; bf16 of FP8 records), row stride free: row t of
    request b, cu_seqlens[b] <= t < cu_seqlens[b + 1], from position starts[b] (0) + t - cu_seqlens[b]."""
    if out is None:
        raise ValueError("out is needed")
    _rows(cache, block_table, cu_seqlens, out, 0, starts, status, stream)


def _rows(cache, block_table, cu_seqlens, out, rows, starts, status, stream):
    """The checks and the call of mla_cache_gather; allocates out, of `rows` rows, if not given, and returns it."""
    dev = cache.get_device()
    ptr, code, pages = _cache(cache, dev, "cache")
    table_ptr = _p(block_table, _INT32, 2, dev, "block_table")
    batch, max_pages = block_table.shape
    cu_ptr = _p(cu_seqlens, _INT32, 1, dev, "cu_seqlens")
    if cu_seqlens.shape[0] != batch + 1:
        raise ValueError("cu_seqlens must have batch + 1 entries")
    starts_ptr = 0
    if starts is not None:
        starts_ptr = _p(starts, _INT32, 1, dev, "starts")
        if starts.shape[0] != batch:
            raise ValueError("starts must have one entry a request")
    want, step = torch.bfloat16 if code == DTYPE_FP8_RECORD else cache.dtype, 576
    if out is None:
        out = torch.empty((rows, 576), dtype=want, device=cache.device)
        at = out.data_ptr()
    else:
        if out.dtype is not want:
            raise TypeError(f"out must be {want}, got {out.dtype}")
        stride = out.stride()
        if len(stride) != 2 or out.shape[1] != 576 or stride[1] != 1 or out.get_device() != dev:
            raise ValueError(f"out must be [rows, 576] with contiguous rows, on cuda:{dev}")
        rows, at = out.shape[0], out.data_ptr()
        if rows > 1:
            step = stride[0]
        if rows and at < ptr + cache.numel() * cache.element_size() and ptr < at + 2 * ((rows - 1) * step + 576):
            raise ValueError("out overlaps the cache")
    _call(_GATHER, "mla_cache_gather", ptr, code, pages, table_ptr, max_pages, cu_ptr, starts_ptr, batch, rows,
          at, step, _p(status, _INT32, 1, dev, "status"), _q(stream, dev))
    return out


def cache_gather(cache, block_table, cu_seqlens, total=None, starts=None, out=None, status=None):
    """Rows of a paged cache as packed rows [total, 576] (see mla_cache_gather).  total defaults to the last offset,
    which reads it from the GPU."""
    st = _status(status, cache)
    if out is None and total is None:
        total = int(cu_seqlens[-1])
    out = _rows(cache, block_table, cu_seqlens, out, total, starts, st, None)
    if status is None:
        check_status(st, "mla_cache_gather")
    return out


# ------------------------------------------------------------------- chunk


class ChunkPlan:
    """The units and runs of a batch of chunks, and its split workspace: reused by every layer of that batch, one
    call at a time."""

    def __init__(self, plan, batch, total_q, h_q, num_parts, causal, workspace):
        self.plan = plan
        self.batch = batch
        self.total_q = total_q
        self.h_q = h_q
        self.num_parts = num_parts
        self.causal = causal
        self.workspace = workspace


def mla_chunk_num_parts() -> int:
    n = load_library().mla_chunk_num_parts()
    if n < 1:
        raise MlaError(-n, "mla_chunk_num_parts")
    return n


def mla_chunk_plan_bytes(batch: int, total_q: int, h_q: int, num_parts: int) -> int:
    return int(load_library().mla_chunk_plan_bytes(int(batch), int(total_q), int(h_q), int(num_parts)))


def mla_chunk_workspace_bytes(num_parts: int) -> int:
    return int(load_library().mla_chunk_workspace_bytes(int(num_parts)))


def mla_chunk_get_plan(cu_seqlens_q, cache_seqlens, total_q, h_q, causal, num_parts, plan, status, stream=None):
    dev = cu_seqlens_q.get_device()
    cu, lens = _p(cu_seqlens_q, _INT32, 1, dev, "cu_seqlens_q"), _p(cache_seqlens, _INT32, 1, dev, "cache_seqlens")
    batch = cache_seqlens.shape[0]
    if cu_seqlens_q.shape[0] != batch + 1:
        raise ValueError("cu_seqlens_q must have batch + 1 entries")
    _check(load_library().mla_chunk_get_plan(
        cu, lens, batch, int(total_q), int(h_q), 1 if causal else 0, int(num_parts),
        _p(plan, _UINT8, 1, dev, "plan"), plan.shape[0], _p(status, _INT32, 1, dev, "status"), _q(stream, dev)),
        "mla_chunk_get_plan")


def _chunk(q, kv, block_table, pl, softmax_scale, status, stream, out=None, lse=None, out_dtype=None,
           cu_seqlens_q=None, cache_seqlens=None, hook=False):
    """The checks and the call of mla_chunk_attention_fwd (hook: mla_test_chunk_timeout); allocates out and lse if
    not given."""
    dt = q.dtype
    if dt not in _DTYPE_CODE16 or (kv.dtype is not dt and not (kv.dtype is _UINT8 and dt is torch.bfloat16)):
        raise TypeError("q and kv must be both bf16 or both fp16, or a bf16 q over FP8 records")
    dev = q.get_device()
    q_ptr = _p(q, dt, 3, dev, "q")
    kv_ptr, code, pages = _cache(kv, dev, "kv")
    table_ptr = _p(block_table, _INT32, 2, dev, "block_table")
    total_q, h_q, d = q.shape
    if d != 576:
        raise ValueError("q must be [total_q, h_q, 576]")
    batch, max_pages = block_table.shape
    if pl.batch != batch or pl.total_q != total_q or pl.h_q != h_q:
        raise ValueError("the plan was made for another batch")
    plan, ws, st = pl.plan, pl.workspace, _p(status, _INT32, 1, dev, "status")
    if out is None and code == DTYPE_FP8_RECORD:
        # room for values that are converted once for three row blocks and more (at most 0.5 GB)
        ws = chunk_workspace(pl, min(min(batch, total_q * h_q // 257) * max_pages, 1 << 13))
    plan_ptr, ws_ptr = _p(plan, _UINT8, 1, dev, "plan"), _p(ws, _UINT8, 1, dev, "workspace")
    queue = _q(stream, dev)
    if out is None:
        out = torch.empty((total_q, h_q, 512), dtype=out_dtype, device=q.device)
        lse = torch.empty((total_q, h_q), dtype=_FP32, device=q.device)
        out_ptr, lse_ptr = out.data_ptr(), lse.data_ptr()
    else:
        out_dtype = out.dtype
        if out_dtype not in _DTYPE_CODE:
            raise TypeError("out must be bf16, fp16 or fp32")
        out_ptr, lse_ptr = _p(out, out_dtype, 3, dev, "out"), _p(lse, _FP32, 2, dev, "lse")
        if out.shape != (total_q, h_q, 512) or lse.shape != (total_q, h_q):
            raise ValueError("out must be [total_q, h_q, 512] and lse [total_q, h_q]")
    cu_ptr = lens_ptr = 0
    if cu_seqlens_q is not None:
        cu_ptr = _p(cu_seqlens_q, _INT32, 1, dev, "cu_seqlens_q")
        if cu_seqlens_q.shape[0] != batch + 1:
            raise ValueError("cu_seqlens_q must have batch + 1 entries")
    if cache_seqlens is not None:
        lens_ptr = _p(cache_seqlens, _INT32, 1, dev, "cache_seqlens")
        if cache_seqlens.shape[0] != batch:
            raise ValueError("block_table / cache_seqlens batch mismatch")
    args = (q_ptr, kv_ptr, table_ptr, max_pages, pages, batch, total_q, h_q, code, softmax_scale, cu_ptr, lens_ptr,
            plan_ptr, plan.shape[0], pl.num_parts, ws_ptr, ws.shape[0], out_ptr, _DTYPE_CODE[out_dtype], lse_ptr, st,
            queue)
    if hook:
        _check(load_library().mla_test_chunk_timeout(*args), "mla_test_chunk_timeout")
    else:
        _call(_CHUNK, "mla_chunk_attention_fwd", *args)
    return out, lse


def mla_chunk_attention_fwd(q, kv, block_table, pl, out, lse, status, softmax_scale=1.0 / 24.0, cu_seqlens_q=None,
                            cache_seqlens=None, stream=None):
    """q [total_q, h_q, 576] and kv [pages, 64, 576], both bf16 or both fp16, or a bf16 q over FP8 records (uint8
    [pages, 64, 656]); pl a ChunkPlan; out [total_q, h_q, 512] bf16, fp16 or fp32, lse fp32 [total_q, h_q].  Offsets
    and lengths that are given are compared with the plan's: others are MLA_ERR_STALE_PLAN in status, the same but out of
    range MLA_ERR_BAD_INDEX."""
    if out is None or lse is None:
        raise ValueError("out and lse are needed")
    _chunk(q, kv, block_table, pl, softmax_scale, status, stream, out, lse, None, cu_seqlens_q, cache_seqlens)


def mla_test_chunk_timeout(q, kv, block_table, pl, out, lse, status, softmax_scale=1.0 / 24.0, stream=None):
    """Test hook: mla_chunk_attention_fwd whose first K stage is never loaded (status: MLA_ERR_TIMEOUT)."""
    if out is None or lse is None:
        raise ValueError("out and lse are needed")
    _chunk(q, kv, block_table, pl, softmax_scale, status, stream, out, lse, hook=True)


def plan_chunks(cu_seqlens_q, cache_seqlens, total_q, h_q, causal=True, num_parts=None, status=None):
    """The plan of a batch of chunks: cu_seqlens_q [batch + 1] the chunks' offsets in the packed queries, of which
    there are total_q, cache_seqlens [batch] the requests' keys, their new tokens among them."""
    parts = mla_chunk_num_parts() if num_parts is None else int(num_parts)
    size = mla_chunk_plan_bytes(cache_seqlens.shape[0], total_q, h_q, parts)
    if size == 0:
        raise ValueError("batch, total_q, h_q or num_parts out of range")
    st = _status(status, cu_seqlens_q)
    plan = torch.empty(size, dtype=torch.uint8, device=cu_seqlens_q.device)
    ws = torch.empty(mla_chunk_workspace_bytes(parts), dtype=torch.uint8, device=cu_seqlens_q.device)
    mla_chunk_get_plan(cu_seqlens_q, cache_seqlens, total_q, h_q, causal, parts, plan, st)
    if status is None:
        check_status(st, "mla_chunk_get_plan")
    return ChunkPlan(plan, cache_seqlens.shape[0], int(total_q), int(h_q), parts, bool(causal), ws)


def chunk_workspace(pl, pages=0):
    """The workspace of a call over FP8 records, with room for the values of `pages` pages: pl.workspace, which
    mla_chunk_attention_fwd takes, is that of calls over 16-bit caches (chunk_attention makes its own)."""
    size = mla_chunk_workspace_bytes(pl.num_parts) + pl.total_q * pl.h_q * CHUNK_QUERY_BYTES + pages * CHUNK_PAGE_BYTES
    return torch.empty(size, dtype=_UINT8, device=pl.plan.device)


def chunk_attention(q, kv, block_table, cache_seqlens, cu_seqlens_q, causal=True, softmax_scale=None, out_fp32=False,
                    pl=None, status=None):
    """Attention of ragged chunks of new tokens over a paged latent cache; returns (out, lse).  softmax_scale defaults
    to 1 / sqrt(576), as decode's does: a model with prompt heads of 192 dims gives 192 ** -0.5.

    A plan holds the offsets and lengths it was made for.  With pl they are compared with cu_seqlens_q and
    cache_seqlens on the device: a plan of others is MLA_ERR_STALE_PLAN, one that is empty because they are out of range
    MLA_ERR_BAD_INDEX (outputs are then not written)."""
    st = _status(status, q)
    cu, lens = cu_seqlens_q, cache_seqlens
    if pl is None:  # a plan made here is that of the offsets
        pl = plan_chunks(cu, lens, q.shape[0], q.shape[1], causal, status=st)
        cu = lens = None
    elif pl.causal != bool(causal):
        raise ValueError("the plan was made with another causal setting")
    out, lse = _chunk(q, kv, block_table, pl, 1.0 / 24.0 if softmax_scale is None else softmax_scale, st, None,
                      out_dtype=_FP32 if out_fp32 else q.dtype, cu_seqlens_q=cu, cache_seqlens=lens)
    if status is None:
        check_status(st, "mla_chunk_attention_fwd")
    return out, lse


__all__ += [n for n in list(globals()) if n.startswith("mla_")]
