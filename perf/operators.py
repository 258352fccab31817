"""Cases of the operators that fill, share and read a paged latent (MLA) cache.

Each case names an operator (``op``) and its sizes; ``prepare`` makes the
inputs of a serving program from a seed, ``run`` makes one call, in plain torch
operations or (``own``) through the framework, and ``exact`` states the same
result in 64 bits.
"""

import math
import random

import numpy as np
import torch

own = False

PAGE, D_C, D_R, D_QK, D_V = 64, 512, 64, 576, 512
RECORD = 656
HEAD_V = 128          # value head of the prompt attention
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------- cases


def listed():
    return [
        # one decode step of a small batch into a cache of FP8 records: latency
        dict(name="append_step_b8_fp8", op="append", requests=8, tokens=8, ctx=1500, cache="fp8", interleaved=True),
        # ragged prompts of a prefill batch, FP8 records
        dict(name="append_prompts_fp8", op="append", requests=13, tokens=24577, ctx=0, cache="fp8", interleaved=True),
        # ragged prompts behind cached contexts, 16-bit rows
        dict(name="append_prompts_bf16", op="append", requests=24, tokens=49153, ctx=900, cache="bf16",
             interleaved=False),
        # parallel sampling: four prompts forked into four samples each, few layers
        dict(name="fork_b16_l4_bf16", op="fork", parents=4, children=16, layers=4, length=700, cache="bf16"),
        # defragmenting a pool that is about half free, eight layers
        dict(name="compact_l8_bf16", op="compact", rows=48, layers=8, length=1500, pages=2001, cache="bf16"),
        # the bookkeeping of one scheduler tick: requests end, others grow (no data moves)
        dict(name="churn_b512", op="churn", rows=512, length=2500, pages=65536, new=130),
        # a short system prompt, a tensor-parallel share of the heads: latency
        dict(name="prefix_b8_h16_1k", op="prefix", requests=8, s_q=1, heads=16, prefix_pages=16, tail=64,
             dtype="bf16", causal=False),
        # a long document that a batch asks questions about, 16 heads on this GPU
        dict(name="prefix_b64_h16_16k", op="prefix", requests=64, s_q=1, heads=16, prefix_pages=256, tail=500,
             dtype="bf16", causal=False),
        # all 128 heads on this GPU
        dict(name="prefix_b64_h128_8k", op="prefix", requests=64, s_q=1, heads=128, prefix_pages=128, tail=1000,
             dtype="bf16", causal=False),
        # a handful of short prompts: latency
        dict(name="prompt_b6_short", op="prompt", requests=6, q_len=130, ctx=0, heads=16, kv_heads=16, d_qk=192,
             dtype="bf16", ragged=True),
        # a ragged prefill batch, one key head for each query head (latent heads expanded)
        dict(name="prompt_b8_ragged_h16", op="prompt", requests=8, q_len=4000, ctx=0, heads=16, kv_heads=16,
             d_qk=192, dtype="bf16", ragged=True),
        # one long prompt
        dict(name="prompt_b1_16k_h16", op="prompt", requests=1, q_len=16384, ctx=0, heads=16, kv_heads=16, d_qk=192,
             dtype="bf16", ragged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "fork", "compact", "churn", "prefix", "prefix", "prompt", "prompt"])
    if op == "append":
        n = _log(rng, 1, 64)
        return dict(op=op, requests=n, tokens=max(n, _log(rng, 1, 40000)), ctx=rng.randint(0, 2000),
                    cache=rng.choice(["fp8", "bf16", "fp16"]), interleaved=rng.random() < 0.5)
    if op == "fork":
        p = _log(rng, 1, 16)
        return dict(op=op, parents=p, children=p * rng.randint(1, 8), layers=rng.randint(1, 8),
                    length=_log(rng, 20, 2000), cache=rng.choice(["fp8", "bf16"]))
    if op == "compact":
        rows, length = _log(rng, 2, 48), _log(rng, 40, 1500)
        return dict(op=op, rows=rows, layers=rng.randint(1, 8), length=length,
                    pages=2 * rows * (length // PAGE + 1) + rng.randint(1, 99), cache=rng.choice(["fp8", "bf16"]))
    if op == "churn":
        rows, length = _log(rng, 4, 512), _log(rng, 64, 2500)
        return dict(op=op, rows=rows, length=length, pages=2 * rows * (length // PAGE + 6) + rng.randint(1, 9999),
                    new=rng.randint(1, 200))
    if op == "prefix":
        heads = rng.choice([16, 32, 64, 128])
        s_q = rng.choice([1, 1, 2])
        return dict(op=op, requests=_log(rng, 2, 64 * 128 // (heads * s_q) if heads * s_q > 64 else 64), s_q=s_q,
                    heads=heads, prefix_pages=_log(rng, 1, 120), tail=_log(rng, 2, 900),
                    dtype=rng.choice(["bf16", "fp16"]), causal=s_q > 1)
    kv = rng.choice([1, 2, 4, 16])
    ctx = rng.choice([0, 0, rng.randint(1, 4000)])
    return dict(op=op, requests=_log(rng, 1, 8), q_len=_log(rng, 2, 3000), ctx=ctx, heads=16, kv_heads=kv,
                d_qk=rng.choice([128, 192]), dtype=rng.choice(["bf16", "fp16"]), ragged=True)


# ---------------------------------------------------------------- lengths (from the case alone: shapes stay)


def _sizes(case):
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _pages(n):
    return -(-n // PAGE)


def _append_lengths(case, rng):
    """New tokens and total length of each request: ragged shares that sum to ``tokens``."""
    n, total = case["requests"], case["tokens"]
    w = [rng.uniform(0.3, 1.0) for _ in range(n)]
    new = [max(1, int(total * x / sum(w))) for x in w]
    new[-1] += total - sum(new)
    if new[-1] < 1:
        new = [1] * (n - 1) + [total - n + 1]
    ctx = [rng.randint(case["ctx"] // 2, case["ctx"]) for _ in range(n)]
    return new, [a + b for a, b in zip(new, ctx)]


def _prompt_lengths(case, rng):
    n, top = case["requests"], case["q_len"]
    lq = [rng.randint(1, top) if case["ragged"] else top for _ in range(n)]
    if case["ragged"]:
        lq[rng.randrange(n)] = top
    lk = [a + (rng.randint(0, case["ctx"]) if case["ctx"] else 0) for a in lq]
    return lq, lk


def _tail_lengths(case, rng):
    """Keys of each request behind the shared pages (its new tokens among them)."""
    return [rng.randint(max(case["s_q"], case["tail"] // 8), max(case["s_q"], case["tail"]))
            for _ in range(case["requests"])]


def _row_lengths(case, rng, n):
    return [rng.randint(1, case["length"]) for _ in range(n)]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cum(v):
    return _i32([0] + list(np.cumsum(v)))


def _table(lengths, width, perm):
    """A block table whose rows take consecutive pages of ``perm``, and the pages used."""
    t = np.full((len(lengths), width), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(lengths):
        k = _pages(n)
        t[b, :k] = perm[at:at + k]
        at += k
    return t, at


def _row_dims(cache):
    return (RECORD,) if cache == "fp8" else (D_QK,)


def _row_bytes(cache):
    return RECORD if cache == "fp8" else 2 * D_QK


def _pool(case, layers, pages, g):
    """A pool of page bytes.  Pages are moved whole, so any bytes serve: held as int16."""
    n = _row_bytes(case["cache"]) // 2
    return torch.randint(-32768, 32767, (layers, pages, PAGE, n), dtype=torch.int16, device="cuda", generator=g)


# ---------------------------------------------------------------- prepare


def prepare(case, seed):
    rng, g = _sizes(case), _gen(seed)
    s = {"case": case}
    op = case["op"]
    if op == "append":
        new, total = _append_lengths(case, rng)
        dt = torch.bfloat16 if case["cache"] == "fp8" else DTYPES[case["cache"]]
        need = sum(_pages(t) for t in total)
        pages = need + need // 5 + 1
        table, _ = _table(total, _pages(max(total)) + 1, np.random.RandomState(seed % 2**32).permutation(pages))
        t = case["tokens"]
        # the projection that a layer computes: 512 latent and 64 RoPE columns of one row
        s["kv_a"] = (torch.randn(t, D_QK, device="cuda", generator=g) *
                     (0.5 + 2.0 * torch.rand(t, 1, device="cuda", generator=g))).to(dt)
        s["weight"] = (1.0 + 0.2 * torch.randn(D_C, device="cuda", generator=g)).to(dt)
        far = max(total) + 1
        angle = torch.arange(far, device="cuda", dtype=torch.float64)[:, None] * \
            (10000.0 ** (-torch.arange(0, 32, device="cuda", dtype=torch.float64) / 32))[None]
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
        s["table"], s["lens"], s["cu"] = torch.from_numpy(table).cuda(), _i32(total), _cum(new)
        if case["cache"] == "fp8":
            s["cache"] = torch.zeros(pages, PAGE, RECORD, dtype=torch.uint8, device="cuda")
        else:
            s["cache"] = torch.zeros(pages, PAGE, D_QK, dtype=dt, device="cuda")
    elif op == "fork":
        lens = _row_lengths(case, rng, case["parents"])
        width = _pages(case["length"]) + 2
        need = sum(_pages(n) for n in lens) + case["children"]
        pages = need + need // 3 + 8
        perm = np.random.RandomState(seed % 2**32).permutation(pages)
        table, used = _table(lens + [0] * case["children"], width, perm)
        ref = np.zeros(pages, dtype=np.int32)
        ref[perm[:used]] = 1
        s["ref0"], s["table0"] = torch.from_numpy(ref).cuda(), torch.from_numpy(table).cuda()
        s["lens0"] = _i32(lens + [0] * case["children"])
        s["parents"] = _i32([i % case["parents"] for i in range(case["children"])])
        s["children"] = _i32([case["parents"] + i for i in range(case["children"])])
        s["pool"] = _pool(case, case["layers"], pages, g)
    elif op == "compact":
        lens = _row_lengths(case, rng, case["rows"])
        width = _pages(case["length"]) + 1
        perm = np.random.RandomState(seed % 2**32).permutation(case["pages"])
        table, used = _table(lens, width, perm)
        ref = np.zeros(case["pages"], dtype=np.int32)
        ref[perm[:used]] = 1
        for b in range(1, case["rows"], 3):  # every third request shares the full pages of the one before it
            k = min(lens[b - 1], lens[b]) // PAGE
            ref[table[b, :k]] -= 1
            table[b, :k] = table[b - 1, :k]
            ref[table[b, :k]] += 1
        s["ref0"], s["table0"], s["lens0"] = torch.from_numpy(ref).cuda(), torch.from_numpy(table).cuda(), _i32(lens)
        s["pool"] = _pool(case, case["layers"], case["pages"], g)
    elif op == "churn":
        lens = _row_lengths(case, rng, case["rows"])
        width = _pages(case["length"] + case["new"]) + 1
        perm = np.random.RandomState(seed % 2**32).permutation(case["pages"])
        table, used = _table(lens, width, perm)
        ref = np.zeros(case["pages"], dtype=np.int32)
        ref[perm[:used]] = 1
        s["ref0"], s["table0"], s["lens0"] = torch.from_numpy(ref).cuda(), torch.from_numpy(table).cuda(), _i32(lens)
        s["gone"] = _i32(list(range(0, case["rows"], 4)))
        stay = [b for b in range(case["rows"]) if b % 4]
        s["stay"] = _i32(stay)
        s["new"] = _i32([rng.randint(1, case["new"]) for _ in stay])
    elif op == "prefix":
        dt, n = DTYPES[case["dtype"]], case["requests"]
        tails = _tail_lengths(case, rng)
        head = case["prefix_pages"]
        pages = head + sum(_pages(t) for t in tails)
        pages += pages // 5 + 1
        perm = np.random.RandomState(seed % 2**32).permutation(pages).astype(np.int32)
        table = np.full((n, head + _pages(max(tails)) + 1), -1, dtype=np.int32)
        table[:, :head] = perm[:head]
        at = head
        for b, t in enumerate(tails):
            table[b, head:head + _pages(t)] = perm[at:at + _pages(t)]
            at += _pages(t)
        s["tails"] = tails
        s["table"], s["lens"] = torch.from_numpy(table).cuda(), _i32([head * PAGE + t for t in tails])
        s["q"] = torch.randn(n, case["s_q"], case["heads"], D_QK, device="cuda", generator=g).to(dt)
        s["kv"] = torch.randn(pages, PAGE, D_QK, device="cuda", generator=g).to(dt)
        if own:
            import mla_paged_kv_gb300 as mla
            s["plan"] = mla.plan_shared_prefix(s["table"], s["lens"], case["s_q"], case["heads"], case["causal"])
            s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    else:
        dt = DTYPES[case["dtype"]]
        lq, lk = _prompt_lengths(case, rng)
        s["lq"], s["lk"] = lq, lk
        s["q"] = torch.randn(sum(lq), case["heads"], case["d_qk"], device="cuda", generator=g).to(dt)
        s["k"] = torch.randn(sum(lk), case["kv_heads"], case["d_qk"], device="cuda", generator=g).to(dt)
        s["v"] = torch.randn(sum(lk), case["kv_heads"], HEAD_V, device="cuda", generator=g).to(dt)
        s["cu_q"], s["cu_k"] = _cum(lq), _cum(lk)
        if own:
            import mla_paged_kv_gb300 as mla
            s["plan"] = mla.plan_prompt(s["cu_q"], s["cu_k"], sum(lq))
            s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if op in ("append", "fork", "compact", "churn"):
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if op in ("fork", "compact", "churn"):  # the tables that a pass changes: it starts from a copy
        s["ref"], s["table"], s["lens"] = (torch.empty_like(s[k]) for k in ("ref0", "table0", "lens0"))
    return s


# ---------------------------------------------------------------- run


def run(s):
    op = s["case"]["op"]
    if op in ("fork", "compact", "churn"):
        s["ref"].copy_(s["ref0"])
        s["table"].copy_(s["table0"])
        s["lens"].copy_(s["lens0"])
    if op == "append":
        return _run_append(s)
    if op == "fork":
        return _run_fork(s)
    if op == "compact":
        return _run_compact(s)
    if op == "churn":
        return _run_churn(s)
    if op == "prefix":
        return _run_prefix(s)
    return _run_prompt(s)


def _cache_views(s):
    c = s["cache"]
    if s["case"]["cache"] != "fp8":
        return c
    return {"codes": c[..., :D_C].view(torch.float8_e4m3fn), "scales": c[..., D_C:D_C + 16].view(torch.float32),
            "rope": c[..., D_C + 16:].view(torch.bfloat16)}


def _run_append(s):
    case = s["case"]
    kv_c, k_pe = s["kv_a"][:, :D_C], s["kv_a"][:, D_C:]
    if own:
        import mla_paged_kv_gb300 as mla
        mla.cache_append(kv_c, k_pe, s["cache"], s["table"], s["lens"], cu_seqlens=s["cu"], norm_weight=s["weight"],
                         norm_eps=EPS, cos_sin=s["cos_sin"], rope_interleaved=case["interleaved"],
                         status=s["status"])
        return _cache_views(s)
    t = torch.arange(kv_c.shape[0], device="cuda")
    b = torch.bucketize(t, s["cu"][1:].long(), right=True)
    pos = s["lens"].long()[b] - s["cu"].long()[b + 1] + t
    slot = s["table"].long()[b, pos // PAGE] * PAGE + pos % PAGE
    x = kv_c.float()
    x = x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * s["weight"].float()
    k, cs = k_pe.float(), s["cos_sin"][pos]
    cos, sin = cs[:, :32], cs[:, 32:]
    if case["interleaved"]:
        lo, hi = k[:, 0::2], k[:, 1::2]
        k = torch.stack([lo * cos - hi * sin, hi * cos + lo * sin], 2).reshape(-1, D_R)
    else:
        lo, hi = k[:, :32], k[:, 32:]
        k = torch.cat([lo * cos - hi * sin, hi * cos + lo * sin], 1)
    if case["cache"] != "fp8":
        s["cache"].view(-1, D_QK)[slot] = torch.cat([x, k], 1).to(s["cache"].dtype)
        return _cache_views(s)
    x = x.view(-1, 4, 128)
    top = x.abs().amax(2)
    scale = torch.where(top > 0, top / 448.0, torch.ones_like(top))
    codes = (x / scale[:, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    rows = s["cache"].view(-1, RECORD)
    rows[slot] = torch.cat([codes.view(torch.uint8).view(-1, D_C), scale.view(torch.uint8).view(-1, 16),
                            k.to(torch.bfloat16).view(torch.uint8).view(-1, 2 * D_R)], 1)
    return _cache_views(s)


def _run_fork(s):
    ref, table, lens, pool = s["ref"], s["table"], s["lens"], s["pool"]
    if own:
        import mla_paged_kv_gb300 as mla
        pairs = mla.cache_fork(ref, table, lens, s["parents"], s["children"], status=s["status"])
        mla.cache_copy_pages(pool, pairs, layered=True, status=s["status"])
        return {"ref": ref, "table": table, "lens": lens, "pairs": pairs, "pool": pool}
    par, chi = s["parents"].long(), s["children"].long()
    n = lens[par].long()
    full, tail = n // PAGE, n % PAGE > 0
    free = (ref == 0).nonzero()[:, 0]
    new = torch.where(tail, free[(tail.long().cumsum(0) - 1).clamp(min=0)], -1)
    col = torch.arange(table.shape[1], device="cuda")[None]
    rows = table[par].long()
    child = torch.where(col < full[:, None], rows, -1)
    child = torch.where((col == full[:, None]) & tail[:, None], new[:, None], child)
    table[chi] = child.int()
    lens[chi] = n.int()
    got = child[child >= 0]
    ref.index_add_(0, got, torch.ones_like(got, dtype=torch.int32))
    old = torch.where(tail, rows.gather(1, full[:, None])[:, 0], -1)
    pool[:, new[tail]] = pool[:, old[tail]]
    return {"ref": ref, "table": table, "lens": lens, "pairs": torch.stack([old, new], 1).int(), "pool": pool}


def _run_compact(s):
    ref, table, lens, pool = s["ref"], s["table"], s["lens"], s["pool"]
    if own:
        import mla_paged_kv_gb300 as mla
        pairs, count = mla.cache_compact(ref, table, lens, status=s["status"])
        mla.cache_copy_pages(pool, pairs, count=count, layered=True, status=s["status"])
        return {"ref": ref, "table": table, "pairs": pairs, "count": count, "pool": pool}
    live = ref > 0
    n = live.sum()
    at = torch.arange(ref.shape[0], device="cuda")
    src, dst = at[live & (at >= n)], at[~live & (at < n)]
    to = at.clone()
    to[src] = dst
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], -1))
    ref[dst] = ref[src]
    ref[src] = 0
    pool[:, dst] = pool[:, src]
    pairs = torch.full((ref.shape[0] // 2, 2), -1, dtype=torch.int32, device="cuda")
    pairs[:src.shape[0]] = torch.stack([src, dst], 1).int()
    return {"ref": ref, "table": table, "pairs": pairs,
            "count": torch.full((1,), src.shape[0], dtype=torch.int32, device="cuda"), "pool": pool}


def _run_churn(s):
    ref, table, lens = s["ref"], s["table"], s["lens"]
    if own:
        import mla_paged_kv_gb300 as mla
        mla.cache_free(ref, table, lens, s["gone"], status=s["status"])
        mla.cache_grow(ref, table, lens, s["stay"], s["new"], status=s["status"])
        return {"ref": ref, "table": table, "lens": lens}
    col = torch.arange(table.shape[1], device="cuda")[None]
    gone, stay = s["gone"].long(), s["stay"].long()
    rows = table[gone].long()
    page = rows[col < (lens[gone].long()[:, None] + PAGE - 1) // PAGE]
    ref.index_add_(0, page, torch.full_like(page, -1, dtype=torch.int32))
    table[gone] = -1
    lens[gone] = 0
    n = lens[stay].long()
    have, want = (n + PAGE - 1) // PAGE, (n + s["new"] + PAGE - 1) // PAGE
    first = (want - have).cumsum(0) - (want - have)
    free = (ref == 0).nonzero()[:, 0]
    take = (col >= have[:, None]) & (col < want[:, None])
    rows = torch.where(take, free[torch.where(take, first[:, None] + col - have[:, None], 0)], table[stay].long())
    table[stay] = rows.int()
    ref[rows[take]] = 1
    lens[stay] += s["new"]
    return {"ref": ref, "table": table, "lens": lens}


def _run_prefix(s):
    case = s["case"]
    if own:
        import mla_paged_kv_gb300 as mla
        return mla.shared_prefix_decode(s["q"], s["kv"], s["table"], s["lens"], causal=case["causal"], pl=s["plan"],
                                        status=s["status"])
    q, kv, head, s_q = s["q"].float(), s["kv"], case["prefix_pages"], case["s_q"]
    n, h = q.shape[0], q.shape[2]
    front = kv[s["table"][0, :head].long()].view(-1, D_QK).float()
    width = s["table"].shape[1] - head
    back = kv[s["table"][:, head:].clamp(min=0).long()].view(n, width * PAGE, D_QK).float()
    scale = 1.0 / math.sqrt(D_QK)
    a = (q.reshape(-1, D_QK) @ front.t()).view(n, s_q, h, -1) * scale
    b = torch.einsum("bihd,bjd->bihj", q, back) * scale
    left = (s["lens"].long() - head * PAGE)[:, None]
    if case["causal"]:
        left = left - s_q + 1 + torch.arange(s_q, device="cuda")[None]
    seen = torch.arange(width * PAGE, device="cuda")[None, None] < left.expand(n, s_q)[:, :, None]
    b = b.masked_fill(~seen[:, :, None], -math.inf)
    top = torch.maximum(a.amax(3), b.amax(3))[..., None]
    a, b = (a - top).exp(), (b - top).exp()
    total = a.sum(3, keepdim=True) + b.sum(3, keepdim=True)
    out = (a.view(-1, a.shape[3]) @ front[:, :D_V]).view(n, s_q, h, D_V)
    out = (out + torch.einsum("bihj,bjd->bihd", b, back[..., :D_V])) / total
    return out.to(s["q"].dtype), (top + total.log())[..., 0]


def _run_prompt(s):
    case = s["case"]
    if own:
        import mla_paged_kv_gb300 as mla
        return mla.prompt_attention(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=True, pl=s["plan"],
                                    status=s["status"])
    scale = 1.0 / math.sqrt(case["d_qk"])
    group = case["heads"] // case["kv_heads"]
    outs, lses = [], []
    for q, k, v in zip(s["q"].split(s["lq"]), s["k"].split(s["lk"]), s["v"].split(s["lk"])):
        q = q.float().transpose(0, 1).reshape(case["kv_heads"], group * q.shape[0], -1)
        k, v = k.float().transpose(0, 1), v.float().transpose(0, 1)
        a = torch.matmul(q, k.transpose(1, 2)).mul_(scale).view(case["heads"], -1, k.shape[1])
        hide = torch.ones(a.shape[1:], dtype=torch.bool, device="cuda").triu_(k.shape[1] - a.shape[1] + 1)
        a.masked_fill_(hide, -math.inf)
        top = a.amax(2, keepdim=True)
        a.sub_(top).exp_()
        total = a.sum(2, keepdim=True)
        o = torch.matmul(a.view(case["kv_heads"], -1, k.shape[1]), v).view(case["heads"], -1, HEAD_V) / total
        outs.append(o.transpose(0, 1).to(s["q"].dtype))
        lses.append((top + total.log())[..., 0].t())
    return torch.cat(outs), torch.cat(lses)


# ---------------------------------------------------------------- work


def work(case):
    op, rng = case["op"], _sizes(case)
    if op == "append":
        return {"bytes": case["tokens"] * (2 * D_QK + _row_bytes(case["cache"]) + 256), "flops": 10 * case["tokens"] * D_QK}
    if op == "fork":
        table = 4 * case["children"] * (_pages(case["length"]) + 2)
        return {"bytes": 2 * case["children"] * case["layers"] * PAGE * _row_bytes(case["cache"]) + 3 * table}
    if op == "compact":
        lens = _row_lengths(case, rng, case["rows"])
        used = sum(_pages(n) for n in lens)
        moved = used * (1 - used / case["pages"])
        table = 4 * case["rows"] * (_pages(case["length"]) + 1)
        return {"bytes": 2 * moved * case["layers"] * PAGE * _row_bytes(case["cache"]) + 8 * case["pages"] + 2 * table}
    if op == "churn":
        table = 4 * case["rows"] * (_pages(case["length"] + case["new"]) + 1)
        return {"bytes": 3 * 4 * case["pages"] + 2 * table}
    if op == "prefix":
        keys = sum(_tail_lengths(case, rng))
        per, rows = case["s_q"] * case["heads"], case["requests"] * case["s_q"] * case["heads"]
        pairs = rows * case["prefix_pages"] * PAGE + per * keys
        return {"bytes": 2 * D_QK * (case["prefix_pages"] * PAGE + keys) + rows * (2 * D_QK + 2 * D_V + 4),
                "flops": 2 * pairs * (D_QK + D_V)}
    lq, lk = _prompt_lengths(case, rng)
    pairs = sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(lq, lk))
    row = case["d_qk"] + HEAD_V
    return {"bytes": 2 * row * (case["heads"] * sum(lq) + case["kv_heads"] * sum(lk)) + 4 * case["heads"] * sum(lq),
            "flops": 2 * case["heads"] * pairs * row}


# ---------------------------------------------------------------- exact


def _e4m3(x):
    """Nearest E4M3 value (ties to even, saturating) of 64-bit values."""
    _, e = torch.frexp(x.abs())
    step = torch.ldexp(torch.ones_like(x), (e - 4).clamp(min=-9))
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def exact(case, seed):
    op = case["op"]
    if op not in ("append", "prefix", "prompt"):
        return None  # whole numbers
    s = prepare(case, seed)
    if op == "append":
        return _exact_append(case, s)
    if op == "prefix":
        return _exact_prefix(case, s)
    return _exact_prompt(case, s)


def _exact_append(case, s):
    cu, lens, table = s["cu"].tolist(), s["lens"].tolist(), s["table"].tolist()
    slot, pos = [], []
    for b, total in enumerate(lens):
        n = cu[b + 1] - cu[b]
        for p in range(total - n, total):
            slot.append(table[b][p // PAGE] * PAGE + p % PAGE)
            pos.append(p)
    slot, pos = torch.tensor(slot, device="cuda"), torch.tensor(pos, device="cuda")
    raw = s["kv_a"].double()
    c = raw[:, :D_C]
    c = c / ((c * c).sum(1, keepdim=True) / D_C + EPS).sqrt() * s["weight"].double()
    rot = torch.complex(s["cos_sin"].double()[pos, :32], s["cos_sin"].double()[pos, 32:])
    k = raw[:, D_C:]
    if case["interleaved"]:
        k = torch.view_as_real(torch.view_as_complex(k.reshape(-1, 32, 2).contiguous()) * rot).reshape(-1, D_R)
    else:
        z = torch.complex(k[:, :32].contiguous(), k[:, 32:].contiguous()) * rot
        k = torch.cat([z.real, z.imag], 1)
    shape = s["cache"].shape[:2]

    def placed(v, dims, start=0.0):
        full = torch.full((shape[0] * PAGE, *dims), start, dtype=torch.float64, device="cuda")
        full[slot] = v.reshape(-1, *dims)
        return full.reshape(*shape, *dims)

    if case["cache"] != "fp8":
        return placed(torch.cat([c, k], 1), (D_QK,))
    c = c.reshape(-1, 4, 128)
    top = c.abs().amax(2)
    scale = torch.where(top > 0, top / 448.0, torch.ones_like(top))
    return {"codes": placed(_e4m3(c / scale[:, :, None]), (D_C,)), "scales": placed(scale, (4,)),
            "rope": placed(k, (D_R,))}


def _exact_prefix(case, s):
    kv, table, lens = s["kv"], s["table"].tolist(), s["lens"].tolist()
    outs, lses = [], []
    for b, total in enumerate(lens):
        keys = kv[torch.tensor(table[b][:_pages(total)], device="cuda")].reshape(-1, D_QK)[:total].double()
        for i in range(case["s_q"]):
            seen = total - case["s_q"] + i + 1 if case["causal"] else total
            a = (s["q"][b, i].double() @ keys[:seen].t()) / math.sqrt(D_QK)
            lse = torch.logsumexp(a, 1)
            outs.append(torch.exp(a - lse[:, None]) @ keys[:seen, :D_V])
            lses.append(lse)
    shape = s["q"].shape[:3]
    return torch.stack(outs).reshape(*shape, D_V), torch.stack(lses).reshape(shape)


def _exact_prompt(case, s):
    out = torch.empty(*s["q"].shape[:2], HEAD_V, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    group = case["heads"] // case["kv_heads"]
    q0 = k0 = 0
    for a, b in zip(s["lq"], s["lk"]):
        for h in range(case["heads"]):
            k, v = (s[n][k0:k0 + b, h // group].double() for n in ("k", "v"))
            for i in range(0, a, 4096):  # rows in blocks: a 64-bit score matrix is large
                m = min(4096, a - i)
                top = b - a + i + m
                x = s["q"][q0 + i:q0 + i + m, h].double() @ k[:top].t() / math.sqrt(case["d_qk"])
                at = torch.arange(top, device="cuda")[None] - torch.arange(m, device="cuda")[:, None]
                x[at > b - a + i] = -math.inf
                z = torch.logsumexp(x, 1)
                out[q0 + i:q0 + i + m, h] = torch.exp(x - z[:, None]) @ v[:top]
                lse[q0 + i:q0 + i + m, h] = z
        q0, k0 = q0 + a, k0 + b
    return out, lse
