"""Cases of the operators that take chunks of new tokens through a paged latent (MLA) cache.

The table of rotary positions, the rotation (and norm) of query and key heads,
rows of the cache as packed rows, and the attention of ragged chunks over the
cache.  Each case names an operator (``op``) and its sizes; ``prepare`` makes the
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
HEAD = 192            # a projected query head: 128 dims and 64 rotary ones
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": torch.bfloat16}


# ---------------------------------------------------------------- cases


def listed():
    return [
        # a model's positions as it is loaded, no scaling
        dict(name="table_4k", op="table", positions=4096, dim=64, base=10000.0, scaling="none", factor=1.0,
             original=4096),
        # a long context, stretched 40 times by parts (YaRN)
        dict(name="table_160k_yarn", op="table", positions=163840, dim=64, base=10000.0, scaling="yarn", factor=40.0,
             original=4096),
        # queries of one decode step: the rotary 64 of each head's 192 into the decode's 576-wide rows; latency
        dict(name="heads_step_b8", op="heads", requests=8, tokens=8, ctx=1500, q_heads=128, k_heads=0, dim=64,
             rope=64, norm=False, interleaved=True, dtype="bf16"),
        # the same for chunks of prompts, all 128 heads
        dict(name="heads_chunks_h128", op="heads", requests=13, tokens=8193, ctx=2000, q_heads=128, k_heads=0, dim=64,
             rope=64, norm=False, interleaved=True, dtype="bf16"),
        # heads of a prompt with grouped keys: norm of every query and key head, then the rotation, out of packed rows
        dict(name="heads_norm_qk", op="heads", requests=24, tokens=24577, ctx=900, q_heads=32, k_heads=8, dim=128,
             rope=128, norm=True, interleaved=False, dtype="bf16"),
        # the cached contexts of a few requests, to be expanded into heads
        dict(name="gather_b4_fp8", op="gather", requests=4, rows=2500, cache="fp8"),
        # contexts of a batch of chunks
        dict(name="gather_b13_fp8", op="gather", requests=13, rows=24577, cache="fp8"),
        dict(name="gather_b24_bf16", op="gather", requests=24, rows=49153, cache="bf16"),
        # a few drafted tokens each, a tensor-parallel share of the heads: latency
        dict(name="chunk_drafts_b8_h16", op="chunk", requests=8, tokens=3, singles=0, ctx=1500, heads=16, cache="bf16",
             causal=True),
        # drafts of a batch to verify, all heads
        dict(name="chunk_drafts_b64_h128", op="chunk", requests=64, tokens=6, singles=0, ctx=4096, heads=128,
             cache="bf16", causal=True),
        # one scheduler step of a mixed batch: chunks of prompts beside single tokens, FP8 records
        dict(name="chunk_mixed_b43_h16_fp8", op="chunk", requests=43, tokens=400, singles=40, ctx=3000, heads=16,
             cache="fp8", causal=True),
        # follow-up turns over long conversations, all heads
        dict(name="chunk_turns_b3_h128", op="chunk", requests=3, tokens=300, singles=0, ctx=8000, heads=128,
             cache="bf16", causal=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["table", "heads", "heads", "gather", "chunk", "chunk", "chunk"])
    if op == "table":
        return dict(op=op, positions=_log(rng, 1, 160000), dim=rng.choice([32, 64, 64, 128]),
                    base=rng.choice([10000.0, 500000.0]), scaling=rng.choice(["none", "linear", "ntk", "yarn",
                                                                              "wavelength"]),
                    factor=rng.uniform(1.5, 40.0), original=rng.choice([2048, 4096, 8192]))
    if op == "heads":
        n = _log(rng, 1, 48)
        if rng.random() < 0.5:  # the rotary part of MLA heads
            q, k, dim, rope, norm = rng.choice([12, 32, 64, 128]), 0, 64, 64, False
        else:
            dim = rng.choice([64, 128, 192])
            q, k, rope, norm = rng.choice([6, 12, 27]), rng.choice([0, 1, 3]), rng.choice([32, 64]), True
        most = 500000 * 128 // (dim * (q + k))
        return dict(op=op, requests=n, tokens=max(n, _log(rng, 1, most)), ctx=rng.randint(0, 2000), q_heads=q,
                    k_heads=k, dim=dim, rope=rope, norm=norm, interleaved=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "fp16"]))
    if op == "gather":
        n = _log(rng, 1, 48)
        return dict(op=op, requests=n, rows=max(n, _log(rng, 1, 45000)), cache=rng.choice(["fp8", "bf16", "fp16"]))
    heads = rng.choice([16, 32, 64, 128])
    cache = rng.choice(["bf16", "fp16", "fp8"])
    n = _log(rng, 1, 48)
    tokens, ctx = _log(rng, 1, 400), _log(rng, 20, 8000)
    # at most about a quarter of the largest listed case's products
    while n * tokens * heads * (ctx + tokens) > 2 ** 28:
        n, tokens, ctx = max(1, n // 2), max(1, 3 * tokens // 4), max(20, 3 * ctx // 4)
    return dict(op=op, requests=n, tokens=tokens, singles=rng.randint(0, n - 1), ctx=ctx, heads=heads, cache=cache,
                causal=rng.random() < 0.8)


# ---------------------------------------------------------------- lengths (from the case alone: shapes stay)


def _sizes(case):
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _pages(n):
    return -(-n // PAGE)


def _shares(total, n, rng):
    """``n`` ragged lengths of at least one that sum to ``total``."""
    w = [rng.uniform(0.3, 1.0) for _ in range(n)]
    part = [max(1, int(total * x / sum(w))) for x in w]
    part[-1] += total - sum(part)
    return part if part[-1] >= 1 else [1] * (n - 1) + [total - n + 1]


def _chunk_lengths(case, rng):
    """New tokens and keys of each request (the new tokens among them)."""
    n, top, alone = case["requests"], case["tokens"], case["singles"]
    new = [rng.randint(max(1, top // 3), top) for _ in range(n - alone)] + [1] * alone
    rng.shuffle(new)
    return new, [a + rng.randint(case["ctx"] // 2, case["ctx"]) for a in new]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cum(v):
    return _i32([0] + list(np.cumsum(v)))


def _table(lengths, pages, seed):
    """A block table whose rows take scattered pages of the pool."""
    perm = np.random.RandomState(seed % 2**32).permutation(pages)
    t = np.full((len(lengths), _pages(max(lengths)) + 1), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(lengths):
        t[b, :_pages(n)] = perm[at:at + _pages(n)]
        at += _pages(n)
    return torch.from_numpy(t).cuda()


def _pool(kind, pages, g):
    """A cache of 16-bit rows, or of FP8 records whose codes and scales are those of normal values."""
    if kind != "fp8":
        return torch.randn(pages, PAGE, D_QK, device="cuda", generator=g).to(DTYPES[kind])
    rec = torch.empty(pages, PAGE, RECORD, dtype=torch.uint8, device="cuda")
    codes = (torch.randn(pages, PAGE, D_C, device="cuda", generator=g) * 120.0).clamp(-448.0, 448.0)
    rec[..., :D_C] = codes.to(torch.float8_e4m3fn).view(torch.uint8)
    scales = (0.5 + torch.rand(pages, PAGE, 4, device="cuda", generator=g)) / 120.0
    rec[..., D_C:D_C + 16] = scales.view(torch.uint8)
    rope = torch.randn(pages, PAGE, D_R, device="cuda", generator=g).to(torch.bfloat16)
    rec[..., D_C + 16:] = rope.view(torch.uint8)
    return rec


def _angles(positions, dim):
    f = 10000.0 ** (-torch.arange(0, dim // 2, device="cuda", dtype=torch.float64) / (dim // 2))
    a = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * f[None]
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


# ---------------------------------------------------------------- prepare


def prepare(case, seed):
    rng, g = _sizes(case), _gen(seed)
    s = {"case": case}
    op = case["op"]
    if op == "table":
        s["first"] = seed % 1000  # the first position
    elif op == "heads":
        dt, t, dim = DTYPES[case["dtype"]], case["tokens"], case["dim"]
        q, k = case["q_heads"], case["k_heads"]
        new = _shares(t, case["requests"], rng)
        total = [a + rng.randint(case["ctx"] // 2, case["ctx"]) for a in new]
        s["lens"], s["cu"] = _i32(total), _cum(new)
        s["cos_sin"] = _angles(max(total) + 1, case["rope"])
        if case["norm"]:  # query, key and value heads of one packed projection
            rows = torch.randn(t, (q + 2 * k) * dim, device="cuda", generator=g)
            rows.mul_(0.5 + 2.0 * torch.rand(t, 1, device="cuda", generator=g))
            rows = rows.to(dt)
            s["q"] = rows[:, :q * dim].view(t, q, dim)
            s["k"] = rows[:, q * dim:(q + k) * dim].view(t, k, dim) if k else None
            s["q_weight"] = (1.0 + 0.2 * torch.randn(dim, device="cuda", generator=g)).to(dt)
            s["k_weight"] = (1.0 + 0.2 * torch.randn(dim, device="cuda", generator=g)).to(dt) if k else None
        else:
            s["q"] = torch.randn(t, q, HEAD, device="cuda", generator=g).to(dt)[..., HEAD - dim:]
            s["rows"] = torch.zeros(t, q, D_QK, dtype=dt, device="cuda")  # the decode's query rows
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    elif op == "gather":
        lens = _shares(case["rows"], case["requests"], rng)
        need = sum(_pages(n) for n in lens)
        pages = need + need // 5 + 1
        s["lens"], s["cu"], s["table"] = _i32(lens), _cum(lens), _table(lens, pages, seed)
        s["cache"] = _pool(case["cache"], pages, g)
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    else:
        dt = DTYPES[case["cache"]]
        new, total = _chunk_lengths(case, rng)
        need = sum(_pages(n) for n in total)
        pages = need + need // 5 + 1
        s["new"], s["total"] = new, total
        s["cu"], s["lens"], s["table"] = _cum(new), _i32(total), _table(total, pages, seed)
        s["q"] = torch.randn(sum(new), case["heads"], D_QK, device="cuda", generator=g).to(dt)
        s["cache"] = _pool(case["cache"], pages, g)
        if own:
            import mla_paged_kv_gb300 as mla
            s["plan"] = mla.plan_chunks(s["cu"], s["lens"], sum(new), case["heads"], causal=case["causal"])
            s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


# ---------------------------------------------------------------- run


def run(s):
    op = s["case"]["op"]
    if op == "table":
        return _run_table(s)
    if op == "heads":
        return _run_heads(s)
    if op == "gather":
        return _run_gather(s)
    return _run_chunk(s)


def _run_table(s):
    c = s["case"]
    n, dim, base, factor = c["positions"], c["dim"], c["base"], c["factor"]
    if own:
        import mla_paged_kv_gb300 as mla
        return mla.rope_table(n, dim, base=base, scaling=c["scaling"], factor=factor, original=c["original"],
                              first=s["first"], device="cuda")
    i = torch.arange(dim // 2, device="cuda", dtype=torch.float64)
    if c["scaling"] == "ntk":
        base = base * factor ** (dim / (dim - 2))
    f = base ** (-2.0 * i / dim)
    size = 1.0
    if c["scaling"] == "linear":
        f = f / factor
    elif c["scaling"] == "yarn":  # 32 turns over the original context and more stay, one and fewer are stretched
        low, high = (dim * math.log(c["original"] / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))
                     for turns in (32.0, 1.0))
        low, high = max(math.floor(low), 0), min(math.ceil(high), dim - 1)
        part = ((i - low) / max(high - low, 0.001)).clamp(0.0, 1.0)
        f = f / factor * part + f * (1.0 - part)
        size = 0.1 * math.log(factor) + 1.0
    elif c["scaling"] == "wavelength":  # 4 turns and more stay, one and fewer are stretched, a blend between
        part = ((c["original"] * f / (2.0 * math.pi) - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        f = (1.0 - part) * f / factor + part * f
    a = torch.arange(s["first"], s["first"] + n, device="cuda", dtype=torch.float64)[:, None] * f[None]
    return (torch.cat([a.cos(), a.sin()], 1) * size).float()


def _positions(s):
    t = torch.arange(s["case"]["tokens"], device="cuda")
    b = torch.bucketize(t, s["cu"][1:].long(), right=True)
    return s["lens"].long()[b] - s["cu"].long()[b + 1] + t


def _heads_plain(s, x, weight):
    case = s["case"]
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt(y.square().mean(2, keepdim=True) + EPS) * weight.float()
    rope = case["rope"]
    cs = s["cos_sin"][_positions(s)]
    cos, sin = cs[:, None, :rope // 2], cs[:, None, rope // 2:]
    r = y[..., y.shape[2] - rope:]
    if case["interleaved"]:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], 3).flatten(2)
    else:
        a, b = r[..., :rope // 2], r[..., rope // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], 2)
    return torch.cat([y[..., :y.shape[2] - rope], r], 2).to(x.dtype)


def _run_heads(s):
    case = s["case"]
    if own:
        import mla_paged_kv_gb300 as mla
        more = dict(cu_seqlens=s["cu"], interleaved=case["interleaved"], status=s["status"])
        if not case["norm"]:
            return mla.rope_heads(s["q"], s["cos_sin"], s["lens"], out=s["rows"][..., D_QK - case["dim"]:], **more)
        return mla.rope_heads(s["q"], s["cos_sin"], s["lens"], norm_weight=s["q_weight"], norm_eps=EPS, k=s["k"],
                              k_norm_weight=s["k_weight"], **more)
    if not case["norm"]:
        out = s["rows"][..., D_QK - case["dim"]:]
        out.copy_(_heads_plain(s, s["q"], None))
        return out
    q = _heads_plain(s, s["q"], s["q_weight"])
    return q if s["k"] is None else (q, _heads_plain(s, s["k"], s["k_weight"]))


def _rows(cache, slots):
    """Rows of the cache at these slots, in 32 bits."""
    r = cache.view(-1, cache.shape[2])[slots]
    if cache.dtype != torch.uint8:
        return r.float()
    codes = r[:, :D_C].contiguous().view(torch.float8_e4m3fn).float().view(-1, 4, 128)
    scales = r[:, D_C:D_C + 16].contiguous().view(torch.float32)
    rope = r[:, D_C + 16:].contiguous().view(torch.bfloat16).float()
    return torch.cat([(codes * scales[:, :, None]).view(-1, D_C), rope], 1)


def _run_gather(s):
    case = s["case"]
    if own:
        import mla_paged_kv_gb300 as mla
        return mla.cache_gather(s["cache"], s["table"], s["cu"], case["rows"], status=s["status"])
    t = torch.arange(case["rows"], device="cuda")
    b = torch.bucketize(t, s["cu"][1:].long(), right=True)
    pos = t - s["cu"].long()[b]
    slot = s["table"].long()[b, pos // PAGE] * PAGE + pos % PAGE
    return _rows(s["cache"], slot).to(DTYPES[case["cache"]])


def _run_chunk(s):
    case = s["case"]
    if own:
        import mla_paged_kv_gb300 as mla
        return mla.chunk_attention(s["q"], s["cache"], s["table"], s["lens"], s["cu"], causal=case["causal"],
                                   pl=s["plan"], status=s["status"])
    h, scale = case["heads"], 1.0 / math.sqrt(D_QK)
    table, at = s["table"].long(), 0
    place = torch.arange(PAGE, device="cuda")
    outs, lses = [], []
    for b, (n, total) in enumerate(zip(s["new"], s["total"])):
        slots = (table[b, :_pages(total), None] * PAGE + place).view(-1)[:total]
        keys = _rows(s["cache"], slots)
        a = s["q"][at:at + n].float().view(n * h, D_QK) @ keys.t()
        a = a.mul_(scale).view(n, h, total)
        if case["causal"]:
            hide = torch.ones(n, total, dtype=torch.bool, device="cuda").triu_(total - n + 1)
            a.masked_fill_(hide[:, None], -math.inf)
        top = a.amax(2, keepdim=True)
        a.sub_(top).exp_()
        sum_ = a.sum(2, keepdim=True)
        outs.append(((a.view(n * h, total) @ keys[:, :D_V]).view(n, h, D_V) / sum_).to(s["q"].dtype))
        lses.append((top + sum_.log())[..., 0])
        at += n
    return torch.cat(outs), torch.cat(lses)


# ---------------------------------------------------------------- work


def _row_bytes(cache):
    return RECORD if cache == "fp8" else 2 * D_QK


def work(case):
    op, rng = case["op"], _sizes(case)
    if op == "table":
        return {"bytes": 4 * case["positions"] * case["dim"]}
    if op == "heads":
        heads = case["q_heads"] + case["k_heads"]
        return {"bytes": case["tokens"] * (4 * heads * case["dim"] + 4 * case["rope"]),
                "flops": case["tokens"] * heads * (3 * case["rope"] + (4 * case["dim"] if case["norm"] else 0))}
    if op == "gather":
        return {"bytes": case["rows"] * (_row_bytes(case["cache"]) + 2 * D_QK)}
    new, total = _chunk_lengths(case, rng)
    if case["causal"]:
        pairs = sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(new, total))
    else:
        pairs = sum(a * b for a, b in zip(new, total))
    rows = case["heads"] * sum(new)
    return {"bytes": _row_bytes(case["cache"]) * sum(total) + rows * (2 * D_QK + 2 * D_V + 4),
            "flops": 2 * case["heads"] * pairs * (D_QK + D_V)}


# ---------------------------------------------------------------- exact


def exact(case, seed):
    s = prepare(case, seed)
    return {"table": _exact_table, "heads": _exact_heads, "gather": _exact_gather, "chunk": _exact_chunk}[case["op"]](
        case, s)


def _exact_table(case, s):
    dim, base, factor, original = case["dim"], case["base"], case["factor"], case["original"]
    pairs = []
    for i in range(dim // 2):
        if case["scaling"] == "ntk":
            pairs.append((base * factor ** (dim / (dim - 2.0))) ** (-i / (dim / 2.0)))
            continue
        f = base ** (-i / (dim / 2.0))
        keep = 1.0  # the share of the unscaled frequency
        if case["scaling"] == "linear":
            keep = 0.0
        elif case["scaling"] == "yarn":
            lo = max(0, math.floor(dim / 2.0 * math.log(original / (64.0 * math.pi), base)))
            hi = min(dim - 1, math.ceil(dim / 2.0 * math.log(original / (2.0 * math.pi), base)))
            keep = 1.0 - min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
        elif case["scaling"] == "wavelength":
            turns = original / (2.0 * math.pi / f)
            keep = min(1.0, max(0.0, (turns - 1.0) / 3.0))
        pairs.append(keep * f + (1.0 - keep) * f / factor)
    p = np.arange(s["first"], s["first"] + case["positions"], dtype=np.float64)
    z = np.exp(1j * np.multiply.outer(p, np.array(pairs)))
    if case["scaling"] == "yarn":
        z *= 1.0 + math.log(factor) / 10.0
    return np.concatenate([z.real, z.imag], 1)


def _exact_heads(case, s):
    rope, half = case["rope"], case["rope"] // 2
    cu, pos = s["cu"].tolist(), []
    for b, n in enumerate(s["lens"].tolist()):
        pos += range(n - (cu[b + 1] - cu[b]), n)
    cs = s["cos_sin"].double()[torch.tensor(pos, device="cuda")]
    turn = torch.complex(cs[:, :half], cs[:, half:])[:, None]

    def one(x, weight):
        x = x.double()
        if weight is not None:
            x = x / ((x * x).sum(2, keepdim=True) / case["dim"] + EPS).sqrt() * weight.double()
        out = x.clone()
        r = x[..., case["dim"] - rope:]
        if case["interleaved"]:
            z = torch.view_as_complex(r.reshape(*r.shape[:2], half, 2).contiguous()) * turn
            out[..., case["dim"] - rope:] = torch.view_as_real(z).reshape(r.shape)
        else:
            z = torch.complex(r[..., :half].contiguous(), r[..., half:].contiguous()) * turn
            out[..., case["dim"] - rope:] = torch.cat([z.real, z.imag], 2)
        return out

    if not case["norm"]:
        return one(s["q"], None)
    q = one(s["q"], s["q_weight"])
    return q if s["k"] is None else (q, one(s["k"], s["k_weight"]))


def _exact_rows(case, s, lengths):
    """All keys of the requests, one after another, in 64 bits."""
    table, parts = s["table"].tolist(), []
    for b, n in enumerate(lengths):
        r = s["cache"][torch.tensor(table[b][:_pages(n)], device="cuda")].flatten(0, 1)[:n]
        if case["cache"] == "fp8":
            scale = r[:, D_C:D_C + 16].contiguous().view(torch.float32).double().repeat_interleave(128, 1)
            r = torch.cat([r[:, :D_C].contiguous().view(torch.float8_e4m3fn).double() * scale,
                           r[:, D_C + 16:].contiguous().view(torch.bfloat16).double()], 1)
        parts.append(r.double())
    return parts


def _exact_gather(case, s):
    return torch.cat(_exact_rows(case, s, s["lens"].tolist()))


def _exact_chunk(case, s):
    outs, lses, at = [], [], 0
    for n, keys in zip(s["new"], _exact_rows(case, s, s["total"])):
        total = keys.shape[0]
        for i in range(0, n, 32):  # tokens in blocks: a 64-bit score matrix is large
            m = min(32, n - i)
            x = torch.einsum("ihd,jd->ihj", s["q"][at + i:at + i + m].double(), keys) / math.sqrt(D_QK)
            if case["causal"]:
                j = torch.arange(total, device="cuda")[None, None]
                last = (total - n + i + torch.arange(m, device="cuda"))[:, None, None]
                x = torch.where(j <= last, x, torch.full_like(x, -math.inf))
            z = torch.logsumexp(x, 2)
            outs.append(torch.einsum("ihj,jd->ihd", (x - z[..., None]).exp(), keys[:, :D_V]))
            lses.append(z)
        at += n
    return torch.cat(outs), torch.cat(lses)
