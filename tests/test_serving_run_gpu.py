"""The serving operators together, as a program uses them: prompts are attended
and appended, one is forked into samples, the samples grow token by token and
decode over their shared prefix, some end, the pool is compacted, and the rest
go on."""

import numpy as np
import pytest
import torch

import mla_paged_kv_gb300 as mla
from oracle import mla_oracle as orc
from oracle import serving_oracle as so
from tests.parity import compare

pytestmark = pytest.mark.gpu

H, LAYERS, PAGES, ROWS, WIDTH = 16, 2, 96, 12, 12


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Program:
    """A pool of `LAYERS` layers with its bookkeeping, and random layers' outputs."""

    def __init__(self, fp8, seed):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.fp8 = fp8
        shape = (LAYERS, PAGES, 64, 656 if fp8 else 576)
        self.pool = torch.zeros(shape, dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
        self.ref = torch.zeros(PAGES, dtype=torch.int32, device="cuda")
        self.table = torch.full((ROWS, WIDTH), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(ROWS, dtype=torch.int32, device="cuda")
        self.weight = (1 + 0.1 * self.rand(512)).to(torch.bfloat16)
        ang = torch.arange(WIDTH * 64)[:, None] * 10000.0 ** (-torch.arange(32) / 32.0)[None]
        self.cos_sin = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
        self.status = i32([0])
        self.count = torch.zeros(PAGES, dtype=torch.int64)

    def rand(self, *s):
        return torch.randn(*s, device="cuda", generator=self.g)

    def append(self, rows, new):
        """New tokens of `rows` in every layer; rows must have grown."""
        idx = torch.tensor(rows, device="cuda")
        cu = None if len(set(new)) == 1 else i32([0] + list(np.cumsum(new)))
        for layer in range(LAYERS):
            kv_a = self.rand(sum(new), 576).to(torch.bfloat16)
            mla.cache_append(kv_a[:, :512], kv_a[:, 512:], self.pool[layer], self.table[idx], self.lens[idx],
                             cu_seqlens=cu, norm_weight=self.weight, cos_sin=self.cos_sin, rope_interleaved=True,
                             refcount=self.ref, status=self.status)

    def oracle(self, q, rows, layer):
        table, lens = self.table[rows].cpu().numpy(), self.lens[rows].cpu().numpy()
        kv = self.pool[layer].cpu()
        kv = kv.numpy() if self.fp8 else kv.float().numpy()
        fn = orc.dense_fp8_decode if self.fp8 else orc.dense_decode
        return fn(q.double().cpu().numpy(), kv, table, lens, False, 1 / 24)[:2]

    def decode(self, rows, check=True):
        idx = torch.tensor(rows, device="cuda")
        table, lens = self.table[idx], self.lens[idx]
        outs = []
        pl = mla.plan_shared_prefix(table, lens, 1, H)
        for layer in range(LAYERS):
            q = torch.randn(len(rows), 1, H, 576, device="cuda",
                            generator=torch.Generator(device="cuda").manual_seed(layer)).to(torch.bfloat16)
            out, lse = mla.shared_prefix_decode(q, self.pool[layer], table, lens, pl=pl, status=self.status)
            if check:
                compare(out, lse, *self.oracle(q, idx, layer))
            outs.append((out, lse))
        return outs

    def audit(self):
        """Every count equals the number of entries that name the page."""
        used = torch.zeros(PAGES, dtype=torch.int32)
        for r, n in enumerate(self.lens.tolist()):
            for p in self.table[r, :-(-n // 64)].tolist():
                used[p] += 1
        assert torch.equal(used, self.ref.cpu())
        assert int(self.status) == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_prompts_samples_and_compaction(fp8):
    p = Program(fp8, seed=21 + fp8)
    prompts = [300, 77]
    # prompts: attention over the expanded heads, then their latent rows into the cache
    q, k, v = (p.rand(sum(prompts), 4, d).to(torch.bfloat16) for d in (192, 192, 128))
    cu = [0, 300, 377]
    out, lse = mla.prompt_attention(q, k, v, i32(cu), status=p.status)
    want, wlse, mix, _ = so.prompt_attention(q.double().cpu().numpy(), k.double().cpu().numpy(),
                                             v.double().cpu().numpy(), cu, cu, True, 192 ** -0.5)
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= 2.0 ** -7 * mix + 2.0 ** -8 * np.abs(want))
    mla.cache_grow(p.ref, p.table, p.lens, i32([0, 1]), i32(prompts), status=p.status)
    p.append([0, 1], prompts)
    p.audit()
    # six samples of the first prompt
    samples = [2, 3, 4, 5, 6, 7]
    pairs = mla.cache_fork(p.ref, p.table, p.lens, i32([0] * 6), i32(samples), status=p.status)
    mla.cache_copy_pages(p.pool, pairs, layered=True, status=p.status)
    p.audit()
    for _ in range(3):
        mla.cache_grow(p.ref, p.table, p.lens, i32(samples), i32([1] * 6), status=p.status)
        p.append(samples, [1] * 6)
        p.decode(samples)
    # a chunk of different lengths for each, past a page
    mla.cache_grow(p.ref, p.table, p.lens, i32(samples), i32([30, 1, 64, 9, 100, 17]), status=p.status)
    p.append(samples, [30, 1, 64, 9, 100, 17])
    p.audit()
    # some end; the pool is compacted; the others read the same keys from other pages
    mla.cache_free(p.ref, p.table, p.lens, i32([0, 3, 6]), status=p.status)
    stay = [2, 4, 5, 7]
    before = p.decode(stay)
    moves, count = mla.cache_compact(p.ref, p.table, p.lens, status=p.status)
    mla.cache_copy_pages(p.pool, moves, count=count, layered=True, status=p.status)
    p.audit()
    live = int((p.ref > 0).sum())
    assert int(count) > 0 and not p.ref[live:].any()
    for (o1, l1), (o2, l2) in zip(before, p.decode(stay)):
        assert torch.equal(o1, o2) and torch.equal(l1, l2)
    # the pages of the shared prompt are still shared: appending into one is refused
    st = i32([0])
    kv = p.rand(1, 576).to(torch.bfloat16)
    snapshot = p.pool.clone()
    mla.cache_append(kv[:, :512], kv[:, 512:], p.pool[0], p.table[2:3], i32([64]), refcount=p.ref, status=st)
    assert int(st) == 5 and torch.equal(snapshot, p.pool)
    mla.cache_free(p.ref, p.table, p.lens, i32(list(range(8))), status=p.status)
    p.audit()
    assert not p.ref.any()


def test_a_decode_step_as_one_graph():
    """Grow, append, plan and decode of a step captured once and replayed: all sizes live on the device."""
    p = Program(False, seed=33)
    mla.cache_grow(p.ref, p.table, p.lens, i32([0]), i32([200]), status=p.status)
    p.append([0], [200])
    samples = [1, 2, 3, 4]
    mla.cache_copy_pages(p.pool, mla.cache_fork(p.ref, p.table, p.lens, i32([0] * 4), i32(samples), status=p.status),
                         layered=True, status=p.status)
    rows, one = i32(samples), i32([1] * 4)
    kv = p.rand(4, 576).to(torch.bfloat16)
    q = p.rand(4, 1, H, 576).to(torch.bfloat16)
    table, lens = p.table[1:5], p.lens[1:5]
    pl = mla.plan_shared_prefix(table, lens, 1, H)
    out = torch.empty(4, 1, H, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(4, 1, H, device="cuda")

    def step():
        mla.mla_cache_grow(p.ref, p.table, p.lens, rows, one, p.status)
        mla.mla_cache_append(kv[:, :512], kv[:, 512:], p.pool[0], table, lens, p.status, cos_sin=p.cos_sin,
                             refcount=p.ref)
        mla.mla_shared_prefix_get_plan(table, lens, 1, H, False, pl.num_parts, pl.plan)
        mla.mla_shared_prefix_decode_fwd(q, p.pool[0], table, pl, out, lse, p.status)

    step()  # (first use of every kernel outside the capture)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in range(202, 270):
        graph.replay()
        if n in (202, 230, 256, 257, 269):
            assert p.lens[1:5].tolist() == [n] * 4
            compare(out, lse, *p.oracle(q, torch.tensor(samples, device="cuda"), 0))
    p.audit()


def test_two_streams_at_once():
    """Every operator on two streams, each with its own tensors, plans and workspaces, as on one."""
    g = torch.Generator().manual_seed(21)
    lens = [300, 1, 700, 130]
    cu = [0, 300, 301, 1001, 1131]

    def state():
        r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
        s = dict(q=r(1131, 4, 192), k=r(1131, 4, 192), v=r(1131, 4, 128), row=r(1131, 576), cu=i32(cu))
        s["table"] = torch.arange(48, dtype=torch.int32).reshape(4, 12).cuda()
        s["lens"], s["cache"] = i32(lens), r(60, 64, 576)
        s["shared"] = torch.arange(96, dtype=torch.int32).reshape(4, 24) % 60
        s["shared"][:, :8] = torch.arange(8, dtype=torch.int32)
        s["shared"] = s["shared"].cuda()
        s["slens"], s["dq"], s["kv"] = i32([700, 1400, 600, 513]), r(4, 1, 16, 576), r(60, 64, 576)
        s["ref"] = (torch.rand(60, generator=g) < 0.6).int().cuda()
        s["pool"], s["status"] = r(2, 60, 64, 16), i32([0])
        return s

    def work(s):
        out, lse = mla.prompt_attention(s["q"], s["k"], s["v"], s["cu"], s["cu"], status=s["status"])
        cache = s["cache"].clone()
        mla.cache_append(s["row"][:, :512], s["row"][:, 512:], cache, s["table"], s["lens"], cu_seqlens=s["cu"],
                         status=s["status"])
        dec, dlse = mla.shared_prefix_decode(s["dq"], s["kv"], s["shared"], s["slens"], status=s["status"])
        ref, table, n, pool = s["ref"].clone(), torch.full_like(s["table"], -1), i32([0, 0, 0, 0]), s["pool"].clone()
        mla.cache_grow(ref, table, n, i32([0, 2]), i32([100, 300]), status=s["status"])
        pairs = mla.cache_fork(ref, table, n, i32([2]), i32([1]), status=s["status"])
        mla.cache_copy_pages(pool, pairs, layered=True, status=s["status"])
        mla.cache_free(ref, table, n, i32([0]), status=s["status"])
        pairs, count = mla.cache_compact(ref, table, n, status=s["status"])
        mla.cache_copy_pages(pool, pairs, count=count, layered=True, status=s["status"])
        return [out, lse, cache, dec, dlse, ref, table, n, pool, pairs, count]

    states = [state(), state()]
    want = [work(s) for s in states]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    for _ in range(5):
        got = []
        for _ in range(3):
            got = []
            for s, stream in zip(states, streams):
                with torch.cuda.stream(stream):
                    got.append(work(s))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert [int(s["status"]) for s in states] == [0, 0]


def test_two_graphs_at_once():
    """Every operator captured into a graph of its own tensors, plans and workspaces, twice; the two replayed
    back to back on two streams, round after round without a wait, give what each gives alone."""
    g = torch.Generator().manual_seed(22)
    lens, slens = [300, 1, 700, 130], [700, 1400, 600, 513]
    cu = [0, 300, 301, 1001, 1131]

    def state():
        r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
        s = dict(q=r(1131, 4, 192), k=r(1131, 4, 192), v=r(1131, 4, 128), row=r(1131, 576), cu=i32(cu))
        s["table"] = torch.arange(48, dtype=torch.int32).reshape(4, 12).cuda()
        s["lens"], s["cache"] = i32(lens), r(60, 64, 576)
        shared = torch.arange(96, dtype=torch.int32).reshape(4, 24) % 60
        shared[:, :8] = torch.arange(8, dtype=torch.int32)
        s["shared"], s["slens"], s["kv"] = shared.cuda(), i32(slens), r(60, 64, 576)
        s["dq"], s["dq128"] = r(4, 1, 16, 576), r(4, 1, 128, 576)
        s["ref0"], s["zero"] = (torch.rand(60, generator=g) < 0.6).int().cuda(), i32([0, 0, 0, 0])
        s["none"], s["pool0"], s["status"] = torch.full_like(s["table"], -1), r(2, 60, 64, 16), i32([0])
        for name, v in (("grow", [0, 2]), ("new", [100, 300]), ("parent", [2]), ("child", [1]), ("gone", [0])):
            s[name] = i32(v)
        return s

    def work(s):
        st = s["status"]
        out = [*mla.prompt_attention(s["q"], s["k"], s["v"], s["cu"], status=st)]
        cache = s["cache"].clone()
        mla.cache_append(s["row"][:, :512], s["row"][:, 512:], cache, s["table"], s["lens"], cu_seqlens=s["cu"],
                         status=st)
        out += [*mla.shared_prefix_decode(s["dq"], s["kv"], s["shared"], s["slens"], status=st),
                *mla.shared_prefix_decode(s["dq128"], s["kv"], s["shared"], s["slens"], status=st)]
        ref, table, n, pool = (s[k].clone() for k in ("ref0", "none", "zero", "pool0"))
        mla.cache_grow(ref, table, n, s["grow"], s["new"], status=st)
        mla.cache_copy_pages(pool, mla.cache_fork(ref, table, n, s["parent"], s["child"], status=st), layered=True,
                             status=st)
        mla.cache_free(ref, table, n, s["gone"], status=st)
        pairs, count = mla.cache_compact(ref, table, n, status=st)
        mla.cache_copy_pages(pool, pairs, count=count, layered=True, status=st)
        return out + [cache, ref, table, n, pool, pairs, count]

    states = [state(), state()]
    want = [[t.clone() for t in work(s)] for s in states]
    torch.cuda.synchronize()
    graphs, got = [], []
    for s in states:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(work(s))
        graphs.append(graph)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    marks = [[torch.cuda.Event(enable_timing=True) for _ in range(2)] for _ in states]
    for _ in range(3):
        for stream, (begin, _) in zip(streams, marks):
            begin.record(stream)
        for _ in range(40):
            for graph, stream in zip(graphs, streams):
                with torch.cuda.stream(stream):
                    graph.replay()
        for stream, (_, end) in zip(streams, marks):
            end.record(stream)
        torch.cuda.synchronize()
        # both were at work for most of the time of either
        alone = max(b.elapsed_time(e) for b, e in marks)
        assert min(marks[0][0].elapsed_time(marks[1][1]), marks[1][0].elapsed_time(marks[0][1])) > 0.5 * alone
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert [int(s["status"]) for s in states] == [0, 0]


@pytest.mark.parametrize("s_q", [1, 3])
def test_decode_continues_the_prompts_attention(s_q):
    """The last queries of prompts, once by prompt attention over expanded heads and once by the decode over the
    appended latent rows: with the same scale the same attention.  The expansions select latent dims (head h: dims
    (37 h + i) % 512 for keys, (53 h + 11 + i) % 512 for values), so both see the same numbers.

    Each side is off by the rounding of its weights and its output, u = 2^-8 of M = sum w |v| and of the value, and
    by its scores, a sum of 576 products at most in fp32: d = 576 2^-23 max scale |q|.|k|, twice that on weights."""
    H, lens, scale = 16, [130, 77, 300, 64], 192 ** -0.5
    g = torch.Generator().manual_seed(5)
    total = sum(lens)
    cu = [0] + [int(x) for x in np.cumsum(lens)]
    lat, rope = (torch.randn(total, n, generator=g).to(torch.bfloat16) for n in (512, 64))
    q = torch.randn(total, H, 192, generator=g).to(torch.bfloat16)
    kdim = torch.stack([(37 * h + torch.arange(128)) % 512 for h in range(H)])
    vdim = torch.stack([(53 * h + 11 + torch.arange(128)) % 512 for h in range(H)])
    k = torch.cat([lat[:, kdim], rope[:, None].expand(-1, H, -1)], 2)
    v = lat[:, vdim]
    out, lse = mla.prompt_attention(q.cuda(), k.cuda(), v.cuda(), i32(cu), softmax_scale=scale)
    # into pages, and the last s_q queries of each with their heads absorbed
    cache = torch.zeros(12, 64, 576, dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[0, 1, 2, -1, -1], [3, 4, -1, -1, -1], [5, 6, 7, 8, 9], [10, -1, -1, -1, -1]],
                         dtype=torch.int32, device="cuda")
    mla.cache_append(lat.cuda(), rope.cuda(), cache, table, i32(lens), cu_seqlens=i32(cu))
    last = torch.tensor([[e - s_q + i for i in range(s_q)] for e in cu[1:]])
    absorbed = torch.zeros(len(lens), s_q, H, 576, dtype=torch.bfloat16)
    absorbed[..., :512].scatter_(3, kdim.expand(len(lens), s_q, H, 128), q[last][..., :128])
    absorbed[..., 512:] = q[last][..., 128:]
    _, _, mix, reach = so.prompt_attention(q.double().numpy(), k.double().numpy(), v.double().numpy(), cu, cu, True,
                                           scale)
    want, wlse = out.double().cpu()[last].numpy(), lse.double().cpu()[last].numpy()
    d = 576 * 2.0 ** -23 * reach[last]
    tol = 2 * ((2.0 ** -8 + 2 * d + 2.0 ** -20)[..., None] * mix[last] + 2.0 ** -8 * (np.abs(want) + 2.0 ** -8))
    pick = vdim.expand(len(lens), s_q, H, 128)
    for name, fn in (("decode", mla.decode), ("shared", mla.shared_prefix_decode)):
        o, l = fn(absorbed.cuda(), cache, table, i32(lens), causal=True, softmax_scale=scale)
        assert np.all(np.abs(o.double().cpu().gather(3, pick).numpy() - want) <= tol), name
        assert np.all(np.abs(l.double().cpu().numpy() - wlse) <= 2 * (d + 2.0 ** -20 + 2.0 ** -23 * np.abs(wlse)))
    # with the decode's default, 1 / sqrt(576), it is another attention
    o, _ = mla.decode(absorbed.cuda(), cache, table, i32(lens), causal=True)
    assert not np.all(np.abs(o.double().cpu().gather(3, pick).numpy() - want) <= tol)
