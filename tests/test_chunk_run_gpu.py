"""Rotary tables, rotated heads, gathered rows and chunk attention as a server
runs them: together, in graphs, on several streams, and where offsets pass 32
bits.  Tolerances are those of the operators' own tests; where the same kernel
reads the same numbers from another place, results are equal to the bit."""

import numpy as np
import pytest
import torch

import mla_paged_kv_gb300 as mla
from oracle import serving_oracle as so
from tests.test_chunk_gpu import Case

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16
H, PAGES, WIDTH = 16, 64, 10


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


caches = pytest.mark.parametrize("fp8", [False, True])


def as_case(q, cache, table, lens, cu):
    """The attention over what the device holds, for Case.check."""
    c = object.__new__(Case)
    c.q, c.table, c.lens, c.cu = q.cpu(), table.cpu().numpy(), list(lens), list(cu)
    rows = c.cache = cache.cpu()
    if cache.dtype != torch.uint8:
        c.values = rows.double().numpy()
    else:
        code = rows[..., :512].contiguous().view(torch.float8_e4m3fn).reshape(-1, 64, 4, 128)
        scale = rows[..., 512:528].contiguous().view(torch.float32)[..., None]
        key = (code.double() * scale.double()).reshape(-1, 64, 512)
        c.scale = scale[..., 0]
        c.values = torch.cat([key, rows[..., 528:].contiguous().view(BF16).double()], 2).numpy()
    return c


@caches
def test_a_servers_steps(fp8):
    """Prompts in chunks beside single tokens, drafts and idle rows: the queries' rotary part is turned in place, the new
    rows are appended with the same table, one plan serves two layers."""
    g = torch.Generator().manual_seed(51)
    r = lambda *s: torch.randn(*s, generator=g).to(BF16).cuda()  # noqa: E731
    cos_sin = mla.rope_table(WIDTH * 64, base=10000.0, scaling="yarn", factor=4.0, original=256)
    weight = (1 + 0.1 * r(512).float()).to(BF16)
    shape, dt = ((2, PAGES, 64, 656), torch.uint8) if fp8 else ((2, PAGES, 64, 576), BF16)
    pool, status = torch.zeros(shape, dtype=dt, device="cuda"), i32([0])
    table = torch.randperm(PAGES, generator=g)[:6 * WIDTH].reshape(6, WIDTH).int().cuda()
    lens = [0] * 6
    for new in ([130, 1, 64, 0, 300, 7], [63, 1, 200, 0, 1, 1], [1, 4, 1, 2, 4, 0], [0, 1, 0, 0, 0, 0]):
        lens = [a + b for a, b in zip(lens, new)]
        cu = [int(x) for x in np.cumsum([0] + new)]
        d_lens, d_cu, total = i32(lens), i32(cu), cu[-1]
        pl = mla.plan_chunks(d_cu, d_lens, total, H, status=status)
        for layer in range(2):
            q, row = r(total, H, 576), r(total, 576)
            before = q.clone()
            rotary = q[..., 512:]
            mla.rope_heads(rotary, cos_sin, d_lens, d_cu, out=rotary, interleaved=True, status=status)
            mla.cache_append(row[:, :512], row[:, 512:], pool[layer], table, d_lens, cu_seqlens=d_cu,
                             norm_weight=weight, cos_sin=cos_sin, rope_interleaved=True, status=status)
            out, lse = mla.chunk_attention(q, pool[layer], table, d_lens, d_cu, pl=pl, status=status)
            assert torch.equal(q[..., :512], before[..., :512])
            host, angles = q.double().cpu().numpy(), cos_sin.cpu().numpy()
            for b in range(6):
                for t in (cu[b], cu[b + 1] - 1):
                    if new[b] == 0:
                        continue
                    want = so.rope_head(before[t, 3, 512:].double().cpu().numpy(),
                                        angles[lens[b] - (cu[b + 1] - t)], 0, True)
                    mag = np.abs(before[t, 3, 512:].double().cpu().numpy()).reshape(-1, 2).sum(1).repeat(2) * 1.2
                    assert np.all(np.abs(host[t, 3, 512:] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -22 * mag)
            as_case(q, pool[layer], table, lens, cu).check(out, lse, True)
    assert int(status) == 0


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_a_chunk_over_its_context_both_ways(kind):
    """Once over latent rows with the heads absorbed, once by prompt attention over the context's rows, gathered and
    expanded.  The expansions select latent dims (head h: dims (37 h + i) % 512 for keys, (53 h + 11 + i) % 512 for
    values), so that both see the same numbers (over FP8 records a 16-bit cache of the gathered rows does).

    Each side is off by the rounding of its weights and its output, u = 2^-8 of M = sum w |v| and of the value, and by
    its scores, a sum of 576 products at most in fp32: d = 576 2^-23 max scale |q|.|k|, twice that on weights."""
    lens, new, scale = [400, 77, 129, 64], [130, 1, 129, 3], 192 ** -0.5
    g = torch.Generator().manual_seed(52)
    cu, cu_k = [0] + [int(x) for x in np.cumsum(new)], [0] + [int(x) for x in np.cumsum(lens)]
    table = torch.cat([torch.randperm(24, generator=g)[:7] for _ in range(4)]).reshape(4, 7).int().cuda()
    c = Case([1], [24 * 64 - 1], spare=0, seed=53, fp8=kind == "fp8")
    cache = c.cache.cuda()
    rows = mla.cache_gather(cache, table, i32(cu_k), cu_k[-1])
    if kind == "fp8":  # the rows at the places where the records are
        pages = torch.arange(24, dtype=torch.int32, device="cuda")[None]
        cache = mla.cache_gather(cache, pages, i32([0, 24 * 64]), 24 * 64).view(24, 64, 576)
    q = torch.randn(cu[-1], H, 192, generator=g).to(BF16)
    kdim = torch.stack([(37 * h + torch.arange(128)) % 512 for h in range(H)])
    vdim = torch.stack([(53 * h + 11 + torch.arange(128)) % 512 for h in range(H)])
    k = torch.cat([rows[:, :512][:, kdim.cuda()], rows[:, None, 512:].expand(-1, H, -1)], 2)
    v = rows[:, :512][:, vdim.cuda()]
    want, wlse = mla.prompt_attention(q.cuda(), k, v, i32(cu), i32(cu_k), softmax_scale=scale)
    absorbed = torch.zeros(cu[-1], H, 576, dtype=BF16)
    absorbed[..., :512].scatter_(2, kdim.expand(cu[-1], H, 128), q[..., :128])
    absorbed[..., 512:] = q[..., 128:]
    out, lse = mla.chunk_attention(absorbed.cuda(), cache, table, i32(lens), i32(cu), True, scale)
    _, _, mix, reach = so.prompt_attention(q.double().numpy(), k.double().cpu().numpy(), v.double().cpu().numpy(), cu,
                                           cu_k, True, scale)
    want, wlse = want.double().cpu().numpy(), wlse.double().cpu().numpy()
    d = 576 * 2.0 ** -23 * reach
    tol = 2 * ((2.0 ** -8 + 2 * d + 2.0 ** -20)[..., None] * mix + 2.0 ** -8 * (np.abs(want) + 2.0 ** -8))
    got = out.double().cpu().gather(2, vdim.expand(cu[-1], H, 128)).numpy()
    assert np.all(np.abs(got - want) <= tol)
    assert np.all(np.abs(lse.double().cpu().numpy() - wlse) <= 2 * (d + 2.0 ** -20 + 2.0 ** -23 * np.abs(wlse)))


class Step:
    """A batch's inputs, and everything that is done with them."""

    def __init__(self, fp8, seed):
        self.c = Case([70, 1, 3, 140], [200, 900, 64, 0], heads=H, seed=seed, fp8=fp8, rest=0.0)
        self.q, self.cache, self.table, self.lens, self.cu = self.c.device()
        self.status, self.weight = i32([0]), torch.ones(64, dtype=BF16, device="cuda")
        self.rows = i32([0, 100, 130, 200, 214])

    def work(self):
        st = self.status
        cos_sin = mla.rope_table(1024, scaling="linear", factor=2.0)
        turned = mla.rope_heads(self.q[..., 512:], cos_sin, self.lens, self.cu, norm_weight=self.weight, status=st)
        rows = mla.cache_gather(self.cache, self.table, self.rows, 214, status=st)
        pl = mla.plan_chunks(self.cu, self.lens, 214, H, status=st)
        return [cos_sin, turned, rows, *mla.chunk_attention(self.q, self.cache, self.table, self.lens, self.cu, pl=pl,
                                                            status=st)]


@caches
def test_a_captured_step_with_other_inputs(fp8):
    """The graph reads the inputs, offsets and lengths of each replay: the plan is made in it."""
    s = Step(fp8, 61)
    s.work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = s.work()
    for lens, cu in (([270, 901, 67, 140], [0, 70, 71, 74, 214]), ([230, 905, 0, 139], [0, 60, 64, 64, 203]),
                     ([100, 300, 67, 2], [0, 99, 212, 213, 214])):
        s.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        s.cu.copy_(torch.tensor(cu, dtype=torch.int32))
        s.q.copy_(torch.randn(s.q.shape, generator=torch.Generator().manual_seed(lens[0])))
        graph.replay()
        have = [t.clone() for t in got]
        want = s.work()
        n = cu[-1]
        for a, b in zip(have, want):
            n_rows = n if a.shape[0] == 214 and a.dim() != 2 or a.shape[-1] == H else a.shape[0]
            assert torch.equal(a[:n_rows], b[:n_rows])
        c = as_case(s.q[:n], s.cache, s.table, lens, cu)
        c.check(have[3][:n], have[4][:n], True)
    assert int(s.status) == 0


@caches
@pytest.mark.parametrize("graphs", [True, False])
def test_two_at_once(fp8, graphs):
    """Two batches with plans and workspaces of their own on two streams, round after round without a wait."""
    steps = [Step(fp8, 71), Step(fp8, 72)]
    want = [[t.clone() for t in s.work()] for s in steps]
    torch.cuda.synchronize()
    streams, ran, got = [torch.cuda.Stream() for _ in steps], [], [None, None]
    if graphs:
        for i, s in enumerate(steps):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                got[i] = s.work()
            ran.append(graph)
        torch.cuda.synchronize()
    for _ in range(20):
        for i, (s, stream) in enumerate(zip(steps, streams)):
            with torch.cuda.stream(stream):
                if graphs:
                    ran[i].replay()
                else:
                    got[i] = s.work()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert [int(s.status) for s in steps] == [0, 0]


@caches
def test_a_stream_that_is_not_the_current_one(fp8):
    s = Step(fp8, 81)
    want = s.work()
    freq, magnitude = mla.rope_frequencies(64, 10000.0, "linear", 2.0)
    side, n = torch.cuda.Stream(), 214
    cos_sin = torch.zeros(1024, 64, device="cuda")
    turned = torch.zeros(n, H, 64, dtype=BF16, device="cuda")
    rows = torch.zeros(n, 576, dtype=BF16, device="cuda")
    parts = mla.mla_chunk_num_parts()
    plan = torch.zeros(mla.mla_chunk_plan_bytes(4, n, H, parts), dtype=torch.uint8, device="cuda")
    pl = mla.ChunkPlan(plan, 4, n, H, parts, True,
                       torch.zeros(mla.mla_chunk_workspace_bytes(parts), dtype=torch.uint8, device="cuda"))
    if fp8:
        pl.workspace = mla.chunk_workspace(pl, 8)
    out, lse = torch.zeros(n, H, 512, dtype=BF16, device="cuda"), torch.zeros(n, H, device="cuda")
    torch.cuda.synchronize()
    # what the operators' inputs wait for is on that stream
    q, cache = s.q.clone(), s.cache.clone()
    s.q.zero_()
    s.cache.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        s.q.copy_(q)
        s.cache.copy_(cache)
    mla.mla_rope_table(freq, magnitude, 0, cos_sin, stream=side)
    mla.mla_rope_heads(s.q[..., 512:], turned, cos_sin, s.status, s.lens, s.cu, x_weight=s.weight, stream=side)
    mla.mla_cache_gather(s.cache, s.table, s.rows, rows, s.status, stream=side)
    mla.mla_chunk_get_plan(s.cu, s.lens, n, H, True, parts, plan, s.status, stream=side)
    mla.mla_chunk_attention_fwd(s.q, s.cache, s.table, pl, out, lse, s.status, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, [cos_sin, turned, rows, out, lse]))
    assert int(s.status) == 0


@caches
def test_pages_behind_32_bits(fp8):
    """Pages whose first element (and, of FP8 records, byte) lies past 2^32."""
    c = Case([3, 40], [130, 900], heads=H, seed=91, fp8=fp8)
    q, cache, table, lens, cu = c.device()
    want = mla.chunk_attention(q, cache, table, lens, cu)
    rows = mla.cache_gather(cache, table, i32([0, 133, 1073]), 1073)
    total = 2 ** 32 // (64 * cache.shape[2]) + 100
    big = torch.empty(total, 64, cache.shape[2], dtype=cache.dtype, device="cuda")
    far = total - cache.shape[0]
    big[far:] = cache
    moved = torch.where(table >= 0, table + far, table)
    got = mla.chunk_attention(q, big, moved, lens, cu)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(mla.cache_gather(big, moved, i32([0, 133, 1073]), 1073), rows)


@caches
def test_rows_behind_32_bits(fp8):
    """Queries and outputs whose first element lies past 2^32, over FP8 records their codes in the workspace too."""
    c = Case([3, 2], [130, 100], heads=128, seed=92, fp8=fp8)
    q, cache, table, lens, cu = c.device()
    want = mla.chunk_attention(q, cache, table, lens, cu)
    before = 2 ** 32 // (128 * 512) + 10
    far = torch.empty(before + 5, 128, 576, dtype=BF16, device="cuda")
    far[before:] = q
    got = mla.chunk_attention(far, cache, table, lens, cu + before)
    assert torch.equal(got[0][before:], want[0]) and torch.equal(got[1][before:], want[1])


def test_strides_behind_32_bits():
    x = torch.randn(5, 2, 64, generator=torch.Generator().manual_seed(93)).to(BF16).cuda()
    cos_sin, lens = mla.rope_table(64), i32([5])
    cache = torch.randn(2, 64, 576, generator=torch.Generator().manual_seed(94)).to(BF16).cuda()
    table = i32([[1]])
    buf = torch.empty(5, 2 ** 30 + 64, dtype=BF16, device="cuda")
    far = buf[:, :128].unflatten(1, (2, 64))
    far.copy_(x)
    want = mla.rope_heads(x, cos_sin, lens)
    assert torch.equal(mla.rope_heads(far, cos_sin, lens), want)
    mla.rope_heads(far, cos_sin, lens, out=far)
    assert torch.equal(far, want)
    mla.cache_gather(cache, table, i32([0, 5]), out=buf[:, :576])
    assert torch.equal(buf[:, :576], cache[1, :5])


@caches
def test_pages_that_several_rows_and_places_share(fp8):
    c = Case([5, 4, 3], [320, 300, 100], heads=H, seed=95, fp8=fp8, rest=0.5)  # (row 0 has the most pages)
    c.table[1] = c.table[0][:c.table.shape[1]]
    c.table[2, :2] = c.table[0, 1]
    q, cache, table, lens, cu = c.device()
    out, lse = mla.chunk_attention(q, cache, table, lens, cu)
    c.check(out, lse, True)


def test_one_plan_for_caches_of_every_kind():
    cases = [Case([70, 1, 3, 140], [200, 900, 64, 0], heads=H, seed=97, dtype=FP16 if k == 1 else BF16, fp8=k == 2)
             for k in range(3)]
    on = [c.device() for c in cases]
    pl = mla.plan_chunks(on[0][4], on[0][3], 214, H)
    for _ in range(2):
        for c, (q, cache, table, lens, cu) in zip(cases, on):
            out, lse = mla.chunk_attention(q, cache, table, lens, cu, pl=pl)
            c.check(out, lse, True)
            alone = mla.chunk_attention(q, cache, table, lens, cu)
            assert torch.equal(out, alone[0]) and torch.equal(lse, alone[1])


@caches
def test_calls_back_to_back(fp8):
    """Each call's first kernel begins while the call before ends: what a call reads is what the one before wrote."""
    c = Case([9, 1, 60], [300, 700, 64], heads=H, seed=98, fp8=fp8)
    q, cache, table, lens, cu = c.device()
    pl, status = mla.plan_chunks(cu, lens, 70, H), i32([0])
    pl.workspace = mla.chunk_workspace(pl, 4)
    outs = [(torch.zeros(70, H, 512, dtype=BF16, device="cuda"), torch.zeros(70, H, device="cuda")) for _ in range(2)]

    def chain(wait):
        x = q.clone()
        for i in range(12):
            out, lse = outs[i % 2]
            mla.mla_chunk_attention_fwd(x, cache, table, pl, out, lse, status)
            if wait:
                torch.cuda.synchronize()
            x[..., :512] = out
            mla.mla_chunk_attention_fwd(x, cache, table, pl, out, lse, status)
            if wait:
                torch.cuda.synchronize()
        return [t.clone() for pair in outs for t in pair]

    want = chain(True)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(chain(False), want))
    assert int(status) == 0


@caches
def test_nothing_to_do(fp8):
    c = Case([2], [100], heads=H, seed=96, fp8=fp8)
    q, cache, table, _, _ = c.device()
    for lens, cu, n in (([0], [0, 0], 0), ([102], [0, 0], 0), ([102], [2, 2], 2), ([0], [0, 2], 2), ([-5], [0, 2], 2)):
        pl = mla.plan_chunks(i32(cu), i32(lens), n, H)
        if fp8:
            pl.workspace = mla.chunk_workspace(pl)
        out, lse = torch.full((n, H, 512), 7.0, dtype=BF16, device="cuda"), torch.full((n, H), 7.0, device="cuda")
        status = i32([0])
        mla.mla_chunk_attention_fwd(q[:n], cache, table, pl, out, lse, status)
        torch.cuda.synchronize()
        written = cu[1] > cu[0]
        assert int(status) == 0 and bool((out == (0.0 if written else 7.0)).all())
        assert bool((lse == (-float("inf") if written else 7.0)).all())
