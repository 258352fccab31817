"""Decode over a shared prefix against the 64-bit oracle of the plain decode
(the same keys in the same order, so the same result), under the decode's own
bars (tests/parity.py)."""

import numpy as np
import pytest
import torch

import mla_paged_kv_gb300 as mla
from oracle import mla_oracle as orc
from tests.parity import compare

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Case:
    def __init__(self, head, tails, s_q, h_q, causal=False, dtype=torch.bfloat16, seed=0, amp=1.0, poison=True,
                 fp8=False):
        """head: shared pages; tails: each request's keys behind them."""
        g = torch.Generator().manual_seed(seed)
        B = len(tails)
        width = head + max(-(-t // 64) for t in tails) + 1
        pages = head + sum(-(-t // 64) for t in tails) + 2
        perm = torch.randperm(pages, generator=g).tolist()
        front = [perm.pop() for _ in range(head)]
        self.table = np.full((B, width), -1, dtype=np.int32)
        for b, t in enumerate(tails):
            self.table[b, :head] = front
            for j in range(-(-t // 64)):
                self.table[b, head + j] = perm.pop()
        self.lens = [head * 64 + t for t in tails]
        self.kv = torch.randn(pages, 64, 576, generator=g).to(dtype)
        for b, n in enumerate(self.lens):  # finite poison behind the last key
            if poison and n % 64:
                self.kv[self.table[b, n // 64], n % 64:] = 1000.0
        if fp8:  # the same rows as records: 128-element groups, scale = max / 448
            x = self.kv.float().reshape(pages * 64, 576)
            rec = torch.empty(pages * 64, 656, dtype=torch.uint8)
            top = x[:, :512].reshape(-1, 4, 128).abs().amax(2)
            scale = torch.where(top > 0, top / 448, torch.ones_like(top))
            rec[:, :512] = (x[:, :512].reshape(-1, 4, 128) / scale[..., None]).clamp(-448, 448).to(
                torch.float8_e4m3fn).view(torch.uint8).reshape(-1, 512)
            rec[:, 512:528] = scale.contiguous().view(torch.uint8)
            rec[:, 528:] = x[:, 512:].to(torch.bfloat16).contiguous().view(torch.uint8)
            self.kv = rec.reshape(pages, 64, 656)
        self.q = (amp * torch.randn(B, s_q, h_q, 576, generator=g)).to(dtype)
        self.causal, self.s_q, self.h_q = causal, s_q, h_q

    def want(self):
        if self.kv.dtype == torch.uint8:
            return orc.dense_fp8_decode(self.q.double().numpy(), self.kv.numpy(), self.table,
                                        np.array(self.lens, dtype=np.int32), self.causal, 1 / 24)[:2]
        return orc.dense_decode(self.q.double().numpy(), self.kv.float().numpy(), self.table,
                                np.array(self.lens, dtype=np.int32), self.causal, 1 / 24)

    def run(self, num_parts=None, out_fp32=False):
        table, lens = torch.from_numpy(self.table).cuda(), i32(self.lens)
        pl = mla.plan_shared_prefix(table, lens, self.s_q, self.h_q, self.causal, num_parts)
        pl.workspace.fill_(0xFF)  # NaN partials: nothing of an earlier call is read
        return mla.shared_prefix_decode(self.q.cuda(), self.kv.cuda(), table, lens, self.causal, out_fp32=out_fp32,
                                        pl=pl)

    def check(self, **kw):
        out, lse = self.run(**kw)
        compare(out, lse, *self.want())
        return out, lse


@pytest.mark.parametrize("head", [1, 2, 17])
@pytest.mark.parametrize("tails", [[1, 64], [65, 3, 130, 64, 1], [0, 5, 0]])
@pytest.mark.parametrize("h_q", [16, 64, 128])
def test_prefix_and_tails(head, tails, h_q):
    Case(head, tails, 1, h_q, seed=head).check()


@pytest.mark.parametrize("s_q,h_q,causal", [(2, 16, True), (2, 128, True), (3, 40, True), (2, 40, False),
                                            (1, 1, False), (5, 7, True), (1, 129, False), (2, 100, True)])
def test_rows_per_request(s_q, h_q, causal):
    Case(5, [s_q, 64, 100, 70, 3 + s_q, 200, 65], s_q, h_q, causal, seed=s_q).check()


@pytest.mark.parametrize("h_q", [111, 112, 113, 120])
@pytest.mark.parametrize("fp8", [False, True])
def test_around_the_rule_for_packing_rows(h_q, fp8):
    """Eight requests: up to 112 heads their rows are packed, above each is attended alone."""
    Case(6, [64, 100, 70, 3, 200, 65, 1, 0], 1, h_q, seed=h_q, fp8=fp8).check()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("out_fp32", [False, True])
def test_types(dtype, out_fp32):
    out, _ = Case(9, [30, 90, 128], 1, 32, dtype=dtype, seed=4).check(out_fp32=out_fp32)
    assert out.dtype == (torch.float32 if out_fp32 else dtype)


@pytest.mark.parametrize("head,tails,s_q,h_q,causal", [
    (1, [1, 64], 1, 16, False), (9, [65, 3, 130, 64, 1], 1, 16, False), (17, [0, 5, 0], 1, 64, False),
    (5, [2, 64, 100, 70, 5, 200, 65], 2, 16, True), (5, [3, 64, 100, 70], 3, 40, True), (5, [5, 7], 1, 128, False),
    (40, [10, 700, 64, 1], 1, 16, False), (30, [64] * 50, 1, 8, False)])
@pytest.mark.parametrize("out_fp32", [False, True])
def test_fp8_records(head, tails, s_q, h_q, causal, out_fp32):
    Case(head, tails, s_q, h_q, causal, seed=head, fp8=True).check(out_fp32=out_fp32)


def test_fp8_records_peaky_and_cut():
    Case(20, [30, 300, 64], 1, 16, seed=6, amp=8.0, fp8=True).check()
    c = Case(6, [64, 100, 5], 2, 16, True, seed=9, fp8=True)
    for n in (3 * 64, 3 * 64 + 1, 65, 2, 1, 0):
        c.lens[1] = n
        c.check()


@pytest.mark.parametrize("num_parts", [1, 2, 7, 300])
def test_split_counts(num_parts):
    Case(40, [10, 700, 64, 1], 1, 16, seed=5).check(num_parts=num_parts)


def test_peaky_scores():
    Case(20, [30, 300, 64], 1, 16, seed=6, amp=8.0).check()


def test_no_common_page():
    c = Case(3, [64, 100, 5], 1, 16, seed=7)
    c.table[1, 0], c.table[1, 1] = c.table[1, 1], c.table[1, 0]
    c.check()


def test_requests_part_inside_the_prefix():
    """Tables that agree in their first 5, 3 and 7 pages: 3 are shared."""
    c = Case(7, [64, 100, 5, 300], 1, 16, seed=8)
    c.table[2, 3:7] = c.table[2, 3:7][::-1].copy()
    c.table[3, 5] = c.table[3, 6]
    c.check()


@pytest.mark.parametrize("causal", [False, True])
def test_a_request_that_ends_inside_the_prefix(causal):
    """Only whole pages that every query of every request sees are shared."""
    c = Case(6, [64, 100, 5], 2, 16, causal, seed=9)
    for n in (3 * 64, 3 * 64 + 1, 3 * 64 - 1, 65, 64, 2, 1):
        c.lens[1] = n
        c.check()


def test_an_empty_request():
    c = Case(6, [64, 100, 5], 1, 16, seed=10)
    c.lens[1] = 0
    out, lse = c.check()
    assert not out[1].any() and torch.isneginf(lse[1]).all()


@pytest.mark.parametrize("empty", [[0], [3], [0, 1, 4], [1, 2, 3, 4], [0, 1, 2, 3, 4]])
@pytest.mark.parametrize("s_q,causal,fp8,few", [(1, False, False, 0), (2, True, False, 3), (2, True, True, 65),
                                                (1, False, True, 63)])
def test_short_slots_stand_apart(empty, s_q, causal, fp8, few):
    """Requests that see less than a page leave the others' prefix alone: their rows of the table and of q
    hold nothing, and no page of the others' prefix is read for them."""
    c = Case(4, [64, 100, 5, 1, 200], s_q, 16, causal, seed=10, fp8=fp8)
    spare = c.kv.shape[0] - 1
    for b in empty:
        c.lens[b] = min(few, 63 if not causal else 64)
        c.table[b] = -1
        c.table[b, 0] = spare
        if c.lens[b] == 0:
            c.q[b] = float("nan")
    out, lse = c.run()
    q = c.q
    c.q = torch.where(torch.isnan(q), torch.zeros_like(q), q)
    ref_out, ref_lse = c.want()
    others = [b for b in range(5) if b not in empty]
    if others:
        compare(out, lse, ref_out, ref_lse, rows=others)
    # The short slots' page may hold rows of 1000 (the poison), beyond what absolute bars are made for.  With
    # M = sum p |v| >= |out|: weights and outputs rounded to bf16 are off by 2^-8 of M each, a sum over the
    # rounded weights by as much again.  A score sums 576 products in fp32, 36 matrix steps and a handful of
    # roundings, each off by 2^-24 of A = scale sum |q k| at most: d = 48 2^-24 max A, so the LSE is off by d
    # and 2^-20 for its own sum, and weights by a factor of e^(2 d) at most.
    for b in empty:
        n = c.lens[b]
        o, l = out[b].double().cpu().numpy(), lse[b].double().cpu().numpy()
        if n == 0:
            assert not o.any() and np.isneginf(l).all()
            continue
        kv = c.kv[spare, :n]
        keys = np.stack([orc.decode_record(r) for r in kv.numpy()]) if fp8 else kv.double().numpy()
        qs = c.q[b].double().numpy()
        scores = np.einsum("shd,kd->shk", qs, keys) / 24
        if causal:
            for s in range(s_q):
                scores[s, :, n - s_q + 1 + s:] = -np.inf
        w = np.exp(scores - scores.max(2, keepdims=True))
        w /= w.sum(2, keepdims=True)
        mag = np.einsum("shk,kd->shd", w, np.abs(keys[:, :512]))
        d = 48 * 2.0**-24 * (np.einsum("shd,kd->shk", np.abs(qs), np.abs(keys)).max() / 24)
        assert np.abs(l - ref_lse[b]).max() <= d + 2.0**-20
        assert (np.abs(o - ref_out[b]) <= (3 * 2.0**-8 + np.expm1(2 * d)) * mag).all()


@pytest.mark.parametrize("empty", [[], [0], [2], [0, 3]])
def test_plan_shares_without_empty_slots(empty):
    """The plan's own units start behind the prefix, except those of the slots that stand apart."""
    c = Case(4, [64, 100, 5, 1], 1, 16, seed=11)
    for b in empty:
        c.lens[b] = 0
        c.table[b] = -1
    pl = mla.plan_shared_prefix(torch.from_numpy(c.table).cuda(), i32(c.lens), 1, 16)
    units = pl.plan[:5 * 32].view(torch.int32).reshape(5, 8).cpu().tolist()
    lens = pl.plan[256:256 + 20].view(torch.int32).cpu().tolist()
    width = c.table.shape[1]
    first = next(b for b in range(4) if b not in empty)
    assert units[0] == [0, 64, -1, first * width, width, 0, 0, 0] and lens[0] == 256
    for b in range(4):
        skip = 0 if b in empty else 4
        assert units[1 + b][:6] == [16 * b, 16, -1, b * width + skip, width - skip, int(b in empty)]
        assert lens[1 + b] == (0 if b in empty else c.lens[b] - 256)


def test_one_request_and_many():
    Case(12, [77], 1, 16, seed=11).check()
    Case(2, [(i * 13) % 90 for i in range(150)], 1, 8, seed=12).check()
    Case(2, [(i * 13) % 90 + 1 for i in range(40)], 1, 128, seed=12).check()


def test_same_as_the_decode_of_each_request():
    c = Case(30, [64, 100, 5, 300], 1, 16, seed=13, poison=False)
    out, lse = c.run(out_fp32=True)
    table, lens = torch.from_numpy(c.table).cuda(), i32(c.lens)
    o2, l2 = mla.decode(c.q.cuda(), c.kv.cuda(), table, lens, out_fp32=True)
    # both round the weights to bf16 against references up to 2^8 apart: 2 * 2^-8 of weights of sum 1
    assert torch.all((out - o2).abs() <= 2.0 ** -6 * c.kv[..., :512].float().abs().max())
    assert torch.all((lse - l2).abs() <= 1e-4)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("where", ["prefix", "tail"])
def test_bad_page_is_masked_and_reported(where, fp8):
    c = Case(4, [64, 100, 130], 1, 16, seed=14, fp8=fp8)
    if where == "prefix":
        c.table[:, 2] = 10 ** 6
    else:
        c.table[2, 5] = -1
    table, lens = torch.from_numpy(c.table).cuda(), i32(c.lens)
    with pytest.raises(mla.MlaError) as e:
        mla.shared_prefix_decode(c.q.cuda(), c.kv.cuda(), table, lens)
    assert e.value.code == 5
    st = i32([0])
    out, lse = mla.shared_prefix_decode(c.q.cuda(), c.kv.cuda(), table, lens, status=st)
    compare(out, lse, *c.want())
    assert int(st) == 5


def test_refusals():
    c = Case(4, [64, 100], 1, 16, seed=15)
    q, kv, table, lens = c.q.cuda(), c.kv.cuda(), torch.from_numpy(c.table).cuda(), i32(c.lens)
    pl = mla.plan_shared_prefix(table, lens, 1, 16)
    for bad in (dict(q=q.half()), dict(kv=kv.float()), dict(table=table[:1]), dict(q=q[:, :, :8]),
                dict(causal=True), dict(lens=None, q=q[..., :512])):
        a = {**dict(q=q, kv=kv, table=table, causal=False), **{k: v for k, v in bad.items() if k != "lens"}}
        with pytest.raises((TypeError, ValueError)):
            mla.shared_prefix_decode(a["q"], a["kv"], a["table"], lens, a["causal"], pl=pl)
    with pytest.raises(ValueError):
        mla.plan_shared_prefix(table, lens, 1, 16, num_parts=1025)
    with pytest.raises(ValueError):
        mla.plan_shared_prefix(table, lens[:1], 1, 16)
    pl.workspace = pl.workspace[:1024]
    with pytest.raises(mla.MlaError):
        mla.shared_prefix_decode(q, kv, table, lens, pl=pl)


@pytest.mark.parametrize("h_q,fp8", [(16, False), (128, False), (16, True), (128, True)])
def test_graph_replays_with_new_lengths(h_q, fp8):
    """Plan and decode captured together: the table and lengths may change between replays."""
    c = Case(10, [64, 100, 5, 300], 1, h_q, seed=16, fp8=fp8)
    q, kv, table, lens = c.q.cuda(), c.kv.cuda(), torch.from_numpy(c.table).cuda(), i32(c.lens)
    pl = mla.plan_shared_prefix(table, lens, 1, h_q)
    st = i32([0])
    out, lse = mla.shared_prefix_decode(q, kv, table, lens, pl=pl, status=st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mla.mla_shared_prefix_get_plan(table, lens, 1, h_q, False, pl.num_parts, pl.plan)
        mla.mla_shared_prefix_decode_fwd(q, kv, table, pl, out, lse, st)
    for lengths in (c.lens, [600, 640, 641, 704], [64, 130, 70, 65], [10, 0, 3, 2]):
        c.lens = lengths
        lens.copy_(i32(lengths))
        out.fill_(float("nan"))
        graph.replay()
        compare(out, lse, *c.want())
    assert int(st) == 0


def test_same_bits_every_time():
    c = Case(64, [500, 100, 5, 300, 64, 9], 1, 16, seed=17)
    first = c.run()
    for _ in range(3):
        again = c.run()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_another_stream():
    c = Case(12, [500, 100, 5], 1, 16, seed=18)
    first = c.run()
    q, kv, table, lens = c.q.cuda(), c.kv.cuda(), torch.from_numpy(c.table).cuda(), i32(c.lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out, lse = mla.shared_prefix_decode(q, kv, table, lens)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


@pytest.mark.parametrize("b,h_q,head,fp8", [(128, 8, 64, False), (256, 16, 32, False), (128, 8, 64, True),
                                            (150, 128, 0, False)])
def test_thousands_of_calls(b, h_q, head, fp8):
    """Partitions of many short units, where a load that is late by some microseconds meets the next units'
    messages: every call ends, without a timeout, in the same bits."""
    c = Case(head, [300 + 3 * (i % 64) for i in range(b)], 1, h_q, seed=3, fp8=fp8)
    q, kv, table, lens = c.q.cuda(), c.kv.cuda(), torch.from_numpy(c.table).cuda(), i32(c.lens)
    pl = mla.plan_shared_prefix(table, lens, 1, h_q)
    plain = mla.plan(lens, b, h_q) if not fp8 else None
    status, bad = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    out, lse = mla.shared_prefix_decode(q, kv, table, lens, pl=pl)
    first = out.clone(), lse.clone()
    if plain is not None:
        pout, plse = torch.empty_like(out), torch.empty_like(lse)

        def decode():
            mla.mla_decode_fwd(q, kv, table, lens, plain.sched, plain.split_offset, plain.num_parts, plain.workspace,
                               pout, plse, status)
        decode()
        pfirst = pout.clone(), plse.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(5):
            mla.mla_shared_prefix_decode_fwd(q, kv, table, pl, out, lse, status)
            bad[0] += (out != first[0]).any() | (lse != first[1]).any()
            if plain is not None:
                decode()
                bad[1] += (pout != pfirst[0]).any() | (plse != pfirst[1]).any()
    for i in range(400):
        g.replay()
        if i % 50 == 49:
            assert int(status) == 0
    assert bad.tolist() == [0, 0]


STALE_PLAN = 7


@pytest.mark.parametrize("h_q,fp8,dtype", [(16, False, torch.bfloat16), (16, False, torch.float16),
                                           (128, False, torch.bfloat16), (128, False, torch.float16),
                                           (16, True, torch.bfloat16), (128, True, torch.bfloat16)])
def test_a_plan_of_other_lengths_is_reported(h_q, fp8, dtype):
    """A plan holds its lengths: with others, longer, shorter or newly empty or live, the call says so (and
    answers by the plan); with the same ones it is silent."""
    c = Case(4, [64, 100, 5, 0, 200], 1, h_q, seed=19, fp8=fp8, dtype=dtype)
    c.lens[3] = 0
    q, kv, table, lens = c.q.cuda(), c.kv.cuda(), torch.from_numpy(c.table).cuda(), i32(c.lens)
    pl = mla.plan_shared_prefix(table, lens, 1, h_q)
    st = i32([0])
    want = mla.shared_prefix_decode(q, kv, table, lens, pl=pl, status=st)
    assert int(st) == 0
    for b, n in ((0, c.lens[0] + 1), (1, c.lens[1] - 1), (2, 0), (3, 1), (4, c.lens[4] + 640), (4, 64)):
        other = list(c.lens)
        other[b] = n
        with pytest.raises(mla.MlaError) as e:
            mla.shared_prefix_decode(q, kv, table, i32(other), pl=pl)
        assert e.value.code == STALE_PLAN
        st = i32([0])
        out, lse = mla.shared_prefix_decode(q, kv, table, i32(other), pl=pl, status=st)
        assert int(st) == STALE_PLAN and torch.equal(out, want[0]) and torch.equal(lse, want[1])
    # rows that grow in place, as mla_cache_grow lets them
    lens[1] += 1
    with pytest.raises(mla.MlaError):
        mla.shared_prefix_decode(q, kv, table, lens, pl=pl)
    mla.shared_prefix_decode(q, kv, table, lens)  # a plan of its own: fine
    lens[1] -= 1
    mla.shared_prefix_decode(q, kv, table, lens, pl=pl)
    if h_q == 16:  # another request of the same length took the slot: it does not start with the prefix
        table[1, :4] = table[1, 4]
        with pytest.raises(mla.MlaError) as e:
            mla.shared_prefix_decode(q, kv, table, lens, pl=pl)
        assert e.value.code == STALE_PLAN


def test_lengths_of_a_given_plan_are_checked_tensors():
    c = Case(4, [64, 100], 1, 16, seed=20)
    q, kv, table, lens = c.q.cuda(), c.kv.cuda(), torch.from_numpy(c.table).cuda(), i32(c.lens)
    pl = mla.plan_shared_prefix(table, lens, 1, 16)
    for bad, error in ((lens.long(), TypeError), (lens[:1], ValueError), (lens.cpu(), ValueError)):
        with pytest.raises(error):
            mla.shared_prefix_decode(q, kv, table, bad, pl=pl)


def test_many_lengths_are_all_compared():
    """More requests than one CTA has threads: the last one's length."""
    c = Case(1, [(i * 13) % 90 for i in range(2000)], 1, 2, seed=21)
    q, kv, table, lens = c.q.cuda(), c.kv.cuda(), torch.from_numpy(c.table).cuda(), i32(c.lens)
    pl = mla.plan_shared_prefix(table, lens, 1, 2)
    st = i32([0])
    mla.shared_prefix_decode(q, kv, table, lens, pl=pl, status=st)
    assert int(st) == 0
    lens[1999] += 1
    mla.shared_prefix_decode(q, kv, table, lens, pl=pl, status=st)
    assert int(st) == STALE_PLAN


@pytest.mark.parametrize("live", [[0], [63], [0, 1], [5, 60], [0, 1, 2, 3, 4, 5, 6, 7, 8], [9, 40, 41]])
@pytest.mark.parametrize("s_q,fp8", [(1, False), (2, False), (1, True)])
def test_padded_batch_attends_the_prefix_for_its_live_rows_alone(live, s_q, fp8):
    """64 slots of 16 heads, few of them live: only row blocks with a request that takes part have the prefix's
    keys, and a single one has all its keys to itself."""
    c = Case(5, [64 + 3 * b for b in range(64)], s_q, 16, s_q > 1, seed=22, fp8=fp8)
    for b in range(64):
        if b not in live:
            c.lens[b] = 0
            c.table[b] = -1
    c.check()
    rows, width = 16 * s_q, c.table.shape[1]
    front = 64 * rows // 128
    pl = mla.plan_shared_prefix(torch.from_numpy(c.table).cuda(), i32(c.lens), s_q, 16, s_q > 1)
    units = pl.plan[:(front + 64) * 32].view(torch.int32).reshape(-1, 8).cpu().tolist()
    at = -(-(front + 64) * 32 // 256) * 256
    keys = pl.plan[at:at + (front + 64) * 4].view(torch.int32).cpu().tolist()
    blocks = {b * rows // 128 for b in live} if len(live) > 1 else set()
    assert keys[:front] == [5 * 64 if u in blocks else 0 for u in range(front)]
    for b in range(64):
        skip = 5 if b in live and len(live) > 1 else 0
        assert units[front + b][3] == b * width + skip and keys[front + b] == c.lens[b] - 64 * skip


def bound_of(c, out_dtype):
    """want, lse and what they may be off by, element by element.  Weights of type `dtype` are rounded once, half a
    step u of each (2^-8 bf16, 2^-11 fp16; FP8 records: bf16, and the sum is that of the rounded ones, once more), so
    the output moves by u M, M = sum w |v|; the output's own rounding is a half step of it.  A score is 576 products in
    fp32, off by 576 2^-23 A, A = max scale |q|.|k|; the exponentials and the merge of the splits add 2^-20.  fp16
    weights below the smallest normal are off by 2^-25 each, of a sum of 1 at least."""
    u = 2.0 ** -11 if c.q.dtype == torch.float16 else 2.0 ** -8
    fp8 = c.kv.dtype == torch.uint8
    want, lse = c.want()
    want, lse = np.asarray(want, dtype=np.float64), np.asarray(lse, dtype=np.float64)
    mix, reach, tiny = np.zeros_like(want), np.zeros_like(lse), np.zeros_like(want)
    for b, n in enumerate(c.lens):
        pages = c.kv[c.table[b, :-(-n // 64)]].reshape(-1, c.kv.shape[2])[:n]
        keys = np.stack([orc.decode_record(r) for r in pages.numpy()]) if fp8 else pages.double().numpy()
        q = c.q[b].double().numpy()
        s = np.einsum("shd,kd->shk", q, keys) / 24
        if c.causal:
            for i in range(c.s_q):
                s[i, :, max(n - c.s_q + 1 + i, 0):] = -np.inf
        w = np.exp(s - lse[b][..., None])
        mix[b] = np.einsum("shk,kd->shd", w, np.abs(keys[:, :512]))
        if c.q.dtype == torch.float16:
            tiny[b] = 2.0 ** -25 * np.abs(keys[:, :512]).sum(0)
        reach[b] = (np.einsum("shd,kd->shk", np.abs(q), np.abs(keys)) / 24).max(2)
    score = 576 * 2.0 ** -23 * reach
    own = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}[out_dtype]
    tiny += 2.0 ** -25 if out_dtype == torch.float16 else 0.0
    return want, lse, ((2 if fp8 else 1) * u + 2 * score + 2.0 ** -20)[..., None] * mix + own * np.abs(want) + tiny, \
        score + 2.0 ** -20 + 2.0 ** -23 * np.abs(lse)


@pytest.mark.parametrize("h_q", [16, 104, 128])  # rows packed twice, requests alone
@pytest.mark.parametrize("dtype,fp8", [(torch.bfloat16, False), (torch.float16, False), (torch.bfloat16, True)])
@pytest.mark.parametrize("out_fp32", [False, True])
@pytest.mark.parametrize("s_q,causal", [(1, False), (2, True)])
def test_every_instance_within_its_roundings(h_q, dtype, fp8, out_fp32, s_q, causal):
    """Every kernel of the call against the bound of its own arithmetic, a fraction of the outputs' spread."""
    c = Case(9, [64, 100, 5, 300, 33, 64, 2, 190], s_q, h_q, causal, dtype=dtype, seed=23 + s_q, poison=False, fp8=fp8)
    out, lse = c.run(out_fp32=out_fp32)
    want, wlse, tol, ltol = bound_of(c, out.dtype)
    assert np.median(tol) < want.std() / 4
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.all(np.abs(o - want) <= tol), np.max(np.abs(o - want) / tol)
    assert np.all(np.abs(l - wlse) <= ltol), np.max(np.abs(l - wlse) / ltol)
    if not fp8 and not causal:  # and so the plain decode of each request
        o2, l2 = mla.decode(c.q.cuda(), c.kv.cuda(), torch.from_numpy(c.table).cuda(), i32(c.lens), out_fp32=out_fp32)
        assert np.all(np.abs(o2.double().cpu().numpy() - o) <= 2 * tol)
        assert np.all(np.abs(l2.double().cpu().numpy() - l) <= 2 * ltol)


@pytest.mark.parametrize("call", ["decode", "shared"])
def test_whole_units_in_one_graph_with_what_follows(call):
    """One partition: every unit is written by the attention kernel itself and the combine has nothing to do, but
    what follows in the graph (a copy of the output, the next plan in the same buffers) still finds it done."""
    c = Case(2, [64 * (i % 7) + 1 for i in range(70)], 1, 128, seed=24, poison=False)
    q, kv, table, lens = c.q.cuda(), c.kv.cuda(), torch.from_numpy(c.table).cuda(), i32(c.lens)
    other = i32([70 + 3 * (i % 40) for i in range(70)])
    st, n = i32([0]), torch.empty_like(lens)
    if call == "shared":
        pl = mla.plan_shared_prefix(table, lens, 1, 128, num_parts=1)
    else:
        pl = mla.plan(lens, 70, 128, num_parts=1)
    out = torch.empty(70, 1, 128, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(70, 1, 128, device="cuda")

    def step(lengths):
        n.copy_(lengths)
        if call == "shared":
            mla.mla_shared_prefix_get_plan(table, n, 1, 128, False, 1, pl.plan)
            mla.mla_shared_prefix_decode_fwd(q, kv, table, pl, out, lse, st)
        else:
            mla.mla_get_metadata(n, 70, 1, pl.sched, pl.split_offset)
            mla.mla_decode_fwd(q, kv, table, n, pl.sched, pl.split_offset, 1, pl.workspace, out, lse, st)
        return out.clone(), lse.clone()

    want = []
    for lengths in (lens, other):
        want.append(step(lengths))
        torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [step(lens), step(other), step(lens)]
    for _ in range(5):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for (o, l), (wo, wl) in zip(got, [want[0], want[1], want[0]]):
            assert torch.equal(o, wo) and torch.equal(l, wl)
    c.lens = other.tolist()
    compare(*want[1], *c.want())
    assert int(st) == 0
