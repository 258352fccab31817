"""Chunk attention calls directly behind one another: a call's first kernel begins
while the call before ends, on the same plan and workspace (partial sums, and over
FP8 records converted queries and pages).  Consecutive calls here differ in their
queries and caches and nothing lies between them, so that a kernel that read or
wrote too early would meet another call's numbers.  Each result equals, to the
bit, that of the call alone."""

import pytest
import torch

import mla_paged_kv_gb300 as mla
from tests.test_chunk_gpu import Case

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
H = 16


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


caches = pytest.mark.parametrize("fp8", [False, True])


class Calls:
    """Four calls' inputs and outputs over two caches, of the same lengths."""

    def __init__(self, new, ctx, fp8, parts=None):
        cases = [Case(new, ctx, heads=H, seed=200 + i, fp8=fp8, rest=0.0) for i in range(4)]
        on = [c.device() for c in cases]
        self.q = [o[0] for o in on]
        self.cache = [on[0][1], on[1][1]]
        self.table, self.lens, self.cu = on[0][2:]
        self.total, self.fp8, self.status = sum(new), fp8, i32([0])
        self.pl = mla.plan_chunks(self.cu, self.lens, self.total, H, num_parts=parts)
        if fp8:
            self.pl.workspace = mla.chunk_workspace(self.pl, 40)

    def outputs(self, n):
        return [(torch.full((self.total, H, 512), 7.0, dtype=BF16, device="cuda"),
                 torch.full((self.total, H), 7.0, device="cuda")) for _ in range(n)]

    def call(self, i, to):
        mla.mla_chunk_attention_fwd(self.q[i % 4], self.cache[i % 2], self.table, self.pl, *to, self.status)

    def alone(self):
        want = self.outputs(4)
        for i in range(4):
            torch.cuda.synchronize()
            self.call(i, want[i])
            torch.cuda.synchronize()
        return want


def same(a, b):
    return torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@caches
@pytest.mark.parametrize("new,ctx,parts", [([9, 1, 60], [300, 700, 64], None), ([1] * 40, [700] * 40, None),
                                           ([2], [3000], None), ([40, 50], [200, 900], 5)])
def test_other_inputs_in_every_call(fp8, new, ctx, parts):
    c = Calls(new, ctx, fp8, parts)
    want = c.alone()
    got = c.outputs(24)
    for i in range(24):
        c.call(i, got[i])
    torch.cuda.synchronize()
    assert all(same(got[i], want[i % 4]) for i in range(24)) and int(c.status) == 0
    assert not same(want[0], want[2])


@caches
def test_other_inputs_in_a_graph(fp8):
    c = Calls([9, 1, 60], [300, 700, 64], fp8)
    want, got = c.alone(), c.outputs(12)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(12):
            c.call(i, got[i])
    for _ in range(3):
        for pair in got:
            pair[0].fill_(7.0)
        graph.replay()
    torch.cuda.synchronize()
    assert all(same(got[i], want[i % 4]) for i in range(12)) and int(c.status) == 0


@caches
def test_a_plan_made_again_behind_a_call(fp8):
    """Between two calls the same plan's memory takes the plan of other lengths: the first call still runs then."""
    c = Calls([9, 1, 60], [300, 700, 64], fp8)
    sets = [(c.cu, c.lens), (i32([0, 2, 40, 70]), i32([64, 700, 90])), (i32([0, 0, 0, 70]), i32([5, 1, 124]))]

    def plan(k):
        mla.mla_chunk_get_plan(*sets[k], 70, H, True, c.pl.num_parts, c.pl.plan, c.status)

    want = c.outputs(12)
    for i in range(12):
        plan(i % 3)
        torch.cuda.synchronize()
        c.call(i, want[i])
        torch.cuda.synchronize()
    got = c.outputs(36)
    for i in range(36):
        plan(i % 3)
        c.call(i, got[i])
    torch.cuda.synchronize()
    assert all(same(got[i], want[i % 12]) for i in range(36)) and int(c.status) == 0
