"""Prompt attention against 64-bit attention, element by element.

Tolerances, from the arithmetic.  Each weight is rounded once to the inputs'
type: half a step, u = 2^-8 (bf16) or 2^-11 (fp16), moves the output by at most
u * mix with mix = sum_j w_j |v_j|; rounding the output adds u |out|.  A score
is a sum of d products in fp32: off by at most d 2^-23 * reach, reach = max_j
scale |q|.|k_j| (each add may lose one last place, truncation allowed for), and
the exponential adds 2^-21; both move weights, hence twice that on the output
(numerator and sum).  lse moves by the score error plus 2^-20 (sum and log) and
one last place of its own value.  fp16 values below the smallest normal are off
by at most 2^-25.
"""

import math

import numpy as np
import pytest
import torch

import mla_paged_kv_gb300 as mla
from oracle import serving_oracle as so

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def make(lq, lk, h, hkv, d, dtype, seed, extra=0, amp=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    q = (amp * r(sum(lq) + extra, h, d)).to(dtype)
    k, v = r(sum(lk) + extra, hkv, d).to(dtype), r(sum(lk) + extra, hkv, 128).to(dtype)
    cum = lambda x: [0] + [int(i) for i in np.cumsum(x)]  # noqa: E731
    return q, k, v, cum(lq), cum(lk)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def check(out, lse, q, k, v, cu_q, cu_k, causal, scale, fill=None):
    u, d = U[q.dtype], q.shape[2]
    want, wlse, mix, reach = so.prompt_attention(q.double().numpy(), k.double().numpy(), v.double().numpy(), cu_q,
                                                 cu_k, causal, scale)
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    live = np.zeros(o.shape[0], dtype=bool)
    for a, b in zip(cu_q[:-1], cu_q[1:]):
        live[a:b] = True
    if fill is not None:
        assert np.all(o[~live] == fill) and np.all(l[~live] == fill), "rows of no sequence were written"
    o, l, want, wlse, mix, reach = (x[live] for x in (o, l, want, wlse, mix, reach))
    none = np.isneginf(wlse)
    assert np.array_equal(np.isneginf(l), none) and not o[none].any()
    score = d * 2.0 ** -23 * reach
    tol = (u + 2 * score + 2.0 ** -20)[..., None] * mix + u * np.abs(want) + \
        (2.0 ** -25 * (1 + np.abs(v.double().numpy()).max()) if q.dtype == torch.float16 else 0)
    assert np.isfinite(o).all() and np.all(np.abs(o - want) <= tol), np.max(np.abs(o - want) / tol)
    l, wlse, score = l[~none], wlse[~none], score[~none]
    assert np.all(np.abs(l - wlse) <= score + 2.0 ** -20 + 2.0 ** -23 * np.abs(wlse))


def run(lq, lk, h=2, hkv=1, d=192, dtype=torch.bfloat16, causal=True, seed=0, scale=None, amp=1.0):
    q, k, v, cu_q, cu_k = make(lq, lk, h, hkv, d, dtype, seed, amp=amp)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    out, lse = mla.prompt_attention(q.cuda(), k.cuda(), v.cuda(), i32(cu_q), i32(cu_k), causal, scale)
    check(out, lse, q, k, v, cu_q, cu_k, causal, scale)


@pytest.mark.parametrize("n", [1, 2, 63, 64, 127, 128, 129, 255, 256, 257, 300, 513, 700])
def test_one_prompt(n):
    run([n], [n], seed=n)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [128, 192])
@pytest.mark.parametrize("causal", [True, False])
def test_types_and_dims(dtype, d, causal):
    run([200, 1, 333], [200, 5, 400], h=4, hkv=2, d=d, dtype=dtype, causal=causal, seed=d)


@pytest.mark.parametrize("h,hkv", [(1, 1), (3, 3), (8, 1), (6, 2), (16, 16)])
def test_head_groups(h, hkv):
    run([150, 270], [150, 270], h=h, hkv=hkv, seed=h)


def test_many_short_prompts():
    lens = [(7 * i) % 50 for i in range(90)]  # empty ones among them
    run(lens, lens, seed=5)


@pytest.mark.parametrize("lens,h,causal", [([1800, 300, 1100, 1, 1700], 24, True), ([1700, 1600], 32, True),
                                           ([200, 1600, 900, 1300], 40, False)])
def test_long_ragged_prompts(lens, h, causal):
    """Three to six rounds of items whose last ones are dealt out by the workers' sums; every row once."""
    run(lens, lens, h=h, hkv=1, causal=causal, seed=len(lens))


@pytest.mark.parametrize("lq,lk", [([1], [1000]), ([129], [1025]), ([300], [301]), ([5, 400], [133, 900])])
def test_chunk_behind_earlier_keys(lq, lk):
    run(lq, lk, h=4, hkv=4, seed=lq[0])


@pytest.mark.parametrize("causal", [True, False])
def test_rows_that_see_no_key(causal):
    """More queries than keys (the first ones see none), and no keys at all."""
    run([300, 40, 7], [130, 0, 7], causal=causal, seed=7)


def test_no_keys_in_the_whole_batch():
    q = torch.randn(9, 2, 192, device="cuda").to(torch.bfloat16)
    k, v = q[:0, :1], q[:0, :1, :128]
    out, lse = mla.prompt_attention(q, k, v, i32([0, 4, 9]), i32([0, 0, 0]))
    assert not out.any() and torch.isneginf(lse).all()


def test_no_queries():
    k = torch.randn(9, 1, 192, device="cuda").to(torch.bfloat16)
    out, lse = mla.prompt_attention(k[:0], k, k[..., :128], i32([0, 0]), i32([0, 9]))
    assert out.shape == (0, 1, 128) and lse.shape == (0, 1)


def test_growing_maxima_rescale_the_output():
    """Scores that rise along the keys by far more than the rescale threshold, and peaky rows."""
    q, k, v, cu, _ = make([600], [600], 2, 1, 192, torch.bfloat16, 11)
    k = (k.float() * 0.02 + torch.linspace(0, 3, 600)[:, None, None] * q[:1, :1].float()).to(torch.bfloat16)
    q = (q.float() * 0.1 + q[:1, :1].float()).to(torch.bfloat16)
    out, lse = mla.prompt_attention(q.cuda(), k.cuda(), v.cuda(), i32(cu), None, True, 0.2)
    check(out, lse, q, k, v, cu, cu, True, 0.2)
    run([400], [400], seed=12, amp=8.0)


@pytest.mark.parametrize("n", [100, 257])
def test_values_outside_the_sequence_may_be_anything(n):
    """Keys, values and queries between and behind the sequences hold NaN and infinities."""
    q, k, v, _, _ = make([n + 200], [n + 300], 2, 1, 192, torch.bfloat16, 13)
    cu_q, cu_k = [30, 30 + n], [55, 55 + n]
    for t, (a, b) in ((q, cu_q), (k, cu_k), (v, cu_k)):
        t[:a] = float("nan")
        t[b:] = float("inf")
    out = torch.full((n + 200, 2, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n + 200, 2), 5.0, device="cuda")
    pl = mla.plan_prompt(i32(cu_q), i32(cu_k), n + 200, n + 300)
    st = i32([0])
    mla.mla_prompt_attention_fwd(q.cuda(), k.cuda(), v.cuda(), pl, out, lse, st)
    assert int(st) == 0
    clean = [torch.where(torch.isfinite(t), t, torch.zeros_like(t)) for t in (q, k, v)]
    check(out, lse, *clean, cu_q, cu_k, True, 1 / math.sqrt(192), fill=5.0)


def test_strided_inputs():
    """Slices of one fused projection, and head-major storage."""
    g = torch.Generator().manual_seed(14)
    n, h = 210, 3
    fused = torch.randn(n, h, 192 + 192 + 128, generator=g).to(torch.bfloat16)
    q, k, v = fused[..., :192], fused[..., 192:384], fused[..., 384:]
    dev = fused.cuda()
    out, lse = mla.prompt_attention(dev[..., :192], dev[..., 192:384], dev[..., 384:], i32([0, 100, n]))
    check(out, lse, q, k, v, [0, 100, n], [0, 100, n], True, 1 / math.sqrt(192))
    major = [t.transpose(0, 1).contiguous().cuda().transpose(0, 1) for t in (q, k, v)]
    out2, lse2 = mla.prompt_attention(*major, i32([0, 100, n]))
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_offsets_out_of_order_give_an_empty_plan():
    q = torch.randn(50, 1, 192, device="cuda").to(torch.bfloat16)
    for cu in ([0, 30, 20, 50], [0, 60], [-1, 50]):
        st = i32([0])
        pl = mla.plan_prompt(i32(cu), i32(cu), 50, 50, status=st)
        assert int(st) == 5
        out = torch.full((50, 1, 128), 2.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((50, 1), 2.0, device="cuda")
        st2 = i32([0])
        mla.mla_prompt_attention_fwd(q, q, q[..., :128], pl, out, lse, st2)
        assert int(st2) == 0 and torch.all(out == 2) and torch.all(lse == 2)
        with pytest.raises(mla.MlaError):
            mla.plan_prompt(i32(cu), i32(cu), 50, 50)


def test_refuses_what_it_cannot_do():
    q = torch.randn(10, 4, 192, device="cuda").to(torch.bfloat16)
    cu = i32([0, 10])
    with pytest.raises(ValueError):
        mla.prompt_attention(q, q[:, :3], q[:, :3, :128], cu)
    with pytest.raises(TypeError):
        mla.prompt_attention(q, q.half(), q[..., :128], cu)
    with pytest.raises(ValueError):
        mla.prompt_attention(q[..., :64], q[..., :64], q[..., :128], cu)
    with pytest.raises(ValueError):
        mla.prompt_attention(q, q, q[..., :128], cu, causal=False, pl=mla.plan_prompt(cu, None, 10))
    with pytest.raises(ValueError):
        mla.prompt_attention(q, q, q[..., :128], cu, pl=mla.plan_prompt(cu, None, 11))
    odd = torch.randn(10, 4, 196, device="cuda").to(torch.bfloat16)[..., :192]  # rows 392 bytes apart
    with pytest.raises(mla.MlaError):
        mla.prompt_attention(odd, q, q[..., :128], cu)


def test_same_result_every_time_and_in_a_graph():
    q, k, v, cu, _ = make([700, 130, 400], [700, 130, 400], 4, 4, 192, torch.bfloat16, 15)
    q, k, v, cu = q.cuda(), k.cuda(), v.cuda(), i32(cu)
    pl = mla.plan_prompt(cu, None, q.shape[0])
    first = mla.prompt_attention(q, k, v, cu, pl=pl)
    st = i32([0])
    out, lse = torch.empty_like(first[0]), torch.empty_like(first[1])
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        mla.mla_prompt_attention_fwd(q, k, v, pl, out, lse, st)
    torch.cuda.current_stream().wait_stream(stream)
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mla.mla_prompt_get_plan(cu, None, q.shape[0], q.shape[0], True, pl.plan, st)
        mla.mla_prompt_attention_fwd(q, k, v, pl, out, lse, st)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    assert int(st) == 0


def test_without_a_plan_the_status_is_the_callers():
    """With a status word nothing waits: offsets that no plan can be made of set it (and give no output), and
    plan and attention can be captured together."""
    q, k, v, cu, _ = make([300, 20], [300, 20], 2, 1, 192, torch.bfloat16, 16)
    q, k, v = q.cuda(), k.cuda(), v.cuda()
    st = i32([0])
    mla.prompt_attention(q, k, v, i32([0, 330, 320]), status=st)
    assert int(st) == 5
    with pytest.raises(mla.MlaError) as e:
        mla.prompt_attention(q, k, v, i32([0, 330, 320]))
    assert e.value.code == 5
    want = mla.prompt_attention(q, k, v, i32(cu))
    st, offsets = i32([0]), i32(cu)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = mla.prompt_attention(q, k, v, offsets, status=st)
    graph.replay()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and int(st) == 0
    offsets.copy_(i32([0, 20, 320]))
    graph.replay()
    assert torch.equal(out[:20], mla.prompt_attention(q, k, v, i32([0, 20, 320]))[0][:20]) and int(st) == 0


@pytest.mark.parametrize("lq,lk", [([300, 20, 0, 5], None), ([700, 900], [700, 1000]), ([3] * 6000, None)])
def test_a_plan_of_other_offsets_is_reported(lq, lk):
    """A plan holds its offsets: with others that end in the same place the call says so (and answers by the
    plan); with the same ones it is silent."""
    q, k, v, cu_q, cu_k = make(lq, lk or lq, 2, 1, 192, torch.bfloat16, 17)
    q, k, v = q.cuda(), k.cuda(), v.cuda()
    dev_q, dev_k = i32(cu_q), i32(cu_k) if lk else None
    pl = mla.plan_prompt(dev_q, dev_k, q.shape[0], k.shape[0])
    want = mla.prompt_attention(q, k, v, dev_q, dev_k, pl=pl)
    for which, at in (("q", 1), ("q", len(lq) - 1), ("k", 1)):
        if which == "k" and lk is None:
            continue
        a, b = dev_q.clone(), None if dev_k is None else dev_k.clone()
        (a if which == "q" else b)[at] += 1
        with pytest.raises(mla.MlaError) as e:
            mla.prompt_attention(q, k, v, a, b, pl=pl)
        assert e.value.code == 7
        st = i32([0])
        out, lse = mla.prompt_attention(q, k, v, a, b, pl=pl, status=st)
        assert int(st) == 7 and torch.equal(out, want[0]) and torch.equal(lse, want[1])
    for bad, error in ((dev_q.long(), TypeError), (dev_q[1:], ValueError), (dev_q.cpu(), ValueError)):
        with pytest.raises(error):
            mla.prompt_attention(q, k, v, bad, dev_k, pl=pl)


# Batches of more than 256 queries a prompt run on pairs of CTAs, in instances of their own by type and dims.


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [128, 192])
@pytest.mark.parametrize("lq,lk,causal", [([600, 1, 333], [600, 5, 400], True), ([600, 1, 333], [600, 5, 400], False),
                                          ([513], [2500], True), ([700, 900], [300, 1000], True),
                                          ([700, 900, 257], [300, 0, 257], False)])
def test_pairs_types_and_dims(dtype, d, lq, lk, causal):
    """Ragged ends, long key rings, queries that see no key (a whole first half of a tile among them), no keys."""
    run(lq, lk, h=4, hkv=2, d=d, dtype=dtype, causal=causal, seed=d + len(lq))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [128, 192])
@pytest.mark.parametrize("h,hkv", [(3, 3), (8, 1), (12, 4)])
def test_pairs_head_groups(dtype, d, h, hkv):
    run([500, 270], [500, 470], h=h, hkv=hkv, d=d, dtype=dtype, seed=h)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [128, 192])
def test_pairs_strided_inputs(dtype, d):
    """Slices of one fused projection, and head-major storage; NaN and infinities between and behind."""
    g = torch.Generator().manual_seed(18)
    n, h, cu = 1000, 2, [3, 420, 960]
    fused = torch.randn(n, h, 2 * d + 128, generator=g).to(dtype)
    fused[:3] = float("nan")
    fused[960:] = float("inf")
    cut = lambda x: (x[..., :d], x[..., d:2 * d], x[..., 2 * d:])  # noqa: E731
    dev = cut(fused.cuda())
    pl = mla.plan_prompt(i32(cu), None, n)
    results = []
    for q, k, v in (dev, [t.transpose(0, 1).contiguous().transpose(0, 1) for t in dev]):
        out = torch.full((n, h, 128), 5.0, dtype=dtype, device="cuda")
        lse, st = torch.full((n, h), 5.0, device="cuda"), i32([0])
        mla.mla_prompt_attention_fwd(q, k, v, pl, out, lse, st)
        assert int(st) == 0
        results.append((out, lse))
    clean = cut(torch.where(torch.isfinite(fused), fused, torch.zeros_like(fused)))
    check(*results[0], *clean, cu, cu, True, 1 / math.sqrt(d), fill=5.0)
    assert torch.equal(results[0][0], results[1][0]) and torch.equal(results[0][1], results[1][1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [128, 192])
def test_pairs_rescale_the_output(dtype, d):
    q, k, v, cu, _ = make([900], [900], 2, 1, d, dtype, 11)
    k = (k.float() * 0.02 + torch.linspace(0, 3, 900)[:, None, None] * q[:1, :1].float()).to(dtype)
    q = (q.float() * 0.1 + q[:1, :1].float()).to(dtype)
    out, lse = mla.prompt_attention(q.cuda(), k.cuda(), v.cuda(), i32(cu), None, True, 0.2)
    check(out, lse, q, k, v, cu, cu, True, 0.2)
    run([600], [600], d=d, dtype=dtype, seed=12, amp=8.0)
