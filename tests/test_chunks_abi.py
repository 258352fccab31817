"""The C boundary of the operators for chunks of new tokens (CPU only): what the
host can see is refused before any launch, and the restatements themselves."""

import ctypes

import numpy as np
import pytest
import torch

import mla_paged_kv_gb300 as mla
from oracle import serving_oracle as so

INVALID, UNSUPPORTED = 1, 2
P = ctypes.c_void_p(4096)  # any aligned address: these calls return before it is used
N = ctypes.c_void_p(0)
ODD = ctypes.c_void_p(4098)
OFF8 = ctypes.c_void_p(4104)

HEADS = dict(x=P, xt=1024, xh=64, out=ctypes.c_void_p(8192), ot=1024, oh=64, heads=16, w=P, k=P, kt=128, kh=64,
             ko=ctypes.c_void_p(8192), kot=128, koh=64, kheads=2, kw=P, dim=64, dt=0, total=4, rope=64, off=0, inter=0,
             eps=1e-6, pos=N, cu=N, lens=P, batch=2, cos=P, maxpos=64, status=P, stream=N)


@pytest.mark.parametrize("change,want", [
    (dict(x=N), INVALID), (dict(out=N), INVALID), (dict(k=N), INVALID), (dict(ko=N), INVALID),
    (dict(status=N), INVALID), (dict(lens=N), INVALID), (dict(heads=0), INVALID), (dict(kheads=-1), INVALID),
    (dict(kheads=0), INVALID), (dict(dim=60), INVALID), (dict(dim=0), INVALID), (dict(dt=1), INVALID),
    (dict(total=-1), INVALID), (dict(total=5), INVALID), (dict(batch=0), INVALID), (dict(rope=24), INVALID),
    (dict(rope=0), INVALID), (dict(rope=80), INVALID), (dict(rope=-16), INVALID), (dict(off=8), INVALID),
    (dict(rope=32, off=4), INVALID), (dict(rope=32, off=-8), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(maxpos=0), INVALID), (dict(pos=P), INVALID), (dict(cos=N), INVALID),
    (dict(xt=1020), INVALID), (dict(oh=60), INVALID), (dict(kt=-8), INVALID), (dict(koh=4), INVALID),
    (dict(x=OFF8), INVALID), (dict(out=OFF8), INVALID), (dict(w=ODD), INVALID), (dict(cos=OFF8), INVALID),
    (dict(lens=ODD), INVALID), (dict(out=P, ot=2048), INVALID), (dict(ko=P, koh=128), INVALID),
    (dict(dim=1032, xh=1032, oh=1032, kh=1032, koh=1032), UNSUPPORTED), (dict(total=1 << 31), INVALID),
    (dict(total=(1 << 30) + 2), UNSUPPORTED), (dict(heads=1 << 21), UNSUPPORTED),
    (dict(total=1 << 30, heads=1 << 12), UNSUPPORTED),
    (dict(dim=512, rope=272, xh=512, oh=512, kh=512, koh=512), UNSUPPORTED)])
def test_heads_refusals(change, want):
    args = {**HEADS, **change}
    args["total"] = ctypes.c_int(args["total"])
    assert mla.load_library().mla_rope_heads(*args.values()) == want


def test_norm_alone_takes_no_positions():
    alone = dict(HEADS, cos=N, rope=0, lens=N, maxpos=0, batch=0)
    for change in (dict(lens=P), dict(pos=P), dict(cu=P), dict(rope=16), dict(w=N, kw=N)):
        assert mla.load_library().mla_rope_heads(*{**alone, **change}.values()) == INVALID


GATHER = dict(cache=P, dt=0, pages=8, table=P, width=4, cu=P, starts=N, batch=2, rows=10, out=P, stride=576, status=P,
              stream=N)


@pytest.mark.parametrize("change,want", [
    (dict(cache=N), INVALID), (dict(table=N), INVALID), (dict(cu=N), INVALID), (dict(out=N), INVALID),
    (dict(status=N), INVALID), (dict(dt=1), INVALID), (dict(dt=4), INVALID), (dict(pages=0), INVALID),
    (dict(width=0), INVALID), (dict(batch=0), INVALID), (dict(rows=-1), INVALID), (dict(stride=570), INVALID),
    (dict(stride=568), INVALID), (dict(out=OFF8), INVALID), (dict(cu=ODD), INVALID), (dict(starts=ODD), INVALID),
    (dict(width=(1 << 18) + 1), UNSUPPORTED), (dict(rows=(1 << 30) + 1), UNSUPPORTED)])
def test_gather_refusals(change, want):
    assert mla.load_library().mla_cache_gather(*{**GATHER, **change}.values()) == want


PLAN = dict(cu=P, lens=P, batch=2, total=10, hq=16, causal=1, parts=4, plan=P, bytes=1 << 16, status=P, stream=N)
CHUNK = dict(q=P, kv=P, table=P, width=4, pages=8, batch=2, total=10, hq=16, dt=0, scale=0.1, cu=N, lens=N, plan=P,
             pbytes=1 << 16, parts=4, ws=P, wbytes=1 << 24, out=P, ot=0, lse=P, status=P, stream=N)
SIZES = [(dict(batch=0), INVALID), (dict(total=-1), INVALID), (dict(hq=0), INVALID), (dict(parts=0), INVALID),
         (dict(parts=1025), UNSUPPORTED), (dict(batch=(1 << 20) + 1), UNSUPPORTED),
         (dict(total=1 << 20, hq=1 << 11), UNSUPPORTED)]


@pytest.mark.parametrize("change,want", SIZES + [
    (dict(cu=N), INVALID), (dict(lens=N), INVALID), (dict(plan=N), INVALID), (dict(status=N), INVALID),
    (dict(bytes=64), INVALID), (dict(plan=OFF8), INVALID), (dict(cu=ODD), INVALID)])
def test_chunk_plan_refusals(change, want):
    assert mla.load_library().mla_chunk_get_plan(*{**PLAN, **change}.values()) == want


@pytest.mark.parametrize("change,want", SIZES + [
    (dict(q=N), INVALID), (dict(kv=N), INVALID), (dict(table=N), INVALID), (dict(plan=N), INVALID),
    (dict(ws=N), INVALID), (dict(out=N), INVALID), (dict(lse=N), INVALID), (dict(status=N), INVALID),
    (dict(dt=1), INVALID), (dict(dt=4), INVALID), (dict(ot=3), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(pbytes=64), INVALID), (dict(wbytes=64), INVALID),
    (dict(pages=0), INVALID), (dict(width=0), INVALID), (dict(q=OFF8), INVALID), (dict(kv=OFF8), INVALID),
    (dict(cu=ODD), INVALID), (dict(lens=ODD), INVALID), (dict(width=(1 << 18) + 1), UNSUPPORTED),
    (dict(dt=3, wbytes=2 * 4 * 128 * 513 * 4 + 160 * 1040 - 1), INVALID)])
@pytest.mark.parametrize("name", ["mla_chunk_attention_fwd", "mla_test_chunk_timeout"])
def test_chunk_refusals(name, change, want):
    assert getattr(mla.load_library(), name)(*{**CHUNK, **change}.values()) == want


def words(values):
    values = [v.value or 0 if isinstance(v, ctypes.c_void_p) else v for v in values]
    return b"".join(np.float64(v).tobytes() if isinstance(v, float) else np.int64(v).tobytes() for v in values)


@pytest.mark.parametrize("op,name,base", [(10, "mla_rope_heads", HEADS), (11, "mla_cache_gather", GATHER),
                                          (12, "mla_chunk_attention_fwd", CHUNK)])
def test_packed_calls(op, name, base):
    """The same arguments as 8-byte words are refused alike, one after another."""
    lib = mla.load_library()
    good = words(base.values())
    assert lib.mla_serving_call(op, good, len(good) - 8) == INVALID
    assert lib.mla_serving_call(op, None, len(good)) == INVALID
    for key, v in base.items():
        change = {key: -1.0} if isinstance(v, float) else {key: N} if isinstance(v, ctypes.c_void_p) else {key: -1}
        args = {**base, **change}
        want = getattr(lib, name)(*args.values()) if key in MUST[name] else None
        if want is not None:
            assert want == INVALID and lib.mla_serving_call(op, words(args.values()), len(good)) == INVALID, key
    for key in ("total", "batch", "pages", "width", "rows", "hq", "heads", "dim"):  # sizes that 32 bits would cut to good ones
        if key in base:
            w = words({**base, key: (1 << 32) + base[key]}.values())
            assert lib.mla_serving_call(op, w, len(w)) == INVALID, key


MUST = {"mla_rope_heads": {"x", "out", "heads", "k", "ko", "kheads", "dim", "dt", "total", "rope", "off", "eps", "lens",
                           "batch", "cos", "maxpos", "status", "xt", "oh"},
        "mla_cache_gather": {"cache", "dt", "pages", "table", "width", "cu", "batch", "rows", "out", "stride", "status"},
        "mla_chunk_attention_fwd": {"q", "kv", "table", "width", "pages", "batch", "total", "hq", "dt", "scale", "plan",
                                    "parts", "ws", "out", "ot", "lse", "status"}}


FREQ = dict(dim=64, base=10000.0, kind=3, factor=4.0, original=4096.0, low=1.0, high=32.0)


@pytest.mark.parametrize("change,want", [
    (dict(dim=4), INVALID), (dict(dim=60), INVALID), (dict(dim=264), UNSUPPORTED), (dict(base=1.0), INVALID),
    (dict(base=float("inf")), INVALID), (dict(kind=5), INVALID), (dict(kind=-1), INVALID), (dict(factor=0.5), INVALID),
    (dict(factor=float("nan")), INVALID), (dict(original=0.0), INVALID), (dict(low=0.0), INVALID),
    (dict(low=32.0), INVALID), (dict(high=float("inf")), INVALID)])
def test_frequency_refusals(change, want):
    with pytest.raises(mla.MlaError) as e:
        mla.mla_rope_frequencies(*{**FREQ, **change}.values())
    assert e.value.code == want


def test_table_refusals():
    lib = mla.load_library()
    freq = (ctypes.c_double * 32)(*[0.5] * 32)
    base = dict(f=freq, dim=64, size=1.0, first=0, n=4, out=P, stream=N)
    for change, want in ((dict(f=None), INVALID), (dict(dim=4), INVALID), (dict(dim=60), INVALID),
                         (dict(size=float("nan")), INVALID), (dict(first=-1), INVALID), (dict(n=-1), INVALID),
                         (dict(out=N), INVALID), (dict(out=OFF8), INVALID), (dict(dim=264), UNSUPPORTED),
                         (dict(first=(1 << 31) - 3), UNSUPPORTED),
                         (dict(f=(ctypes.c_double * 32)(*[-0.5] * 32)), INVALID),
                         (dict(f=(ctypes.c_double * 32)(*[float("nan")] * 32)), INVALID),
                         (dict(f=(ctypes.c_double * 32)(*[2000.0] * 32)), INVALID)):
        assert lib.mla_rope_table(*{**base, **change}.values()) == want, change
    with pytest.raises(ValueError):
        mla.rope_table(4, scaling="other")


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn", "wavelength"])
@pytest.mark.parametrize("dim,base,factor,original", [(64, 10000.0, 40.0, 4096), (128, 500000.0, 8.0, 8192),
                                                      (8, 100.0, 1.0, 100), (256, 1e6, 3.5, 333)])
def test_frequencies(scaling, dim, base, factor, original):
    got, size = mla.rope_frequencies(dim, base, scaling, factor, original)
    want, wsize = so.rope_frequencies(dim, base, scaling, factor, original, 1.0, 4.0 if scaling == "wavelength" else 32.0)
    # both are a few 64-bit operations on a power: 2^-53 each, its exponent's rounding times ln(base) more
    np.testing.assert_allclose(got, want, rtol=2.0 ** -46, atol=0)
    assert abs(size - wsize) <= 2.0 ** -50 * wsize


def test_sizes():
    assert mla.mla_chunk_workspace_bytes(76) == 2 * 76 * 128 * 513 * 4
    assert mla.mla_chunk_workspace_bytes(0) == 0 and mla.mla_chunk_workspace_bytes(1025) == 0
    assert mla.mla_chunk_plan_bytes(0, 1, 16, 76) == 0
    assert mla.mla_chunk_plan_bytes(3, 0, 16, 76) > 0


def test_python_refuses_wrong_tensors():
    st = torch.zeros(1, dtype=torch.int32)
    x, table = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(8, 64)
    lens, cu = torch.full((2,), 4, dtype=torch.int32), torch.tensor([0, 2, 4], dtype=torch.int32)

    def refuses(kind, *args, **more):
        with pytest.raises(kind):
            mla.rope_heads(*args, status=st, **more)

    refuses(ValueError, x, table, lens)  # not on a GPU
    refuses(TypeError, x.float(), table, lens)
    refuses(TypeError, x, table.half(), lens)
    refuses(ValueError, x[0], table, lens)
    refuses(ValueError, x, table)
    refuses(ValueError, x, table, lens, positions=torch.zeros(4, dtype=torch.int32))
    refuses(ValueError, x, table, lens, cu[:2])
    refuses(ValueError, x, table, positions=torch.zeros(3, dtype=torch.int32))
    refuses(ValueError, x, None, lens)
    refuses(ValueError, x, table, lens, out=x[:3])
    refuses(TypeError, x, table, lens, out=x.half())
    refuses(ValueError, x, table, lens, k_norm_weight=torch.zeros(64, dtype=torch.bfloat16))
    refuses(ValueError, x, table, lens, norm_weight=torch.zeros(32, dtype=torch.bfloat16))
    # outputs that overlap what is read, or themselves
    both = torch.zeros(5, 3, 128, dtype=torch.bfloat16)
    refuses(ValueError, both[:4, :2, :64], table, lens, out=both[:4, :2, 8:72])
    refuses(ValueError, both[:4, :2, :64], table, lens, out=both[:4, 1:, :64])
    refuses(ValueError, both[:4, :2, :64], table, lens, out=both[1:, :2, :64])
    refuses(ValueError, x, table, lens, out=torch.zeros(4, 1, 64, dtype=torch.bfloat16).expand(4, 2, 64))
    refuses(ValueError, x, table, lens, k=x.clone(), k_out=x)

    cache, block = torch.zeros(8, 64, 576, dtype=torch.bfloat16), torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError):
        mla.cache_gather(cache, block, cu, 4, status=st)  # not on a GPU
    with pytest.raises(TypeError):
        mla.cache_gather(cache.float(), block, cu, 4, status=st)
    with pytest.raises(TypeError):
        mla.cache_gather(cache, block, cu, out=torch.zeros(4, 576), status=st)
    with pytest.raises(ValueError):
        mla.cache_gather(cache[..., :512].contiguous(), block, cu, 4, status=st)
    with pytest.raises(ValueError):
        mla.cache_gather(cache, block, cu[:2], 4, status=st)
    with pytest.raises(ValueError):
        mla.cache_gather(cache, block, cu, out=cache.view(-1, 576)[:4], status=st)

    q = torch.zeros(4, 16, 576, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mla.plan_chunks(cu, lens, 4, 0, num_parts=4, status=st)
    with pytest.raises(ValueError):
        mla.plan_chunks(cu[:2], lens, 4, 16, num_parts=4, status=st)
    pl = mla.ChunkPlan(torch.zeros(1 << 16, dtype=torch.uint8), 2, 4, 16, 4, True, torch.zeros(16, dtype=torch.uint8))
    for bad in (dict(q=q.half()), dict(q=q[:3]), dict(q=q[:, :8].contiguous()), dict(cache=cache.half()),
                dict(block=block[:1]), dict(causal=False)):
        a = dict(q=q, cache=cache, block=block, causal=True, **{}) | bad
        with pytest.raises((ValueError, TypeError)):
            mla.chunk_attention(a["q"], a["cache"], a["block"], lens, cu, a["causal"], pl=pl, status=st)


# ---------------------------------------------------------------- the plain forms themselves


def test_chunk_oracle_against_torch_attention():
    g = torch.Generator().manual_seed(3)
    q = torch.randn(6, 2, 576, dtype=torch.float64, generator=g)
    keys = [torch.randn(n, 576, dtype=torch.float64, generator=g).numpy() for n in (9, 2)]
    seen = [np.ones(9, dtype=bool), np.ones(2, dtype=bool)]
    seen[0][4] = False
    out, lse, _, _ = so.chunk_attention(q.numpy(), keys, seen, [0, 3, 6], [9, 2], True, 0.1)
    for b, (cu, total) in enumerate(((0, 9), (3, 2))):
        for i in range(3):
            see = torch.from_numpy(seen[b].copy()) & (torch.arange(total) <= total - 3 + i)
            if not see.any():
                assert not out[cu + i].any() and np.all(np.isneginf(lse[cu + i]))
                continue
            k = torch.from_numpy(keys[b])[see]
            want = torch.nn.functional.scaled_dot_product_attention(q[cu + i][None, :, None], k[None, None].expand(1, 2, -1, -1),
                                                                    k[None, None, :, :512].expand(1, 2, -1, -1), scale=0.1)
            np.testing.assert_allclose(out[cu + i], want[0, :, 0].numpy(), rtol=0, atol=1e-12)


def test_rope_oracle_turns_by_the_angle():
    z = np.array([1.0, 2.0, 3.0, 4.0]) + 1j * np.array([0.5, -1.0, 2.0, 0.0])
    row = np.concatenate([np.cos([0.3, 1.1, 2.0, 5.0]), np.sin([0.3, 1.1, 2.0, 5.0])])
    want = z * np.exp(1j * np.array([0.3, 1.1, 2.0, 5.0]))
    half = so.rope_head(np.concatenate([[9.0], z.real, z.imag]), row, 1, False)
    np.testing.assert_allclose(half, np.concatenate([[9.0], want.real, want.imag]), atol=1e-15)
    pairs = so.rope_head(np.stack([z.real, z.imag], 1).reshape(-1), row, 0, True)
    np.testing.assert_allclose(pairs, np.stack([want.real, want.imag], 1).reshape(-1), atol=1e-15)


def test_record_rows_are_codes_times_scales():
    rec = np.zeros((1, 656), dtype=np.uint8)
    rec[0, :512] = 0x38  # 1.0
    rec[0, 512:528] = np.array([1.0, 2.0, 3.0, 0.5], dtype=np.float32).view(np.uint8)
    rec[0, 528:] = np.full(64, 0x3F80, dtype=np.uint16).view(np.uint8)
    np.testing.assert_array_equal(so.record_rows(rec)[0], np.repeat([1.0, 2.0, 3.0, 0.5, 1.0], [128] * 4 + [64]))
