"""The serving operators' C boundary (CPU only): every declared function is
exported and bound, and what the host can see is refused before any launch."""

import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import mla_paged_kv_gb300 as mla
from oracle import serving_oracle as so

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mla_serving.h")
INVALID, UNSUPPORTED = 1, 2


def declared():
    text = open(HEADER).read()
    return set(re.findall(r"^(?:int|size_t)\s+(mla_\w+)\(", text, flags=re.M))


def test_declared_functions_are_exported_and_bound():
    lib = mla.load_library()
    out = subprocess.run(["nm", "-D", "--defined-only", mla.LIB_PATH], capture_output=True, text=True, check=True)
    exported = set(re.findall(r"\sT\s(mla_\w+)$", out.stdout, flags=re.M))
    assert declared() <= exported
    assert declared() == set(mla.SERVING_SYMBOLS)
    for name in declared():
        assert callable(getattr(mla, name)) and getattr(lib, name) is not None


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "mla_serving.h"\nint main(void) { return MLA_ERR_NO_PAGES == 6 ? 0 : 1; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-c", str(src), "-o",
                    str(tmp_path / "t.o")], check=True)


P = ctypes.c_void_p(4096)  # any aligned address: these calls return before it is used
N = ctypes.c_void_p(0)
ODD = ctypes.c_void_p(4098)

APPEND = dict(c=P, cs=576, r=P, rs=576, dt=0, total=4, cu=N, lens=P, batch=2, table=P, width=4, cache=P, cdt=0, pages=8,
              w=P, eps=1e-6, cos=P, maxpos=64, inter=0, ref=N, status=P, stream=N)


@pytest.mark.parametrize("change,want", [
    (dict(c=N), INVALID), (dict(lens=N), INVALID), (dict(table=N), INVALID), (dict(cache=N), INVALID),
    (dict(status=N), INVALID), (dict(dt=1), INVALID), (dict(cdt=2), INVALID), (dict(cs=577), INVALID),
    (dict(rs=-8), INVALID), (dict(total=-1), INVALID), (dict(total=5), INVALID), (dict(batch=0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=-1.0), INVALID), (dict(maxpos=0), INVALID), (dict(c=ODD), INVALID),
    (dict(cache=ctypes.c_void_p(4104)), INVALID), (dict(width=(1 << 18) + 1), UNSUPPORTED),
    (dict(total=(1 << 30) + 2), UNSUPPORTED)])
def test_append_refusals(change, want):
    assert mla.load_library().mla_cache_append(*{**APPEND, **change}.values()) == want


GROW = dict(ref=P, pages=8, table=P, rows=4, width=4, lens=P, list=P, new=P, n=2, status=P, stream=N)
FORK = dict(ref=P, pages=8, table=P, rows=4, width=4, lens=P, par=P, chi=P, n=2, pairs=P, status=P, stream=N)
FREE = dict(ref=P, pages=8, table=P, rows=4, width=4, lens=P, list=P, n=2, status=P, stream=N)
COMPACT = dict(ref=P, pages=8, table=P, rows=4, width=4, lens=P, pairs=P, count=P, ws=P, bytes=1 << 12, status=P,
               stream=N)
COPY = dict(pool=P, layers=2, stride=8 * 1024, pages=8, page=1024, pairs=P, count=N, n=2, status=P, stream=N)
SHARED = [(dict(ref=N), INVALID), (dict(table=N), INVALID), (dict(lens=N), INVALID), (dict(status=N), INVALID),
          (dict(pages=0), INVALID), (dict(rows=0), INVALID), (dict(width=0), INVALID), (dict(ref=ODD), INVALID),
          (dict(rows=65537), UNSUPPORTED), (dict(width=(1 << 18) + 1), UNSUPPORTED)]
LIST = [(dict(n=-1), INVALID), (dict(n=4097), UNSUPPORTED)]


@pytest.mark.parametrize("name,base,change,want",
                         [("grow", GROW, c, w) for c, w in SHARED + LIST + [(dict(new=N), INVALID)]] +
                         [("fork", FORK, c, w) for c, w in SHARED + LIST + [(dict(pairs=N), INVALID)]] +
                         [("free", FREE, c, w) for c, w in SHARED + LIST + [(dict(list=N), INVALID)]] +
                         [("compact", COMPACT, c, w) for c, w in SHARED + [
                             (dict(pairs=N), INVALID), (dict(count=N), INVALID), (dict(ws=N), INVALID),
                             (dict(bytes=16), INVALID)]] +
                         [("copy_pages", COPY, c, w) for c, w in [
                             (dict(pool=N), INVALID), (dict(status=N), INVALID), (dict(pairs=N), INVALID),
                             (dict(n=-1), INVALID), (dict(page=1000), INVALID), (dict(stride=8 * 1024 - 16), INVALID),
                             (dict(stride=8 * 1024 + 8), INVALID), (dict(layers=0), INVALID),
                             (dict(pool=ODD), INVALID),
                             (dict(page=1 << 25, layers=1), UNSUPPORTED), (dict(n=1 << 25), UNSUPPORTED)]])
def test_page_refusals(name, base, change, want):
    assert getattr(mla.load_library(), "mla_cache_" + name)(*{**base, **change}.values()) == want


PLAN = dict(cuq=P, cuk=N, batch=2, tq=10, tk=10, causal=1, plan=P, bytes=1 << 12, status=P, stream=N)
PROMPT = dict(q=P, qt=192, qh=192, k=P, kt=192, kh=192, v=P, vt=128, vh=128, dt=0, tq=10, tk=10, batch=2, hq=1, hkv=1,
              d=192, scale=0.1, plan=P, bytes=1 << 12, out=P, lse=P, status=P, stream=N)


@pytest.mark.parametrize("change,want", [
    (dict(cuq=N), INVALID), (dict(plan=N), INVALID), (dict(status=N), INVALID), (dict(batch=0), INVALID),
    (dict(tk=11), INVALID), (dict(tq=-1), INVALID), (dict(bytes=64), INVALID), (dict(plan=ODD), INVALID)])
def test_plan_refusals(change, want):
    assert mla.load_library().mla_prompt_get_plan(*{**PLAN, **change}.values()) == want


@pytest.mark.parametrize("change,want", [
    (dict(q=N), INVALID), (dict(k=N), INVALID), (dict(v=N), INVALID), (dict(plan=N), INVALID), (dict(out=N), INVALID),
    (dict(lse=N), INVALID), (dict(status=N), INVALID), (dict(dt=1), INVALID), (dict(dt=3), INVALID),
    (dict(hq=3, hkv=2, qh=192), INVALID), (dict(scale=0.0), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(qt=190), INVALID), (dict(kt=196), INVALID), (dict(vt=64), INVALID), (dict(q=ODD), INVALID),
    (dict(hq=2, qh=100), INVALID), (dict(bytes=64), INVALID), (dict(d=64, qt=64, kt=64), UNSUPPORTED)])
def test_prompt_refusals(change, want):
    assert mla.load_library().mla_prompt_attention_fwd(*{**PROMPT, **change}.values()) == want


SPLAN = dict(table=P, width=4, lens=P, batch=2, s_q=1, h_q=16, causal=0, parts=4, plan=P, bytes=1 << 16, stream=N)
SDEC = dict(q=P, kv=P, table=P, width=4, pages=8, batch=2, s_q=1, h_q=16, dt=0, causal=0, scale=0.1, plan=P, pbytes=1 << 16,
            parts=4, ws=P, wbytes=1 << 24, out=P, ot=0, lse=P, status=P, stream=N)


@pytest.mark.parametrize("change,want", [
    (dict(table=N), INVALID), (dict(lens=N), INVALID), (dict(plan=N), INVALID), (dict(batch=0), INVALID),
    (dict(s_q=0), INVALID), (dict(width=0), INVALID), (dict(parts=0), INVALID), (dict(parts=1025), UNSUPPORTED),
    (dict(batch=65536), UNSUPPORTED), (dict(bytes=64), INVALID), (dict(width=1 << 18, batch=1 << 14), UNSUPPORTED),
    (dict(s_q=1 << 17), UNSUPPORTED)])
def test_shared_plan_refusals(change, want):
    assert mla.load_library().mla_shared_prefix_get_plan(*{**SPLAN, **change}.values()) == want


@pytest.mark.parametrize("change,want", [
    (dict(q=N), INVALID), (dict(kv=N), INVALID), (dict(table=N), INVALID), (dict(plan=N), INVALID),
    (dict(ws=N), INVALID), (dict(out=N), INVALID), (dict(lse=N), INVALID), (dict(status=N), INVALID),
    (dict(dt=1), INVALID), (dict(dt=4), INVALID), (dict(ot=3), INVALID), (dict(scale=-1.0), INVALID),
    (dict(pbytes=64), INVALID), (dict(wbytes=64), INVALID), (dict(pages=0), INVALID), (dict(q=ODD), INVALID)])
def test_shared_decode_refusals(change, want):
    assert mla.load_library().mla_shared_prefix_decode_fwd(*{**SDEC, **change}.values()) == want


def test_packed_call():
    """mla_serving_call takes the same arguments as 8-byte words, and refuses another number of them."""
    lib = mla.load_library()
    for op, base in enumerate((APPEND, GROW, FORK, FREE, COMPACT, COPY, PROMPT, SDEC)):
        values = [v.value or 0 if isinstance(v, ctypes.c_void_p) else v for v in base.values()]
        words = b"".join(np.float64(v).tobytes() if isinstance(v, float) else np.int64(v).tobytes() for v in values)
        assert lib.mla_serving_call(op, words, len(words) - 8) == INVALID
        assert lib.mla_serving_call(op, None, len(words)) == INVALID
        # refused for the same reason as the call itself: one pointer or size at a time
        for i, v in enumerate(values):
            if isinstance(v, float) or v in (0, 4096):
                continue
            bad = words[:8 * i] + np.int64(-1).tobytes() + words[8 * i + 8:]
            args = [x if j != i else -1 for j, x in enumerate(base.values())]
            got = lib.mla_serving_call(op, bad, len(bad))
            assert got == getattr(lib, NAMES[op])(*args)
            if got == INVALID:
                break
        else:
            raise AssertionError("no refusal compared")
        for i, key in enumerate(base):  # a size that 32 bits would cut to a good one
            if key in ("batch", "pages", "n", "rows", "width", "layers", "total", "tq", "tk", "hq", "h_q", "s_q"):
                big = words[:8 * i] + np.int64((1 << 32) + 2).tobytes() + words[8 * i + 8:]
                assert lib.mla_serving_call(op, big, len(big)) == INVALID, key
    assert lib.mla_serving_call(8, b"", 0) == INVALID and lib.mla_serving_call(-1, b"", 0) == INVALID
    with pytest.raises(mla.MlaError):
        mla.mla_serving_call(0, b"")


NAMES = ["mla_cache_append", "mla_cache_grow", "mla_cache_fork", "mla_cache_free", "mla_cache_compact",
         "mla_cache_copy_pages", "mla_prompt_attention_fwd", "mla_shared_prefix_decode_fwd"]


def test_shared_prefix_sizes():
    # 64 requests of 16 rows: 8 prefix blocks and 64 own ones; (units + parts) slots of 128 rows
    assert mla.mla_shared_prefix_workspace_bytes(64, 1, 16, 76) == (72 + 76) * 128 * 513 * 4
    # rows that fill their blocks: the plain decode and its workspace
    assert mla.mla_shared_prefix_workspace_bytes(64, 1, 128, 76) == mla.mla_workspace_bytes(64, 128, 76)
    assert mla.mla_shared_prefix_workspace_bytes(1, 1, 16, 5) == mla.mla_workspace_bytes(1, 16, 5)
    assert mla.mla_shared_prefix_plan_bytes(0, 1, 16, 76) == 0


def test_python_refuses_wrong_tensors():
    c, r = torch.zeros(4, 512, dtype=torch.bfloat16), torch.zeros(4, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(2, 4, dtype=torch.int32), torch.full((2,), 2, dtype=torch.int32)
    cache, st = torch.zeros(8, 64, 576, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        mla.mla_cache_append(c, r, cache, table, lens, st)
    with pytest.raises(TypeError):
        mla.mla_cache_append(c, r.half(), cache, table, lens, st)
    with pytest.raises(TypeError):
        mla.mla_cache_append(c, r, cache.half(), table, lens, st)
    with pytest.raises(ValueError):
        mla.mla_cache_append(c, r[:3], cache, table, lens, st)
    with pytest.raises(ValueError):
        mla.mla_cache_append(c[:, ::1], r, cache[:, :, :512].contiguous(), table, lens, st)
    with pytest.raises(ValueError):
        mla.mla_cache_append(c[:3], r[:3], cache, table, lens, st)
    ref = torch.zeros(8, dtype=torch.int32)
    with pytest.raises(ValueError):
        mla.cache_grow(ref, table, lens[:1], lens, lens, st)
    with pytest.raises(TypeError):
        mla.cache_free(ref, table, lens, lens.long(), st)
    with pytest.raises(ValueError):
        mla.cache_copy_pages(torch.zeros(8, 64, 576)[:, ::2], torch.zeros(2, 2, dtype=torch.int32), status=st)
    with pytest.raises(ValueError):
        mla.plan_prompt(torch.zeros(1, dtype=torch.int32), total_q=0, status=st)


# ---------------------------------------------------------------- the plain forms themselves


def test_e4m3_values_agree_with_torch():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(so.e4m3_value(codes), want)


def test_page_oracle_on_a_hand_made_pool():
    # pages:      0  1  2  3  4  5
    p = so.Pool([0, 1, 0, 1, 0, 1], [[3, 5, -1], [1, -1, -1], [-1, -1, -1]], [100, 64, 0])
    assert p.fork([0], [2]) == [(5, 0)]
    assert p.table[2] == [3, 0, -1] and p.ref == [1, 1, 0, 2, 0, 1] and p.lens == [100, 64, 100]
    p.grow([1, 2], [1, 28])
    assert p.table[1] == [1, 2, -1] and p.table[2] == [3, 0, -1] and p.lens == [100, 65, 128]
    p.free([0])
    assert p.ref == [1, 1, 1, 1, 0, 0] and p.table[0] == [-1, -1, -1]
    p.free([1])
    assert p.compact() == [(3, 1)] and p.table[2] == [1, 0, -1] and p.ref == [1, 1, 0, 0, 0, 0]
    assert not p.bad and not p.empty


def test_prompt_oracle_against_torch_attention():
    g = torch.Generator().manual_seed(3)
    q = torch.randn(9, 2, 128, dtype=torch.float64, generator=g)
    k = torch.randn(14, 1, 128, dtype=torch.float64, generator=g)
    v = torch.randn(14, 1, 128, dtype=torch.float64, generator=g)
    out, lse, _, _ = so.prompt_attention(q, k, v, [0, 4, 9], [0, 6, 14], True, 0.1)
    for qs, ks in ((slice(0, 4), slice(0, 6)), (slice(4, 9), slice(6, 14))):
        lq, lk = qs.stop - qs.start, ks.stop - ks.start
        mask = torch.ones(lq, lk, dtype=torch.bool).tril(lk - lq)
        want = torch.nn.functional.scaled_dot_product_attention(
            q[qs].transpose(0, 1), k[ks].transpose(0, 1).expand(2, -1, -1), v[ks].transpose(0, 1).expand(2, -1, -1),
            attn_mask=mask, scale=0.1)
        np.testing.assert_allclose(out[qs], want.transpose(0, 1).numpy(), rtol=0, atol=1e-12)


# ---------------------------------------------------------------- calls that compare their plan


def checked(base, names, at):
    """The arguments of a call with further pointers before `at`."""
    out = {}
    for k, v in base.items():
        if k == at:
            out.update({n: P for n in names})
        out[k] = v
    return out


CHECKED = [(8, "mla_shared_prefix_decode_checked_fwd", checked(SDEC, ["lens"], "plan"), "lens"),
           (9, "mla_prompt_attention_checked_fwd", checked(PROMPT, ["cuq", "cuk"], "plan"), "cuq")]


@pytest.mark.parametrize("op,name,base,own", CHECKED)
def test_checked_calls_refuse_as_the_plain_ones(op, name, base, own):
    lib = mla.load_library()
    for change in ({own: N}, {own: ODD}, dict(q=N), dict(plan=N), dict(status=N), dict(batch=0), dict(scale=-1.0)):
        args = {**base, **change}
        assert getattr(lib, name)(*args.values()) == INVALID
        values = [v.value or 0 if isinstance(v, ctypes.c_void_p) else v for v in args.values()]
        words = b"".join(np.float64(v).tobytes() if isinstance(v, float) else np.int64(v).tobytes() for v in values)
        assert lib.mla_serving_call(op, words, len(words)) == INVALID
        assert lib.mla_serving_call(op, words, len(words) - 8) == INVALID
    assert lib.mla_serving_call(CHECKED[-1][0] + 1, b"", 0) == INVALID


def test_status_words_have_names():
    for code, name in ((6, "MLA_ERR_NO_PAGES"), (7, "MLA_ERR_STALE_PLAN")):
        assert mla.mla_status_string(code).startswith(name)
