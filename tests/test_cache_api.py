"""CPU-only checks of the cache operators' C ABI and binding: exported symbols, the attention's plan,
refusals (every call here is rejected on the host before any CUDA call), and the 64-bit forms that the
GPU tests compare with, against torch's own conversion and softmax."""

import ctypes
import math
import os
import re

import pytest
import torch

import cache_reference as ref
import exact_top_selection_gb300 as etk
from exact_top_selection_gb300 import cache as binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GB300 = etk.DeviceInfo(152, 3, 3, 1, 2)


def test_header_declares_what_the_library_exports():
    with open(os.path.join(ROOT, "include", "exact_topk_cache.h")) as f:
        declared = set(re.findall(r"^int\s+(exact_topk\w*)\s*\(", f.read(), re.M))
    assert declared == set(etk.CACHE_SYMBOLS)
    lib = etk.library()
    for name in declared:
        assert hasattr(lib, name), name


def test_error_strings():
    for code in (-9, -10, -11):
        assert etk.error_string(code) != "unknown exact_topk status"
    assert etk.error_string(-12) == "unknown exact_topk status"


@pytest.mark.parametrize("tokens,seqs,single,q_heads,heads,columns,tile_tokens,tile_heads", [
    (64, 64, True, 32, 4, 8, 1, 8), (64, 64, True, 4, 4, 8, 1, 1), (3, 3, True, 12, 1, 16, 1, 12),
    (24, 8, False, 8, 2, 8, 2, 4), (4096, 1, False, 16, 2, 16, 2, 8), (100, 1, False, 1, 1, 8, 8, 1),
    (7, 7, True, 80, 2, 32, 1, 32), (100, 1, False, 6, 2, 8, 2, 3), (0, 1, False, 1, 1, 8, 8, 1),
    (64, 16, False, 16, 4, 8, 2, 4), (1024, 256, False, 16, 4, 16, 4, 4), (24, 3, False, 24, 1, 32, 1, 24),
])
def test_plan(tokens, seqs, single, q_heads, heads, columns, tile_tokens, tile_heads):
    p = etk.make_attention_plan(tokens, seqs, q_heads, heads, 128, 64, 100, 0, single, GB300)
    assert (p.columns, p.tile_tokens, p.tile_heads) == (columns, tile_tokens, tile_heads)
    assert p.tile_tokens * p.tile_heads <= p.columns and p.workers % 152 == 0
    assert p.counter_bytes >= 4 * p.workers and p.counter_bytes % 16 == 0
    assert p.workspace_bytes >= p.workers * 2 * p.columns * 128 * 4


def test_plan_refusals():
    good = dict(num_tokens=8, num_seqs=8, q_heads=8, kv_heads=2, head_dim=128, page_size=64, table_width=10,
                num_blocks=4, single_rows=True, device_info=GB300)
    etk.make_attention_plan(**good)
    for code, bad in ((-9, dict(head_dim=96)), (-9, dict(page_size=48)), (-9, dict(kv_heads=0)), (-10, dict(num_tokens=9)),
                      (-10, dict(num_seqs=0, num_tokens=0)), (-10, dict(num_seqs=4097, num_tokens=4097)), (-10, dict(table_width=0)),
                      (-10, dict(table_width=65537)), (-10, dict(num_tokens=-1)), (-10, dict(table_width=1 << 25)),
                      (-11, dict(q_heads=7)), (-11, dict(q_heads=0)), (-3, dict(num_blocks=-1)), (-3, dict(num_blocks=16385))):
        with pytest.raises(etk.ExactTopKError) as e:
            etk.make_attention_plan(**{**good, **bad})
        assert e.value.code == code, bad
    etk.make_attention_plan(**{**good, "table_width": 65537, "num_blocks": 0})
    with pytest.raises(etk.ExactTopKError) as e:
        etk.make_attention_plan(**{**good, "table_width": 24577, "prompt": 1})
    assert e.value.code == -7


@pytest.mark.parametrize("tokens,seqs,q_heads,heads,blocks,width,prompt,expect", [
    (4096, 1, 16, 2, 32, 2048, -1, (16, 8)), (4096, 1, 16, 2, 0, 2048, -1, (16, 8)), (4096, 1, 16, 2, 32, 2048, 0, (0, 0)),
    (4096, 1, 16, 2, 32, 30000, -1, (0, 0)), (100, 1, 16, 2, 32, 2048, -1, (0, 0)), (100, 1, 16, 2, 32, 2048, 1, (16, 8)),
    (6400, 1, 2, 2, 0, 100, -1, (32, 1)), (4096, 4096, 16, 2, 0, 100, -1, (0, 0)), (2000, 1, 260, 1, 0, 100, -1, (1, 128)),
    (512, 64, 32, 4, 0, 100, -1, (0, 0)),
])
def test_plan_of_prompts(tokens, seqs, q_heads, heads, blocks, width, prompt, expect):
    p = etk.make_attention_plan(tokens, seqs, q_heads, heads, 128, 64, width, blocks, tokens == seqs, GB300, prompt)
    assert (p.prompt_tokens, p.prompt_heads) == expect
    group = q_heads // heads
    flags = tokens * heads * -(-group // p.prompt_heads) if expect[0] else 0
    assert p.workspace_bytes >= p.workers * 2 * p.columns * 130 * 4 + flags


def fake(i):
    return 0x100000 * i  # an address that no check may dereference


def structs():
    cache = binding._Cache(fake(1), fake(2), fake(3), fake(4), fake(5), 10, 2, 64, 128, 0, 0)
    batch = binding._Batch(fake(6), fake(7), None, 4, 3, 3)
    return cache, batch, binding._Rows(fake(8), 256, 128), binding._Rows(fake(9), 256, 128)


def test_c_entry_points_refuse_bad_arguments():
    lib = binding._lib()

    def calls(cache, batch, a, b, tokens=4):
        ref_ = ctypes.byref
        yield lib.exact_topk_cache_write(ref_(cache), ref_(batch), tokens, ref_(a), ref_(b), None)
        yield lib.exact_topk_cache_read(ref_(cache), ref_(batch), tokens, ref_(a), ref_(b), None)
        yield lib.exact_topk_block_scores(ref_(cache), ref_(batch), tokens, 8, ref_(a), 0, 0, fake(10), 3, fake(11), None, None)
        plan = etk.make_attention_plan(4, 4, 8, 2, 128, 64, 3, 0, True, GB300)
        plan.num_tokens = tokens
        yield lib.exact_topk_attention_run(ref_(plan), ref_(cache), ref_(batch), ref_(a), ref_(b), None, 1.0, fake(12),
                                           plan.counter_bytes, fake(13), plan.workspace_bytes, None)

    def check(code, which=range(4), tokens=4, **changes):
        cache, batch, a, b = structs()
        for name, value in changes.items():
            part, field = name.split("__")
            setattr({"cache": cache, "batch": batch, "a": a, "b": b}[part], field, value)
        got = list(calls(cache, batch, a, b, tokens))
        assert [got[i] for i in which] == [code] * len(list(which)), (changes, got)

    for field in ("k", "v", "k_scale", "v_scale"):
        check(-1, **{"cache__" + field: None})
    check(-1, which=[2], cache__key_bounds=None)
    check(-1, batch__page_table=None)
    check(-1, batch__kv_len=None)
    check(-1, a__data=None)
    check(-1, which=[0, 1, 3], b__data=None)
    for field, value in (("num_pages", 0), ("kv_heads", 0), ("kv_heads", 1025), ("page_size", 8), ("head_dim", 32), ("type", 2)):
        check(-9, **{"cache__" + field: value})
    for field, value in (("num_seqs", 0), ("num_seqs", 5000), ("table_width", 0), ("table_pitch", 2), ("table_width", 1 << 26)):
        check(-10, **{"batch__" + field: value})
    check(-10, tokens=5)  # without q_start: one row each
    check(-10, tokens=-1)
    for name in ("cache__k", "cache__v", "cache__key_bounds", "a__data"):
        check(-6, **{name: fake(1) + 8})
    check(-6, cache__k_scale=fake(3) + 2)
    check(-6, batch__kv_len=fake(7) + 1)
    check(-6, a__token_stride=257)
    check(-6, a__head_stride=4)
    for i, lib_call in enumerate(("exact_topk_cache_write", "exact_topk_cache_read")):
        cache, batch, a, b = structs()
        f = getattr(lib, lib_call)
        assert f(None, ctypes.byref(batch), 4, ctypes.byref(a), ctypes.byref(b), None) == -1
        assert f(ctypes.byref(cache), None, 4, ctypes.byref(a), ctypes.byref(b), None) == -1
        assert f(ctypes.byref(cache), ctypes.byref(batch), 4, None, ctypes.byref(b), None) == -1


def test_scores_refuse_bad_arguments():
    lib = binding._lib()
    cache, batch, a, _ = structs()

    def call(q_heads=8, first=0, last=0, scores=fake(10), pitch=3, ke=fake(11), live=None):
        return lib.exact_topk_block_scores(ctypes.byref(cache), ctypes.byref(batch), 4, q_heads, ctypes.byref(a), first, last,
                                           scores, pitch, ke, live, None)

    assert call(scores=None) == -1 and call(ke=None) == -1
    assert call(q_heads=7) == -11 and call(q_heads=0) == -11
    assert call(first=-1) == -2 and call(last=-1) == -2 and call(pitch=2) == -2
    assert call(scores=fake(10) + 2) == -6 and call(ke=fake(11) + 2) == -6 and call(live=fake(12) + 1) == -6


def test_attention_refuses_bad_plans_and_buffers():
    lib = binding._lib()
    cache, batch, a, b = structs()

    def call(blocks=None, scale=1.0, counters=fake(12), less=0, workspace=fake(13), less_work=0, num_blocks=0, **fields):
        plan = etk.make_attention_plan(4, 4, 8, 2, 128, 64, 3, num_blocks, True, GB300)
        for name, value in fields.items():
            setattr(plan, name, value)
        return lib.exact_topk_attention_run(ctypes.byref(plan), ctypes.byref(cache), ctypes.byref(batch), ctypes.byref(a),
                                            ctypes.byref(b), blocks, scale, counters, plan.counter_bytes - less, workspace,
                                            plan.workspace_bytes - less_work, None)

    assert call(counters=None) == -1 and call(workspace=None) == -1 and call(num_blocks=2) == -1
    assert call(less=16) == -4 and call(less_work=4) == -5
    assert call(counters=fake(12) + 8) == -6 and call(workspace=fake(13) + 8) == -6
    assert call(num_blocks=2, blocks=fake(14) + 2) == -6
    assert call(blocks=fake(14)) == -7
    for bad in (dict(scale=math.inf), dict(scale=math.nan), dict(scale=3e38), dict(scale=-3e38), dict(kv_heads=1), dict(head_dim=64), dict(page_size=32), dict(table_width=4),
                dict(num_seqs=3), dict(columns=24), dict(tile_tokens=0), dict(tile_tokens=9), dict(tile_heads=0), dict(tile_heads=5),
                dict(tile_tokens=3), dict(prompt_tokens=33, prompt_heads=1), dict(prompt_tokens=-1),
                dict(prompt_tokens=1, prompt_heads=0), dict(prompt_tokens=1, prompt_heads=3), dict(workers=609), dict(workers=0), dict(workers=1 << 20), dict(min_units=0)):
        assert call(**bad) == -7, bad
    # a plan whose sizes were made smaller by hand does not get past the buffers' checks
    assert call(counter_bytes=16) == -4 and call(workspace_bytes=16) == -5
    assert call(prompt_tokens=8, prompt_heads=4) == -5  # no room for the marks
    assert call(q_heads=9) == -11


def test_binding_refuses_tensors_on_the_cpu_and_of_wrong_types():
    k = torch.zeros(2, 1, 16, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    scale = torch.ones(2, 1)
    bounds = torch.zeros(2, 1, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        etk.KVCache(k, k, scale, scale, bounds)  # not on a CUDA device
    with pytest.raises(TypeError):
        etk.KVCache(k, k, scale, scale, bounds.float())
    with pytest.raises(ValueError):
        etk.KVCache(k[:, :, :8], k[:, :, :8], scale, scale, bounds)
    table = torch.zeros(2, 3, dtype=torch.int32)
    lens = torch.zeros(2, dtype=torch.int32)
    etk.SequenceBatch(table, lens)
    for bad in ((table.long(), lens, None), (table, lens.long(), None), (table[0], lens, None), (table, lens[:1], None),
                (table, lens, lens), (table.t(), lens, None), (table[:, :0], lens, None)):
        with pytest.raises((TypeError, ValueError)):
            etk.SequenceBatch(*bad)


def test_outputs_that_overlap_are_refused():
    x, apart = torch.zeros(4 * 64 * 4, dtype=torch.bfloat16), torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    binding._written(x.view(4, 4, 64), "out", apart)
    binding._written(x.as_strided((4, 4, 64), (64, 256, 1)), "out", apart)
    for size, stride in (((4, 4, 64), (0, 64, 1)), ((4, 4, 64), (64, 64, 1)), ((4, 2, 64), (96, 64, 1)), ((4, 2, 64), (64, 32, 1))):
        with pytest.raises(ValueError):
            binding._written(x.as_strided(size, stride), "out", apart)
    with pytest.raises(ValueError):
        binding._written(x.view(4, 4, 64), "out", x.view(4, 4, 64)[1:])
    y = x.view(2, 2, 4, 64)
    binding._written(y[0], "out", y[1])


# ---- the 64-bit forms ----

def test_reference_codes_are_torchs_conversion():
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    fine = every[every.isfinite()]
    between = torch.cat([fine, (fine[:, None] + fine[None]).flatten() / 2, torch.randn(5000, dtype=torch.float64) * 50])
    between = between[between.abs() <= 448].float()
    assert torch.equal(ref.e4m3(between.double()), between.to(torch.float8_e4m3fn).double())
    assert ref.e4m3(torch.tensor([math.inf, math.nan], dtype=torch.float64)).isnan().all()


def test_reference_attention_is_softmax():
    lens, new = [40, 7], [3, 2]
    tensors, batch = ref.make(1, lens, new, 2, 16, 64, torch.float16)
    q = ref.rows(2, 5, 4, 64, torch.float16)
    out, tol = ref.attention(ref.Cache(*tensors), batch, q, None, 0.125, 0.0)
    k, v = tensors[0].double() * tensors[2].double()[..., None, None], tensors[1].double() * tensors[3].double()[..., None, None]
    t, h, pos = 1, 3, 38
    rows = [(int(batch[0][0, p // 16]), p % 16) for p in range(pos + 1)]
    kk, vv = (torch.stack([x[a, h // 2, o] for a, o in rows]) for x in (k, v))
    want = torch.nn.functional.scaled_dot_product_attention(q[t, h].double()[None], kk, vv, scale=0.125)[0]
    assert torch.allclose(out[t, h], want, rtol=1e-12) and (tol[t, h] < 0.02 * vv.abs().max()).all()


def test_reference_scores_bound_the_products():
    lens, new = [40], [4]
    tensors, batch = ref.make(3, lens, new, 1, 16, 64, torch.bfloat16, poison=False)
    cache = ref.Cache(*tensors)
    k = ref.rows(4, 40, 1, 64, torch.bfloat16)
    ref.write(cache, (batch[0], batch[1], torch.tensor([0, 40])), k, k)
    q = ref.rows(5, 4, 2, 64, torch.bfloat16)
    got, ke, _ = ref.scores(cache, batch, q, 0, 0, 0.0)
    dots = torch.einsum("tgd,pd->tgp", q.double(), k[:, 0].double()).amax(1)
    for t in range(4):
        for j in range(int(ke[t])):
            assert got[t, j] >= dots[t, j * 16:min(40, (j + 1) * 16)].max() - 1e-12
