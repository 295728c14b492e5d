"""CPU-only checks of the operators around a batch and of the 4-bit cache: refusals (every call here is rejected on the host before
any CUDA call), and the 64-bit forms that the GPU tests compare with."""

import ctypes
import math

import pytest
import torch

import cache_reference as ref
import exact_top_selection_gb300 as etk
import serving_reference as srv
from exact_top_selection_gb300 import batch as binding
from exact_top_selection_gb300 import cache as cache_binding

GB300 = etk.DeviceInfo(152, 3, 3, 1, 2)


def fake(i):
    return 0x100000 * i  # an address that no check may dereference


def test_cache4_entry_points_refuse_bad_arguments():
    lib, byref = cache_binding._lib(), ctypes.byref

    def check(code, which=range(4), tokens=4, scale=1.0, **changes):
        cache = cache_binding._Cache4(fake(1), fake(2), fake(3), fake(4), fake(5), 10, 2, 64, 128, 0, 1.0, 1.0)
        batch = cache_binding._Batch(fake(6), fake(7), None, 4, 3, 3)
        a, b = cache_binding._Rows(fake(8), 256, 128), cache_binding._Rows(fake(9), 256, 128)
        for name, value in changes.items():
            part, field = name.split("__")
            setattr({"cache": cache, "batch": batch, "a": a, "b": b}[part], field, value)
        plan = etk.make_attention_plan(4, 4, 8, 2, 128, 64, 3, 0, True, GB300)
        plan.num_tokens = tokens
        got = [lib.exact_topk_cache4_write(byref(cache), byref(batch), tokens, byref(a), byref(b), None) if 0 in which else 0,
               lib.exact_topk_cache4_read(byref(cache), byref(batch), tokens, byref(a), byref(b), None) if 1 in which else 0,
               lib.exact_topk_cache4_block_scores(byref(cache), byref(batch), tokens, 8, byref(a), 0, 0, fake(10), 3, fake(11), None, None)
               if 2 in which else 0,
               lib.exact_topk_cache4_attention_run(byref(plan), byref(cache), byref(batch), byref(a), byref(b), None, scale, fake(12),
                                                   plan.counter_bytes, fake(13), plan.workspace_bytes, None) if 3 in which else 0]
        assert [got[i] for i in which] == [code] * len(list(which)), (changes, got)

    for field in ("k", "v", "k_scale", "v_scale"):
        check(-1, **{"cache__" + field: None})
    check(-1, which=[2], cache__key_bounds=None)
    check(-1, batch__kv_len=None)
    check(-1, a__data=None)
    for field, value in (("num_pages", 0), ("kv_heads", 0), ("page_size", 8), ("head_dim", 96), ("type", 2), ("k_unit", 3.0), ("k_unit", 0.0),
                         ("v_unit", -1.0), ("v_unit", math.inf), ("v_unit", math.nan), ("k_unit", 2.0 ** 41), ("k_unit", 2.0 ** -41)):
        check(-9, **{"cache__" + field: value})
    check(-10, tokens=5)
    check(-10, batch__num_seqs=5000)
    for name in ("cache__k", "cache__v", "cache__key_bounds", "a__data"):
        check(-6, **{name: fake(1) + 8})
    for name in ("cache__k_scale", "cache__v_scale"):
        check(-6, **{name: fake(3) + 4})
    check(-6, a__token_stride=257)
    check(-7, which=[3], scale=math.inf)
    check(-7, which=[3], scale=1e30, cache__k_unit=2.0 ** 40)
    check(-7, which=[3], scale=math.nan)


@pytest.mark.parametrize("tokens,blocks,four,eight", [(300, 0, False, False), (320, 0, False, True), (383, 0, False, True), (384, 0, True, True),
                                                      (1023, 32, False, False), (1024, 32, True, True)])
def test_plans_of_prompts_by_bits(tokens, blocks, four, eight):
    for bits, prompt in ((4, four), (8, eight)):
        p = etk.make_attention_plan(tokens, 1, 16, 2, 128, 64, 2048, blocks, False, GB300, bits=bits)
        assert (p.prompt_tokens > 0) == prompt, bits
    with pytest.raises(ValueError):
        etk.make_attention_plan(tokens, 1, 16, 2, 128, 64, 2048, blocks, False, GB300, bits=16)
    with pytest.raises(etk.ExactTopKError):
        etk.make_attention_plan(tokens, 1, 15, 2, 128, 64, 2048, blocks, False, GB300, bits=4)


def test_rotary_refuses_bad_arguments():
    lib, byref = binding._lib(), ctypes.byref

    def call(positions=fake(2), tokens=4, q_heads=2, k_heads=1, batch=None, q=(fake(3), 256, 128), q_out=(fake(4), 256, 128),
             k=(fake(5), 128, 128), k_out=(fake(6), 128, 128), **fields):
        spec = binding._Spec(fake(1), 1.0, 128, 64, 0, 0)
        for name, value in fields.items():
            setattr(spec, name, value)
        rows = [None if r is None else byref(cache_binding._Rows(*r)) for r in (q, q_out, k, k_out)]
        b = None if batch is None else byref(batch)
        return lib.exact_topk_rotary(byref(spec), b, positions, tokens, q_heads, rows[0], rows[1], k_heads, rows[2], rows[3], 0, None)

    batch = cache_binding._Batch(None, fake(7), None, 4, 1, 1)
    assert lib.exact_topk_rotary(None, None, fake(2), 4, 1, None, None, 0, None, None, 0, None) == -1
    assert call(turns=None) == -1 and call(positions=None) == -1 and call(batch=batch) == -1  # one of the two
    assert call(q=None) == -1 and call(q_out=(None, 256, 128)) == -1 and call(k=None) == -1 and call(k_out=None) == -1
    assert call(tokens=-1) == -10 and call(tokens=(1 << 24) + 1) == -10 and call(positions=None, batch=batch, tokens=5) == -10
    for bad in (dict(num_seqs=0), dict(num_seqs=4097)):
        assert call(positions=None, batch=cache_binding._Batch(None, fake(7), fake(8), bad["num_seqs"], 1, 1)) == -10
    assert call(positions=None, batch=cache_binding._Batch(None, None, None, 4, 1, 1)) == -1
    assert call(positions=None, batch=cache_binding._Batch(None, fake(7) + 2, None, 4, 1, 1)) == -6
    for bad in (dict(head_dim=0), dict(head_dim=100), dict(head_dim=1032), dict(rotary_dim=0), dict(rotary_dim=3), dict(rotary_dim=130),
                dict(rotary_dim=-2), dict(head_dim=1024, rotary_dim=514), dict(type=2), dict(amplitude=math.inf), dict(amplitude=math.nan)):
        assert call(**bad) == -2, bad
    assert call(q_heads=0) == -11 and call(q_heads=65537) == -11 and call(k_heads=-1) == -11 and call(k_heads=65537) == -11
    assert call(q=(fake(3) + 8, 256, 128)) == -6 and call(k_out=(fake(3), 257, 128)) == -6 and call(q_out=(fake(3), 256, 4)) == -6
    assert call(turns=fake(1) + 4) == -6 and call(positions=fake(2) + 2) == -6
    assert call(tokens=0) == 0 and call(tokens=0, positions=None, k=None, k_heads=0, q=(None, 0, 0)) == 0


def test_rotary_refuses_bad_page_sizes():
    lib, byref = binding._lib(), ctypes.byref

    def call(page_size, width=1, positions=None):
        spec = binding._Spec(fake(1), 1.0, 128, 64, 0, 0, page_size)
        batch = cache_binding._Batch(None, fake(7), fake(8), 4, width, width)
        rows = byref(cache_binding._Rows(fake(3), 256, 128))
        return lib.exact_topk_rotary(byref(spec), None if positions else byref(batch), positions, 0, 2, rows, rows, 0, None, None, 0, None)

    for bad in (-1, 1, 8, 48, 256, 2 ** 30):
        assert call(bad) == -2 and call(bad, positions=fake(2)) == -2, bad
    assert call(16, 0) == -10 and call(16, -1) == -10 and call(128, (1 << 23) + 1) == -10 and call(16, 2 ** 31 - 1) == -10
    for good in ((0, 0), (0, 2 ** 31 - 1), (16, 1), (128, 1 << 23)):
        assert call(*good) == 0, good


def test_tables_refuse_bad_arguments():
    lib, byref = binding._lib(), ctypes.byref
    def call(change=fake(20), **fields):
        t = binding._Tables(*(fake(i) for i in range(1, 10)), 16, 8, 100, 4, 8, 10, 16)
        for name, value in fields.items():
            setattr(t, name, value)
        return lib.exact_topk_update_tables(byref(t), change, 0, None)

    assert lib.exact_topk_update_tables(None, fake(20), 0, None) == -1 and call(change=None) == -1
    for name in ("page_table", "kv_len", "q_start", "free_pages", "free_range", "counters"):
        assert call(**{name: None}) == -1, name
    for bad in (dict(page_size=8), dict(page_size=48), dict(num_pages=0), dict(num_pages=1 << 27)):
        assert call(**bad) == -9, bad
    for bad in (dict(num_seqs=0), dict(num_seqs=4097), dict(table_width=0), dict(table_width=9), dict(table_width=1 << 27, table_pitch=1 << 27),
                dict(max_tokens=-1), dict(max_tokens=(1 << 24) + 1)):
        assert call(**bad) == -10, bad
    assert call(counter_bytes=3) == -4
    for name in ("page_table", "kv_len", "q_start", "applied", "slots", "positions", "free_pages", "free_range", "counters"):
        assert call(**{name: fake(3) + 2}) == -6, name
    assert call(change=fake(20) + 1) == -6


def test_bindings_refuse_wrong_tensors_and_numbers():
    k = torch.zeros(2, 1, 16, 32, dtype=torch.uint8)
    scale = torch.zeros(2, 1, 16, 4, dtype=torch.uint8).view(torch.float8_e4m3fn)
    bounds = torch.zeros(2, 1, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        etk.KVCache4(k, k, scale, scale, bounds)
    with pytest.raises(TypeError):
        etk.KVCache4(k, k, scale, scale, bounds.float())
    for bad in (k[:, :, :8], k[..., :24], k[0]):
        with pytest.raises(ValueError):
            etk.KVCache4(bad, bad, scale, scale, bounds)
    for unit in (3.0, 0.0, -1.0, math.inf, math.nan, 2.0 ** 41):
        with pytest.raises(ValueError, match="unit"):
            etk.KVCache4(k, k, scale, scale, bounds, k_unit=unit)
    for args in (dict(head_dim=100), dict(head_dim=0), dict(head_dim=2048), dict(head_dim=64, rotary_dim=65), dict(head_dim=64, rotary_dim=66),
                 dict(head_dim=64, rotary_dim=0), dict(head_dim=64, base=0.0), dict(head_dim=64, factor=-1.0), dict(head_dim=64, factor=math.inf),
                 dict(head_dim=64, original_length=0), dict(head_dim=64, original_length=5, slow=2.0, fast=2.0), dict(head_dim=64, frequencies=[1.0]),
                 dict(head_dim=64, frequencies=[math.nan] * 32), dict(head_dim=64, amplitude=math.inf), dict(head_dim=64, device="cpu")):
        with pytest.raises(ValueError):
            etk.Rotary(**{"device": "cuda:0", **args})
    table, lens, free = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(9, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        etk.PageTables(table, lens, free, lens, 16, 10)
    with pytest.raises(ValueError):
        etk.PageTables(table, lens, free, lens, 24, 10)
    for most in (-1, (1 << 24) + 1):
        with pytest.raises(ValueError):
            etk.PageTables(table, lens, free, lens, 16, most)


def test_rows_that_interleave_are_apart():
    x = torch.zeros(6, 10, 64, dtype=torch.bfloat16)
    for a, b in ((x[:, :4], x[:, 4:6]), (x[:, 4:6], x[:, :4]), (x[:2], x[2:]), (x[..., :32], x[..., 32:]), (x[1:, 2:4], x[:-1, 8:]), (x[:0], x),
                 (x[:, ::2], x[:, 1::2])):
        binding._apart(a, b, "out")
    for a, b in ((x[:, :4], x[:, 3:6]), (x, x), (x[1:, :4], x[:-1, 2:3]), (x[:, 8:], x.view(30, 2, 64)[:6]), (x[..., :40], x[..., 32:])):
        with pytest.raises(ValueError):
            binding._apart(a, b, "out")


def test_rows_of_one_token_or_head_that_interleave_are_apart():
    """Heads of one projection in turn ([tokens, heads, 3, dim]) and channels side by side, by tokens and by heads, one of either among them."""
    for tokens in (1, 2, 5):
        for heads in (1, 2, 4):
            x = torch.zeros(tokens, heads, 3, 64, dtype=torch.bfloat16)
            for i, j in ((0, 1), (1, 0), (0, 2), (2, 1)):
                binding._apart(x[:, :, i], x[:, :, j], "out")
            wide = torch.zeros(tokens, heads, 128, dtype=torch.bfloat16)
            binding._apart(wide[..., :64], wide[..., 64:], "out")
            binding._apart(wide[..., 64:], wide[..., :64], "out")
            rows = torch.zeros(tokens, 2 * heads + 1, 64, dtype=torch.bfloat16)
            binding._apart(rows[:, :2 * heads], rows[:, 2 * heads:], "out")
            binding._apart(rows[:, 2 * heads:], rows[:, :2 * heads], "out")
            for a, b in ((x[:, :, 1], x[:, :, 1]), (wide[..., :72], wide[..., 64:]), (wide[..., 64:], wide[..., :72]), (rows[:, :heads + 1], rows[:, heads:])):
                with pytest.raises(ValueError):
                    binding._apart(a, b, "out")
    x = torch.zeros(1, 9, 64, dtype=torch.bfloat16)  # a head each of one array between those of the other, and one beside them
    binding._apart(x[:, ::3], x[:, 1::3], "out")
    binding._apart(x[:, ::3], x[:, 4:5], "out")
    for a, b in ((x[:, ::3], x[:, 1:]), (x[:, ::3], x[:, 3:4]), (x[:, ::2], x[:, 1::3])):
        with pytest.raises(ValueError):
            binding._apart(a, b, "out")


def test_rows_that_are_taken_for_apart_share_no_element():
    """Random slices of one buffer: where the check passes, no element is in both."""
    g = torch.Generator().manual_seed(1)

    def pick(lo, hi):
        return int(torch.randint(lo, hi + 1, (1,), generator=g))

    passed = 0
    for _ in range(4000):
        x = torch.arange(pick(1, 4) * 240, dtype=torch.int32)
        both = []
        for _ in range(2):
            shape = pick(1, 3), pick(1, 3), pick(1, 3) * 4
            strides = pick(0, 12) * 8, pick(0, 12) * 8, 1
            most = sum((n - 1) * s for n, s in zip(shape, strides)) + 1
            both.append(x.as_strided(shape, strides, pick(0, (x.numel() - most) // 4) * 4) if most <= x.numel() else x.view(-1, 3, 80)[:, :1])
        try:
            binding._apart(*both, "out")
        except ValueError:
            continue
        passed += 1
        assert not set(both[0].flatten().tolist()) & set(both[1].flatten().tolist())
    assert passed > 1000


# ---- the 64-bit forms ----

def test_reference_values_and_rounding():
    every = torch.arange(256, dtype=torch.uint8)[:, None].expand(256, 8)
    x = srv.values(every, torch.ones(256, 1).to(torch.float8_e4m3fn))
    assert x[0x31, 0] == 0.5 and x[0x31, 1] == 1.5 and x[0xF9, 0] == -0.5 and x[0xF9, 15] == -6.0
    assert srv.SCALES[1] == 2.0 ** -9 and srv.SCALES[-1] == 448 and (srv.SCALES.diff() > 0).all()
    a = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.26, 4.99, 100.0], dtype=torch.float64)
    assert srv.GRID[srv.nearest(a, srv.GRID)].tolist() == [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 0.5, 4.0, 6.0]
    near = torch.rand(4000, dtype=torch.float64, generator=torch.Generator().manual_seed(1)) * 448
    near = torch.cat([near, (srv.SCALES[1:] + srv.SCALES[:-1]) / 2]).float()
    assert torch.equal(srv.SCALES[srv.nearest(near.double(), srv.SCALES)], near.to(torch.float8_e4m3fn).double())


def test_reference_quantises_within_half_a_step():
    x = ref.rows(1, 50, 2, 64, torch.bfloat16, 5.0).double()
    for unit in (1.0, 2.0 ** -5):
        code, value = srv.quantise(x, unit)
        scale = srv.SCALES[code.long()][..., None]
        off = (value * unit - x).abs().unflatten(-1, (-1, 16)) / (scale * unit)
        top = x.abs().unflatten(-1, (-1, 16)) / (scale * unit)
        # half a step of the codes: 1 above 4, and what the scale's own rounding (2^-4 of it) cuts off above 6
        assert (off <= torch.where(top < 2, 0.25, torch.where(top < 4, 0.5, 1.0)) + 1e-12).all() and (top <= 6 * (1 + 2.0 ** -3)).all()
    for bad in (math.inf, math.nan):
        x[0, 0, 3] = bad
        code, value = srv.quantise(x, 1.0)
        assert code[0, 0, 0] == 0x7F and value[0, 0, :16].isnan().all() and value[0, 0, 16:].isfinite().all()


def test_reference_tables_hand_out_each_page_once():
    t = srv.Tables(torch.full((2, 4), -1), torch.zeros(2, dtype=torch.int32), torch.arange(6), torch.tensor([0, 6]), 16, 100)
    t.update([17, 1])
    assert t.table == [[0, 1, -1, -1], [2, -1, -1, -1]] and t.slots[:18] == list(range(17)) + [32] and t.range == [3, 3]
    t.update([-17, 40])
    assert t.table[1] == [2, 3, 4, -1] and t.range == [5, 3] and t.ring == [0, 1, 2, 3, 4, 5] and t.applied == [-17, 40]
    t.update([33, 20])
    assert t.table[0][:3] == [5, 0, 1] and t.kv_len == [33, 41] and t.applied == [33, 0]


def test_reference_rotary_keeps_lengths():
    x = ref.rows(2, 3, 2, 64, torch.float16)
    got, tol = srv.rotary(x, [0, 7, 10 ** 6], [0.5 ** i for i in range(32)], 1.0, False, 0.0)
    assert torch.equal(got[0], x[0].double()) and torch.allclose(got.norm(dim=-1), x.double().norm(dim=-1), rtol=1e-12)
    back, _ = srv.rotary(got.half(), [0, 7, 10 ** 6], [0.5 ** i for i in range(32)], 1.0, False, 0.0, inverse=True)
    assert ((back - x.double()).abs() <= 4 * 2.0 ** -11 * (1 + x.double().abs().amax())).all()


def test_reference_attention_of_many_rows_is_the_other_one():
    lens, new = [40, 7, 90], [3, 9, 20]
    tensors, batch = srv.make(1, lens, new, 2, 16, 64, torch.float16)
    tensors[3].view(torch.uint8)[batch[0][2, 1].long(), 0, 5, 2] = 0x7F
    batch[0][2, 0] = -1
    q = ref.rows(2, 34, 4, 64, torch.float16)
    blocks = torch.randint(-1, 7, (68, 4), generator=torch.Generator().manual_seed(3), dtype=torch.int32)
    for lists in (None, blocks):
        want, tol = ref.attention(srv.Cache4(*tensors), batch, q, lists, 0.125, -7.0)
        got, got_tol = srv.attention(srv.Cache4(*tensors), batch, q, lists, 0.125, -7.0)
        assert torch.allclose(got, want, rtol=1e-12, equal_nan=True) and torch.equal(got.isnan(), want.isnan()) and want.isnan().any()
        fine = ~want.isnan()
        assert torch.allclose(got_tol[fine], tol[fine], rtol=1e-9)
