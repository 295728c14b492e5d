"""The 4-bit cache against its 64-bit definitions (tests/serving_reference.py): writing, reading, page scores, attention over
the whole cache and over listed pages, by the kernel for decoding and by the one for prompts.

Everything that an operator must not read holds NaN (scales behind a sequence's end, pages of no sequence, rows of no
sequence); everything that it must not write holds a mark that is looked for."""

import math

import pytest
import torch

import cache_reference as ref
import exact_top_selection_gb300 as etk
import serving_reference as srv
from exact_top_selection_gb300 import cache as binding

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16
MARK = -7.0


def device_cache(tensors, k_unit=1.0, v_unit=1.0):
    return etk.KVCache4(*(t.cuda() for t in tensors), k_unit, v_unit)


def device_batch(batch, single=False):
    table, kv_len, q_start = (t.cuda() for t in batch)
    return etk.SequenceBatch(table, kv_len, None if single else q_start)


def rows_to_device(x, strided):
    """Rows on the device; strided: a slice of a wider projection, the rest of it NaN."""
    if not strided:
        return x.cuda()
    T, H, D = x.shape
    wide = torch.full((T, 2 * H + 1, D + 24), math.nan, dtype=x.dtype, device="cuda")
    wide[:, 1:2 * H:2, 8:8 + D] = x.cuda()
    return wide[:, 1:2 * H:2, 8:8 + D]


def same(a, b):
    a, b = a.detach().cpu().double(), b.detach().cpu().double()
    return a.shape == b.shape and bool(((a == b) | (a.isnan() & b.isnan())).all())


def check_cache(cache, plain):
    assert torch.equal(cache.k_scale.view(torch.uint8).cpu(), plain.k_codes)
    assert torch.equal(cache.v_scale.view(torch.uint8).cpu(), plain.v_codes)
    assert same(srv.values(cache.k.cpu(), cache.k_scale.cpu()), plain.k)
    assert same(srv.values(cache.v.cpu(), cache.v_scale.cpu()), plain.v)
    assert same(cache.key_bounds, plain.bounds)


# ---- write and read ----

WRITES = [([1], [1]), ([64], [64]), ([65], [1]), ([200], [200]), ([17], [3]), ([130, 1, 16, 64], [1, 1, 1, 1]),
          ([300, 5, 40, 129], [130, 0, 40, 64]), ([3, 0, 70], [5, 2, 70])]


@pytest.mark.parametrize("lens,new", WRITES)
@pytest.mark.parametrize("page,dim,heads,dtype", [(16, 64, 3, BF16), (32, 128, 1, FP16), (64, 128, 2, BF16),
                                                  (128, 64, 2, FP16), (16, 128, 5, FP16), (128, 128, 1, BF16),
                                                  (32, 64, 2, BF16), (64, 64, 1, FP16)])
def test_write_and_read(lens, new, page, dim, heads, dtype):
    tensors, batch = srv.make(1, lens, new, heads, page, dim, dtype, poison=False)
    T = sum(new) + 3  # rows behind the last sequence
    k, v = ref.rows(2, T, heads, dim, dtype, 3.0), ref.rows(3, T, heads, dim, dtype, 0.01)
    k[sum(new):], v[sum(new):] = math.nan, math.nan
    units = 2.0 ** (page // 32 - 1), 2.0 ** -(dim // 16)
    plain = srv.Cache4(*tensors, *units)
    srv.write(plain, batch, k, v)
    cache, b = device_cache(tensors, *units), device_batch(batch)
    strided = len(lens) % 2 == 0
    etk.cache_write(cache, b, rows_to_device(k, strided), rows_to_device(v, not strided))
    check_cache(cache, plain)
    out = tuple(torch.full((T, heads, dim), MARK, dtype=dtype, device="cuda") for _ in range(2))
    etk.cache_read(cache, b, out=out)
    for got, want in zip(out, ref.read(plain, batch, T, MARK)):
        assert same(got, want)
    wide = torch.full((2, T, heads + 1, dim + 8), MARK, dtype=dtype, device="cuda")
    etk.cache_read(cache, b, out=(wide[0, :, 1:, :dim], wide[1, :, :heads, 8:]))
    assert same(wide[0, :, 1:, :dim], out[0]) and same(wide[1, :, :heads, 8:], out[1])
    assert (wide[0, :, 0] == MARK).all() and (wide[0, ..., dim:] == MARK).all() and (wide[1, :, heads] == MARK).all()


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("unit", [1.0, 2.0 ** -40, 2.0 ** 40, 2.0 ** -7])
def test_write_of_extreme_rows(dtype, unit):
    """Infinities, NaN, zeros, subnormals, the type's largest number, and every border between codes and between scales."""
    page, dim, heads = 16, 64, 2
    info = torch.finfo(dtype)
    borders = (srv.GRID[1:] + srv.GRID[:-1]) / 2
    scale_borders = (srv.SCALES[1:] + srv.SCALES[:-1]) / 2 * 6
    special = [0.0, -0.0, math.inf, -math.inf, math.nan, float(info.max), -float(info.max), float(info.tiny), float(info.smallest_normal) / 4]
    rows = [torch.full((16,), x, dtype=torch.float64) for x in special]
    for x in special:
        rows.append(torch.linspace(-2, 2, 16, dtype=torch.float64))
        rows[-1][3] = x
    for s in srv.SCALES[1:]:  # a group that has this scale, with all borders between codes
        rows.append(torch.cat([torch.tensor([6.0]), borders, -borders, torch.tensor([0.0])]).double() * s)
        rows.append(rows[-1] * (1 + 2.0 ** -7))
    for s in scale_borders:  # groups whose largest number is 6 times a border between two scales
        rows.append(torch.linspace(0, 1, 16, dtype=torch.float64) * s)
        rows.append(-rows[-1] * (1 - 2.0 ** -8))
    x = torch.cat(rows)
    x = torch.where(torch.isfinite(x) & (x.abs() < float(info.max)), x * unit, x)
    x = torch.cat([x, torch.zeros(-len(x) % (2 * heads * dim))]).to(dtype).reshape(2, -1, heads, dim)
    lens = [x.shape[1]]
    tensors, batch = srv.make(6, lens, lens, heads, page, dim, dtype, poison=False)
    plain, cache = srv.Cache4(*tensors, unit, unit), device_cache(tensors, unit, unit)
    srv.write(plain, batch, x[0], x[1])
    etk.cache_write(cache, device_batch(batch), x[0].cuda(), x[1].cuda())
    check_cache(cache, plain)
    assert cache.key_bounds.isfinite().all()
    for got, want in zip(etk.cache_read(cache, device_batch(batch), num_tokens=lens[0]), ref.read(plain, batch, lens[0])):
        assert same(got, want)


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_every_number_of_a_type(dtype):
    """All 65536 bit patterns, in groups with one another."""
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dtype)
    x = torch.stack([x, x[torch.randperm(65536, generator=torch.Generator().manual_seed(3))]]).reshape(2, 512, 1, 128)
    tensors, batch = srv.make(7, [512], [512], 1, 64, 128, dtype, poison=False)
    plain, cache = srv.Cache4(*tensors), device_cache(tensors)
    srv.write(plain, batch, x[0], x[1])
    etk.cache_write(cache, device_batch(batch), x[0].cuda(), x[1].cuda())
    check_cache(cache, plain)


def test_every_page_of_a_long_batch():
    lens, new = [700, 3000, 64, 1111], [650, 2999, 1, 0]
    tensors, batch = srv.make(8, lens, new, 4, 64, 128, BF16, poison=False)
    T = sum(new)
    k, v = ref.rows(9, T, 4, 128, BF16, 2.0), ref.rows(10, T, 4, 128, BF16, 5.0)
    plain, cache = srv.Cache4(*tensors), device_cache(tensors)
    srv.write(plain, batch, k, v)
    etk.cache_write(cache, device_batch(batch), k.cuda(), v.cuda())
    check_cache(cache, plain)
    for x, y in zip(etk.cache_read(cache, device_batch(batch), num_tokens=T), ref.read(plain, batch, T)):
        assert same(x, y)


def test_scores_are_of_the_bounds():
    """As of an 8-bit cache with the same bounds: steps and prompts."""
    for lens, new in (([700, 3], [1, 1]), ([300, 5, 40, 129], [130, 0, 40, 2])):
        tensors, batch = srv.make(11, lens, new, 2, 16, 64, BF16)
        eight, _ = ref.make(11, lens, new, 2, 16, 64, BF16)
        q = ref.rows(12, sum(new), 16, 64, BF16).cuda()
        b = device_batch(batch)
        got, ke = etk.block_scores(device_cache(tensors), b, q, 1, 2, scores=torch.full((sum(new) * 2, b.table_width), MARK, device="cuda"))
        want, want_ke = etk.block_scores(etk.KVCache(*(t.cuda() for t in eight[:4]), tensors[4].cuda()), b, q, 1, 2,
                                         scores=torch.full((sum(new) * 2, b.table_width), MARK, device="cuda"))
        assert torch.equal(got, want) and torch.equal(ke, want_ke)


# ---- attention ----

def check_attention(tensors, batch, q, blocks=None, scale=None, single=False, strided=False, units=(1.0, 1.0), **overrides):
    T, QH, D = q.shape
    plain, cache = srv.Cache4(*tensors, *units), device_cache(tensors, *units)
    behind = 0 if single else 2
    rows = torch.cat([q, torch.full((behind, QH, D), math.nan, dtype=q.dtype)])
    lists = None if blocks is None else torch.cat([blocks, torch.zeros(behind * plain.heads, blocks.shape[1], dtype=torch.int32)])
    want, tol = ref.attention(plain, batch, rows, lists, 1 / math.sqrt(D) if scale is None else scale, MARK)
    b = device_batch(batch, single)
    attend = etk.CacheAttention(cache, b.num_seqs, T + behind, QH, b.table_width,
                                num_blocks=0 if blocks is None else blocks.shape[1], **overrides)
    out = rows_to_device(torch.full(rows.shape, MARK, dtype=q.dtype), strided)
    for _ in range(2):  # the second call finds the counters as the first left them
        attend(rows_to_device(rows, strided), b, blocks=None if blocks is None else lists.cuda(), out=out, scale=scale)
    assert not attend.counters.any()
    got = out.cpu().double()
    assert torch.equal(got.isnan(), want.isnan())
    fine = ~want.isnan()
    bad = ((got - want).abs() > tol) & fine
    assert not bad.any(), (bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), want[bad][:4].tolist(), tol[bad][:4].tolist())


SHAPES = [([1], [1]), ([0, 1, 2], [1, 1, 1]), ([700], [1]), ([3000, 16, 17, 64], [1, 1, 1, 1]),
          ([300, 5, 40, 129], [13, 0, 40, 2]), ([3, 0, 70], [5, 2, 9]), ([1500], [3])]
LAYOUTS = [(16, 64, 2, 8, BF16), (32, 128, 1, 1, FP16), (64, 128, 2, 3, BF16), (128, 64, 1, 5, FP16),
           (64, 128, 1, 16, BF16), (16, 128, 1, 12, FP16), (64, 64, 1, 40, BF16), (128, 128, 2, 4, BF16),
           (32, 64, 1, 20, FP16), (16, 64, 1, 9, FP16), (32, 128, 1, 33, BF16)]


def some_lists(seed, lens, rows, page, count=9):
    g = torch.Generator().manual_seed(seed)
    blocks = torch.randint(-1, max(1, -(-max(lens) // page)) + 1, (rows, count), generator=g, dtype=torch.int32)
    blocks[0] = -1
    if len(blocks) > 1:
        blocks[1] = 0
    blocks[-1, 0], blocks[-1, 1] = 2 ** 31 - 1, -2 ** 31
    return blocks


@pytest.mark.parametrize("lens,new", SHAPES)
@pytest.mark.parametrize("page,dim,heads,group,dtype", LAYOUTS)
def test_dense(lens, new, page, dim, heads, group, dtype):
    tensors, batch = srv.make(30, lens, new, heads, page, dim, dtype)
    q = ref.rows(31, sum(new), heads * group, dim, dtype, 3.0)
    check_attention(tensors, batch, q, single=all(n == 1 for n in new), strided=len(lens) % 2 == 1, units=(2.0, 2.0 ** -9))


@pytest.mark.parametrize("lens,new", SHAPES)
@pytest.mark.parametrize("page,dim,heads,group,dtype", LAYOUTS)
def test_listed_pages(lens, new, page, dim, heads, group, dtype):
    """Lists with -1, repeats, pages behind the token's own and out of the table, all-empty rows."""
    tensors, batch = srv.make(32, lens, new, heads, page, dim, dtype)
    q = ref.rows(33, sum(new), heads * group, dim, dtype, 3.0)
    check_attention(tensors, batch, q, some_lists(34, lens, sum(new) * heads, page), single=all(n == 1 for n in new), strided=len(lens) % 2 == 0)


PROMPTS = [([1], [1]), ([90, 0, 2], [40, 2, 2]), ([700, 64], [130, 17]), ([200, 5], [200, 9])]


@pytest.mark.parametrize("lens,new", PROMPTS)
@pytest.mark.parametrize("page,dim,heads,group,dtype", LAYOUTS + [(64, 128, 1, 130, BF16), (32, 64, 2, 7, FP16)])
@pytest.mark.parametrize("listed", [False, True])
def test_prompt(lens, new, page, dim, heads, group, dtype, listed):
    tensors, batch = srv.make(62, lens, new, heads, page, dim, dtype)
    q = ref.rows(63, sum(new), heads * group, dim, dtype, 3.0)
    blocks = some_lists(64, lens, sum(new) * heads, page) if listed else None
    check_attention(tensors, batch, q, blocks, strided=len(lens) % 2 == 0, prompt=1, units=(1.0, 2.0 ** 5))


@pytest.mark.parametrize("prompt", [0, 1])
def test_long_lists_and_long_caches_pass_the_pages_held_at_a_time(prompt):
    lens, new, page, heads = [16 * 1400 + 5], [2], 16, 1
    tensors, batch = srv.make(38, lens, new, heads, page, 64, BF16)
    g = torch.Generator().manual_seed(39)
    blocks = torch.stack([torch.randperm(1401, generator=g)[:1300] for _ in range(2)]).to(torch.int32)
    q = ref.rows(40, 2, 3, 64, BF16, 3.0)
    check_attention(tensors, batch, q, blocks, prompt=prompt)
    check_attention(tensors, batch, q, prompt=prompt)


@pytest.mark.parametrize("prompt", [0, 1])
@pytest.mark.parametrize("size,units", [(2.0 ** -9, (1.0, 1.0)), (200.0, (1.0, 2.0 ** -40)), (0.3, (2.0 ** -30, 2.0 ** 20)), (448.0, (2.0 ** 12, 1.0))])
def test_scales_and_units_of_any_size(prompt, size, units):
    """Scales from the smallest, which are below the type's normal numbers, to the largest."""
    lens, new = [500, 64], [2, 3]
    tensors, batch = srv.make(41, lens, new, 2, 32, 128, FP16 if units[1] == 1.0 and size < 1 else BF16, size=size)
    q = ref.rows(42, 5, 8, 128, tensors[4].dtype)
    check_attention(tensors, batch, q, units=units, scale=0.3 / size / units[0] / 16, prompt=prompt)


@pytest.mark.parametrize("prompt", [0, 1])
@pytest.mark.parametrize("size", [1e-30, 1e-3, 30.0, 3000.0])
def test_queries_of_any_size(prompt, size):
    lens, new = [300, 64], [2, 1]
    tensors, batch = srv.make(43, lens, new, 2, 32, 128, BF16)
    q = ref.rows(44, 3, 8, 128, BF16, 1.0) * size
    for scale in (min(1.0, 0.05 / size), -min(1.0, 0.05 / size), 0.0):
        check_attention(tensors, batch, q, scale=scale, prompt=prompt)


@pytest.mark.parametrize("prompt", [0, 1])
def test_peaked_scores_raise_the_maximum_late(prompt):
    """Keys that grow along the sequence, so that the running maximum moves all the time; then ones that shrink."""
    for sign in (1, -1):
        lens, new, page, dim = [2000], [2], 64, 64
        tensors, batch = srv.make(45, lens, new, 1, page, dim, FP16)
        grow = torch.exp2(torch.linspace(-7, 3, 32).round())
        for j in range(32):
            s = tensors[2].view(torch.uint8)[batch[0][0, j].long()]
            s[s != 0x7F] = grow[j if sign > 0 else 31 - j].to(torch.float8_e4m3fn).view(torch.uint8)
            tensors[2].view(torch.uint8)[batch[0][0, j].long()] = s
        check_attention(tensors, batch, ref.rows(46, 2, 4, dim, FP16, 2.0), prompt=prompt)


@pytest.mark.parametrize("page,dim,group", [(16, 64, 4), (64, 128, 4), (32, 128, 1), (64, 128, 2), (128, 64, 12)])
def test_nan_reaches_the_rows_that_see_it_and_no_other(page, dim, group):
    """NaN scales among the keys and values of tokens that only some rows of a tile see: by position and by list."""
    lens, new, heads = [page * 6 + 5], [7], 1
    tensors, batch = srv.make(47, lens, new, heads, page, dim, BF16)
    k, v = tensors[2].view(torch.uint8), tensors[3].view(torch.uint8)

    def put(codes, position, channel, code=0x7F):
        codes[batch[0][0, position // page].long(), 0, position % page, channel // 16] = code

    last = lens[0] - 1
    put(v, last, 3)                 # seen by the last row alone
    put(v, last - 2, dim - 1, 0xFF)  # by three
    put(k, last - 4, 0)             # by five
    q = ref.rows(48, 7, group, dim, BF16, 2.0)
    check_attention(tensors, batch, q)
    check_attention(tensors, batch, q, prompt=1)
    put(v, 2 * page + 1, 5)    # by those that list page 2
    put(k, 3 * page, 1)        # page 3
    blocks = torch.tensor([[0, 1, -1], [0, 2, 1], [1, 0, 5], [3, 0, 1], [0, 1, 2], [6, 0, 1], [4, 5, 0]], dtype=torch.int32)
    check_attention(tensors, batch, q, blocks)
    check_attention(tensors, batch, q, blocks, prompt=1)
    q[2], q[4, 0, 0] = math.nan, math.inf
    check_attention(tensors, batch, q, blocks)
    check_attention(tensors, batch, q, blocks, prompt=1)


@pytest.mark.parametrize("prompt", [0, 1])
@pytest.mark.parametrize("page,dim,group,dtype", [(64, 128, 4, BF16), (16, 128, 12, FP16), (16, 64, 3, BF16), (32, 64, 20, FP16)])
def test_infinite_queries_under_every_sign_of_the_scale(page, dim, group, dtype, prompt):
    """One key stands against all others in the infinite channel, so that a single score is +inf where the others are -inf, or the
    other way round, in the first step and in a late one; a scale of 0 makes NaN of each."""
    lens, new, heads = [page * 5 + 3], [3], 2
    for at in (1, page * 4 + 2):
        tensors, batch = srv.make(140, lens, new, heads, page, dim, dtype)
        codes = tensors[0]
        codes[..., 0] = codes[..., 0] & 0xF0 | 2  # channel 0: +1
        where = batch[0][0, at // page].long()
        codes[where, :, at % page, 0] |= 8
        q = ref.rows(141, 3, heads * group, dim, dtype)
        q[0, 0, 0], q[2, -1, 0], q[1, group, 0] = math.inf, -math.inf, math.inf
        for scale in (0.1, -0.1, 0.0):
            check_attention(tensors, batch, q, scale=scale, prompt=prompt)
            some = torch.tensor([[0, 1, 4, -1]], dtype=torch.int32).expand(3 * heads, 4).contiguous()
            check_attention(tensors, batch, q, some, scale=scale, prompt=prompt)


@pytest.mark.parametrize("prompt", [0, 1])
def test_absent_pages_are_not_seen(prompt):
    lens, new = [300, 100, 64], [3, 1, 1]
    tensors, batch = srv.make(49, lens, new, 2, 16, 64, BF16)
    batch[0][0, 3] = -1
    batch[0][0, 18] = 10 ** 6
    batch[0][1, :] = -5       # nothing at all
    check_attention(tensors, batch, ref.rows(50, 5, 8, 64, BF16, 2.0), prompt=prompt)
    plain, cache, b = srv.Cache4(*tensors), device_cache(tensors), device_batch(batch)
    k = ref.rows(51, 5, 2, 64, BF16)
    srv.write(plain, batch, k, k)
    etk.cache_write(cache, b, k.cuda(), k.cuda())
    check_cache(cache, plain)
    for x, y in zip(etk.cache_read(cache, b, num_tokens=5), ref.read(plain, batch, 5)):
        assert same(x, y)


def test_row_ranges_and_lengths_out_of_range_are_clamped():
    lens, new = [100, 64, 30], [2, 2, 2]
    tensors, batch = srv.make(52, lens, new, 1, 16, 64, BF16, poison=False)
    q = ref.rows(53, 6, 4, 64, BF16)
    for bad_len, bad_start in (([10 ** 6, -3, 2 ** 31 - 1], [0, 2, 4, 6]), ([100, 64, 30], [-5, 2, 4, 100]), ([100, 64, 30], [1, 3, 3, 5])):
        changed = (batch[0], torch.tensor(bad_len, dtype=torch.int32), torch.tensor(bad_start, dtype=torch.int32))
        cache, b = device_cache(tensors), device_batch(changed)
        want, tol = ref.attention(srv.Cache4(*tensors), changed, q, None, 0.125, MARK)
        for prompt in (0, 1):
            a = etk.CacheAttention(cache, 3, 6, 4, b.table_width, prompt=prompt)
            out = a(q.cuda(), b, out=torch.full_like(q, MARK, device="cuda")).cpu().double()
            assert ((out - want).abs() <= tol).all()
        k = ref.rows(54, 6, 1, 64, BF16)
        plain = srv.Cache4(*tensors)
        srv.write(plain, changed, k, k)
        etk.cache_write(cache, b, k.cuda(), k.cuda())
        check_cache(cache, plain)


def test_many_sequences():
    """More sequences than a CTA has threads, some without rows, some without tokens."""
    g = torch.Generator().manual_seed(55)
    lens = torch.randint(0, 70, (301,), generator=g).tolist()
    new = [min(n, int(x)) for n, x in zip(lens, torch.randint(0, 3, (301,), generator=g))]
    tensors, batch = srv.make(56, lens, new, 1, 16, 64, BF16)
    q = ref.rows(57, sum(new), 4, 64, BF16, 3.0)
    check_attention(tensors, batch, q)
    check_attention(tensors, batch, q, torch.randint(-1, 5, (sum(new), 3), generator=g, dtype=torch.int32))


def test_a_cache_whose_offsets_pass_32_bits():
    """Pages at the end of a cache of more than 2^32 numbers, and of more than 2^32 bytes of codes."""
    heads, page, dim = 8, 128, 128
    pages = (1 << 33) // (heads * page * dim) + 40
    cache = etk.KVCache4.allocate(pages, heads, page, dim, device="cuda")
    lens = [700, 260]
    table = torch.tensor([[pages - 1 - 2 * j - b for j in range(6)] for b in range(2)], dtype=torch.int32)
    kv_len = torch.tensor(lens, dtype=torch.int32)
    k, v = ref.rows(58, sum(lens), heads, dim, BF16), ref.rows(59, sum(lens), heads, dim, BF16)
    q_start = torch.tensor([0, 700, 960], dtype=torch.int32)
    etk.cache_write(cache, device_batch((table, kv_len, q_start)), k.cuda(), v.cuda())
    low = pages - 13
    part = srv.Cache4(*(t[low:] for t in (cache.k, cache.v, cache.k_scale, cache.v_scale, cache.key_bounds)))
    small = (table - low, kv_len, q_start)
    plain = srv.Cache4(*(torch.zeros_like(t[low:]) for t in (cache.k, cache.v, cache.k_scale, cache.v_scale, cache.key_bounds)))
    srv.write(plain, small, k, v)
    assert same(part.k, plain.k) and same(part.v, plain.v) and same(part.bounds, plain.bounds)
    for x, y in zip(etk.cache_read(cache, device_batch((table, kv_len, q_start)), num_tokens=960), ref.read(part, small, 960)):
        assert same(x, y)
    one = torch.tensor([0, 1, 2], dtype=torch.int32)
    q = ref.rows(60, 2, heads * 2, dim, BF16, 2.0)
    want, tol = ref.attention(part, (small[0], kv_len, one), q, None, 1 / math.sqrt(dim), 0.0)
    for prompt in (0, 1):
        a = etk.CacheAttention(cache, 2, 2, heads * 2, 6, prompt=prompt)
        assert ((a(q.cuda(), device_batch((table, kv_len, one))).cpu().double() - want).abs() <= tol).all()


@pytest.mark.parametrize("page,dim,heads,group,dtype", LAYOUTS[:5])
def test_a_prompt_whose_waits_run_out(page, dim, heads, group, dtype):
    """What the prompt's kernel gives up is left to the other one."""
    lens, new = [700, 64], [130, 17]
    tensors, batch = srv.make(65, lens, new, heads, page, dim, dtype)
    q = ref.rows(66, sum(new), heads * group, dim, dtype, 3.0)
    lib = binding._lib()
    try:
        for blocks in (None, some_lists(67, lens, sum(new) * heads, page)):
            assert lib.exact_topk_set_wait_limit(0) == 0
            check_attention(tensors, batch, q, blocks, prompt=1)
            assert lib.exact_topk_set_wait_limit(-1) == 0
            check_attention(tensors, batch, q, blocks, prompt=1)
    finally:
        assert lib.exact_topk_set_wait_limit(-1) == 0


@pytest.mark.parametrize("prompt", [0, 1])
def test_a_captured_call_replays_with_new_contents(prompt):
    heads, group, page, dim, B, width, T = 2, 8, 32, 128, 3, 30, 70
    tensors, batch = srv.make(85, [width * page] * B, [30, 20, 20], heads, page, dim, BF16, poison=False)
    cache, dev_batch = device_cache(tensors), device_batch(batch)
    q, out, listed_out = (torch.zeros(T, heads * group, dim, dtype=BF16, device="cuda") for _ in range(3))
    k, v, rk, rv = (torch.zeros(T, heads, dim, dtype=BF16, device="cuda") for _ in range(4))
    blocks = torch.zeros(T * heads, 5, dtype=torch.int32, device="cuda")
    whole = etk.CacheAttention(cache, B, T, heads * group, width, prompt=prompt)
    listed = etk.CacheAttention(cache, B, T, heads * group, width, num_blocks=5, prompt=prompt)

    def run():
        etk.cache_write(cache, dev_batch, k, v)
        etk.cache_read(cache, dev_batch, out=(rk, rv))
        whole(q, dev_batch, out=out)
        listed(q, dev_batch, blocks=blocks, out=listed_out)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        run()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        run()
    for rep, (lens, new) in enumerate((([960, 70, 31], [30, 39, 1]), ([33, 500, 900], [33, 0, 30]), ([0, 1, 960], [0, 1, 69]))):
        tensors, batch = srv.make(86 + rep, [width * page] * B, [0] * B, heads, page, dim, BF16, poison=False)
        start = [sum(new[:i]) for i in range(B + 1)]
        batch = (batch[0], torch.tensor(lens, dtype=torch.int32), torch.tensor(start, dtype=torch.int32))
        for mine, other in zip((cache.k, cache.v, cache.k_scale, cache.v_scale, cache.key_bounds), tensors):
            mine.copy_(other)
        for mine, other in zip((dev_batch.page_table, dev_batch.kv_len, dev_batch.q_start), batch):
            mine.copy_(other)
        hq, hk, hv = (ref.rows(s + rep, T, h, dim, BF16, 2.0) for s, h in ((89, heads * group), (93, heads), (97, heads)))
        lists = torch.randint(-1, width, (T * heads, 5), generator=torch.Generator().manual_seed(rep), dtype=torch.int32)
        q.copy_(hq), k.copy_(hk), v.copy_(hv), blocks.copy_(lists)
        for x in (out, listed_out, rk, rv):
            x.fill_(MARK)
        torch.cuda.synchronize()
        graph.replay()
        graph.replay()  # writing the same rows again changes nothing
        torch.cuda.synchronize()
        plain = srv.Cache4(*tensors)
        srv.write(plain, batch, hk, hv)
        check_cache(cache, plain)
        for x, y in zip((rk, rv), ref.read(plain, batch, T, MARK)):
            assert same(x, y)
        for got, which in ((out, None), (listed_out, lists)):
            want, tol = ref.attention(plain, batch, hq, which, 1 / math.sqrt(dim), MARK)
            assert ((got.cpu().double() - want).abs() <= tol).all()


def test_streams_and_objects_of_their_own():
    """Two streams at once, an object each; objects and a cache made behind other work and used on another stream."""
    lens, new = [4000, 100, 900], [1, 1, 1]
    tensors, batch = srv.make(100, lens, new, 2, 32, 64, BF16)
    cache, b = device_cache(tensors), device_batch(batch, single=True)
    q = ref.rows(101, 3, 8, 64, BF16, 3.0).cuda()
    want = etk.CacheAttention(cache, 3, 3, 8, b.table_width)(q, b)
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    objects = [etk.CacheAttention(cache, 3, 3, 8, b.table_width) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.empty_like(q) for _ in range(20)] for _ in range(2)]
    for i in range(20):
        for a, s, o in zip(objects, streams, outs):
            a(q, b, out=o[i], stream=s)
    torch.cuda.synchronize()
    for o in outs:
        for x in o:
            assert torch.equal(x, want)
    torch.cuda._sleep(20_000_000)
    fresh = etk.KVCache4.allocate(10, 2, 32, 64, device="cuda")
    k = ref.rows(102, 3, 2, 64, BF16).cuda()
    table = torch.tensor([[0], [1], [2]], dtype=torch.int32, device="cuda")
    one = etk.SequenceBatch(table, torch.ones(3, dtype=torch.int32, device="cuda"))
    torch.cuda.current_stream().synchronize()
    etk.cache_write(fresh, one, k, k, stream=streams[0])
    torch.cuda.synchronize()
    plain = srv.Cache4(*(torch.zeros_like(t) for t in (fresh.k, fresh.v, fresh.k_scale, fresh.v_scale, fresh.key_bounds)))
    srv.write(plain, (table.cpu(), torch.ones(3, dtype=torch.int32), None), k.cpu(), k.cpu())
    check_cache(fresh, plain)


def test_empty_calls_do_nothing():
    tensors, batch = srv.make(110, [30, 20], [0, 0], 1, 16, 64, BF16)
    cache, b = device_cache(tensors), device_batch(batch)
    empty = torch.empty(0, 1, 64, dtype=BF16, device="cuda")
    etk.cache_write(cache, b, empty, empty)
    assert etk.cache_read(cache, b, num_tokens=0)[0].shape[0] == 0
    assert etk.CacheAttention(cache, 2, 0, 4, b.table_width)(torch.empty(0, 4, 64, dtype=BF16, device="cuda"), b).shape[0] == 0
    some = torch.full((4, 1, 64), math.nan, dtype=BF16, device="cuda")  # rows, but of no sequence
    etk.cache_write(cache, b, some, some)
    assert torch.equal(cache.k.cpu(), tensors[0]) and torch.equal(cache.k_scale.view(torch.uint8).cpu(), tensors[2].view(torch.uint8))
    out = torch.full((4, 4, 64), MARK, dtype=BF16, device="cuda")
    etk.CacheAttention(cache, 2, 4, 4, b.table_width)(torch.full_like(out, math.nan), b, out=out)
    assert (out == MARK).all()


def far_rows(x, apart):
    """x's rows, `apart` numbers from one token to the next."""
    T, H, D = x.shape
    wide = torch.empty((T - 1) * apart + H * D, dtype=x.dtype, device="cuda").as_strided((T, H, D), (apart, D, 1))
    wide.copy_(x)
    return wide


@pytest.mark.parametrize("dim", [64, 128])
def test_rows_whose_offsets_pass_32_bits(dim):
    """Every row argument of a step with its last tokens more than 2^32 numbers behind its first."""
    T, heads, group, page, apart = 40, 2, 4, 16, 1 << 27
    tensors, batch = srv.make(130, [T + 30], [T], heads, page, dim, BF16, poison=False)
    plain, cache, b = srv.Cache4(*tensors), device_cache(tensors), device_batch(batch)
    near = [ref.rows(131 + i, T, h, dim, BF16, 2.0) for i, h in enumerate((heads * group, heads, heads))]
    q, k, v = (far_rows(x, apart) for x in near)
    rotary = etk.Rotary(dim, device="cuda")
    turned = rotary(near[0].cuda(), near[1].cuda(), batch=b)
    rotary(q, k, batch=b, out=(q, k))
    assert torch.equal(q, turned[0]) and torch.equal(k, turned[1])
    etk.cache_write(cache, b, k, v)
    srv.write(plain, batch, turned[1].cpu(), near[2])
    check_cache(cache, plain)
    scores = [etk.block_scores(cache, b, x, scores=torch.full((T * heads, b.table_width), MARK, device="cuda"))[0] for x in (q, turned[0])]
    assert torch.equal(*scores)
    want, tol = ref.attention(plain, batch, turned[0].cpu(), None, 1 / math.sqrt(dim), 0.0)
    out = far_rows(torch.zeros_like(near[0]), apart)
    for prompt in (0, 1):
        etk.CacheAttention(cache, 1, T, heads * group, b.table_width, prompt=prompt)(q, b, out=out.fill_(MARK))
        assert ((out.cpu().double() - want).abs() <= tol).all()
    for x, y in zip(etk.cache_read(cache, b, out=(k.fill_(MARK), v.fill_(MARK))), ref.read(plain, batch, T)):
        assert same(x, y)


# Two tiles of 128 rows share a CTA, more of them than SMs: 160, 160, 348, 156, 170 and 510 tiles; small groups over the whole
# cache alone.
@pytest.mark.parametrize("page,dim,heads,group,dtype", [(16, 64, 10, 8, BF16), (64, 128, 5, 16, FP16), (128, 64, 4, 40, BF16),
                                                        (32, 128, 6, 12, FP16), (64, 128, 10, 9, BF16), (16, 128, 1, 130, BF16),
                                                        (64, 128, 16, 2, BF16), (32, 64, 9, 5, FP16)])
@pytest.mark.parametrize("listed", [False, True])
def test_two_tiles_a_cta(page, dim, heads, group, dtype, listed):
    """Sequences that end in a tile's first tokens, in its second half and in a first tile alone; NaN scales; waits that run out."""
    lens, new = [330, 0, 200, 40, 700, 64], [150, 2, 90, 21, 1, 3]
    tensors, batch = srv.make(120, lens, new, heads, page, dim, dtype)
    T = sum(new)
    q = ref.rows(121, T, heads * group, dim, dtype, 3.0)
    blocks = some_lists(122, lens, T * heads, page, 12) if listed else None
    lib = binding._lib()
    for nan in (False, True):
        if nan:
            tensors[3].view(torch.uint8)[batch[0][0, 250 // page].long(), heads - 1, 250 % page, 1] = 0x7F
            tensors[2].view(torch.uint8)[batch[0][2, 150 // page].long(), 0, 150 % page, 3] = 0x7F
        units = (2.0, 2.0 ** -3)
        want, tol = srv.attention(srv.Cache4(*tensors, *units), batch, q, blocks, 1 / math.sqrt(dim), MARK)
        cache, b = device_cache(tensors, *units), device_batch(batch)
        attend = etk.CacheAttention(cache, len(lens), T, heads * group, b.table_width, 0 if blocks is None else 12, prompt=1)
        for limit in (-1, 0, -1):
            out = torch.full(q.shape, MARK, dtype=dtype, device="cuda")
            try:
                assert lib.exact_topk_set_wait_limit(limit) == 0
                attend(q.cuda(), b, blocks=None if blocks is None else blocks.cuda(), out=out)
            finally:
                assert lib.exact_topk_set_wait_limit(-1) == 0
            got = out.cpu().double()
            assert torch.equal(got.isnan(), want.isnan()) and want.isnan().any() == nan
            fine = ~want.isnan()
            bad = ((got - want).abs() > tol) & fine
            assert not bad.any(), (limit, bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), want[bad][:4].tolist())
            assert not attend.counters.any()


@pytest.mark.parametrize("page,dim,dtype", [(64, 128, BF16), (16, 64, FP16)])
def test_more_sequences_of_a_tile_than_sms(page, dim, dtype):
    """A tile a CTA: 100 sequences of up to 16 tokens, two heads; NaN scales; waits that run out."""
    g = torch.Generator().manual_seed(130)
    new = torch.randint(1, 17, (100,), generator=g).tolist()
    lens = [n + int(torch.randint(0, 200, (1,), generator=g)) for n in new]
    tensors, batch = srv.make(131, lens, new, 2, page, dim, dtype)
    tensors[3].view(torch.uint8)[batch[0][3, 0].long(), 1, 0, 1] = 0x7F
    q = ref.rows(132, sum(new), 16, dim, dtype, 3.0)
    want, tol = srv.attention(srv.Cache4(*tensors), batch, q, None, 1 / math.sqrt(dim), MARK)
    cache, b = device_cache(tensors), device_batch(batch)
    attend = etk.CacheAttention(cache, 100, sum(new), 16, b.table_width, prompt=1)
    lib = binding._lib()
    for limit in (-1, 0, -1):
        out = torch.full(q.shape, MARK, dtype=dtype, device="cuda")
        try:
            assert lib.exact_topk_set_wait_limit(limit) == 0
            attend(q.cuda(), b, out=out)
        finally:
            assert lib.exact_topk_set_wait_limit(-1) == 0
        got = out.cpu().double()
        assert torch.equal(got.isnan(), want.isnan()) and want.isnan().any()
        assert ((got - want).abs() <= tol)[~want.isnan()].all() and not attend.counters.any()


def test_two_tiles_a_cta_over_long_caches():
    """More parts of pages than are held at a time, running maxima that rise late, queries of a size that needs it."""
    lens, new, heads, group, page, dim = [16 * 150 + 5, 700], [200, 100], 10, 8, 16, 64
    tensors, batch = srv.make(125, lens, new, heads, page, dim, FP16)
    for j in range(150):
        s = tensors[2].view(torch.uint8)[batch[0][0, j].long()]
        s[s != 0x7F] = torch.tensor(2.0 ** (j // 15 - 6)).to(torch.float8_e4m3fn).view(torch.uint8)
        tensors[2].view(torch.uint8)[batch[0][0, j].long()] = s
    q = ref.rows(126, 300, heads * group, dim, FP16, 2.0)
    for blocks in (None, torch.stack([torch.randperm(151, generator=torch.Generator().manual_seed(i))[:140] for i in range(3000)]).to(torch.int32)):
        want, tol = srv.attention(srv.Cache4(*tensors), batch, q, blocks, 0.125, MARK)
        cache, b = device_cache(tensors), device_batch(batch)
        attend = etk.CacheAttention(cache, 2, 300, heads * group, b.table_width, 0 if blocks is None else 140, prompt=1)
        got = attend(q.cuda(), b, blocks=None if blocks is None else blocks.cuda()).cpu().double()
        assert ((got - want).abs() <= tol).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("width", [16384, 16385, 24576])
def test_prompts_over_lists_of_wide_tables(width, dim):
    """The widest tables of the kernel of two tiles a CTA and of the one of a tile, and their largest shared memory; the last pages are listed."""
    page, group, new = 16, 8, 20
    lens = [width * page - 3]
    tensors, batch = srv.make(150, lens, [new], 1, page, dim, BF16, width=width)
    g = torch.Generator().manual_seed(151)
    some = torch.randint(0, width, (40,), generator=g)  # neighbours share pages
    blocks = torch.stack([torch.cat([some[torch.randint(0, 40, (9,), generator=g)], torch.tensor([0, width - 1, width - 2 + i % 3])]) for i in range(new)])
    q = ref.rows(152, new, group, dim, BF16, 3.0)
    check_attention(tensors, batch, q, blocks.to(torch.int32), prompt=1)


def test_prompts_over_lists_of_wider_tables_are_refused():
    with pytest.raises(etk.ExactTopKError):
        etk.make_attention_plan(20, 1, 8, 1, 64, 16, 24577, 12, False, prompt=1, bits=4)
    assert etk.make_attention_plan(4096, 1, 16, 1, 64, 16, 24577, 12, False, bits=4).prompt_tokens == 0


@pytest.mark.parametrize("prompt", [0, 1])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("page,dim,group,dtype", [(64, 128, 4, BF16), (16, 128, 12, FP16), (16, 64, 3, BF16), (32, 64, 20, FP16)])
def test_a_query_with_an_infinity_gives_nan(page, dim, group, dtype, bits, prompt):
    """Every score of such a row is an infinity or NaN: also where all are -inf the weights are 0 / 0. Its neighbours are not touched, and
    a row that sees nothing gives zeros."""
    lens, new, heads = [page * 5 + 3, 1], [6, 2], 2
    if bits == 4:
        tensors, batch = srv.make(160, lens, new, heads, page, dim, dtype)
        tensors[0][..., 0] = tensors[0][..., 0] & 0xF0 | 2  # channel 0: +1
        cache = device_cache(tensors)
        plain = srv.Cache4(*tensors)
    else:
        tensors, batch = ref.make(160, lens, new, heads, page, dim, dtype)
        codes = tensors[0].view(torch.uint8)
        codes[..., 0] = torch.where(codes[..., 0] & 0x7F == 0x7F, codes[..., 0], 0x38)
        cache = etk.KVCache(*(t.cuda() for t in tensors))
        plain = ref.Cache(*tensors)
    q = ref.rows(161, 8, heads * group, dim, dtype)
    q[0, 0, 0], q[2, -1, 0], q[4, group, 0], q[6] = math.inf, -math.inf, -math.inf, math.inf  # row 6 has no token
    q[3, 1, 5], q[3, 1, 0] = math.inf, 3.0
    for scale in (0.1, -0.1, 0.0):
        for blocks in (None, torch.tensor([[0, 1, 4, -1]], dtype=torch.int32).expand(8 * heads, 4).contiguous()):
            want, tol = ref.attention(plain, batch, q, blocks, scale, MARK)
            b = device_batch(batch)
            attend = etk.CacheAttention(cache, 2, 8, heads * group, b.table_width, 0 if blocks is None else 4, prompt=prompt)
            got = attend(q.cuda(), b, blocks=None if blocks is None else blocks.cuda(), out=torch.full_like(q, MARK, device="cuda"), scale=scale).cpu().double()
            assert want.isnan().any() and torch.equal(got.isnan(), want.isnan())
            assert ((got - want).abs() <= tol)[~want.isnan()].all()
