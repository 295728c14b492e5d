"""The cache operators against their 64-bit definitions (tests/cache_reference.py): writing, reading,
page scores, attention over the whole cache and over listed pages, and the step that runs them together.

Everything that an operator must not read holds NaN (codes behind a sequence's end, pages of no
sequence, rows of no sequence); everything that it must not write holds a mark that is looked for."""

import math

import pytest
import torch

import cache_reference as ref
import exact_top_selection_gb300 as etk

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16
MARK = -7.0


def device_cache(tensors):
    return etk.KVCache(*(t.cuda() for t in tensors))


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


# ---- write and read ----

WRITES = [
    # lens, new
    ([1], [1]), ([64], [64]), ([65], [1]), ([200], [200]), ([17], [3]), ([130, 1, 16, 64], [1, 1, 1, 1]),
    ([300, 5, 40, 129], [130, 0, 40, 64]), ([3, 0, 70], [5, 2, 70]),
]


@pytest.mark.parametrize("lens,new", WRITES)
@pytest.mark.parametrize("page,dim,heads,dtype", [(16, 64, 3, BF16), (32, 128, 1, FP16), (64, 128, 2, BF16),
                                                  (128, 64, 2, FP16), (16, 128, 5, FP16), (128, 128, 1, BF16),
                                                  (32, 64, 2, BF16), (64, 64, 1, FP16)])
def test_write_and_read(lens, new, page, dim, heads, dtype):
    tensors, batch = ref.make(1, lens, new, heads, page, dim, dtype, poison=False)
    T = sum(new) + 3  # rows behind the last sequence
    k, v = ref.rows(2, T, heads, dim, dtype, 3.0), ref.rows(3, T, heads, dim, dtype, 0.01)
    k[sum(new):], v[sum(new):] = math.nan, math.nan
    plain = ref.Cache(*tensors)
    ref.write(plain, batch, k, v)
    cache, b = device_cache(tensors), device_batch(batch)
    strided = len(lens) % 2 == 0
    etk.cache_write(cache, b, rows_to_device(k, strided), rows_to_device(v, not strided))
    for name in ("k", "v", "k_scale", "v_scale"):
        assert same(getattr(cache, name).float(), getattr(plain, name)), name
    assert same(cache.key_bounds, plain.bounds)
    out = tuple(torch.full((T, heads, dim), MARK, dtype=dtype, device="cuda") for _ in range(2))
    etk.cache_read(cache, b, out=out)
    for got, want in zip(out, ref.read(plain, batch, T, MARK)):
        assert same(got, want)


def test_a_page_is_continued_and_its_scale_grows():
    """Tokens one at a time, each larger than the last by a random factor: earlier codes are brought to
    the new scale each time. Then smaller ones: the scale stays. Then the page starts anew."""
    page, dim, heads = 32, 128, 2
    tensors, batch = ref.make(5, [1], [1], heads, page, dim, BF16, poison=False)
    plain, cache = ref.Cache(*tensors), device_cache(tensors)
    table = batch[0].cuda()
    for t in range(20):
        size = 10.0 ** (t % 13 - 6)
        k, v = ref.rows(10 + t, 1, heads, dim, BF16, size), ref.rows(50 + t, 1, heads, dim, BF16, 1 / size)
        kv_len = torch.tensor([t + 1], dtype=torch.int32)
        ref.write(plain, (batch[0], kv_len, None), k, v)
        etk.cache_write(cache, etk.SequenceBatch(table, kv_len.cuda()), k.cuda(), v.cuda())
        for name in ("k", "v", "k_scale", "v_scale"):
            assert same(getattr(cache, name).float(), getattr(plain, name)), (t, name)
        assert same(cache.key_bounds, plain.bounds), t
    k = ref.rows(99, 1, heads, dim, BF16, 1e-3)
    one = torch.tensor([1], dtype=torch.int32)
    ref.write(plain, (batch[0], one, None), k, k)
    etk.cache_write(cache, etk.SequenceBatch(table, one.cuda()), k.cuda(), k.cuda())
    assert same(cache.k_scale, plain.k_scale) and same(cache.key_bounds, plain.bounds)
    assert same(cache.k.float(), plain.k)


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_write_of_extreme_rows(dtype):
    """Infinities, NaN, zeros, subnormals, the type's largest number, and every border of the scale."""
    page, dim, heads = 16, 64, 1
    special = [0.0, -0.0, math.inf, -math.inf, math.nan, float(torch.finfo(dtype).max), float(torch.finfo(dtype).tiny),
               float(torch.finfo(dtype).smallest_normal) / 4, 448.0, 449.0, 450.0, -448.0, 1.75, 1.7578125, 464.0, 3.5]
    lens = [len(special) * 3]
    tensors, batch = ref.make(6, lens, lens, heads, page, dim, dtype, poison=False)
    k = ref.rows(7, lens[0], heads, dim, dtype, 0.3)
    v = torch.zeros_like(k)
    for i, s in enumerate(special):
        k[16 * (i % 3) + i % 16, 0, i] = s
        v[i * 3:i * 3 + 3] = torch.tensor(s, dtype=dtype)
    plain, cache = ref.Cache(*tensors), device_cache(tensors)
    ref.write(plain, batch, k, v)
    etk.cache_write(cache, device_batch(batch), k.cuda(), v.cuda())
    for name in ("k", "v", "k_scale", "v_scale"):
        assert same(getattr(cache, name).float(), getattr(plain, name)), name
    assert same(cache.key_bounds, plain.bounds) and cache.key_bounds.isfinite().all()
    got = etk.cache_read(cache, device_batch(batch), num_tokens=lens[0])
    for x, y in zip(got, ref.read(plain, batch, lens[0])):
        assert same(x, y)


def test_every_page_of_a_long_batch():
    lens, new = [700, 3000, 64, 1111], [650, 2999, 1, 0]
    tensors, batch = ref.make(8, lens, new, 4, 64, 128, BF16, poison=False)
    T = sum(new)
    k, v = ref.rows(9, T, 4, 128, BF16, 2.0), ref.rows(10, T, 4, 128, BF16, 5.0)
    plain, cache = ref.Cache(*tensors), device_cache(tensors)
    ref.write(plain, batch, k, v)
    etk.cache_write(cache, device_batch(batch), k.cuda(), v.cuda())
    for name in ("k", "v", "k_scale", "v_scale"):
        assert same(getattr(cache, name).float(), getattr(plain, name)), name
    assert same(cache.key_bounds, plain.bounds)
    for x, y in zip(etk.cache_read(cache, device_batch(batch), num_tokens=T), ref.read(plain, batch, T)):
        assert same(x, y)


# ---- scores ----

@pytest.mark.parametrize("lens,new", [([1], [1]), ([700], [1]), ([300, 5, 40, 129], [130, 0, 40, 64]),
                                      ([3, 0, 70], [5, 2, 9]), ([2000, 64, 65], [1, 1, 1])])
@pytest.mark.parametrize("page,dim,heads,group,dtype", [(16, 64, 2, 8, BF16), (32, 128, 1, 1, FP16),
                                                        (64, 128, 2, 3, BF16), (16, 128, 1, 12, FP16),
                                                        (128, 64, 3, 4, FP16), (16, 128, 2, 16, BF16),
                                                        (32, 64, 1, 40, FP16)])
def test_scores(lens, new, page, dim, heads, group, dtype):
    tensors, batch = ref.make(20, lens, new, heads, page, dim, dtype)
    T = sum(new) + 2
    q = ref.rows(21, T, heads * group, dim, dtype, 2.0)
    q[sum(new):] = math.nan
    for first, last, strided in ((0, 0, False), (1, 2, True)):
        want, ke, size = ref.scores(ref.Cache(*tensors), batch, q, first, last, MARK)
        cache, b = device_cache(tensors), device_batch(batch)
        wide = torch.full((T * heads, b.table_width + 5), MARK, device="cuda")
        out = wide[:, :b.table_width] if strided else wide[:, :b.table_width].contiguous()
        got_ke = torch.full((T * heads,), int(MARK), dtype=torch.int32, device="cuda")
        live = torch.zeros(1, dtype=torch.int32, device="cuda")
        etk.block_scores(cache, b, rows_to_device(q, strided), first, last, out, got_ke, live)
        assert torch.equal(got_ke.cpu(), ke) and int(live) == sum(new) * heads
        got = out.cpu().double()
        same_kind = torch.isfinite(want) == torch.isfinite(got)
        assert same_kind.all() and torch.equal(got[~want.isfinite()], want[~want.isfinite()])
        # 2 D exact products summed in FP32, each sum within 2^-23 of the terms' magnitudes
        fine = want.isfinite()
        assert ((got - want).abs()[fine] <= (2 * dim * 2.0 ** -23 * size)[fine]).all()
        assert (wide[:, b.table_width:] == MARK).all()


@pytest.mark.parametrize("heads,group,page,dim,dtype", [(2, 4, 64, 128, BF16), (1, 8, 16, 64, FP16), (1, 1, 32, 128, FP16),
                                                        (1, 5, 16, 128, BF16), (1, 12, 16, 64, BF16), (1, 20, 64, 128, FP16),
                                                        (1, 2, 16, 64, FP16), (1, 33, 32, 64, BF16)])
def test_scores_of_a_prompt(heads, group, page, dim, dtype):
    """Hundreds of rows of a sequence against hundreds of pages, causally ragged."""
    lens, new = [5000, 777], [391, 300]
    tensors, batch = ref.make(22, lens, new, heads, page, dim, dtype)
    T = sum(new)
    q = ref.rows(23, T, heads * group, dim, dtype)
    cache, b = device_cache(tensors), device_batch(batch)
    out = torch.full((T * heads, b.table_width), MARK, device="cuda")
    ke = torch.zeros(T * heads, dtype=torch.int32, device="cuda")
    etk.block_scores(cache, b, q.cuda(), 1, 1, out, ke)
    plain = ref.Cache(*tensors)
    at = 0
    for i, (n, length) in enumerate(zip(new, lens)):
        ends = plain.bounds[batch[0][i, :-(-length // page)].long()]
        for h in range(heads):
            u = q[at:at + n, h * group:(h + 1) * group].double()
            terms = torch.einsum("tgd,jd->tgj", u.clamp(min=0), ends[:, h, 0]) + torch.einsum("tgd,jd->tgj", u.clamp(max=0), ends[:, h, 1])
            size = torch.einsum("tgd,jd->tgj", u.abs(), ends[:, h].abs().amax(1)).amax(1)
            for t in range(n):
                seen = (length - n + t) // page + 1
                want = terms[t].amax(0)
                want[0] = want[seen - 1] = math.inf
                row = out[(at + t) * heads + h].cpu().double()
                assert (row[seen:] == MARK).all() and int(ke[(at + t) * heads + h]) == seen
                assert math.isinf(row[0]) and math.isinf(row[seen - 1])
                assert ((row[1:seen - 1] - want[1:seen - 1]).abs() <= 2 * dim * 2.0 ** -23 * size[t, 1:seen - 1]).all()
        at += n


# ---- attention ----

def check_attention(tensors, batch, q, blocks=None, scale=None, single=False, strided=False, **overrides):
    cache, b = device_cache(tensors), device_batch(batch, single)
    T, QH, D = q.shape
    heads = cache.kv_heads
    K = 0 if blocks is None else blocks.shape[1]
    a = etk.CacheAttention(cache, b.num_seqs, T, QH, b.table_width, num_blocks=K, **overrides)
    out = rows_to_device(torch.full_like(q, MARK), strided)
    got = a(rows_to_device(q, strided), b, blocks=None if blocks is None else blocks.cuda(), out=out, scale=scale)
    assert got is out
    want, tol = ref.attention(ref.Cache(*tensors), (batch[0], batch[1], None if single else batch[2]), q, blocks,
                              1 / math.sqrt(D) if scale is None else scale, MARK)
    got = got.cpu().double()
    kind = torch.isnan(want) == torch.isnan(got)
    assert kind.all(), f"NaN at {(~kind).nonzero()[:5].tolist()}"
    fine = ~want.isnan()
    over = (got - want).abs()[fine] > tol[fine]
    assert not over.any(), (float((got - want).abs()[fine].max()), float(tol[fine].max()), int(over.sum()))
    assert not a.counters.any()
    # the same again, from the counters that the first call left
    again = a(rows_to_device(q, strided), b, blocks=None if blocks is None else blocks.cuda(), scale=scale)
    assert same(again[:int(batch[2][-1])], got[:int(batch[2][-1])])


SHAPES = [([1], [1]), ([0, 1, 2], [1, 1, 1]), ([700], [1]), ([3000, 16, 17, 64], [1, 1, 1, 1]),
          ([300, 5, 40, 129], [13, 0, 40, 2]), ([3, 0, 70], [5, 2, 9]), ([1500], [3])]
LAYOUTS = [(16, 64, 2, 8, BF16), (32, 128, 1, 1, FP16), (64, 128, 2, 3, BF16), (128, 64, 1, 5, FP16),
           (64, 128, 1, 16, BF16), (16, 128, 1, 12, FP16), (64, 64, 1, 40, BF16), (128, 128, 2, 4, BF16)]


@pytest.mark.parametrize("lens,new", SHAPES)
@pytest.mark.parametrize("page,dim,heads,group,dtype", LAYOUTS)
def test_dense(lens, new, page, dim, heads, group, dtype):
    tensors, batch = ref.make(30, lens, new, heads, page, dim, dtype)
    q = ref.rows(31, sum(new), heads * group, dim, dtype, 3.0)
    check_attention(tensors, batch, q, single=all(n == 1 for n in new), strided=len(lens) % 2 == 1)


@pytest.mark.parametrize("lens,new", SHAPES)
@pytest.mark.parametrize("page,dim,heads,group,dtype", LAYOUTS)
def test_listed_pages(lens, new, page, dim, heads, group, dtype):
    """Lists with -1, repeats, pages behind the token's own and out of the table, all-empty rows."""
    tensors, batch = ref.make(32, lens, new, heads, page, dim, dtype)
    T, K = sum(new), 9
    q = ref.rows(33, T, heads * group, dim, dtype, 3.0)
    g = torch.Generator().manual_seed(34)
    most = max(1, -(-max(lens) // page))
    blocks = torch.randint(-1, most + 1, (T * heads, K), generator=g, dtype=torch.int32)
    blocks[0] = -1
    if len(blocks) > 1:
        blocks[1] = 0
    blocks[-1, 0], blocks[-1, 1] = 2 ** 31 - 1, -2 ** 31
    check_attention(tensors, batch, q, blocks, single=all(n == 1 for n in new), strided=len(lens) % 2 == 0)


@pytest.mark.parametrize("group,dtype", [(1, BF16), (2, FP16), (4, BF16), (8, FP16), (16, BF16)])
def test_neighbouring_tokens_share_pages(group, dtype):
    """Tokens of one tile with lists that overlap in part."""
    lens, new, page, heads = [2100, 900], [21, 6], 16, 2
    tensors, batch = ref.make(35, lens, new, heads, page, 64, dtype)
    T, K = sum(new), 40
    g = torch.Generator().manual_seed(36)
    score = torch.rand(1, heads, 131, generator=g) + 0.3 * torch.rand(T, heads, 131, generator=g)
    blocks = score.topk(K, -1).indices.to(torch.int32).reshape(T * heads, K)
    check_attention(tensors, batch, ref.rows(37, T, heads * group, 64, dtype, 3.0), blocks.contiguous())


def test_long_lists_pass_the_ids_held_at_a_time():
    lens, new, page, heads = [16 * 1400 + 5], [2], 16, 1
    tensors, batch = ref.make(38, lens, new, heads, page, 64, BF16)
    g = torch.Generator().manual_seed(39)
    blocks = torch.stack([torch.randperm(1401, generator=g)[:1300] for _ in range(2)]).to(torch.int32)
    q = ref.rows(40, 2, 3, 64, BF16, 3.0)
    check_attention(tensors, batch, q, blocks)
    check_attention(tensors, batch, q)


@pytest.mark.parametrize("spread", [0, 30])
def test_scales_far_apart(spread):
    """Pages whose scales differ by up to 2^30: small values keep their precision beside large ones."""
    lens, new = [500, 64], [1, 1]
    tensors, batch = ref.make(41, lens, new, 2, 16, 64, BF16, spread=spread)
    k_scale = torch.full_like(tensors[2], 2.0 ** -8)
    q = ref.rows(42, 2, 8, 64, BF16)
    check_attention((tensors[0], tensors[1], k_scale, tensors[3], tensors[4]), batch, q, single=True)


@pytest.mark.parametrize("size", [1e-30, 1e-3, 30.0, 3000.0])
def test_queries_of_any_size(size):
    lens, new = [300, 64], [2, 1]
    tensors, batch = ref.make(43, lens, new, 2, 32, 128, BF16)
    q = ref.rows(44, 3, 8, 128, BF16, 1.0) * size
    check_attention(tensors, batch, q, scale=min(1.0, 0.05 / size))
    check_attention(tensors, batch, q, scale=-min(1.0, 0.05 / size))
    check_attention(tensors, batch, q, scale=0.0)


def test_peaked_scores_raise_the_maximum_late():
    """Keys that grow along the sequence, so that the running maximum moves all the time; then ones that shrink."""
    for sign in (1, -1):
        lens, new, page, dim = [2000], [1], 64, 64
        tensors, batch = ref.make(45, lens, new, 1, page, dim, FP16)
        grow = torch.exp2(torch.linspace(-12, -4, 32).round())
        for j in range(32):
            tensors[2][batch[0][0, j]] = grow[j if sign > 0 else 31 - j]
        check_attention(tensors, batch, ref.rows(46, 1, 4, dim, FP16, 4.0), single=True)


@pytest.mark.parametrize("page,dim,group", [(16, 64, 4), (64, 128, 4), (32, 128, 1), (64, 128, 2)])
def test_nan_reaches_the_rows_that_see_it_and_no_other(page, dim, group):
    """NaN among the keys and values of tokens that only some rows of a tile see: by position and by list."""
    lens, new, heads = [page * 6 + 5], [7], 1
    tensors, batch = ref.make(47, lens, new, heads, page, dim, BF16)
    k8, v8 = tensors[0].view(torch.uint8), tensors[1].view(torch.uint8)

    def put(codes, position, channel):
        codes[batch[0][0, position // page].long(), 0, position % page, channel] = 0xFF

    last = lens[0] - 1
    put(v8, last, 3)            # seen by the last row alone
    put(v8, last - 2, dim - 1)  # by three
    put(k8, last - 4, 0)        # by five
    q = ref.rows(48, 7, group, dim, BF16, 2.0)
    check_attention(tensors, batch, q)
    check_attention(tensors, batch, q, prompt=1)
    put(v8, 2 * page + 1, 5)    # by those that list page 2
    put(k8, 3 * page, 1)        # page 3
    blocks = torch.tensor([[0, 1, -1], [0, 2, 1], [1, 0, 5], [3, 0, 1], [0, 1, 2], [6, 0, 1], [4, 5, 0]], dtype=torch.int32)
    check_attention(tensors, batch, q, blocks)
    check_attention(tensors, batch, q, blocks, prompt=1)
    q[2], q[4, 0, 0] = math.nan, math.inf
    check_attention(tensors, batch, q, blocks)
    check_attention(tensors, batch, q, blocks, prompt=1)


def test_absent_pages_are_not_seen():
    lens, new = [300, 100, 64], [3, 1, 1]
    tensors, batch = ref.make(49, lens, new, 2, 16, 64, BF16)
    batch[0][0, 3] = -1
    batch[0][0, 18] = 10 ** 6
    batch[0][1, :] = -5       # nothing at all
    q = ref.rows(50, 5, 8, 64, BF16, 2.0)
    check_attention(tensors, batch, q)
    plain, cache, b = ref.Cache(*tensors), device_cache(tensors), device_batch(batch)
    k = ref.rows(51, 5, 2, 64, BF16)
    before = cache.k.view(torch.uint8).clone()
    ref.write(plain, batch, k, k)
    etk.cache_write(cache, b, k.cuda(), k.cuda())
    assert same(cache.k.float(), plain.k) and same(cache.k_scale, plain.k_scale)
    assert not torch.equal(before, cache.k.view(torch.uint8))
    for x, y in zip(etk.cache_read(cache, b, num_tokens=5), ref.read(plain, batch, 5)):
        assert same(x, y)


def test_row_ranges_and_lengths_out_of_range_are_clamped():
    """Lengths beyond the table and negative, row ranges beyond the rows and descending: clamped as documented."""
    lens, new = [100, 64, 30], [2, 2, 2]
    tensors, batch = ref.make(52, lens, new, 1, 16, 64, BF16, poison=False)
    table, kv_len, q_start = batch
    q = ref.rows(53, 6, 4, 64, BF16)
    for bad_len, bad_start in (([10 ** 6, -3, 2 ** 31 - 1], [0, 2, 4, 6]), ([100, 64, 30], [-5, 2, 4, 100]), ([100, 64, 30], [1, 3, 3, 5])):
        changed = (table, torch.tensor(bad_len, dtype=torch.int32), torch.tensor(bad_start, dtype=torch.int32))
        cache, b = device_cache(tensors), device_batch(changed)
        a = etk.CacheAttention(cache, 3, 6, 4, b.table_width)
        out = a(q.cuda(), b, out=torch.full_like(q, MARK, device="cuda")).cpu().double()
        want, tol = ref.attention(ref.Cache(*tensors), changed, q, None, 0.125, MARK)
        assert ((out - want).abs() <= tol).all()
        want, ke, size = ref.scores(ref.Cache(*tensors), changed, q, 0, 1, MARK)
        got = torch.full(want.shape, MARK, device="cuda")
        got_ke = torch.full(ke.shape, int(MARK), dtype=torch.int32, device="cuda")
        etk.block_scores(cache, b, q.cuda(), 0, 1, got, got_ke)
        assert torch.equal(got_ke.cpu(), ke)
        fine = want.isfinite()
        assert ((got.cpu().double() - want).abs()[fine] <= (128 * 2.0 ** -23 * size)[fine]).all()
        k = ref.rows(54, 6, 1, 64, BF16)
        plain = ref.Cache(*tensors)
        ref.write(plain, changed, k, k)
        etk.cache_write(cache, b, k.cuda(), k.cuda())
        assert same(cache.k.float(), plain.k)


def test_many_sequences():
    """More sequences than a CTA has threads, some without rows, some without tokens."""
    g = torch.Generator().manual_seed(55)
    lens = torch.randint(0, 70, (301,), generator=g).tolist()
    new = [min(n, int(x)) for n, x in zip(lens, torch.randint(0, 3, (301,), generator=g))]
    tensors, batch = ref.make(56, lens, new, 1, 16, 64, BF16)
    q = ref.rows(57, sum(new), 4, 64, BF16, 3.0)
    check_attention(tensors, batch, q)
    blocks = torch.randint(-1, 5, (sum(new), 3), generator=g, dtype=torch.int32)
    check_attention(tensors, batch, q, blocks)
    want, ke, _ = ref.scores(ref.Cache(*tensors), batch, q, 0, 0, MARK)
    cache = device_cache(tensors)
    got, got_ke = etk.block_scores(cache, device_batch(batch), q.cuda(), ke=torch.full((sum(new),), -7, dtype=torch.int32, device="cuda"))
    assert torch.equal(got_ke.cpu(), ke)
    assert torch.allclose(torch.where(want == MARK, 0, got.cpu().double()), torch.where(want == MARK, 0, want), rtol=1e-4, atol=1e-4)


def test_a_cache_whose_offsets_pass_32_bits():
    """Pages at the end of a cache of more than 2^32 codes."""
    heads, page, dim = 8, 128, 128
    pages = (1 << 32) // (heads * page * dim) + 40
    cache = etk.KVCache.allocate(pages, heads, page, dim, device="cuda")
    lens = [700, 260]
    table = torch.tensor([[pages - 1 - 2 * j - b for j in range(6)] for b in range(2)], dtype=torch.int32)
    kv_len = torch.tensor(lens, dtype=torch.int32)
    k, v = ref.rows(58, sum(lens), heads, dim, BF16), ref.rows(59, sum(lens), heads, dim, BF16)
    q_start = torch.tensor([0, 700, 960], dtype=torch.int32)
    etk.cache_write(cache, device_batch((table, kv_len, q_start)), k.cuda(), v.cuda())
    low = pages - 13
    part = ref.Cache(cache.k[low:].float(), cache.v[low:].float(), cache.k_scale[low:], cache.v_scale[low:], cache.key_bounds[low:])
    small = (table - low, kv_len, q_start)
    for x, y in zip(etk.cache_read(cache, device_batch((table, kv_len, q_start)), num_tokens=960), ref.read(part, small, 960)):
        assert same(x, y)
    assert (ref.read(part, small, 960)[0].float() - k.float()).abs().max() <= 2.0 ** -4 * k.float().abs().max()
    one = torch.tensor([0, 1, 2], dtype=torch.int32)
    q = ref.rows(60, 2, heads * 2, dim, BF16, 2.0)
    a = etk.CacheAttention(cache, 2, 2, heads * 2, 6)
    got = a(q.cuda(), device_batch((table, kv_len, one), single=True)).cpu().double()
    want, tol = ref.attention(part, (table - low, kv_len, one), q, None, 1 / math.sqrt(dim), MARK)
    assert ((got - want).abs() <= tol).all()
    scores, _ = etk.block_scores(cache, device_batch((table, kv_len, one)), q.cuda())
    want, ke, size = ref.scores(part, (table - low, kv_len, one), q, 0, 0, MARK)
    seen = want != MARK
    assert ((scores.cpu().double() - want).abs()[seen] <= (2 * dim * 2.0 ** -23 * size)[seen]).all()


# ---- the prompt's kernel, on tiles that fill it and ones that do not ----

PROMPTS = [([1], [1]), ([90, 0, 2], [40, 2, 2]), ([700, 64], [130, 17]), ([200, 5], [200, 9])]


@pytest.mark.parametrize("lens,new", PROMPTS)
@pytest.mark.parametrize("page,dim,heads,group,dtype", LAYOUTS + [(64, 128, 1, 130, BF16), (32, 64, 2, 7, FP16)])
def test_prompt_over_the_whole_cache(lens, new, page, dim, heads, group, dtype):
    tensors, batch = ref.make(130, lens, new, heads, page, dim, dtype)
    q = ref.rows(131, sum(new), heads * group, dim, dtype, 3.0)
    check_attention(tensors, batch, q, strided=len(lens) % 2 == 1, prompt=1)


@pytest.mark.parametrize("lens,new", PROMPTS)
@pytest.mark.parametrize("page,dim,heads,group,dtype", LAYOUTS + [(32, 64, 2, 7, FP16)])
def test_prompt_over_listed_pages(lens, new, page, dim, heads, group, dtype):
    tensors, batch = ref.make(132, lens, new, heads, page, dim, dtype)
    T, K = sum(new), 9
    q = ref.rows(133, T, heads * group, dim, dtype, 3.0)
    most = max(1, -(-max(lens) // page))
    blocks = torch.randint(-1, most + 1, (T * heads, K), generator=torch.Generator().manual_seed(134), dtype=torch.int32)
    blocks[0] = -1
    blocks[-1, 0], blocks[-1, 1] = 2 ** 31 - 1, -2 ** 31
    check_attention(tensors, batch, q, blocks, prompt=1)


@pytest.mark.parametrize("page,dim,dtype", [(16, 64, BF16), (64, 128, FP16)])
def test_prompt_passes_the_parts_held_at_a_time(page, dim, dtype):
    """More parts of pages than the kernel holds at once, with scales that grow along the sequence."""
    lens, new = [page * 300 + 7], [5]
    tensors, batch = ref.make(135, lens, new, 1, page, dim, dtype)
    for j in range(301):
        tensors[3][batch[0][0, j]] = 2.0 ** (j // 60 - 8)
    q = ref.rows(136, 5, 3, dim, dtype, 3.0)
    check_attention(tensors, batch, q, prompt=1)
    blocks = torch.stack([torch.randperm(301, generator=torch.Generator().manual_seed(k))[:260] for k in range(5)]).to(torch.int32)
    check_attention(tensors, batch, q, blocks, prompt=1)


def test_prompt_leaves_what_it_cannot_do_to_the_other_kernel():
    """NaN among the values, scales far apart and of no power of two, absent pages: the same results."""
    lens, new, page, dim = [400, 300], [40, 20], 16, 64
    for case in range(4):
        tensors, batch = ref.make(137 + case, lens, new, 2, page, dim, BF16, spread=0 if case == 2 else 4)
        if case == 0:
            for position in (399, 390, 370, 10):
                tensors[1].view(torch.uint8)[batch[0][0, position // page].long(), 1, position % page, 7] = 0x7F
        elif case == 1:
            tensors[3][batch[0][1, 3]] = 2.0 ** 20
            tensors[3][batch[0][0, 2]] = 2.0 ** -30
        elif case == 2:
            g = torch.Generator().manual_seed(5)
            for t in tensors[2:4]:
                t.mul_(1 + torch.rand(t.shape, generator=g))
        else:
            batch[0][0, 4], batch[0][1, :] = -1, 10 ** 6
        q = ref.rows(141, 60, 16, dim, BF16, 2.0)
        check_attention(tensors, batch, q, prompt=1)
        blocks = torch.randint(-1, 25, (120, 6), generator=torch.Generator().manual_seed(142), dtype=torch.int32)
        check_attention(tensors, batch, q, blocks, prompt=1)


@pytest.mark.parametrize("size", [1e-30, 30.0, 3000.0])
def test_prompt_with_queries_of_any_size(size):
    lens, new = [300, 64], [20, 9]
    tensors, batch = ref.make(143, lens, new, 2, 32, 128, BF16)
    q = ref.rows(144, 29, 8, 128, BF16, 1.0) * size
    check_attention(tensors, batch, q, scale=min(1.0, 0.05 / size), prompt=1)
    check_attention(tensors, batch, q, scale=-min(1.0, 0.05 / size), prompt=1)


def test_the_planner_takes_the_prompts_kernel_and_both_agree():
    lens, new, heads, group, page, dim = [4000], [1300], 2, 8, 64, 128
    tensors, batch = ref.make(145, lens, new, heads, page, dim, BF16)
    cache, b = device_cache(tensors), device_batch(batch)
    q = ref.rows(146, 1300, heads * group, dim, BF16, 3.0).cuda()
    g = torch.Generator().manual_seed(147)
    score = torch.rand(1, heads, 43, generator=g) + 0.3 * torch.rand(1300, heads, 43, generator=g)
    blocks = score.topk(12, -1).indices.to(torch.int32).reshape(-1, 12).cuda()
    for K, lists in ((0, None), (12, blocks)):
        objects = [etk.CacheAttention(cache, 1, 1300, heads * group, b.table_width, num_blocks=K, prompt=p) for p in (-1, 0)]
        assert objects[0].plan.prompt_tokens == 16 and objects[1].plan.prompt_tokens == 0
        x, y = (a(q, b, blocks=lists).double() for a in objects)
        # two roundings to bf16 (2^-9 of the value each way) and the two kernels' probabilities in FP16
        bound = float(tensors[1].float().nan_to_num(0.0).abs().max()) * float(tensors[3].max())
        assert ((x - y).abs() <= 2.0 ** -8 * y.abs() + 2.0 ** -9 * bound).all()


# ---- together, streams, graphs ----

def plain_step(plain, batch, q, num_blocks, first, last, picked):
    """The attention of the step over the pages that were picked, which must be a Top-K of the scores."""
    want, ke, size = ref.scores(plain, batch, q, first, last, MARK)
    for r in range(want.shape[0]):
        got = [int(x) for x in picked[r] if x >= 0]
        n = int(ke[r])
        assert len(set(got)) == len(got) == min(n, num_blocks) and all(0 <= x < n for x in got)
        rest = [j for j in range(n) if j not in got]
        if rest and got:  # up to the rounding of the scores
            slack = 2 * plain.dim * 2.0 ** -22 * float(size[r].max())
            assert float(want[r, got].min()) >= float(want[r, rest].max()) - slack
    return ref.attention(plain, batch, q, picked, 1 / math.sqrt(plain.dim), MARK)


@pytest.mark.parametrize("group,page,dtype", [(4, 16, BF16), (8, 32, FP16), (1, 16, FP16)])
def test_a_prompt_and_the_tokens_after_it(group, page, dtype):
    """Prompts in two chunks, then single tokens: write, scores, exact Top-K and attention as one object."""
    heads, dim, B, K = 2, 64, 3, 8
    width = 30
    cache = etk.KVCache.allocate(B * width, heads, page, dim, dtype=dtype, device="cuda")
    plain = ref.Cache(cache.k.float(), cache.v.float(), cache.k_scale, cache.v_scale, cache.key_bounds)
    table = torch.randperm(B * width, generator=torch.Generator().manual_seed(61)).int().reshape(B, width)
    have = torch.zeros(B, dtype=torch.int32)
    seed = 62
    for new in ([130, 17, 1], [200, 0, 33], [1, 1, 1], [1, 1, 1], [1, 1, 1], [3, 2, 4]):
        T = sum(new)
        have = have + torch.tensor(new, dtype=torch.int32)
        batch = (table, have, torch.tensor([sum(new[:i]) for i in range(B + 1)], dtype=torch.int32))
        q = ref.rows(seed, T, heads * group, dim, dtype, 2.0)
        k, v = ref.rows(seed + 1, T, heads, dim, dtype), ref.rows(seed + 2, T, heads, dim, dtype)
        seed += 3
        step = etk.SparseAttention(cache, B, T, heads * group, width, K, keep_first=1, keep_last=2)
        out = step(q.cuda(), device_batch(batch, single=new == [1, 1, 1]), k=k.cuda(), v=v.cuda())
        ref.write(plain, batch, k, v)
        want, tol = plain_step(plain, batch, q, K, 1, 2, step.blocks.cpu())
        assert ((out.cpu().double() - want).abs() <= tol).all()


def test_a_captured_step_replays_with_new_contents():
    """One captured decoding step: lengths, tables, rows and caches change between its replays."""
    heads, group, page, dim, B, width, K = 2, 8, 16, 128, 5, 40, 6
    tensors, batch = ref.make(70, [width * page] * B, [1] * B, heads, page, dim, BF16, poison=False)
    cache, dev_batch = device_cache(tensors), device_batch(batch, single=True)
    q = torch.zeros(B, heads * group, dim, dtype=BF16, device="cuda")
    k, v = (torch.zeros(B, heads, dim, dtype=BF16, device="cuda") for _ in range(2))
    out, dense = torch.zeros_like(q), torch.zeros_like(q)
    step = etk.SparseAttention(cache, B, B, heads * group, width, K)
    whole = etk.CacheAttention(cache, B, B, heads * group, width)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step(q, dev_batch, k, v, out=out)
        whole(q, dev_batch, out=dense)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step(q, dev_batch, k, v, out=out)
        whole(q, dev_batch, out=dense)
    for rep, lens in enumerate(([640, 1, 16, 17, 333], [5, 640, 640, 2, 100], [0, 1, 1, 1, 1])):
        tensors, batch = ref.make(71 + rep, [width * page] * B, [1] * B, heads, page, dim, BF16, poison=False)
        batch = (batch[0], torch.tensor(lens, dtype=torch.int32), None)
        for mine, new in zip((cache.k, cache.v, cache.k_scale, cache.v_scale, cache.key_bounds), tensors):
            mine.copy_(new)
        hq, hk, hv = ref.rows(80 + rep, B, heads * group, dim, BF16), ref.rows(90 + rep, B, heads, dim, BF16), ref.rows(95 + rep, B, heads, dim, BF16)
        dev_batch.page_table.copy_(batch[0])
        dev_batch.kv_len.copy_(batch[1])
        q.copy_(hq), k.copy_(hk), v.copy_(hv)
        torch.cuda.synchronize()
        graph.replay()
        graph.replay()  # writing the same rows again changes nothing
        torch.cuda.synchronize()
        plain = ref.Cache(*tensors)
        ref.write(plain, batch, hk, hv)
        want, tol = plain_step(plain, batch, hq, K, 0, 1, step.blocks.cpu())
        assert ((out.cpu().double() - want).abs() <= tol).all()
        want, tol = ref.attention(plain, batch, hq, None, 1 / math.sqrt(dim), MARK)
        assert ((dense.cpu().double() - want).abs() <= tol).all()
    assert not whole.counters.any() and not step.attention.counters.any()


def test_a_captured_prompt_replays_with_new_contents():
    """Scores and attention of prompts in one graph: lengths, row ranges, rows and caches change."""
    heads, group, page, dim, B, width, T = 1, 8, 32, 64, 3, 30, 100
    tensors, batch = ref.make(85, [width * page] * B, [40, 30, 30], heads, page, dim, FP16, poison=False)
    cache, dev_batch = device_cache(tensors), device_batch(batch)
    q = torch.zeros(T, heads * group, dim, dtype=FP16, device="cuda")
    out = torch.zeros_like(q)
    scores = torch.zeros(T * heads, width, device="cuda")
    ke = torch.zeros(T * heads, dtype=torch.int32, device="cuda")
    blocks = torch.zeros(T * heads, 5, dtype=torch.int32, device="cuda")
    whole = etk.CacheAttention(cache, B, T, heads * group, width, prompt=1)
    listed = etk.CacheAttention(cache, B, T, heads * group, width, num_blocks=5, prompt=1)
    listed_out = torch.zeros_like(q)

    def run():
        etk.block_scores(cache, dev_batch, q, 0, 1, scores, ke)
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
    for rep, (lens, new) in enumerate((([960, 70, 31], [60, 39, 1]), ([33, 500, 900], [33, 0, 60]), ([0, 1, 960], [0, 1, 99]))):
        tensors, batch = ref.make(86 + rep, [width * page] * B, [0] * B, heads, page, dim, FP16, poison=False)
        if rep == 1:  # what the prompt's kernel leaves to the other one
            tensors[1].view(torch.uint8)[batch[0][2, 3].long(), 0, 5, 9] = 0x7F
        start = [sum(new[:i]) for i in range(B + 1)]
        batch = (batch[0], torch.tensor(lens, dtype=torch.int32), torch.tensor(start, dtype=torch.int32))
        for mine, other in zip((cache.k, cache.v, cache.k_scale, cache.v_scale, cache.key_bounds), tensors):
            mine.copy_(other)
        for mine, other in zip((dev_batch.page_table, dev_batch.kv_len, dev_batch.q_start), batch):
            mine.copy_(other)
        hq = ref.rows(89 + rep, T, heads * group, dim, FP16, 2.0)
        lists = torch.randint(-1, width, (T * heads, 5), generator=torch.Generator().manual_seed(rep), dtype=torch.int32)
        q.copy_(hq), blocks.copy_(lists)
        for x in (out, listed_out, scores):
            x.fill_(MARK)
        ke.fill_(int(MARK))
        graph.replay()
        torch.cuda.synchronize()
        plain = ref.Cache(*tensors)
        for got, which in ((out, None), (listed_out, lists)):
            want, tol = ref.attention(plain, batch, hq, which, 1 / math.sqrt(dim), MARK)
            got = got.cpu().double()
            assert torch.equal(got.isnan(), want.isnan())
            fine = ~want.isnan()
            assert ((got - want).abs()[fine] <= tol[fine]).all()
        want, want_ke, size = ref.scores(plain, batch, hq, 0, 1, MARK)
        assert torch.equal(ke.cpu(), want_ke)
        got, fine = scores.cpu().double(), want.isfinite()
        assert torch.equal(got[~fine], want[~fine])
        assert ((got - want).abs()[fine] <= (2 * dim * 2.0 ** -23 * size)[fine]).all()


def test_more_slots_than_pages():
    """A selection of more pages than the table has: every page is taken, the rest is -1."""
    lens, new, width = [40, 7], [3, 1], 3
    tensors, batch = ref.make(115, lens, new, 2, 16, 64, BF16, width=width, poison=False)
    cache, b = device_cache(tensors), device_batch(batch)
    q = ref.rows(116, 4, 8, 64, BF16, 2.0)
    step = etk.SparseAttention(cache, 2, 4, 8, width, 20, keep_first=2, keep_last=5)
    out = step(q.cuda(), b).cpu().double()
    want, tol = ref.attention(ref.Cache(*tensors), batch, q, None, 0.125, MARK)
    assert ((out - want).abs() <= tol).all()
    assert int((step.blocks >= 0).sum()) == 2 * (3 + 3 + 3 + 1)


def test_host_threads_with_an_object_each():
    import threading

    lens, new = [2000, 300], [20, 9]
    tensors, batch = ref.make(117, lens, new, 2, 16, 64, FP16)
    cache, b = device_cache(tensors), device_batch(batch)
    q = ref.rows(118, 29, 16, 64, FP16, 3.0).cuda()
    objects = [etk.CacheAttention(cache, 2, 29, 16, b.table_width, prompt=i % 2) for i in range(4)]
    want = [a(q, b).clone() for a in objects]
    read = etk.cache_read(cache, b, num_tokens=29)
    torch.cuda.synchronize()
    failed = []

    def work(a, expect):
        stream = torch.cuda.Stream()
        for _ in range(25):
            got = a(q, b, stream=stream)
            rows = etk.cache_read(cache, b, num_tokens=29, stream=stream)
            scores, ke = etk.block_scores(cache, b, q, stream=stream)
            stream.synchronize()
            if not torch.equal(got, expect) or not torch.equal(rows[0], read[0]):
                failed.append(1)

    threads = [threading.Thread(target=work, args=x) for x in zip(objects, want)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    assert not failed


def test_two_streams_with_an_object_each():
    lens, new = [4000, 100, 900], [1, 1, 1]
    tensors, batch = ref.make(100, lens, new, 2, 32, 64, BF16)
    cache, b = device_cache(tensors), device_batch(batch, single=True)
    q = ref.rows(101, 3, 8, 64, BF16, 3.0).cuda()
    objects = [etk.CacheAttention(cache, 3, 3, 8, b.table_width) for _ in range(2)]
    want = objects[0](q, b)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.empty_like(q) for _ in range(20)] for _ in range(2)]
    for i in range(20):
        for a, s, o in zip(objects, streams, outs):
            a(q, b, out=o[i], stream=s)
    torch.cuda.synchronize()
    for o in outs:
        for x in o:
            assert torch.equal(x, want)


def test_an_object_made_behind_other_work_and_used_on_another_stream():
    lens, new, width = [4000, 100, 900], [1, 1, 1], 130
    tensors, batch = ref.make(120, lens, new, 2, 32, 64, BF16, width=width, poison=False)
    cache, b = device_cache(tensors), device_batch(batch, single=True)
    q = ref.rows(121, 3, 8, 64, BF16, 3.0).cuda()
    want = etk.CacheAttention(cache, 3, 3, 8, width)(q, b)
    sparse = etk.SparseAttention(cache, 3, 3, 8, width, 6)(q, b)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    stale = [torch.full((1 << 18,), 7, dtype=torch.uint8, device="cuda") for _ in range(64)]  # for the buffers to land in
    del stale
    torch.cuda._sleep(20_000_000)
    attention = etk.CacheAttention(cache, 3, 3, 8, width)
    got = attention(q, b, stream=stream)
    torch.cuda._sleep(20_000_000)
    step = etk.SparseAttention(cache, 3, 3, 8, width, 6)
    got_sparse = step(q, b, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(got_sparse, sparse)


def test_empty_calls_do_nothing():
    tensors, batch = ref.make(110, [30, 20], [0, 0], 1, 16, 64, BF16)
    cache, b = device_cache(tensors), device_batch(batch)
    before = cache.k.view(torch.uint8).clone()
    empty = torch.empty(0, 1, 64, dtype=BF16, device="cuda")
    etk.cache_write(cache, b, empty, empty)
    assert etk.cache_read(cache, b, num_tokens=0)[0].shape[0] == 0
    live = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    etk.block_scores(cache, b, torch.empty(0, 4, 64, dtype=BF16, device="cuda"), num_valid_rows=live)
    assert int(live) == 0
    assert etk.CacheAttention(cache, 2, 0, 4, b.table_width)(torch.empty(0, 4, 64, dtype=BF16, device="cuda"), b).shape[0] == 0
    # rows, but of no sequence
    some = torch.full((4, 1, 64), math.nan, dtype=BF16, device="cuda")
    etk.cache_write(cache, b, some, some)
    assert torch.equal(before, cache.k.view(torch.uint8))
    out = torch.full((4, 4, 64), MARK, dtype=BF16, device="cuda")
    etk.CacheAttention(cache, 2, 4, 4, b.table_width)(torch.full_like(out, math.nan), b, out=out)
    assert (out == MARK).all()
