"""Page tables on the GPU against a plain form that goes sequence by sequence (tests/serving_reference.py), and the whole step:
tables, rotary positions, the 4-bit cache and attention, captured and replayed."""

import math

import pytest
import torch

import cache_reference as ref
import exact_top_selection_gb300 as etk
import serving_reference as srv

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


def check(tables, plain):
    for name in ("kv_len", "q_start", "applied", "slots", "positions"):
        assert getattr(tables, name).tolist() == getattr(plain, name), name
    assert tables.free_pages.tolist() == plain.ring and tables.free_range.tolist() == plain.range
    assert tables.page_table.tolist() == plain.table and not tables.counters.any()


def pair(pages, seqs, width, page, max_tokens, strided=False, head=0):
    tables = etk.PageTables.allocate(pages, seqs, width, page, max_tokens, device="cuda")
    if strided or head:
        table = tables.page_table
        if strided:
            table = torch.full((seqs, width + 5), -9, dtype=torch.int32, device="cuda")[:, 2:2 + width]
        ring = tables.free_pages.roll(head)
        tables = etk.PageTables(table, tables.kv_len, ring, torch.tensor([head, pages], dtype=torch.int32, device="cuda"), page, max_tokens)
    for x in (tables.slots, tables.positions):
        x.fill_(-7)
    return tables, srv.Tables(tables.page_table, tables.kv_len, tables.free_pages, tables.free_range, page, max_tokens)


# pages, sequences, table width, page size, most rows: one CTA alone, then many; pools and tables that run out
CASES = [(40, 1, 30, 16, 300), (20, 7, 6, 16, 200), (300, 64, 12, 64, 700), (5000, 300, 40, 32, 20000), (900, 1030, 9, 16, 5000),
         (12000, 4096, 5, 128, 100000), (64, 3, 64, 128, 70), (1, 2, 3, 16, 16), (3000, 20, 400, 16, 60000)]


@pytest.mark.parametrize("pages,seqs,width,page,max_tokens", CASES)
@pytest.mark.parametrize("seed", [0, 1])
def test_sequences_grow_and_shrink(pages, seqs, width, page, max_tokens, seed):
    g = torch.Generator().manual_seed(seed)
    tables, plain = pair(pages, seqs, width, page, max_tokens, strided=seed == 1, head=seed * (pages // 2))
    assert tables.batch.num_seqs == seqs
    for step in range(8):
        most = max(1, min(width * page, 2 * max_tokens // seqs) + 2) if step % 2 == 0 else 3
        change = torch.randint(-most // 2, most + 1, (seqs,), generator=g, dtype=torch.int32)
        change[torch.rand(seqs, generator=g) < 0.2] = 0
        change[torch.rand(seqs, generator=g) < 0.1] = -2 ** 31
        if step == 5:
            change[-1] = 2 ** 31 - 1  # fits no table
        batch = tables.update(change.cuda())
        plain.update(change.tolist())
        assert batch is tables.batch
        check(tables, plain)
        used = [p for row, n in zip(plain.table, plain.kv_len) for p in row[:-(-n // page)]]
        free = [plain.ring[(plain.range[0] + i) % pages] for i in range(plain.range[1])]
        assert sorted(used + free) == list(range(pages))
        if step % 3 == 2:
            counts = torch.randint(-2, most, (seqs,), generator=g, dtype=torch.int32)
            tables.drop(counts.cuda())
            plain.update([-c for c in counts.tolist()])
            check(tables, plain)
    tables.drop(tables.kv_len)  # everything goes back; the counts are a tensor that the call writes
    plain.update([-n for n in plain.kv_len])
    check(tables, plain)
    assert plain.range[1] == pages


def test_what_a_call_took_is_given_back():
    tables, plain = pair(100, 5, 20, 16, 400)
    for change in ([100, 1, 16, 17, 0], [3, 30, 0, 200, 1], [400, 400, 1, 1, 1]):
        tables.update(torch.tensor(change, dtype=torch.int32, device="cuda"))
        plain.update(change)
        check(tables, plain)
        tables.drop(tables.applied)
        plain.update([-c for c in plain.applied])
        check(tables, plain)
        assert tables.kv_len.tolist() == [0] * 5


def test_pages_given_back_serve_in_the_same_call():
    """With nothing free: the pages of a sequence that ends go to one that begins, in one CTA and in many."""
    for width, page, max_tokens in ((8, 16, 128), (400, 16, 30000)):
        tables, plain = pair(width, 2, width, page, max_tokens, head=3)
        for change in ([width * page, 0], [-2 ** 31, width * page - 5], [width * page, -2 ** 31], [-page * 3, 2 * page + 1], [0, page]):
            tables.update(torch.tensor(change, dtype=torch.int32, device="cuda"))
            plain.update(change)
            check(tables, plain)


def test_refusals_by_the_rule():
    """A sequence that asks for too much counts for those behind it that need pages, and not for those that need none."""
    tables, plain = pair(10, 5, 8, 16, 1000)
    for change, applied in (([20, 3, 30, 1, 1], [20, 3, 30, 1, 1]), ([0, 100, 1, 16, 15], [0, 0, 1, 0, 15]), ([200, 1, 0, 0, 0], [0, 1, 0, 0, 0])):
        tables.update(torch.tensor(change, dtype=torch.int32, device="cuda"))
        plain.update(change)
        check(tables, plain)
        assert plain.applied == applied
    tables, plain = pair(100, 4, 20, 16, 50)
    change = [20, 40, 10, -3]
    tables.update(torch.tensor(change, dtype=torch.int32, device="cuda"))
    plain.update(change)
    check(tables, plain)
    assert plain.applied == [20, 0, 0, 0]


def test_contents_out_of_range_are_clamped():
    """Lengths beyond the table and negative, a ring's range out of range: nothing outside the buffers is touched."""
    for seqs, max_tokens in ((6, 200), (6, 40000)):
        guard = torch.full((3, 64), -9, dtype=torch.int32, device="cuda")
        tables = etk.PageTables.allocate(20, seqs, 7, 16, max_tokens, device="cuda")
        for lens, where in (([2 ** 31 - 1, -5, 112, 10 ** 6, 0, 3], [-7, 50]), ([112] * 6, [2 ** 31 - 1, -3]), ([-2 ** 31] * 6, [5, 2 ** 31 - 1])):
            tables.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
            tables.free_range.copy_(torch.tensor(where, dtype=torch.int32))
            for change in ([-2 ** 31] * 6, [16, 1, -1, 2 ** 31 - 1, -2 ** 31, 5]):
                tables.update(torch.tensor(change, dtype=torch.int32, device="cuda"))
                assert 0 <= int(tables.kv_len.min()) and int(tables.kv_len.max()) <= 112
                assert 0 <= int(tables.free_range[0]) < 20 and 0 <= int(tables.free_range[1]) <= 20
        assert (guard == -9).all()


@pytest.mark.parametrize("max_tokens", [100, 30000])
def test_a_captured_update_replays(max_tokens):
    tables, plain = pair(500, 6, 80, 16, max_tokens)
    change = torch.zeros(6, dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        tables.update(change)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        tables.update(change)
    plain.update([0] * 6)
    for values in ([10, 20, 0, 1, 16, 17], [1] * 6, [1] * 6, [-1, -2 ** 31, 30, 0, 1, -16], [17] * 6):
        change.copy_(torch.tensor(values, dtype=torch.int32))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        plain.update(values)
        check(tables, plain)


def test_tables_made_behind_other_work_and_used_on_another_stream():
    stream = torch.cuda.Stream()
    change = torch.tensor([5, 40], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    tables = etk.PageTables.allocate(10, 2, 4, 16, 64, device="cuda")
    tables.update(change, stream=stream)
    torch.cuda.synchronize()
    assert tables.kv_len.tolist() == [5, 40] and tables.page_table.tolist() == [[0, -1, -1, -1], [1, 2, 3, -1]]
    assert tables.slots[:45].tolist() == list(range(5)) + list(range(16, 56))


@pytest.mark.parametrize("seqs,max_tokens", [(6, 200), (6, 40000), (1500, 3000)])
def test_nothing_around_the_buffers_is_touched(seqs, max_tokens):
    """Every buffer lies between marked entries, the tables' rows too: ordinary changes, then contents out of every range."""
    pages, width, page, margin = 20 * seqs, 7, 16, 37
    whole = []

    def between(values):
        x = torch.full((len(values) + 2 * margin,), -9, dtype=torch.int32, device="cuda")
        x[margin:-margin] = torch.as_tensor(values, dtype=torch.int32)
        whole.append(x)
        return x[margin:-margin]

    wide = torch.full((seqs + 2, width + 2 * margin), -9, dtype=torch.int32, device="cuda")
    tables = etk.PageTables(wide[1:-1, margin:margin + width], between([0] * seqs), between(range(pages)), between([0, pages]), page, max_tokens,
                            q_start=between([0] * (seqs + 1)), slots=between([0] * max_tokens), positions=between([0] * max_tokens))

    def untouched():
        assert all(bool((x[:margin] == -9).all()) and bool((x[-margin:] == -9).all()) for x in whole)
        assert (wide[0] == -9).all() and (wide[-1] == -9).all() and (wide[:, :margin] == -9).all() and (wide[:, margin + width:] == -9).all()

    g = torch.Generator().manual_seed(seqs)
    for _ in range(4):
        tables.update(torch.randint(-40, 60, (seqs,), generator=g, dtype=torch.int32).cuda())
        untouched()
    assert tables.positions.max() > 0
    edges = torch.tensor([2 ** 31 - 1, -5, 112, 10 ** 6, 0, -2 ** 31], dtype=torch.int32).repeat(-(-seqs // 6))[:seqs]
    steps = torch.tensor([-2 ** 31, 16, 1, -1, 2 ** 31 - 1, 5, 0], dtype=torch.int32).repeat(-(-seqs // 7))[:seqs]
    for lens, where in ((edges, [-7, 2 ** 31 - 1]), (edges.roll(1), [2 ** 31 - 1, -3]), (edges.roll(2), [-2 ** 31, pages]), (edges.roll(3), [pages - 1, pages])):
        tables.kv_len.copy_(lens)
        tables.free_range.copy_(torch.tensor(where, dtype=torch.int32))
        for change in (steps, -1 - steps, steps.roll(3), edges):
            tables.update(change.cuda())
            untouched()
            tables.drop(change.cuda())
            untouched()
            assert 0 <= int(tables.kv_len.min()) and int(tables.kv_len.max()) <= width * page
            assert 0 <= int(tables.free_range[0]) < pages and 0 <= int(tables.free_range[1]) <= pages
            assert 0 <= int(tables.q_start.min()) and int(tables.q_start.max()) <= max_tokens and not tables.counters.any()


def test_more_pages_than_the_ctas_fill_at_once():
    """Three million tokens in pages of 16: each CTA goes through its units more than once. Checked by tensor arithmetic."""
    page, width, most = 16, 80000, 3_000_000
    pages = 240_000
    tables = etk.PageTables.allocate(pages, 5, width, page, most, device="cuda")
    ring = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    tables.free_pages.copy_(ring)
    lens, head, free = torch.zeros(5, dtype=torch.long), 0, pages
    held = [torch.zeros(0, dtype=torch.int32, device="cuda") for _ in range(5)]
    for change in ([700_001, 1_279_999, 16, 0, 1_000_001 - 17], [-650_007, 1, -2 ** 31, 1_240_000, 0], [1_000_000, -1_279_999, 77, -1_240_000, 31]):
        tables.update(torch.tensor(change, dtype=torch.int32, device="cuda"))
        want = torch.maximum(torch.tensor(change), -lens)
        new = lens + want
        have = [-(-int(n) // page) for n in new]
        back = [h[n:] for h, n in zip(held, have)]
        ring_now = torch.cat([ring.roll(-head)[:free], *back])  # the free pages in order, those given back behind them
        taken, start = 0, 0
        for b in range(5):
            held[b], need = held[b][:have[b]], have[b] - len(held[b][:have[b]])
            held[b] = torch.cat([held[b], ring_now[taken:taken + need]])
            taken += need
            assert torch.equal(tables.page_table[b, :have[b]], held[b])
            got = int(max(want[b], 0))
            pos = torch.arange(int(lens[b]), int(lens[b]) + got, device="cuda")
            assert torch.equal(tables.positions[start:start + got].long(), pos)
            assert torch.equal(tables.slots[start:start + got].long(), held[b][pos // page].long() * page + pos % page)
            start += got
            assert int(tables.q_start[b + 1]) == start
        assert tables.kv_len.tolist() == new.tolist() and tables.applied.tolist() == want.tolist() and not tables.counters.any()
        lens, free, ring = new, len(ring_now) - taken, tables.free_pages.clone()
        head = int(tables.free_range[0])
        assert tables.free_range.tolist()[1] == free and torch.equal(ring.roll(-head)[:free], ring_now[taken:])
        assert torch.equal(torch.cat([*held, ring_now[taken:]]).sort().values, torch.arange(pages, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("bits", [4, 8])
def test_a_step_from_tables_to_attention(bits):
    """Prompts, then tokens one at a time with tokens taken back and a sequence that ends and another that begins, all in
    one captured step: tables, rotary positions, write, page scores, selection, attention over all and over selected pages."""
    heads, group, page, dim, B, width, T, picked = 2, 4, 16, 64, 3, 12, 60, 4
    make = etk.KVCache4 if bits == 4 else etk.KVCache
    cache = make.allocate(B * width, heads, page, dim, device="cuda")
    tables = etk.PageTables.allocate(B * width, B, width, page, T, device="cuda")
    rotary = etk.Rotary(dim, base=500000.0, device="cuda")
    step = etk.SparseAttention(cache, B, T, heads * group, width, picked, 1, 1, rotary=rotary)
    whole = etk.CacheAttention(cache, B, T, heads * group, width)
    q = torch.zeros(T, heads * group, dim, dtype=BF16, device="cuda")
    k, v = (torch.zeros(T, heads, dim, dtype=BF16, device="cuda") for _ in range(2))
    out, dense = torch.zeros_like(q), torch.zeros_like(q)
    change = torch.zeros(B, dtype=torch.int32, device="cuda")

    def run():
        batch = tables.update(change)
        step(q, batch, k, v, out=out)
        whole(step.turned[0], batch, out=dense)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        run()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        run()
    plain_tables = srv.Tables(tables.page_table, tables.kv_len, tables.free_pages, tables.free_range, page, T)
    for rep, values in enumerate(([30, 10, 20], [1, 1, 1], [-5, 1, 25], [3, -2 ** 31, 0], [1, 40, 1], [1, 1, 1])):
        hq, hk, hv = (ref.rows(10 * rep + s, T, h, dim, BF16, 2.0) for s, h in ((1, heads * group), (2, heads), (3, heads)))
        change.copy_(torch.tensor(values, dtype=torch.int32))
        q.copy_(hq), k.copy_(hk), v.copy_(hv)
        torch.cuda.synchronize()
        before = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale, cache.key_bounds)]
        graph.replay()
        torch.cuda.synchronize()
        plain_tables.update(values)
        table, kv_len = tables.page_table.cpu(), tables.kv_len.cpu()
        assert kv_len.tolist() == plain_tables.kv_len and table.tolist() == plain_tables.table
        batch = table, kv_len, torch.tensor(plain_tables.q_start, dtype=torch.int32)
        rows = plain_tables.q_start[-1]
        pos = plain_tables.positions[:rows] + [None] * (T - rows)
        turned = [x.cpu() for x in step.turned]
        for x, y in zip((hq, hk), turned):
            want, tol = srv.rotary(x, pos, rotary.frequencies, 1.0, False, 0.0)
            assert ((y.double() - want).abs() <= tol)[:rows].all()
        # the cache as written from the rows that the rotation gave, then attention over it
        plain = srv.Cache4(*before) if bits == 4 else ref.Cache(*before)
        (srv if bits == 4 else ref).write(plain, batch, turned[1], hv)
        got = srv.values(cache.k.cpu(), cache.k_scale.cpu()) if bits == 4 else cache.k.cpu().double()
        assert torch.equal(got, plain.k)
        for got, blocks in ((out, step.blocks.cpu()), (dense, None)):
            want, tol = ref.attention(plain, batch, turned[0], blocks, 1 / math.sqrt(dim), 0.0)
            assert ((got.cpu().double() - want).abs() <= tol)[:rows].all()
        for t in range(rows):  # the newest page is always among the selected ones
            for h in range(heads):
                assert pos[t] // page in step.blocks[t * heads + h].tolist()
