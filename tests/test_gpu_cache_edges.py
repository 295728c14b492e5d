"""The cache operators where the sizes of test_gpu_cache.py do not lead."""

import contextlib
import ctypes
import math
import threading

import pytest
import torch

import cache_reference as ref
import exact_top_selection_gb300 as etk
from exact_top_selection_gb300 import cache as binding
from test_gpu_cache import BF16, FP16, LAYOUTS, check_attention, device_batch, device_cache, same

pytestmark = pytest.mark.gpu


# ---- small probabilities ----

def tailed(lens, new, page, dim, dtype, dominant):
    """Sequences of one key head. Tokens at `dominant` (a function of the position) have a key of 1 in channel 0
    and no value; all others a key of zeros and values of 32 to 64 in steps of 4."""
    tensors, batch = ref.make(200, lens, new, 1, page, dim, dtype, poison=False)
    k, v, k_scale, v_scale, _ = tensors
    g = torch.Generator().manual_seed(201)
    values = torch.randint(8, 17, (v.shape[0], 1, page, dim), generator=g).float() * 4
    keys = torch.zeros(k.shape)
    k_scale.fill_(2.0 ** -4), v_scale.fill_(1.0)
    for b, n in enumerate(lens):
        for p in (p for p in range(n) if dominant(p)):
            at = int(batch[0][b, p // page])
            keys[at, 0, p % page, 0] = 16.0
            values[at, 0, p % page] = 0.0
    k.copy_(keys.to(ref.FP8)), v.copy_(values.to(ref.FP8))
    return tensors, batch


def far(tokens, heads, dim, dtype, powers):
    """Queries whose product with the key of a dominant token is each of `powers` in turn, in powers of two."""
    q = torch.zeros(tokens, heads, dim, dtype=dtype)
    q[:, :, 0] = torch.tensor([powers[i % len(powers)] for i in range(tokens * heads)]).view(tokens, heads).to(dtype)
    return q


def tail_bound(p, v, dim, terms, dtype, want):
    """How far an output may be from `want` = p @ v, for probabilities p that add up to 1.

    A probability is held in FP16 against a largest one of at least 2^6. It is off by 2^-11 of itself, or, where
    it is below FP16's normal range, by half of FP16's smallest step, 2^-25: by 2^-31 of the largest. Their sum
    is that of the unrounded ones. Scores are off as cache_reference.attention says (2^-23 of the terms'
    magnitudes for each of D + 3 roundings, 2^-21 for the power of two), in the sum too, and the FP32
    sums by 2^-24 for each of n + 40 steps. The result is rounded to its type once."""
    n = len(p)
    rel = 2 * (2.0 ** -11 + 2.0 ** -21 + terms * (dim + 3) * 2.0 ** -23) + (n + 40) * 2.0 ** -24
    small = n * 2.0 ** -31 * p.max() * v.abs().amax(0)
    return rel * (p @ v.abs()) + small + want.abs() * torch.finfo(dtype).eps / 2 + torch.finfo(dtype).tiny * torch.finfo(dtype).eps


POWERS = [20.0, 25.5, 26.25, 28.0, 12.0, 24.75]


@pytest.mark.parametrize("page,dim,group,dtype", [(16, 64, 3, FP16), (64, 128, 8, BF16), (32, 128, 12, BF16), (128, 64, 20, FP16)])
@pytest.mark.parametrize("prompt", [0, 1])
@pytest.mark.parametrize("listed", [False, True])
def test_a_flat_tail_beside_dominant_tokens(page, dim, group, dtype, prompt, listed):
    """In every 32 tokens one whose probability is 2^12 to 2^28 times that of each other, and whose value is zero:
    the outputs are what the others add up to."""
    lens, new = [700, 33, 1300], [5, 2, 9]
    tensors, batch = tailed(lens, new, page, dim, dtype, lambda p: p % 32 == 0)
    T, width = sum(new), batch[0].shape[1]
    q = far(T, group, dim, dtype, POWERS)
    blocks = None
    if listed:
        g = torch.Generator().manual_seed(202)
        blocks = torch.stack([torch.randperm(width, generator=g)[:max(1, width * 2 // 3)] for _ in range(T)]).to(torch.int32)
    scale = math.log(2.0)
    cache = device_cache(tensors)
    a = etk.CacheAttention(cache, len(lens), T, group, width, num_blocks=0 if blocks is None else blocks.shape[1], prompt=prompt)
    got = a(q.cuda(), device_batch(batch), blocks=None if blocks is None else blocks.cuda(), scale=scale).cpu().double()
    plain, row = ref.Cache(*tensors), 0
    for b, (n, length) in enumerate(zip(new, lens)):
        for i in range(n):
            pos = length - n + i
            at = [p for p in range(pos + 1) if blocks is None or p // page in blocks[row].tolist()]
            if at:
                k, v = (plain.rows(name, batch[0][b], 0, at)[0] for name in ("k", "v"))
            for h in range(group):
                if not at:
                    assert not got[row, h].any()
                    continue
                x = k @ q[row, h].double() * scale
                p = torch.softmax(x, 0)
                want = p @ v
                bound = tail_bound(p, v, dim, float(x.abs().max()), dtype, want)
                off = (got[row, h] - want).abs()
                assert (off <= bound).all(), (row, h, float(off.max()), float(want.max()), float(bound.max()))
            row += 1


@pytest.mark.parametrize("prompt", [0, 1])
def test_a_long_tail_beside_one_dominant_token(prompt):
    """Half a million tokens of 2^-26 each, a hundredth of the whole, beside one that was there before them. Many
    sequences of the same pages, so that a CTA of the kernel of single tokens goes over a whole one alone;
    its four warps take 32 tokens of a page in turn, so four tokens are dominant."""
    page, dim, group = 128, 64, 8
    length = 524288 if prompt else 65536
    seqs, each = (1, 16) if prompt else (1300, 1)
    tensors, batch = tailed([length], [each], page, dim, BF16, lambda p: p in (0, 32, 64, 96))
    table = batch[0].expand(seqs, -1).contiguous()
    T = seqs * each
    q = far(T, group, dim, BF16, [26.25, 24.75, 25.5, 26.5])
    scale = math.log(2.0)
    cache = device_cache(tensors)
    kv_len = torch.full((seqs,), length, dtype=torch.int32)
    dev = device_batch((table, kv_len, torch.tensor([i * each for i in range(seqs + 1)], dtype=torch.int32)), single=each == 1)
    got = etk.CacheAttention(cache, seqs, T, group, table.shape[1], prompt=prompt)(q.cuda(), dev, scale=scale)
    order = batch[0][0].long()
    k, v = (tensors[i].float()[order, 0].flatten(0, 1).cuda().double() * s for i, s in ((0, 2.0 ** -4), (1, 1.0)))
    for t in range(each):
        n = length - each + 1 + t
        for h in range(group):
            x = k[:n] @ q[t, h].cuda().double() * scale
            p = torch.softmax(x, 0)
            want = p @ v[:n]
            bound = tail_bound(p, v[:n], dim, float(x.abs().max()), BF16, want)
            off = (got[t::each, h].double() - want).abs()  # every sequence has the same queries
            assert (off <= bound).all(), (t, h, float(off.max()), float(want.max()), float(bound.max()))


# ---- host threads ----

@pytest.mark.parametrize("prompt", [0, 1])
def test_host_threads_with_calls_of_different_sizes(prompt):
    """Objects whose tables and numbers of sequences differ: what a call sets for its launch must not be too
    small for another thread's. The entry point is called as the binding does, without the binding's
    checks, which hold the interpreter's lock most of the time."""
    tensors, batch = ref.make(210, [500, 90], [12, 9], 1, 16, 64, BF16)
    cache, lib = device_cache(tensors), binding._lib()
    pages = torch.where(batch[0] < cache.num_pages, batch[0], 0)
    jobs = []
    for seqs, width in ((2, 32), (700, 24576 if prompt else 65536), (2, 4000), (4096, 24000)):
        table = torch.zeros(seqs, width, dtype=torch.int32)
        table[:2, :pages.shape[1]] = pages
        lens, start = torch.zeros(seqs, dtype=torch.int32), torch.full((seqs + 1,), 21, dtype=torch.int32)
        lens[:2], start[:2] = batch[1], batch[2][:2]
        b = device_batch((table, lens, start))
        q = ref.rows(211, 21, 8, 64, BF16).cuda()
        blocks = torch.randint(0, 32, (21, 6), generator=torch.Generator().manual_seed(212), dtype=torch.int32).cuda()
        a = etk.CacheAttention(cache, seqs, 21, 8, width, num_blocks=6, prompt=prompt)
        jobs.append((a, b, q, blocks, a(q, b, blocks=blocks).clone()))
    torch.cuda.synchronize()
    assert all(torch.equal(j[-1], jobs[0][-1]) for j in jobs)
    failed = []
    ready = threading.Barrier(len(jobs))

    def work(a, b, q, blocks, want):
        stream, out = torch.cuda.Stream(), torch.zeros_like(want)
        torch.cuda.synchronize()
        ref_ = ctypes.byref
        args = (ref_(a.plan), cache._ref, b._ref, ref_(binding._rows(q, "q", cache, 8)), ref_(binding._rows(out, "out", cache, 8)),
                blocks.data_ptr(), 0.125, *a._buffers, stream.cuda_stream)
        ready.wait()
        for _ in range(3000):
            rc = lib.exact_topk_attention_run(*args)
            if rc != 0:
                failed.append(rc)
                break
        stream.synchronize()
        if not torch.equal(out, want):
            failed.append("differs")

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


# ---- streams ----

def test_a_cache_made_behind_other_work_and_written_on_another_stream():
    page, dim, heads, pages = 16, 64, 2, 40
    stream = torch.cuda.Stream()
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, pages)
    n = pages * page
    b = etk.SequenceBatch(table, torch.tensor([n], dtype=torch.int32, device="cuda"),
                          torch.tensor([0, n], dtype=torch.int32, device="cuda"))
    k, v = (ref.rows(s, n, heads, dim, BF16).cuda() for s in (220, 221))
    want = etk.KVCache.allocate(pages, heads, page, dim, device="cuda")
    etk.cache_write(want, b, k, v)
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    cache = etk.KVCache.allocate(pages, heads, page, dim, device="cuda")
    etk.cache_write(cache, b, k, v, stream=stream)
    torch.cuda.synchronize()
    for name in ("k", "v", "k_scale", "v_scale", "key_bounds"):
        agree = same(getattr(cache, name).float(), getattr(want, name).float())
        assert agree, name


# ---- waits that run out ----

@contextlib.contextmanager
def waits(polls):
    """Waits within a CTA give up after so many polls (0: at once)."""
    lib = binding._lib()
    assert lib.exact_topk_set_wait_limit(polls) == 0
    try:
        yield
    finally:
        assert lib.exact_topk_set_wait_limit(-1) == 0


@pytest.mark.parametrize("page,dim,heads,group,dtype", LAYOUTS + [(64, 128, 1, 130, BF16)])
def test_a_prompt_whose_waits_run_out(page, dim, heads, group, dtype):
    """The kernel behind the prompt's computes all that was left: its own results, bit for bit. The tensor memory
    is given back each time."""
    lens, new = [page * 9 + 3, 64], [23, 9]
    tensors, batch = ref.make(230, lens, new, heads, page, dim, dtype)
    T, K = sum(new), 5
    q = ref.rows(231, T, heads * group, dim, dtype, 3.0)
    blocks = torch.randint(-1, 10, (T * heads, K), generator=torch.Generator().manual_seed(232), dtype=torch.int32)
    cache, b = device_cache(tensors), device_batch(batch)
    for lists in (None, blocks):
        with waits(0):
            check_attention(tensors, batch, q, lists, prompt=1)
        dev = None if lists is None else lists.cuda()
        plain, prompt = (etk.CacheAttention(cache, 2, T, heads * group, b.table_width, num_blocks=0 if dev is None else K, prompt=p)
                         for p in (0, 1))
        want = plain(q.cuda(), b, blocks=dev)
        with waits(0):
            for _ in range(10):
                got = prompt(q.cuda(), b, blocks=dev)
        assert torch.equal(got, want)
        check_attention(tensors, batch, q, lists, prompt=1)


# ---- page scores ----

def check_scores(lens, new, page, dim, heads, group, dtype, first, last, absent=0.0, before=lambda: contextlib.nullcontext()):
    """All rows against the definition in 64 bits, computed on the GPU by one product for each sequence and
    head. `absent`: share of the table's entries, the first and the newest among them, that name no page."""
    g = torch.Generator().manual_seed(240)
    held = [-(-n // page) for n in lens]
    total = sum(held) + 1
    mid, half = torch.randn(total, heads, dim, generator=g), torch.rand(total, heads, dim, generator=g)
    bounds = torch.stack([mid + half, mid - half], 2).to(dtype).cuda()
    codes = torch.zeros(total, heads, page, dim, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    one = torch.ones(total, heads, device="cuda")
    cache = etk.KVCache(codes, codes, one, one, bounds)
    table = torch.full((len(lens), max(held)), total + 3, dtype=torch.int32)
    order, at = torch.randperm(total, generator=g).int(), 0
    for b, n in enumerate(held):
        table[b, :n] = order[at:at + n]
        gone = torch.rand(n, generator=g) < absent
        if absent and n > 2:
            gone[0] = gone[n - 1] = True
        table[b, :n][gone] = torch.tensor([-1, total, 2 ** 31 - 1], dtype=torch.int32)[torch.arange(int(gone.sum())) % 3]
        at += n
    T = sum(new)
    start = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32)
    dev = device_batch((table, torch.tensor(lens, dtype=torch.int32), start))
    q = ref.rows(241, T + 5, heads * group, dim, dtype, 2.0).cuda()
    q[T:] = math.nan
    got = torch.full(((T + 5) * heads, max(held)), -7.0, device="cuda")
    ke = torch.full(((T + 5) * heads,), -7, dtype=torch.int32, device="cuda")
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    with before():
        etk.block_scores(cache, dev, q, first, last, got, ke, live)
        torch.cuda.synchronize()
    assert int(live) == T * heads
    assert bool((got[T * heads:] == -7).all()) and bool((ke[T * heads:] == -7).all())
    got, ke = got.view(T + 5, heads, -1), ke.view(T + 5, heads)
    page_ids = dev.page_table.long()
    for b, (n, length) in enumerate(zip(new, lens)):
        if n == 0:
            continue
        lo = int(start[b])
        pos = length - n + torch.arange(n, device="cuda")
        newest = torch.where(pos >= 0, torch.div(pos, page, rounding_mode="floor"), -1)[:, None]
        assert bool((ke[lo:lo + n] == newest + 1).all())
        j = torch.arange(held[b], device="cuda")[None]
        there = (page_ids[b, :held[b]] >= 0) & (page_ids[b, :held[b]] < total)
        ends = bounds[torch.where(there, page_ids[b, :held[b]], 0)].double()
        for h in range(heads):
            u = q[lo:lo + n, h * group:(h + 1) * group].double().flatten(0, 1)
            hi, low = ends[:, h, 0].T, ends[:, h, 1].T
            want = (u.clamp(min=0) @ hi + u.clamp(max=0) @ low).view(n, group, -1).amax(1)
            size = (u.abs() @ torch.maximum(hi.abs(), low.abs())).view(n, group, -1).amax(1)
            want = torch.where((j < first) | (j > newest - last), math.inf, want)
            want = torch.where(there[None], want, -math.inf)
            want = torch.where(j > newest, -7.0, want)
            mine = got[lo:lo + n, h].double()
            assert bool((mine[:, held[b]:] == -7).all())
            mine = mine[:, :held[b]]
            fine = want.isfinite() & (j <= newest)
            # 2 D exact products summed in FP32, each sum within 2^-23 of the terms' magnitudes
            good = torch.where(fine, (mine - want).abs() <= 2 * dim * 2.0 ** -23 * size, mine == want)
            assert bool(good.all()), (b, h, (~good).nonzero()[:4].tolist(), mine[~good][:4].tolist(), want[~good][:4].tolist())


@pytest.mark.parametrize("lens,new,page,dim,heads,group,dtype", [
    ([777], [300], 16, 64, 2, 4, BF16), ([3, 9000, 64], [70, 700, 33], 64, 128, 3, 5, FP16), ([10300], [4096], 16, 64, 10, 16, BF16),
    ([6000], [1000], 32, 128, 1, 1, BF16), ([2500, 2100], [300, 256], 16, 128, 2, 32, FP16)])
def test_scores_of_a_prompt_whose_waits_run_out(lens, new, page, dim, heads, group, dtype):
    """Everything is computed again, the lengths are written all the same, and the tensor memory is given back."""
    for first, last, absent in ((1, 2, 0.1), (0, 0, 0.0)):
        check_scores(lens, new, page, dim, heads, group, dtype, first, last, absent, before=lambda: waits(0))
    check_scores(lens, new, page, dim, heads, group, dtype, 1, 2, 0.1)


# Items (256 columns x a run of page tiles) of each: 2570 of 6 tiles, more than 16 for each CTA; 1020 of 16 tiles; 420 of
# 2 tiles; 864 of 2 tiles; 1004 of 2 tiles; 1060 of 4 and fewer.
@pytest.mark.parametrize("lens,new,page,dim,heads,group,dtype", [
    ([10300], [4096], 16, 64, 10, 16, BF16), ([32768, 500], [1500, 100], 16, 128, 10, 16, FP16),
    ([70000, 3000, 200], [700, 0, 130], 64, 128, 3, 5, BF16), ([20000], [9000], 32, 64, 8, 1, FP16),
    ([6000], [2000], 16, 64, 2, 32, BF16), ([16000, 1, 900, 15000], [800, 1, 333, 500], 16, 64, 5, 12, FP16)])
@pytest.mark.parametrize("absent", [0.0, 0.15])
def test_scores_of_more_items_than_ctas(lens, new, page, dim, heads, group, dtype, absent):
    """A CTA goes from item to item: accumulators, column lines and barriers are used again and again."""
    check_scores(lens, new, page, dim, heads, group, dtype, 1, 2, absent)


@pytest.mark.parametrize("page,dim,heads,group,dtype", [(16, 64, 2, 8, BF16), (64, 128, 1, 3, FP16), (32, 128, 2, 12, BF16), (16, 64, 1, 40, FP16)])
def test_scores_of_absent_pages(page, dim, heads, group, dtype):
    """Pages that no id names score -inf, also where they are to be kept: single tokens, tokens to verify, prompts."""
    for lens, new in (([page * 90, 5, page * 7 + 3], [1, 1, 1]), ([page * 40 + 1, page * 9], [5, 2]), ([page * 50, 300], [270, 190])):
        for first, last in ((0, 0), (2, 3), (1000, 0)):
            check_scores(lens, new, page, dim, heads, group, dtype, first, last, 0.25)
