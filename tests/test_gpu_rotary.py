"""Rotary positions against their definition with exact angles (tests/serving_reference.py)."""

import math

import pytest
import torch

import cache_reference as ref
import exact_top_selection_gb300 as etk
import serving_reference as srv

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16
MARK = -7.0


def close(got, want, tol):
    off = (got.detach().cpu().double() - want).abs()
    bad = off > tol
    assert not bad.any(), (bad.nonzero()[:4].tolist(), off[bad][:4].tolist(), tol[bad][:4].tolist())


def device_batch(batch, single=False):
    table = torch.zeros(len(batch[1]), 1, dtype=torch.int32, device="cuda")  # not looked at
    return etk.SequenceBatch(table, batch[1].cuda(), None if single else batch[2].cuda())


def sequences(lens, new):
    start = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32)
    return None, torch.tensor(lens, dtype=torch.int32), start


SHAPES = [([1], [1]), ([65536, 1, 2048], [1, 1, 1]), ([300, 5, 40, 129], [130, 0, 40, 2]), ([3, 0, 70], [5, 2, 9]),
          ([131072, 2 ** 24], [3, 700])]


@pytest.mark.parametrize("lens,new", SHAPES)
@pytest.mark.parametrize("dim,rot,q_heads,k_heads,dtype", [(128, 128, 32, 4, BF16), (64, 64, 7, 1, FP16), (128, 64, 3, 3, BF16), (96, 24, 5, 2, FP16),
                                                           (80, 20, 2, 1, BF16), (64, 2, 1, 1, BF16), (8, 6, 2, 2, FP16), (1024, 512, 1, 1, BF16), (72, 50, 3, 1, FP16)])
@pytest.mark.parametrize("neighbours", [False, True])
def test_rows_of_a_batch(lens, new, dim, rot, q_heads, k_heads, dtype, neighbours):
    batch, single = sequences(lens, new), all(n == 1 for n in new)
    T = sum(new) + (0 if single else 2)  # rows behind the last sequence
    q, k = ref.rows(1, T, q_heads, dim, dtype, 3.0), ref.rows(2, T, k_heads, dim, dtype)
    if not single:
        q[-2:] = math.nan
    rotary = etk.Rotary(dim, rot, neighbours=neighbours, device="cuda")
    out = torch.full_like(q, MARK, device="cuda"), torch.full_like(k, MARK, device="cuda")
    got = rotary(q.cuda(), k.cuda(), batch=device_batch(batch, single), out=out)
    assert got[0] is out[0] and got[1] is out[1]
    pos = srv.positions(batch, T, page=1 << 30)
    for x, y in zip((q, k), got):
        close(y, *srv.rotary(x, pos, rotary.frequencies, 1.0, neighbours, MARK))
    # without k, without out; then in place on slices of one projection
    assert torch.equal(rotary(q.cuda(), batch=device_batch(batch, single))[:sum(new)], out[0][:sum(new)]) or not all(p is not None for p in pos)
    wide = torch.cat([q, k, k], 1).cuda()
    a, b = wide[:, :q_heads], wide[:, q_heads:q_heads + k_heads]
    rotary(a, b, batch=device_batch(batch, single), out=(a, b))
    there = torch.tensor([p is not None for p in pos])
    assert torch.equal(a[there], out[0][there]) and torch.equal(b[there], out[1][there])
    assert torch.equal(a[~there].nan_to_num(1.0), q.cuda()[~there].nan_to_num(1.0))
    assert torch.equal(wide[:, q_heads + k_heads:], k.cuda())


@pytest.mark.parametrize("neighbours", [False, True])
def test_positions_of_any_size(neighbours):
    """Far and negative positions: the angles are exact. Strided rows."""
    pos = [0, 1, -1, 65536, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, 123456789, 5, 5]
    q = ref.rows(3, len(pos), 2, 64, FP16)
    wide = torch.full((len(pos), 5, 88), math.nan, dtype=FP16, device="cuda")
    wide[:, 1:5:2, 8:72] = q.cuda()
    rotary = etk.Rotary(64, neighbours=neighbours, device="cuda")
    positions = torch.tensor(pos, dtype=torch.int32, device="cuda")
    got = rotary(wide[:, 1:5:2, 8:72], positions=positions)
    close(got, *srv.rotary(q, pos, rotary.frequencies, 1.0, neighbours, MARK))
    rotary(wide[:, 1:5:2, 8:72], positions=positions, out=wide[:, 1:5:2, 8:72])
    assert torch.equal(wide[:, 1:5:2, 8:72], got) and wide[:, ::2].isnan().all()


def test_many_tokens_share_a_cta():
    lens, new = [9000, 40000, 3], [6001, 17, 3]
    batch = sequences(lens, new)
    T = sum(new)
    q, k = ref.rows(4, T, 3, 64, BF16), ref.rows(5, T, 1, 64, BF16)
    rotary = etk.Rotary(64, 32, base=500000.0, device="cuda")
    pos = srv.positions(batch, T, page=1 << 30)
    for x, y in zip((q, k), rotary(q.cuda(), k.cuda(), batch=device_batch(batch))):
        close(y, *srv.rotary(x, pos, rotary.frequencies, 1.0, False, 0.0))


def test_scaled_contexts():
    """Kept, ramp and slowed pairs by the definition; the amplitude; plain interpolation; given frequencies."""
    dim, base, s, length = 128, 10000.0, 8.0, 4096
    rotary = etk.Rotary(dim, base=base, factor=s, original_length=length, slow=1.0, fast=32.0, device="cuda")
    for i, got in enumerate(rotary.frequencies):
        f = base ** (-2 * i / dim)
        g = min(1.0, max(0.0, (length / (2 * math.pi / f) - 1.0) / 31.0))
        assert math.isclose(got, (1 - g) * f / s + g * f, rel_tol=1e-14)
    assert rotary.frequencies[0] == 1.0 and math.isclose(rotary.frequencies[-1] * s, base ** (-126 / 128))
    assert math.isclose(rotary.amplitude, 0.1 * math.log(s) + 1)
    plain = etk.Rotary(dim, base=base, factor=s, device="cuda")
    assert plain.amplitude == 1.0 and math.isclose(plain.frequencies[5] * s, base ** (-10 / 128))
    given = etk.Rotary(dim, frequencies=[-0.25 * i for i in range(64)], amplitude=-2.5, device="cuda")
    pos = [32000, 7, 100001]
    q = ref.rows(6, 3, 2, dim, BF16)
    for r in (rotary, plain, given):
        got = r(q.cuda(), positions=torch.tensor(pos, dtype=torch.int32, device="cuda"))
        close(got, *srv.rotary(q, pos, r.frequencies, r.amplitude, False, MARK))


@pytest.mark.parametrize("neighbours", [False, True])
def test_the_inverse_is_the_gradient(neighbours):
    """Against the formula's gradient (autograd of it in 64 bits) and against differences of the kernel's own outputs."""
    pos, dim, rot = [3, 4096, 70000, 11], 64, 48
    rotary = etk.Rotary(dim, rot, neighbours=neighbours, factor=4.0, original_length=2048, device="cuda")
    positions = torch.tensor(pos, dtype=torch.int32, device="cuda")
    g = ref.rows(7, 4, 3, dim, FP16)
    back = rotary(g.cuda(), positions=positions, inverse=True)
    close(back, *srv.rotary(g, pos, rotary.frequencies, rotary.amplitude, neighbours, MARK, inverse=True))
    x = torch.zeros(4, 3, dim, dtype=torch.float64, requires_grad=True)
    i = torch.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if neighbours else (i, i + rot // 2)
    angle = torch.tensor(pos, dtype=torch.float64)[:, None, None] * torch.tensor(rotary.frequencies, dtype=torch.float64)
    c, s = angle.cos() * rotary.amplitude, angle.sin() * rotary.amplitude
    loss = (g.double()[..., a] * (x[..., a] * c - x[..., b] * s) + g.double()[..., b] * (x[..., b] * c + x[..., a] * s)).sum() \
        + (g.double()[..., rot:] * x[..., rot:]).sum()
    loss.backward()
    _, tol = srv.rotary(g, pos, rotary.frequencies, rotary.amplitude, neighbours, MARK, inverse=True)
    close(back, x.grad, tol + 1e-9)
    # The operator is linear: a step of one along channel j changes the outputs by its column. Each of a column's entries is an
    # output rounded to FP16 with the tolerance of a row with a single 1.
    for j in (0, 1, 23, 24, 47, 60):
        one = torch.zeros(4, 3, dim, dtype=FP16)
        one[..., j] = 1.0
        column = rotary(one.cuda(), positions=positions).cpu().double()
        _, off = srv.rotary(one, pos, rotary.frequencies, rotary.amplitude, neighbours, MARK)
        want, slack = (column * g.double()).sum(-1), (off * g.double().abs()).sum(-1)
        assert ((back.cpu().double()[..., j] - want).abs() <= slack + tol[..., j]).all(), j


def test_infinities_and_nan_stay_in_their_pair():
    q = ref.rows(8, 1, 1, 64, BF16)
    q[0, 0, 3], q[0, 0, 40] = math.nan, math.inf
    got = etk.Rotary(64, device="cuda")(q.cuda(), positions=torch.tensor([9], dtype=torch.int32, device="cuda")).cpu()
    bad = ~got[0, 0].isfinite()
    assert bad.nonzero().flatten().tolist() == [3, 8, 35, 40]


def test_a_captured_call_replays_with_new_positions():
    T, dim = 6, 128
    q, k = torch.zeros(T, 4, dim, dtype=BF16, device="cuda"), torch.zeros(T, 2, dim, dtype=BF16, device="cuda")
    out = torch.zeros_like(q), torch.zeros_like(k)
    batch = sequences([10, 20], [3, 3])
    dev = device_batch(batch)
    rotary = etk.Rotary(dim, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        rotary(q, k, batch=dev, out=out)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        rotary(q, k, batch=dev, out=out)
    for rep, (lens, new) in enumerate((([9000, 2], [4, 2]), ([1, 131072], [1, 5]), ([0, 50], [0, 4]))):
        batch = sequences(lens, new)
        dev.kv_len.copy_(batch[1]), dev.q_start.copy_(batch[2])
        hq, hk = ref.rows(20 + rep, T, 4, dim, BF16), ref.rows(30 + rep, T, 2, dim, BF16)
        q.copy_(hq), k.copy_(hk)
        for x in out:
            x.fill_(MARK)
        graph.replay()
        torch.cuda.synchronize()
        pos = srv.positions(batch, T, page=1 << 30)
        for x, y in zip((hq, hk), out):
            close(y, *srv.rotary(x, pos, rotary.frequencies, 1.0, False, MARK))


def test_other_streams_and_an_object_made_behind_other_work():
    q = ref.rows(9, 5, 2, 64, BF16).cuda()
    positions = torch.arange(5, dtype=torch.int32, device="cuda")
    want = etk.Rotary(64, device="cuda")(q, positions=positions)
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    rotary = etk.Rotary(64, device="cuda")
    stream = torch.cuda.Stream()
    got = rotary(q, positions=positions, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_empty_calls_and_overlaps():
    rotary = etk.Rotary(64, device="cuda")
    none = torch.zeros(0, 2, 64, dtype=BF16, device="cuda")
    assert rotary(none, positions=torch.zeros(0, dtype=torch.int32, device="cuda")).shape == (0, 2, 64)
    x = torch.zeros(8, 4, 64, dtype=BF16, device="cuda")
    positions = torch.zeros(4, dtype=torch.int32, device="cuda")
    for q, k, out in ((x[:4], None, x[1:5]), (x[:4, :2], x[:4, 2:], (x[4:, :2], x[4:, 1:3])), (x[:4, :2], x[:4, 2:], (x[:4, 2:], x[:4, :2])),
                      (x[:4], x[:4], (x[:4], x[:4])), (x[:4], x[:4], (x[:4], x[4:])), (x[:4], x[:4], (x[4:], x[:4])), (x[:4, :, :], None, x[:1].expand(4, 4, 64))):
        with pytest.raises(ValueError):
            rotary(q, k, positions=positions, out=out)
    rotary(x[:4, :2], x[:4, 2:], positions=positions, out=(x[:4, :2], x[4:, 1:3]))


@pytest.mark.parametrize("T", [1, 2])
def test_in_place_on_heads_that_interleave(T):
    """Queries, keys and values of a projection [tokens, heads, 3, channels], turned in place: a single token, as a batch of one decodes."""
    x = ref.rows(10, T, 12, 64, BF16).view(T, 4, 3, 64)
    wide = x.cuda()
    rotary = etk.Rotary(64, device="cuda")
    positions = torch.arange(7, 7 + T, dtype=torch.int32, device="cuda")
    rotary(wide[:, :, 0], wide[:, :, 1], positions=positions, out=(wide[:, :, 0], wide[:, :, 1]))
    for i in range(2):
        close(wide[:, :, i], *srv.rotary(x[:, :, i], range(7, 7 + T), rotary.frequencies, 1.0, False, MARK))
    assert torch.equal(wide[:, :, 2].cpu(), x[:, :, 2])


@pytest.mark.parametrize("new", [[3, 1, 2, 5], [1, 1, 1, 1]])
def test_lengths_beyond_the_table_are_clamped_to_it(new):
    """As by the cache's operators, where the page size is given; as they are without."""
    lens, width = [100, 64, 2 ** 31 - 1, 30], 4
    single = all(n == 1 for n in new)
    for page_size, most in ((16, 64), (32, 128), (None, 1 << 30)):
        batch = sequences([min(n, most) for n in lens], new)
        table = torch.zeros(4, width, dtype=torch.int32, device="cuda")
        dev = etk.SequenceBatch(table, torch.tensor(lens, dtype=torch.int32, device="cuda"), None if single else batch[2].cuda())
        q = ref.rows(11, sum(new), 3, 64, BF16)
        rotary = etk.Rotary(64, device="cuda")
        got = rotary(q.cuda(), batch=dev, page_size=page_size)
        close(got, *srv.rotary(q, srv.positions(batch, sum(new), page=1 << 30), rotary.frequencies, 1.0, False, MARK))
    for bad in (0, 17, 256):
        with pytest.raises(ValueError, match="page_size"):
            rotary(q.cuda(), batch=dev, page_size=bad)


@pytest.mark.parametrize("make", [etk.KVCache, etk.KVCache4])
def test_a_step_on_lengths_beyond_the_table_is_one_on_the_clamped_lengths(make):
    """Angles, the places that are written and the tokens that are attended to go together."""
    page, dim, width, heads, group, new = 16, 64, 4, 2, 4, [3, 1]
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, width)
    start = torch.tensor([0, 3, 4], dtype=torch.int32, device="cuda")
    q, k, v = (ref.rows(12 + i, 4, h, dim, BF16).cuda() for i, h in enumerate((heads * group, heads, heads)))
    old = [ref.rows(15 + i, 2 * width * page, heads, dim, BF16).cuda() for i in range(2)]
    full = etk.SequenceBatch(table, torch.full((2,), width * page, dtype=torch.int32, device="cuda"),
                             torch.tensor([0, width * page, 2 * width * page], dtype=torch.int32, device="cuda"))
    got = []
    for lens in ([width * page, 50], [100, 50], [2 ** 31 - 1, 50]):
        cache = make.allocate(8, heads, page, dim, device="cuda")
        etk.cache_write(cache, full, *old)
        step = etk.SparseAttention(cache, 2, 4, heads * group, width, 3, 1, 1, rotary=etk.Rotary(dim, device="cuda"))
        out = step(q, etk.SequenceBatch(table, torch.tensor(lens, dtype=torch.int32, device="cuda"), start), k, v)
        got.append([out, cache.k.view(torch.uint8), cache.v.view(torch.uint8), step.blocks.sort(-1).values])
    for other in got[1:]:
        for x, y in zip(got[0], other):
            assert torch.equal(x, y)


@pytest.mark.parametrize("amplitude", [1.0, 1.25, -0.5])
def test_there_and_back_gives_the_amplitudes_square(amplitude):
    """The way back is off by its own tolerance and by what the way there rounded: turned back, that of a pair's two numbers."""
    pos, dim, rot = [0, 5, 70000], 64, 48
    rotary = etk.Rotary(dim, rot, amplitude=amplitude, device="cuda")
    positions = torch.tensor(pos, dtype=torch.int32, device="cuda")
    x = ref.rows(20, 3, 2, dim, FP16)
    there = rotary(x.cuda(), positions=positions)
    _, tol = srv.rotary(x, pos, rotary.frequencies, amplitude, False, MARK)
    _, back_tol = srv.rotary(there.cpu(), pos, rotary.frequencies, amplitude, False, MARK, inverse=True)
    pair = tol[..., :rot // 2] + tol[..., rot // 2:rot]
    tol = torch.cat([pair, pair, tol[..., rot:]], -1) * abs(amplitude) + back_tol
    by = torch.ones(dim, dtype=torch.float64)
    by[:rot] = amplitude ** 2
    close(rotary(there, positions=positions, inverse=True), x.double() * by, tol)


@pytest.mark.parametrize("lens,new", [([300, 5, 40, 129], [130, 0, 40, 2]), ([3, 0, 70], [5, 2, 9]), ([1], [1])])
def test_outputs_that_the_call_makes(lens, new):
    """Without `out`: as into tensors of the caller's where a row has a position, zeros elsewhere; without k, as with it."""
    batch = sequences(lens, new)
    T = sum(new) + 3  # rows behind the last sequence
    q, k = ref.rows(30, T, 5, 64, BF16, 3.0), ref.rows(31, T, 2, 64, BF16)
    q[-3:], k[-3:] = math.nan, math.inf
    rotary, dev = etk.Rotary(64, 48, device="cuda"), device_batch(batch)
    there = torch.tensor([p is not None for p in srv.positions(batch, T, page=1 << 30)])
    assert not there.all() and there.any()
    into = torch.full_like(q, MARK, device="cuda"), torch.full_like(k, MARK, device="cuda")
    rotary(q.cuda(), k.cuda(), batch=dev, out=into)
    for got, want in zip((*rotary(q.cuda(), k.cuda(), batch=dev), rotary(q.cuda(), batch=dev)), (*into, into[0])):
        assert got.is_contiguous() and torch.equal(got[there], want[there])
        assert (got[~there] == 0).all() and (want[~there] == MARK).all()
