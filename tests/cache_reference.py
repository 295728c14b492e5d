"""Plain 64-bit forms of the cache operators, written out token by token on the CPU, and the
inputs of their tests."""

import math

import numpy as np
import torch

FP8 = torch.float8_e4m3fn
LOW, HIGH = -40, 40


def e4m3(y):
    """The nearest e4m3 value of each |y| <= 448, ties to the even one; NaN and infinities give NaN."""
    a = y.abs()
    e = torch.floor(torch.log2(torch.where(a > 2.0 ** -6, a, 2.0 ** -6)))
    step = torch.exp2(e - 3)
    r = torch.copysign(torch.round(a / step) * step, y)
    return torch.where(y.isfinite(), r.clamp(-448, 448), math.nan)


def scale_for(rows):
    a = rows.abs()
    top = float(torch.where(a.isfinite(), a, 0.0).max()) if rows.numel() else 0.0
    e = LOW
    while e < HIGH and top > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** e


class Cache:
    """A cache in 64 bits: k, v hold the codes' values."""

    def __init__(self, k, v, k_scale, v_scale, bounds):
        self.k, self.v, self.k_scale, self.v_scale, self.bounds = (
            t.detach().cpu().double().clone() for t in (k, v, k_scale, v_scale, bounds))
        self.dtype = bounds.dtype
        self.pages, self.heads, self.page, self.dim = k.shape

    def page_of(self, table, j):
        p = int(table[j])
        return p if 0 <= p < self.pages else None

    def rows(self, name, table, head, positions):
        """Stored numbers [n, dim] and which positions have a page."""
        codes, scale = getattr(self, name), getattr(self, name + "_scale")
        x = torch.zeros(len(positions), self.dim, dtype=torch.float64)
        there = torch.zeros(len(positions), dtype=torch.bool)
        for j in sorted({p // self.page for p in positions}):
            at = self.page_of(table, j)
            if at is None:
                continue
            which = [i for i, p in enumerate(positions) if p // self.page == j]
            x[which] = codes[at, head, [positions[i] % self.page for i in which]] * scale[at, head]
            there[which] = True
        return x, there


def spans(batch, tokens, page):
    """(sequence, first row, rows, length) with everything clamped as the kernels do."""
    table, kv_len, q_start = batch
    width = table.shape[1]
    for b in range(table.shape[0]):
        lo, hi = (b, b + 1) if q_start is None else (min(max(int(q_start[b + i]), 0), tokens) for i in (0, 1))
        yield b, lo, max(0, hi - lo), min(max(int(kv_len[b]), 0), width * page)


def write(cache, batch, k, v):
    table = batch[0]
    k, v = k.detach().cpu().double(), v.detach().cpu().double()
    most = torch.finfo(cache.dtype).max
    for b, lo, n, length in spans(batch, k.shape[0], cache.page):
        first = max(length - n, 0)
        while first < length:
            j, o = divmod(first, cache.page)
            m = min(cache.page - o, length - first)
            at = cache.page_of(table[b], j)
            r = lo + first - (length - n)
            if at is not None:
                for name, src in (("k", k), ("v", v)):
                    codes, scales = getattr(cache, name), getattr(cache, name + "_scale")
                    for h in range(cache.heads):
                        rows = src[r:r + m, h]
                        s = scale_for(rows)
                        if o:
                            was = float(scales[at, h])
                            s = max(s, was)
                            codes[at, h, :o] = e4m3(codes[at, h, :o] * (was / s))
                        y = rows / s
                        y = torch.where(y.isfinite(), y.clamp(-448, 448), y)
                        codes[at, h, o:o + m] = e4m3(y)
                        scales[at, h] = s
                x = torch.where(k[r:r + m].isnan(), 0.0, k[r:r + m]).clamp(-most, most)
                hi, lo_ = x.amax(0), x.amin(0)
                if o:
                    hi, lo_ = torch.maximum(hi, cache.bounds[at, :, 0]), torch.minimum(lo_, cache.bounds[at, :, 1])
                cache.bounds[at, :, 0], cache.bounds[at, :, 1] = hi, lo_
            first += m


def read(cache, batch, tokens, fill=0.0):
    out = [torch.full((tokens, cache.heads, cache.dim), fill, dtype=torch.float64) for _ in range(2)]
    for b, lo, n, length in spans(batch, tokens, cache.page):
        pos = [length - n + i for i in range(n)]
        for x, name in zip(out, ("k", "v")):
            x[lo:lo + n] = 0.0
            good = [i for i in range(n) if pos[i] >= 0]
            for h in range(cache.heads):
                x[[lo + i for i in good], h] = cache.rows(name, batch[0][b], h, [pos[i] for i in good])[0]
    return [x.to(cache.dtype) for x in out]


def scores(cache, batch, q, keep_first, keep_last, fill):
    """(scores, ke, the sum of the terms' magnitudes of each score)."""
    q = q.detach().cpu().double()
    T, QH, D = q.shape
    G, width = QH // cache.heads, batch[0].shape[1]
    out = torch.full((T * cache.heads, width), fill, dtype=torch.float64)
    size = torch.zeros_like(out)
    ke = torch.full((T * cache.heads,), int(fill), dtype=torch.int32)
    for b, lo, n, length in spans(batch, T, cache.page):
        for i in range(n):
            pos = length - n + i
            for h in range(cache.heads):
                r = (lo + i) * cache.heads + h
                ke[r] = pos // cache.page + 1 if pos >= 0 else 0
                for j in range(int(ke[r])):
                    at = cache.page_of(batch[0][b], j)
                    if at is None:
                        out[r, j] = -math.inf
                    elif j < keep_first or j >= int(ke[r]) - keep_last:
                        out[r, j] = math.inf
                    else:
                        u = q[lo + i, h * G:(h + 1) * G]
                        terms = torch.maximum(u * cache.bounds[at, h, 0], u * cache.bounds[at, h, 1])
                        out[r, j] = terms.sum(-1).max()
                        size[r, j] = terms.abs().sum(-1).max()
    return out, ke, size


def attention(cache, batch, q, blocks, scale, fill):
    """(out, tolerance): the definition, and how far a kernel of this design may be from it.

    The kernel rounds each probability to FP16: 2^-11 of it where it is normal, 2^-25 where it is
    below FP16's normal range, against a largest one of at least 1. Its FP32 scores are sums
    of D exact products with errors of at most 2^-23 of the terms' magnitudes for each term,
    with three roundings more (2^-24 each), and exp2 is within 2^-21: e^x carries the absolute error of x as its
    relative one. The sum l of the probabilities has the same relative errors. The FP32 sums of
    the second product, the rescaling and the joins add 2^-24 for each of n + 40 steps. The result
    is rounded to the output's type once."""
    q = q.detach().cpu().double()
    T, QH, D = q.shape
    G = QH // cache.heads
    out = torch.full(q.shape, fill, dtype=torch.float64)
    tol = torch.zeros_like(out)
    eps = torch.finfo(cache.dtype).eps / 2
    tiny = torch.finfo(cache.dtype).smallest_normal * eps * 2
    lists = None if blocks is None else blocks.detach().cpu()
    for b, lo, n, length in spans(batch, T, cache.page):
        for i in range(n):
            pos = length - n + i
            for h in range(cache.heads):
                if lists is None:
                    at = list(range(pos + 1))
                else:
                    want = {int(x) for x in lists[(lo + i) * cache.heads + h] if pos >= 0 and 0 <= x <= pos // cache.page}
                    at = [p for j in sorted(want) for p in range(j * cache.page, min((j + 1) * cache.page, pos + 1))]
                k, there = cache.rows("k", batch[0][b], h, at)
                v, _ = cache.rows("v", batch[0][b], h, at)
                k, v = k[there], v[there]
                for g in range(h * G, (h + 1) * G):
                    if not len(k):
                        out[lo + i, g] = 0.0
                        continue
                    u = q[lo + i, g]
                    x = k @ u * scale
                    p = torch.softmax(x, 0)
                    out[lo + i, g] = p @ v
                    terms = float((k.abs() @ u.abs()).max() * abs(scale))
                    rel = 2.0 ** -11 + 2.0 ** -21 + terms * (D + 3) * 2.0 ** -23
                    rel = 2 * rel + (len(k) + 40) * 2.0 ** -24
                    tol[lo + i, g] = rel * (p @ v.abs()) + len(k) * 2.0 ** -25 * v.abs().max(0).values * 2
    tol = tol + out.abs().nan_to_num(0.0, 0.0, 0.0) * eps + tiny
    return out, tol


# ---- inputs ----

def make(seed, lens, new, heads, page, dim, dtype, spare=2, width=None, spread=4, poison=True, pages=None):
    """A cache with the pages of sequences of `lens` tokens, `new` of each new; tables in no order. Codes behind a
    sequence's end, pages of no sequence and (with poison) everything else that nothing may read hold NaN."""
    g = torch.Generator().manual_seed(seed)
    held = [-(-n // page) for n in lens]
    total = sum(held) + spare if pages is None else pages
    width = max(1, max(held)) if width is None else width
    order = torch.randperm(total, generator=g)
    table = torch.full((len(lens), width), total + 7 if poison else 0, dtype=torch.int32)
    at = 0
    codes = [(torch.randn(total, heads, page, dim, generator=g) * 100).clamp(-448, 448).to(FP8) for _ in range(2)]
    used = torch.zeros(total, page, dtype=torch.bool)
    for b, n in enumerate(held):
        table[b, :n] = order[at:at + n].int()
        for j in range(n):
            used[order[at + j], :max(0, min(page, lens[b] - j * page))] = True
        at += n
    if poison:
        for c in codes:
            c.view(torch.uint8)[~used[:, None, :].expand(total, heads, page)] = 0x7F
    scale = [torch.exp2(torch.randint(-7 - spread, -6, (total, heads), generator=g).float()) for _ in range(2)]
    mid, half = torch.randn(total, heads, dim, generator=g), torch.rand(total, heads, dim, generator=g)
    bounds = torch.stack([mid + half, mid - half], 2).to(dtype)
    q_start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
    return (codes[0], codes[1], scale[0], scale[1], bounds), (table, torch.tensor(lens, dtype=torch.int32), q_start)


def rows(seed, tokens, heads, dim, dtype, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(tokens, heads, dim, generator=g) * size).to(dtype)
