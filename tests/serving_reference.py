"""Plain 64-bit forms of the 4-bit cache, of rotary positions and of the page tables, written out on the CPU, and the
inputs of their tests. What the 4-bit cache shares with the 8-bit one is cache_reference's."""

import math

import torch

import cache_reference as ref

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
SCALES = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()  # 0 to 448, ascending
GROUP = 16


def nearest(a, grid):
    """The place in an ascending grid nearest to each a, ties to the even place; beyond the last one, the last."""
    i = torch.searchsorted(grid, a.contiguous()).clamp(1, len(grid) - 1)
    below, above = a - grid[i - 1], grid[i] - a
    return torch.where((above < below) | ((above == below) & (i % 2 == 0)), i, i - 1)


def values(codes, scale):
    """Numbers [..., dim] of codes [..., dim / 2] and scales [..., dim / 16], without the unit."""
    both = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    x = GRID[both & 7] * torch.where(both >= 8, -1.0, 1.0).double()
    return (x.unflatten(-1, (-1, GROUP)) * scale.double()[..., None]).flatten(-2)


def quantise(x, unit):
    """Scales' codes [..., dim / 16] and the values (without the unit) of rows x [..., dim]."""
    x = x.double().unflatten(-1, (-1, GROUP))
    top = x.abs().amax(-1)
    fine = x.isfinite().all(-1)
    code = nearest(torch.where(fine, top, 0.0) / 6 / unit, SCALES).clamp(min=1)
    scale = SCALES[code]
    y = GRID[nearest(x.abs().nan_to_num(0.0, 0.0) / unit / scale[..., None], GRID)]
    value = torch.copysign(y, x) * scale[..., None]
    value = torch.where(fine[..., None], value, math.nan)
    return torch.where(fine, code, 0x7F).to(torch.uint8), value.flatten(-2)


class Cache4(ref.Cache):
    """As ref.Cache: k and v hold code * scale, k_scale and v_scale the units; scale codes beside them."""

    def __init__(self, k, v, k_scale, v_scale, bounds, k_unit=1.0, v_unit=1.0):
        k, v, k_scale, v_scale = (t.detach().cpu().clone() for t in (k, v, k_scale, v_scale))
        self.k, self.v = values(k, k_scale), values(v, v_scale)
        self.k_codes, self.v_codes = k_scale.view(torch.uint8), v_scale.view(torch.uint8)
        self.bounds, self.dtype = bounds.detach().cpu().double().clone(), bounds.dtype
        self.pages, self.heads, self.page, self.dim = *k.shape[:3], k.shape[3] * 2
        self.k_unit, self.v_unit = k_unit, v_unit
        self.k_scale, self.v_scale = (torch.full((self.pages, self.heads), u, dtype=torch.float64) for u in (k_unit, v_unit))


def write(cache, batch, k, v):
    table = batch[0]
    k, v = k.detach().cpu().double(), v.detach().cpu().double()
    most = torch.finfo(cache.dtype).max
    for b, lo, n, length in ref.spans(batch, k.shape[0], cache.page):
        first = max(length - n, 0)
        while first < length:
            j, o = divmod(first, cache.page)
            m = min(cache.page - o, length - first)
            at = cache.page_of(table[b], j)
            r = lo + first - (length - n)
            if at is not None:
                for name, src in (("k", k), ("v", v)):
                    codes, value = quantise(src[r:r + m].transpose(0, 1), getattr(cache, name + "_unit"))
                    getattr(cache, name)[at, :, o:o + m] = value
                    getattr(cache, name + "_codes")[at, :, o:o + m] = codes
                x = torch.where(k[r:r + m].isnan(), 0.0, k[r:r + m]).clamp(-most, most)
                hi, lo_ = x.amax(0), x.amin(0)
                if o:
                    hi, lo_ = torch.maximum(hi, cache.bounds[at, :, 0]), torch.minimum(lo_, cache.bounds[at, :, 1])
                cache.bounds[at, :, 0], cache.bounds[at, :, 1] = hi, lo_
            first += m


def make(seed, lens, new, heads, page, dim, dtype, size=0.3, **kw):
    """As ref.make: codes of every kind, scales around `size`; what nothing may read has NaN scales."""
    poison = kw.get("poison", True)
    tensors, batch = ref.make(seed, lens, new, heads, page, dim, dtype, **kw)
    total = tensors[0].shape[0]
    g = torch.Generator().manual_seed(seed + 1000)
    codes = [torch.randint(0, 256, (total, heads, page, dim // 2), generator=g, dtype=torch.uint8) for _ in range(2)]
    scales = [(torch.exp(torch.randn(total, heads, page, dim // GROUP, generator=g) * 0.5) * size).clamp(max=448).to(torch.float8_e4m3fn)
              for _ in range(2)]
    if poison:
        behind = (tensors[0].view(torch.uint8)[:, 0, :, 0] == 0x7F) & (tensors[1].view(torch.uint8)[:, 0, :, 0] == 0x7F)
        for s in scales:
            s.view(torch.uint8)[behind[:, None, :].expand(total, heads, page)] = 0x7F
    return (codes[0], codes[1], scales[0], scales[1], tensors[4]), batch


def positions(batch, tokens, page=1 << 24):
    """Position of each row, None where it has none."""
    out = [None] * tokens
    for b, lo, n, length in ref.spans((torch.zeros(len(batch[1]), 64), *batch[1:]), tokens, page):
        for i in range(n):
            if length - n + i >= 0:
                out[lo + i] = length - n + i
    return out


def rotary(x, pos, frequencies, amplitude, neighbours, fill, inverse=False):
    """(rows turned, tolerance). FP32: the angle's fraction of a turn is rounded by 2^-24 of itself, which moves a cosine or sine
    by at most pi 2^-24; the function is within 2 units of 2^-23 of one; the amplitude, two products and a sum round by 2^-24
    each: 11 * 2^-24 of amplitude * (|x1| + |x2|) in all. Then one rounding to the type."""
    from fractions import Fraction

    x64, R = x.detach().cpu().double(), 2 * len(frequencies)
    out, tol = x64.clone(), torch.zeros_like(x64)
    i = torch.arange(R // 2)
    a, b = (2 * i, 2 * i + 1) if neighbours else (i, i + R // 2)
    pi = Fraction("3.14159265358979323846264338327950288419716939937510")
    eps = torch.finfo(x.dtype).eps / 2
    tiny = torch.finfo(x.dtype).smallest_normal * eps * 2
    for t, p in enumerate(pos):
        if p is None:
            out[t] = fill
            continue
        turns = [Fraction(f) * (-p if inverse else p) / (2 * pi) for f in frequencies]
        angle = torch.tensor([float((u - math.floor(u)) * 2 * pi) for u in turns], dtype=torch.float64)
        c, s = angle.cos() * amplitude, angle.sin() * amplitude
        out[t, :, a] = x64[t][:, a] * c - x64[t][:, b] * s
        out[t, :, b] = x64[t][:, b] * c + x64[t][:, a] * s
        both = (x64[t][:, a].abs() + x64[t][:, b].abs()) * abs(amplitude) * 11 * 2.0 ** -24
        tol[t, :, a], tol[t, :, b] = both, both
    turned = torch.zeros(x.shape[-1], dtype=torch.bool)
    turned[:R] = True
    tol += torch.where(turned, out.abs() * eps + tiny, 0.0)
    return out, tol


class Tables:
    """Page tables and a ring of free pages as lists, changed sequence by sequence."""

    def __init__(self, table, kv_len, free_pages, free_range, page, max_tokens):
        self.table, self.kv_len = table.tolist(), kv_len.tolist()
        self.ring, self.range = free_pages.tolist(), free_range.tolist()
        self.page, self.max_tokens = page, max_tokens
        self.slots, self.positions = [-7] * max_tokens, [-7] * max_tokens
        self.q_start, self.applied = [0] * (len(self.kv_len) + 1), [0] * len(self.kv_len)

    def update(self, change):
        n, P, width = len(self.ring), self.page, len(self.table[0])
        head, free = self.range
        pages = lambda x: -(-x // P)  # noqa: E731
        want = [max(c, -x) for c, x in zip(change, self.kv_len)]
        want = [c if x + c <= width * P else 0 for c, x in zip(want, self.kv_len)]
        back = []
        for b, c in enumerate(want):
            if c < 0:
                back += self.table[b][pages(self.kv_len[b] + c):pages(self.kv_len[b])]
        for i, page in enumerate(back):
            self.ring[(head + free + i) % n] = page
        free += len(back)
        asked_pages = asked_rows = row = taken = 0
        for b, c in enumerate(want):
            self.q_start[b] = row
            self.applied[b] = c
            old = self.kv_len[b]
            if c > 0:
                need = pages(old + c) - pages(old)
                asked_pages += need
                asked_rows += c
                if (need and asked_pages > free) or asked_rows > self.max_tokens:
                    self.applied[b] = 0
                    continue
                for j in range(pages(old), pages(old) + need):
                    self.table[b][j] = self.ring[(head + taken) % n]
                    taken += 1
                for p in range(old, old + c):
                    self.slots[row] = self.table[b][p // P] * P + p % P
                    self.positions[row] = p
                    row += 1
            self.kv_len[b] = old + c
        self.q_start[-1] = row
        self.range = [(head + taken) % n, free - taken]


def attention(cache, batch, q, blocks, scale, fill):
    """cache_reference.attention and its tolerance, many rows at a time: for calls of thousands of rows."""
    q = q.detach().cpu().double()
    T, QH, D = q.shape
    G = QH // cache.heads
    out, tol = torch.full(q.shape, fill, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    eps = torch.finfo(cache.dtype).eps / 2
    tiny = torch.finfo(cache.dtype).smallest_normal * eps * 2
    for b, lo, n, length in ref.spans(batch, T, cache.page):
        if n == 0:
            continue
        if length == 0:
            out[lo:lo + n] = 0.0
            continue
        pos = length - n + torch.arange(n)
        at = list(range(length))
        for h in range(cache.heads):
            k, there = cache.rows("k", batch[0][b], h, at)
            v, _ = cache.rows("v", batch[0][b], h, at)
            seen = (torch.arange(length) <= pos[:, None]) & there
            if blocks is not None:
                lists = blocks.detach().cpu().reshape(-1, cache.heads, blocks.shape[1])[lo:lo + n, h].long()
                width = -(-length // cache.page) + 1
                taken = torch.zeros(n, width, dtype=torch.bool)
                good = (lists >= 0) & (lists <= pos[:, None].div(cache.page, rounding_mode="floor"))
                taken.scatter_(1, torch.where(good, lists, width - 1), True)
                taken[:, -1] = False
                seen &= taken[:, torch.arange(length) // cache.page]
            u = q[lo:lo + n, h * G:(h + 1) * G]
            bad_v = v.isnan().any(-1)  # a NaN value reaches the rows that see it, and no other
            x = torch.where(seen[:, None], u @ k.T * scale, -math.inf)
            p = torch.softmax(x, -1)
            none = ~seen.any(-1)
            p = torch.where(none[:, None, None], 0.0, p)
            fine = v.nan_to_num(0.0)
            y = p @ fine
            hit = (seen & bad_v).double() @ v.isnan().double() > 0  # [n, D]
            out[lo:lo + n, h * G:(h + 1) * G] = torch.where(hit[:, None], math.nan, y)
            count = seen.sum(-1).double()[:, None, None]
            terms = torch.where(seen[:, None], u.abs() @ k.abs().T, 0.0).nan_to_num(0.0).amax(-1, keepdim=True) * abs(scale)
            rel = 2.0 ** -11 + 2.0 ** -21 + terms * (D + 3) * 2.0 ** -23
            rel = 2 * rel + (count + 40) * 2.0 ** -24
            most = torch.where(seen[:, :, None], fine.abs(), 0.0).amax(1)[:, None]
            tol[lo:lo + n, h * G:(h + 1) * G] = rel * (p.nan_to_num(0.0) @ fine.abs()) + count * 2.0 ** -25 * most * 2
    return out, tol + out.abs().nan_to_num(0.0, 0.0, 0.0) * eps + tiny
