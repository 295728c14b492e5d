"""What surrounds attention over a paged cache in 4 bits: the cases it is measured on.

Five operators, in the order of a serving step:

  tables  sequences grow and shrink: pages come from a ring of free ones and go back to it, with the lengths, the
          row ranges, and for each new row its slot in the cache and its position
  rotary  queries and keys turned by their positions
  write   new keys and values go into pages of e2m1 codes with one e4m3 scale for 16 channels of a token and one unit
          for the cache; they are read back as the values that their codes stand for
  read    the stored tokens of each sequence come back as rows of bf16 or fp16
  attend  attention of each sequence's last tokens over its whole cache, or over the pages that a list names for each
          token and key head

`own` selects between the plain torch form and the framework's kernels; `exact` is the definition in 64 bits.
"""

import math
import random

import torch

own = False

FP8 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
GROUP = 16  # channels that share a scale
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # magnitudes of the codes


def case(name, op, dtype, dim, page, heads, group, seqs, lo, hi, new_lo=1, new_hi=1, blocks=0, drift=0.0, rot=0, base=10000.0, factor=1.0, pairs="half"):
    """heads: key heads, group: query heads for each, seqs sequences of lo..hi tokens, new_lo..new_hi of them new."""
    c = {"op": op, "dtype": dtype, "dim": dim, "page": page, "heads": heads, "group": group, "seqs": seqs, "lo": lo, "hi": hi, "new_lo": new_lo,
         "new_hi": new_hi, "blocks": blocks, "drift": drift, "rot": rot, "base": base, "factor": factor, "pairs": pairs}
    return dict(c, name=name) if name else c


def listed():
    return [
        # a decoding batch takes a token each, and gives it back: latency
        case("tables_step", "tables", "bf16", 128, 64, 4, 8, 64, 2048, 65536),
        # a thousand prompts are admitted at once, with small pages, and leave again
        case("tables_prompts", "tables", "bf16", 64, 16, 8, 1, 1000, 1, 2047, 1, 2047),
        # one decoding step's queries and keys, positions up to 65536 under a scaled context: latency
        case("rotary_step", "rotary", "bf16", 128, 64, 4, 8, 64, 2048, 65536, 1, 1, 0, 0.0, 128, 500000.0, 8.0),
        # prompts of a batch behind long prefixes, neighbouring channels in pairs, half of each head turned
        case("rotary_prompts", "rotary", "fp16", 128, 64, 4, 8, 8, 100000, 131072, 4001, 4999, 0, 0.0, 64, 10000.0, 1.0, "neighbours"),
        # one decoding step's keys and values of 64 sequences: latency
        case("write_step", "write", "bf16", 128, 64, 8, 1, 64, 2048, 65536),
        # prompts of a batch, ragged, written at once behind what is cached
        case("write_prompts", "write", "bf16", 128, 64, 8, 1, 24, 5000, 8192, 4001, 4999),
        # a few short sequences copied out, as before a page is moved to another pool
        case("read_short", "read", "bf16", 128, 64, 4, 1, 4, 100, 1000, 100, 100),
        # long shared prefixes read back for a prompt that runs on unquantised rows
        case("read_prefixes", "read", "fp16", 64, 16, 8, 1, 8, 32768, 65536, 32768, 32768),
        # a decoding batch, ragged between 2048 and 65536 tokens
        case("dense_step", "attend", "bf16", 128, 64, 4, 8, 64, 2048, 65536),
        # a prompt's chunk over everything before it
        case("dense_chunk", "attend", "bf16", 128, 64, 2, 8, 1, 16384, 16384, 2048, 2048),
        # a decoding step over 32 selected pages (2048 tokens) of each sequence
        case("sparse_step", "attend", "bf16", 128, 64, 4, 8, 64, 2048, 65536, 1, 1, 32),
        # a prompt's chunk: every token with its own 32 pages, most of them shared with its neighbours
        case("sparse_chunk", "attend", "bf16", 128, 64, 2, 8, 1, 131072, 131072, 4096, 4096, 32, 0.05),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "rotary", "write", "read", "attend", "attend", "attend"])
    dtype, dim, page = rng.choice(["bf16", "fp16"]), rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    seqs = _log(rng, 1, 64)
    if op == "tables":
        seqs = _log(rng, 1, 4096)
        new = max(1, _log(rng, 1, 1_000_000) // seqs)
        lo = new + _log(rng, 1, min(65536, 4_000_000 // seqs)) - 1
        return case("", op, dtype, dim, page, heads, group, seqs, max(1, lo // 3), lo, 1 + new // 2, new)
    if op == "rotary":
        new = max(1, _log(rng, 1, 32768) // seqs)
        lo = new + _log(rng, 1, 1_000_000) - 1
        rot = rng.choice([dim, dim, dim // 2, dim // 4])
        return case("", op, dtype, dim, page, heads, min(group, 8), seqs, lo, lo + _log(rng, 1, 2000), 1 + new // 2, new, 0, 0.0, rot,
                    rng.choice([10000.0, 500000.0, 1000000.0]), rng.choice([1.0, 4.0, 8.0, 32.0]), rng.choice(["half", "neighbours"]))
    if op in ("write", "read"):
        new = max(1, _log(rng, 1, 100000) // seqs)
        lo = new + _log(rng, 1, 4096) - 1
        return case("", op, dtype, dim, page, heads, 1, seqs, lo, lo + _log(rng, 1, 2000), 1 + new // 2, new)
    longest = _log(rng, 16, min(131072, 2_000_000 // seqs // max(1, heads // 4)))
    lo = max(1, int(longest * rng.uniform(0.05, 1.0)))
    if rng.random() < 0.5:
        most = max(1, min(256, 30_000_000 // (longest * seqs)))
        new = min(lo, rng.choice([1, 1, 2, rng.randint(1, 9), _log(rng, 1, most)]))
        return case("", op, dtype, dim, page, heads, group, seqs, lo, longest, 1 + new // 2, new)
    new = min(lo, rng.choice([1, rng.randint(1, 9), max(1, _log(rng, 8, 2048) // seqs)]))
    blocks = max(1, min(_log(rng, 128, 4096) // page, -(-lo // page)))
    return case("", op, dtype, dim, page, heads, min(group, 8), seqs, lo, longest, 1 + new // 2, new, blocks, rng.choice([0.01, 0.05, 0.3]))


def _lengths(c):
    """Tokens and new tokens of each sequence: the case's own, the same for each seed."""
    r = random.Random("%(seqs)d %(lo)d %(hi)d %(new_lo)d %(new_hi)d" % c)
    total = [r.randint(c["lo"], c["hi"]) for _ in range(c["seqs"])]
    return total, [min(t, r.randint(c["new_lo"], c["new_hi"])) for t in total]


def _pages(c):
    """Pages that the pool of a case holds for each sequence. A write reaches the last tokens' pages alone: its pool holds no others."""
    total, new = _lengths(c)
    if c["op"] == "write":
        return [(t - 1) // c["page"] - (t - n) // c["page"] + 1 for t, n in zip(total, new)]
    return [-(-t // c["page"]) for t in total]


def _frequencies(c):
    """Radians a position of each pair. Scaled by parts: pairs that turn often within the original 8192 positions are kept, those that
    turn less than once are slowed by the factor, a ramp between; and the factor that the result is brought to."""
    R, s = c["rot"], c["factor"]
    f = [c["base"] ** (-2 * i / R) for i in range(R // 2)]
    if s == 1.0:
        return f, 1.0
    ramp = [min(1.0, max(0.0, (8192 * x / (2 * math.pi) - 1) / (32 - 1))) for x in f]
    return [x * g + x / s * (1 - g) for x, g in zip(f, ramp)], 0.1 * math.log(s) + 1


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev, dt, D, P, H = "cuda", TYPES[c["dtype"]], c["dim"], c["page"], c["heads"]
    total, new = _lengths(c)
    held = _pages(c)
    width, pool, T = max(-(-t // P) for t in total), sum(held), sum(new)
    s = dict(c, most=max(new))

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    if c["op"] == "rotary":
        f, s["amplitude"] = _frequencies(c)
        s["f"] = torch.tensor(f, dtype=torch.float64, device=dev)
    if c["op"] == "tables":  # the new tokens are still to come; a ring of free pages, begun somewhere, holds one spare page in eight
        before = [t - n for t, n in zip(total, new)]
        used = sum(-(-t // P) for t in before)
        pool += pool // 8 + 1
        order = torch.randperm(pool, device=dev, generator=g).to(torch.int32)
        head = seed % pool
        s["pages"], s["change"] = pool, ints(new)
        s["free"] = torch.full((pool,), -1, dtype=torch.int32, device=dev)
        s["free"][(torch.arange(pool - used, device=dev) + head) % pool] = order[used:]
        s["range"] = ints([head, pool - used])
        s["slots"], s["positions"] = (torch.zeros(T, dtype=torch.int32, device=dev) for _ in range(2))
        s["kv_len"], s["q_start"] = ints(before), ints([0] * (c["seqs"] + 1))
        held = [-(-t // P) for t in before]
    else:
        order = torch.randperm(pool, device=dev, generator=g).to(torch.int32)  # pages lie in the pool in no order
        s["kv_len"] = ints(total)
        s["q_start"] = ints([sum(new[:b]) for b in range(len(new) + 1)])
    if c["op"] != "rotary":
        n = ints(held)
        end = ints([-(-t // P) for t in total]) if c["op"] != "tables" else n
        j = torch.arange(width, device=dev)
        mine = (j < end[:, None]) & (j >= (end - n)[:, None])
        at = (n.cumsum(0) - n)[:, None] + j - (end - n)[:, None]
        s["table"] = torch.where(mine, order[at.clamp(0, order.shape[0] - 1)], 0).to(torch.int32)
    single = all(n == 1 for n in new)
    if c["op"] in ("write", "read", "attend"):
        LUT = torch.tensor([16 * a + b for a in range(16) for b in range(16)], dtype=torch.uint8, device=dev).reshape(16, 16)

        def codes():  # normal values that fill the codes' range, about a thousand draws shared out at random
            edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=dev)
            x = torch.randn(1 << 20, 2, device=dev, generator=g) * 2
            q = torch.bucketize(x.abs(), edges) + 8 * (x < 0)
            pairs = LUT[q[:, 1], q[:, 0]]
            return pairs[torch.randint(0, 1 << 20, (pool, H, P, D // 2), device=dev, generator=g, dtype=torch.int32)]

        def scales():
            return (torch.exp(torch.randn(pool, H, P, D // GROUP, device=dev, generator=g) * 0.5) * 0.3).to(FP8)

        s["k"], s["v"], s["k_scale"], s["v_scale"] = codes(), codes(), scales(), scales()
        mid, half = torch.randn(pool, H, D, device=dev, generator=g), torch.rand(pool, H, D, device=dev, generator=g) * 2
        s["bounds"] = torch.stack([mid + half, mid - half], 2).to(dt)
        s["k_unit"], s["v_unit"] = 1.0, 0.25
    if c["op"] in ("rotary", "write"):
        s["new_k"] = (torch.randn(T, H, D, device=dev, generator=g) * torch.exp(torch.randn(H, D, device=dev, generator=g) * 0.5)).to(dt)
    if c["op"] == "write":
        s["new_v"] = torch.randn(T, H, D, device=dev, generator=g).to(dt)
    if c["op"] in ("write", "read"):
        s["out_k"], s["out_v"] = (torch.zeros(T, H, D, dtype=dt, device=dev) for _ in range(2))
    if c["op"] in ("rotary", "attend"):
        s["q"] = (torch.randn(T, H * c["group"], D, device=dev, generator=g) * 3).to(dt)
        s["out"] = torch.zeros_like(s["q"])
    if c["op"] == "rotary":
        s["out_k"] = torch.zeros_like(s["new_k"])
    if c["blocks"]:
        # What a token attends to drifts from token to token: a page's interest is a smooth function of the token with some noise on
        # it, so that neighbours share most of their pages. The first page and the newest two are always taken, and rows with fewer
        # pages than slots are padded with -1, as the selection leaves them.
        seq, pos = _tokens(s, T)
        score = torch.randn(c["seqs"], H, width, device=dev, generator=g)[seq]
        turn = torch.randn(c["seqs"], H, width, device=dev, generator=g)[seq]
        angle = (torch.arange(T, device=dev) * c["drift"] * 0.05)[:, None, None]
        score = score * angle.cos() + turn * angle.sin() + c["drift"] * torch.randn(T, H, width, device=dev, generator=g)
        page, newest = torch.arange(width, device=dev), (pos // P)[:, None, None]
        score = score.masked_fill((page < 1) | (page > newest - 2), math.inf).masked_fill(page > newest, -math.inf)
        best = score.topk(c["blocks"], -1)
        s["list"] = torch.where(best.values == -math.inf, -1, best.indices).to(torch.int32).reshape(T * H, c["blocks"])
        s["list"] = s["list"][:, torch.randperm(c["blocks"], device=dev, generator=g)].contiguous()
    if own:
        import exact_top_selection_gb300 as etk
        if c["op"] == "tables":
            s["tables"] = etk.PageTables(s["table"], s["kv_len"], s["free"], s["range"], P, T, slots=s["slots"], positions=s["positions"], q_start=s["q_start"])
        elif c["op"] == "rotary":
            s["table"] = torch.zeros(c["seqs"], 1, dtype=torch.int32, device=dev)
            s["batch"] = etk.SequenceBatch(s["table"], s["kv_len"], None if single else s["q_start"])
            s["rotary"] = etk.Rotary(D, c["rot"], c["base"], neighbours=c["pairs"] == "neighbours", factor=c["factor"],
                                     original_length=8192 if c["factor"] != 1.0 else None, device=dev)
        else:
            s["cache"] = etk.KVCache4(s["k"], s["v"], s["k_scale"], s["v_scale"], s["bounds"], s["k_unit"], s["v_unit"])
            s["batch"] = etk.SequenceBatch(s["table"], s["kv_len"], None if single else s["q_start"])
            if c["op"] == "attend":
                s["attention"] = etk.CacheAttention(s["cache"], c["seqs"], T, c["group"] * H, width, num_blocks=c["blocks"])
    return s


def run(s):
    if own:
        import exact_top_selection_gb300 as etk
        if s["op"] == "tables":
            t = s["tables"]
            t.update(s["change"])
            t.drop(t.applied)
            return s["table"], s["kv_len"], s["q_start"], s["slots"], s["positions"], s["free"], s["range"]
        if s["op"] == "rotary":
            return s["rotary"](s["q"], s["new_k"], batch=s["batch"], out=(s["out"], s["out_k"]))
        if s["op"] == "write":
            etk.cache_write(s["cache"], s["batch"], s["new_k"], s["new_v"])
            return etk.cache_read(s["cache"], s["batch"], out=(s["out_k"], s["out_v"])) + (s["k_scale"], s["v_scale"], s["bounds"])
        if s["op"] == "read":
            return etk.cache_read(s["cache"], s["batch"], out=(s["out_k"], s["out_v"]))
        return s["attention"](s["q"], s["batch"], blocks=s.get("list"), out=s["out"])
    return {"tables": _tables, "rotary": _rotary, "write": _write, "read": _read, "attend": _sparse if s["blocks"] else _dense}[s["op"]](s)


def _tokens(s, T):
    """Sequence and position of each of the T new tokens."""
    t = torch.arange(T, device=s["kv_len"].device)
    seq = torch.searchsorted(s["q_start"][1:].long(), t, right=True)
    return seq, (s["kv_len"] - s["q_start"][1:])[seq].long() + t


def _update(s, change):
    """Lengths changed by `change`, in place; what each sequence really got or gave back."""
    table, P, n, T = s["table"], s["page"], s["pages"], s["slots"].shape[0]
    B, width = table.shape
    head, free = s["range"].long().unbind()
    length, change = s["kv_len"].long(), change.long()
    less = torch.minimum(-change, length).clamp(min=0)
    asked = (change > 0) & (length + change <= width * P)
    old, small = -(-length // P), -(-(length - less) // P)
    need = torch.where(asked, -(-(length + change) // P) - old, 0)
    back = old - small
    # refused where the pages, or the rows, of a sequence and those asked for by the ones before it are more than there are
    fits = asked & ((need == 0) | (need.cumsum(0) <= free + back.sum())) & (torch.where(asked, change, 0).cumsum(0) <= T)
    got = torch.where(fits, change, 0)
    need = torch.where(fits, need, 0)
    # pages given back go behind the free ones, in the sequences' order; new ones come from the front
    j = torch.arange(width, device=table.device)
    given = (j >= small[:, None]) & (j < old[:, None])
    at = (head + free + (back.cumsum(0) - back)[:, None] + j - small[:, None]) % n
    ring = torch.cat([s["free"], s["free"][:1]])
    ring[torch.where(given, at, n)] = table
    s["free"].copy_(ring[:n])
    new = (j >= old[:, None]) & (j < (old + need)[:, None])
    at = (head + (need.cumsum(0) - need)[:, None] + j - old[:, None]) % n
    table.copy_(torch.where(new, s["free"][at], table))
    taken = need.sum()
    s["range"].copy_(torch.stack([(head + taken) % n, free + back.sum() - taken]))
    s["q_start"][1:] = got.cumsum(0)
    s["kv_len"].copy_(length + got - less)
    row = torch.arange(T, device=table.device)
    seq = torch.searchsorted(s["q_start"][1:].long(), row, right=True).clamp(max=B - 1)
    pos = length[seq] + row - s["q_start"][seq]
    there = row < s["q_start"][B]
    slot = table[seq, (pos // P).clamp(0, width - 1)] * P + pos % P
    s["slots"].copy_(torch.where(there, slot, s["slots"]))
    s["positions"].copy_(torch.where(there, pos, s["positions"]))
    return got - less


def _tables(s):
    _update(s, -_update(s, s["change"]))
    return s["table"], s["kv_len"], s["q_start"], s["slots"], s["positions"], s["free"], s["range"]


def _turned(x, cos, sin, R, pairs):
    """The first R channels of x [T, H, D] turned: pairs (i, i + R/2), or (2i, 2i + 1)."""
    a, b = (x[..., :R // 2], x[..., R // 2:R]) if pairs == "half" else (x[..., 0:R:2], x[..., 1:R:2])
    a, b = a * cos - b * sin, b * cos + a * sin
    y = torch.cat([a, b], -1) if pairs == "half" else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([y, x[..., R:]], -1)


def _rotary(s):
    _, pos = _tokens(s, s["q"].shape[0])
    angle = pos.double()[:, None, None] * s["f"]  # 32 bits lose the angles of far positions
    cos, sin = (angle.cos() * s["amplitude"]).float(), (angle.sin() * s["amplitude"]).float()
    s["out"].copy_(_turned(s["q"].float(), cos, sin, s["rot"], s["pairs"]))
    s["out_k"].copy_(_turned(s["new_k"].float(), cos, sin, s["rot"], s["pairs"]))
    return s["out"], s["out_k"]


def _quantise(x, unit):
    """x [T, H, D] as codes (two a byte), scales and the values that they stand for."""
    T, H, D = x.shape
    x = x.float().reshape(T, H, D // GROUP, GROUP)
    top = x.abs().amax(-1)
    scale = (top / 6 / unit).clamp(2.0 ** -9, 448)
    scale = torch.where(top.isfinite(), scale, math.nan).to(FP8)
    by = scale.float()[..., None] * unit
    a = (x / by).abs().clamp(max=6)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = torch.round(a / step) * step
    code = torch.where(a <= 2, a * 2, torch.where(a <= 3, 5, torch.where(a <= 4, 6, 7))).nan_to_num(7)
    code = (code + 8 * torch.signbit(x)).to(torch.uint8).reshape(T, H, D // 2, 2)
    return code[..., 0] | code[..., 1] << 4, scale, (torch.copysign(a, x) * by).reshape(T, H, D)


def _write(s):
    T, P = s["new_k"].shape[0], s["page"]
    seq, pos = _tokens(s, T)
    page, off = s["table"][seq, pos // P].long(), pos % P
    for name in ("k", "v"):
        codes, scale, value = _quantise(s["new_" + name], s[name + "_unit"])
        s[name][page, :, off] = codes
        s[name + "_scale"].view(torch.uint8)[page, :, off] = scale.view(torch.uint8)
        s["out_" + name].copy_(value)
    start = torch.full((s["k"].shape[0],), P, device=page.device).index_reduce_(0, page, off, "amin")
    most = torch.finfo(s["bounds"].dtype).max
    x = torch.where(s["new_k"].isnan(), 0, s["new_k"]).float().clamp(-most, most)
    fresh = (start == 0)[:, None, None]
    old = s["bounds"].float()
    hi = torch.where(fresh, -math.inf, old[:, :, 0]).index_reduce_(0, page, x, "amax")
    lo = torch.where(fresh, math.inf, old[:, :, 1]).index_reduce_(0, page, x, "amin")
    s["bounds"].copy_(torch.stack([hi, lo], 2))
    return s["out_k"], s["out_v"], s["k_scale"], s["v_scale"], s["bounds"]


def _values(codes, scale, unit, dtype=torch.float32):
    """The numbers that codes [..., D/2] with scales [..., D/16] stand for."""
    grid = torch.tensor(GRID + tuple(-x for x in GRID), dtype=dtype, device=codes.device)
    both = torch.stack([grid[None].expand(16, 16), grid[:, None].expand(16, 16)], -1).reshape(256, 2)
    x = both[codes.int()]  # [..., D/2, 2]
    x = x.reshape(*scale.shape, GROUP).mul_(scale.to(dtype).mul_(unit)[..., None])
    return x.flatten(-2)


def _read(s):
    T, P = s["out_k"].shape[0], s["page"]
    seq, pos = _tokens(s, T)
    page, off = s["table"][seq, pos // P].long(), pos % P
    for name in ("k", "v"):
        scale = s[name + "_scale"].view(torch.uint8)[page, :, off].view(FP8)
        s["out_" + name].copy_(_values(s[name][page, :, off], scale, s[name + "_unit"]))
    return s["out_k"], s["out_v"]


def _dense(s):
    T, H, G, P, D = s["q"].shape[0], s["heads"], s["group"], s["page"], s["dim"]
    B, width = s["table"].shape
    seq, pos = _tokens(s, T)
    i = torch.arange(T, device=pos.device) - s["q_start"][seq]
    most = s["most"]
    q = torch.zeros(B, H, most, G, D, device=pos.device)
    q[seq, :, i] = s["q"].float().reshape(T, H, G, D)
    end = torch.zeros(B, most, dtype=torch.long, device=pos.device)
    end[seq, i] = pos + 1
    at = s["table"].long()

    def rows(name):
        x = _values(s[name][at], s[name + "_scale"].view(torch.uint8)[at].view(FP8), s[name + "_unit"])  # [B, width, H, P, D]
        return x.transpose(1, 2).reshape(B, H, width * P, D)

    x = torch.matmul(q.reshape(B, H, most * G, D), rows("k").transpose(2, 3)) / math.sqrt(D)
    x = x.reshape(B, H, most, G, width * P)
    x = x.masked_fill(torch.arange(width * P, device=q.device) >= end[:, None, :, None, None], -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-1e30))
    total = x.sum(-1, keepdim=True)
    x = torch.matmul(x.reshape(B, H, most * G, -1), rows("v")).reshape(B, H, most, G, D) / torch.where(total > 0, total, 1)
    s["out"].copy_(x[seq, :, i].reshape(T, H * G, D))
    return s["out"]


def _sparse(s):
    T, H, G, P, D = s["q"].shape[0], s["heads"], s["group"], s["page"], s["dim"]
    K = s["blocks"]
    seq, pos = _tokens(s, T)
    want = s["list"].reshape(T, H, K).long().sort(-1).values
    newest = (pos // P)[:, None, None]
    good = (want >= 0) & (want <= newest)
    good[..., 1:] &= want[..., 1:] != want[..., :-1]
    want = want.clamp(0, s["table"].shape[1] - 1)
    at = s["table"][seq[:, None, None], want].long()
    head = torch.arange(H, device=at.device)[None, :, None]

    def rows(name):
        x = _values(s[name][at, head], s[name + "_scale"].view(torch.uint8)[at, head].view(FP8), s[name + "_unit"])  # [T, H, K, P, D]
        return x.reshape(T, H, K * P, D)

    place = want[..., None] * P + torch.arange(P, device=at.device)
    seen = (good[..., None] & (place <= pos[:, None, None, None])).reshape(T, H, 1, K * P)
    x = torch.matmul(s["q"].float().reshape(T, H, G, D), rows("k").transpose(2, 3)) / math.sqrt(D)
    x = x.masked_fill(~seen, -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-1e30))
    total = x.sum(-1, keepdim=True)
    x = torch.matmul(x, rows("v")) / torch.where(total > 0, total, 1)
    s["out"].copy_(x.reshape(T, H * G, D))
    return s["out"]


def work(c):
    """Each stored byte that the operator needs once, each new one once; products of the pairs that are seen."""
    total, new = _lengths(c)
    D, P, H, G, T = c["dim"], c["page"], c["heads"], c["group"], sum(new)
    number = 9 / 16  # bytes
    if c["op"] == "tables":
        pages = sum(-(-t // P) - -(-(t - n) // P) for t, n in zip(total, new))
        # pages read from the ring and put into the table, and the other way; slots and positions; change, lengths and row ranges twice
        return {"bytes": pages * 4 * 4 + T * 8 + 2 * c["seqs"] * 16, "flops": T * 4}
    if c["op"] == "rotary":
        return {"bytes": T * H * (1 + G) * D * 4, "flops": T * H * (1 + G) * c["rot"] * 3}
    if c["op"] == "write":
        return {"bytes": 2 * T * H * D * (2 + number + 2) + sum(_pages(c)) * H * 2 * 2 * D, "flops": T * H * D * 12}
    if c["op"] == "read":
        return {"bytes": 2 * T * H * D * (2 + number), "flops": T * H * D * 4}
    seen = [[t - n + i + 1 for i in range(n)] for t, n in zip(total, new)]  # tokens that each new token sees
    if not c["blocks"]:
        pairs = sum(sum(v) for v in seen)
        return {"bytes": sum(total) * H * D * 2 * number + T * H * G * D * 4, "flops": 4 * pairs * H * G * D}
    pairs = sum(min(x, c["blocks"] * P) for v in seen for x in v)
    # the cached bytes of a list's pages: those of one token alone are its own, a longer run's are at most the whole cache
    held = sum(min(t, sum(min(x, c["blocks"] * P) for x in v)) for t, v in zip(total, seen))
    return {"bytes": held * H * D * 2 * number + T * H * (c["blocks"] * 4 + G * D * 4), "flops": 4 * pairs * H * G * D}


def _nearest(a, grid):
    """The place in an ascending grid nearest to each a, ties to the even place; beyond the last one, the last."""
    grid = torch.tensor(grid, dtype=torch.float64, device=a.device)
    i = torch.searchsorted(grid, a).clamp(1, len(grid) - 1)
    below, above = a - grid[i - 1], grid[i] - a
    return torch.where((above < below) | ((above == below) & (i % 2 == 0)), i, i - 1)


E4M3 = tuple(m * 2.0 ** -9 for m in range(8)) + tuple((8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8))[:-1]


def exact(c, seed):
    total, new = _lengths(c)
    D, P, H, G, T = c["dim"], c["page"], c["heads"], c["group"], sum(new)
    if c["op"] == "tables" or (c["op"] == "write" and T * H * D > 1.5e8):
        return None
    s = prepare(c, seed)
    first = [sum(new[:b]) for b in range(len(new))]
    where = [(b, t - n + i) for b, (t, n) in enumerate(zip(total, new)) for i in range(n)]
    if c["op"] == "rotary":
        f, by = _frequencies(c)
        pos = torch.tensor([p for _, p in where], dtype=torch.float64, device="cuda")
        angle = pos[:, None] * torch.tensor(f, dtype=torch.float64, device="cuda")
        turn = torch.polar(torch.full_like(angle, by), angle)[:, None]
        out = []
        for x in (s["q"].double(), s["new_k"].double()):
            y, R = x.clone(), c["rot"]
            i = torch.arange(R // 2, device="cuda")
            a, b = (i, i + R // 2) if c["pairs"] == "half" else (2 * i, 2 * i + 1)
            z = torch.complex(x[..., a], x[..., b]) * turn
            y[..., a], y[..., b] = z.real, z.imag
            out.append(y)
        return tuple(out)
    if c["op"] == "write":
        grid, scales, rows = torch.tensor(GRID, dtype=torch.float64, device="cuda"), torch.tensor(E4M3, dtype=torch.float64, device="cuda"), []
        page = torch.tensor([s["table"][b].tolist()[p // P] for b, p in where] if T < 3000 else [], dtype=torch.long)
        held = []
        for name in ("k", "v"):
            x = s["new_" + name].double().reshape(T, H, -1, GROUP)
            scale = scales[_nearest(x.abs().amax(-1) / 6 / s[name + "_unit"], E4M3).clamp(min=1)]
            by = scale[..., None] * s[name + "_unit"]
            rows.append((torch.copysign(grid[_nearest(x.abs() / by, GRID)], x) * by).reshape(T, H, D))
            if T < 3000:
                all_ = s[name + "_scale"].double().cpu()
                all_[page, :, [p % P for _, p in where]] = scale.cpu()
                held.append(all_)
        return rows[0], rows[1], *(held or (None, None)), None

    def stored(name, b, h, at):  # pages `at` of sequence b in 64 bits, one token a row
        p = s["table"][b].long()[at]
        codes, scale = s[name][p, h], s[name + "_scale"].view(torch.uint8)[p, h].view(FP8).double()
        signs = torch.tensor([1.0, -1.0], dtype=torch.float64, device="cuda")
        grid = torch.tensor(GRID, dtype=torch.float64, device="cuda")
        x = torch.stack([grid[(c_ & 7).int()] * signs[(c_ >> 3).int()] for c_ in (codes & 15, codes >> 4)], -1)
        return (x.reshape(*scale.shape, GROUP) * scale[..., None] * s[name + "_unit"]).reshape(-1, D)

    if c["op"] == "read":
        got = []
        for name in ("k", "v"):
            x = torch.empty(T, H, D, dtype=torch.float64, device="cuda")
            for b, (t, n) in enumerate(zip(total, new)):
                begin = (t - n) // P
                at = torch.arange(begin, -(-t // P), device="cuda")
                for h in range(H):
                    x[first[b]:first[b] + n, h] = stored(name, b, h, at)[t - n - begin * P:][:n]
            got.append(x)
        return tuple(got)
    q = s["q"].double()
    if work(c)["flops"] / 4 / D > 6e8 or T > 4096:
        return None
    got = torch.zeros(T, H * G, D, dtype=torch.float64, device="cuda")
    for b, (t, n) in enumerate(zip(total, new)):
        every = torch.arange(-(-t // P), device="cuda")
        for h in range(H):
            if not c["blocks"]:
                k, v = stored("k", b, h, every), stored("v", b, h, every)
                for i in range(0, n, 64):
                    m = min(64, n - i)
                    x = torch.einsum("mgd,kd->mgk", q[first[b] + i:first[b] + i + m, h * G:(h + 1) * G], k) / math.sqrt(D)
                    ends = t - n + i + torch.arange(m, device="cuda")
                    x = x.masked_fill(torch.arange(k.shape[0], device="cuda") > ends[:, None, None], -math.inf)
                    got[first[b] + i:first[b] + i + m, h * G:(h + 1) * G] = torch.softmax(x, -1) @ v
                continue
            for i in range(n):
                r, end = first[b] + i, t - n + i + 1
                want = sorted({x for x in s["list"][r * H + h].tolist() if 0 <= x <= (end - 1) // P})
                at = torch.tensor(want, device="cuda")
                place = (at[:, None] * P + torch.arange(P, device="cuda")).reshape(-1)
                k, v = stored("k", b, h, at)[place < end], stored("v", b, h, at)[place < end]
                got[r, h * G:(h + 1) * G] = torch.softmax(q[r, h * G:(h + 1) * G] @ k.T / math.sqrt(D), -1) @ v
    return got
