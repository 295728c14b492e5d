"""The 8-bit paged cache and the attention over it: the cases they are measured on.

Five operators surround the exact Top-K selection in a sparse-attention step:

  write    new keys and values go into pages of e4m3 codes with one power-of-two scale for each page
           and head; the page's per-channel key extremes are kept beside it
  read     the stored tokens of each sequence come back as rows of bf16 or fp16
  scores   an upper bound of q.k over each page, the largest of the heads that share it: the score rows
           that the selection reads, with their lengths
  dense    attention of each sequence's last tokens over its whole cache
  sparse   the same over the pages that a list names for each token and key head

`own` selects between the plain torch form and the framework's kernels; `exact` is the definition in 64 bits.
"""

import math
import random

import torch

own = False

FP8 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
LOW, HIGH = -40, 40  # exponents that a scale may have


def case(name, op, dtype, dim, page, heads, group, seqs, lo, hi, new_lo=1, new_hi=1, blocks=0, first=0, last=0, drift=0.0):
    """heads: key heads, group: query heads for each, seqs sequences of lo..hi stored tokens, new_lo..new_hi of them new."""
    c = {"op": op, "dtype": dtype, "dim": dim, "page": page, "heads": heads, "group": group, "seqs": seqs, "lo": lo, "hi": hi,
         "new_lo": new_lo, "new_hi": new_hi, "blocks": blocks, "first": first, "last": last, "drift": drift}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decoding step's keys and values of 64 sequences: latency
        case("write_step", "write", "bf16", 128, 64, 8, 1, 64, 2048, 65536),
        # prompts of a batch, ragged, written at once behind what is cached
        case("write_prompts", "write", "bf16", 128, 64, 8, 1, 24, 5000, 8192, 4001, 4999),
        # a few short sequences copied out, as before a page is moved to another pool
        case("read_short", "read", "bf16", 128, 64, 4, 1, 4, 100, 1000, 100, 100),
        # long shared prefixes read back for a prompt that runs on unquantised rows
        case("read_prefixes", "read", "fp16", 64, 16, 8, 1, 8, 32768, 65536, 32768, 32768),
        # score rows of one decoding step: 64 sequences of up to 65536 tokens
        case("scores_step", "scores", "bf16", 128, 64, 4, 8, 64, 2048, 65536, 1, 1, 0, 1, 2),
        # score rows of a prompt's chunk of 4096 tokens at the end of 131072
        case("scores_chunk", "scores", "bf16", 128, 64, 4, 8, 1, 131072, 131072, 4096, 4096, 0, 1, 2),
        # four short sequences: the smallest attention call, latency
        case("dense_short", "dense", "bf16", 128, 64, 4, 8, 4, 1, 8192),
        # a decoding batch, ragged between 2048 and 65536 tokens
        case("dense_step", "dense", "bf16", 128, 64, 4, 8, 64, 2048, 65536),
        # few very long sequences with some tokens to verify, narrow heads
        case("dense_verify", "dense", "fp16", 64, 128, 2, 4, 8, 500000, 524288, 3, 3),
        # a decoding step over 32 selected pages (2048 tokens) of each sequence
        case("sparse_step", "sparse", "bf16", 128, 64, 4, 8, 64, 2048, 65536, 1, 1, 32, 1, 2),
        # a prompt's chunk: every token with its own 32 pages, most of them shared with its neighbours
        case("sparse_chunk", "sparse", "bf16", 128, 64, 2, 8, 1, 131072, 131072, 4096, 4096, 32, 1, 2, 0.05),
        # tokens to verify of some sequences, small pages, narrow heads, an odd group
        case("sparse_verify", "sparse", "fp16", 64, 16, 2, 7, 9, 3000, 20001, 1, 5, 100, 1, 4, 0.05),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "scores", "dense", "sparse"])
    dtype, dim, page = rng.choice(["bf16", "fp16"]), rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    seqs = _log(rng, 1, 64)
    first, last = rng.randint(0, 2), rng.randint(0, 3)
    if op in ("write", "read"):
        new = max(1, _log(rng, 1, 131072) // seqs)
        lo = new + _log(rng, 1, 4096) - 1
        return case("", op, dtype, dim, page, heads, 1, seqs, lo, lo + _log(rng, 1, 2000), 1 + new // 2, new)
    longest = _log(rng, 16, min(131072, 2_000_000 // seqs // max(1, heads // 4)))
    lo = max(1, int(longest * rng.uniform(0.05, 1.0)))
    if op == "dense":
        new = min(lo, rng.choice([1, 1, 2, rng.randint(1, 9)]))
        return case("", op, dtype, dim, page, heads, group, seqs, lo, longest, 1 + new // 2, new)
    if op == "scores":
        page = rng.choice([32, 64, 128])
        new = min(lo, rng.choice([1, rng.randint(1, 9), max(1, _log(rng, 8, 4096) // seqs)]))
        return case("", op, dtype, dim, page, heads, group, seqs, lo, longest, 1 + new // 2, new, 0, first, last)
    new = min(lo, rng.choice([1, rng.randint(1, 9), max(1, _log(rng, 8, 2048) // seqs)]))
    blocks = max(1, min(_log(rng, 128, 4096) // page, -(-lo // page)))
    return case("", op, dtype, dim, page, heads, min(group, 8), seqs, lo, longest, 1 + new // 2, new, blocks, min(first, blocks // 3), min(last, blocks // 3),
                rng.choice([0.01, 0.05, 0.3]))


def _lengths(c):
    """Stored tokens and new tokens of each sequence: the case's own, the same for each seed."""
    r = random.Random("%(seqs)d %(lo)d %(hi)d %(new_lo)d %(new_hi)d" % c)
    total = [r.randint(c["lo"], c["hi"]) for _ in range(c["seqs"])]
    return total, [min(t, r.randint(c["new_lo"], c["new_hi"])) for t in total]


def _pages(c):
    """Pages that the pool of a case holds for each sequence. A write reaches the last tokens' pages alone: its pool holds no others."""
    total, new = _lengths(c)
    if c["op"] == "write":
        return [(t - 1) // c["page"] - (t - n) // c["page"] + 1 for t, n in zip(total, new)]
    return [-(-t // c["page"]) for t in total]


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev, dt, D, P, H = "cuda", TYPES[c["dtype"]], c["dim"], c["page"], c["heads"]
    total, new = _lengths(c)
    held = _pages(c)
    width, pool, T = max(-(-t // P) for t in total), sum(held), sum(new)
    # pages lie in the pool in no order
    order = torch.randperm(pool, device=dev, generator=g).to(torch.int32)
    table = torch.zeros(c["seqs"], width, dtype=torch.int32, device=dev)
    at = 0
    for b, (t, n) in enumerate(zip(total, held)):
        end = -(-t // P)
        table[b, end - n:end] = order[at:at + n]
        at += n
    s = dict(c, most=max(new), table=table, kv_len=torch.tensor(total, dtype=torch.int32, device=dev),
             q_start=torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32, device=dev))
    single = all(n == 1 for n in new)

    def codes(n):  # normal values that fill the codes' range
        x = torch.empty(n, H, P, D, dtype=FP8, device=dev)
        for i in range(0, n, 8192):
            x[i:i + 8192] = (torch.randn(x[i:i + 8192].shape, device=dev, generator=g) * 100).clamp(-448, 448).to(FP8)
        return x

    def scales(n):
        return torch.exp2(torch.randint(-8, -5, (n, H), device=dev, generator=g).float())

    s["k"], s["v"] = (codes(pool), codes(pool)) if c["op"] != "scores" else (torch.zeros(pool, H, P, D, dtype=FP8, device=dev),) * 2
    s["k_scale"], s["v_scale"] = scales(pool), scales(pool)
    mid, half = torch.randn(pool, H, D, device=dev, generator=g), torch.rand(pool, H, D, device=dev, generator=g) * 2
    s["bounds"] = torch.stack([mid + half, mid - half], 2).to(dt)
    if c["op"] == "write":
        s["new_k"], s["new_v"] = ((torch.randn(T, H, D, device=dev, generator=g) * torch.exp(torch.randn(H, D, device=dev, generator=g) * 0.5)).to(dt) for _ in range(2))
    elif c["op"] == "read":
        s["out_k"], s["out_v"] = (torch.zeros(T, H, D, dtype=dt, device=dev) for _ in range(2))
    else:
        s["q"] = (torch.randn(T, H * c["group"], D, device=dev, generator=g) * 3).to(dt)
    if c["op"] == "scores":
        s["scores"] = torch.zeros(T * H, width, device=dev)
        s["ke"] = torch.zeros(T * H, dtype=torch.int32, device=dev)
    if c["op"] == "sparse":
        # What a token attends to drifts from token to token: a page's interest is a smooth function of the token with
        # some noise on it, so that neighbours share most of their pages. The first and the newest pages are always
        # taken, and rows with fewer pages than slots are padded with -1, as the selection leaves them.
        seq, pos = _tokens(s, T)
        score = torch.randn(c["seqs"], 1, H, width, device=dev, generator=g)[seq, 0]
        turn = torch.randn(c["seqs"], 1, H, width, device=dev, generator=g)[seq, 0]
        angle = (torch.arange(T, device=dev) * c["drift"] * 0.05)[:, None, None]
        score = score * angle.cos() + turn * angle.sin() + c["drift"] * torch.randn(T, H, width, device=dev, generator=g)
        page = torch.arange(width, device=dev)
        newest = (pos // P)[:, None, None]
        score = score.masked_fill((page < c["first"]) | (page > newest - c["last"]), math.inf).masked_fill(page > newest, -math.inf)
        best = score.topk(c["blocks"], -1)
        s["list"] = torch.where(best.values == -math.inf, -1, best.indices).to(torch.int32).reshape(T * H, c["blocks"])
        s["list"] = s["list"][:, torch.randperm(c["blocks"], device=dev, generator=g)].contiguous()
    if c["op"] in ("dense", "sparse"):
        s["out"] = torch.zeros_like(s["q"])
    if own:
        import exact_top_selection_gb300 as etk
        s["cache"] = etk.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"], s["bounds"])
        s["batch"] = etk.SequenceBatch(s["table"], s["kv_len"], None if single else s["q_start"])
        if c["op"] in ("dense", "sparse"):
            s["attention"] = etk.CacheAttention(s["cache"], c["seqs"], T, c["group"] * H, width, num_blocks=c["blocks"])
    return s


def run(s):
    if own:
        import exact_top_selection_gb300 as etk
        if s["op"] == "write":
            etk.cache_write(s["cache"], s["batch"], s["new_k"], s["new_v"])
        elif s["op"] == "read":
            return etk.cache_read(s["cache"], s["batch"], out=(s["out_k"], s["out_v"]))
        elif s["op"] == "scores":
            return etk.block_scores(s["cache"], s["batch"], s["q"], keep_first=s["first"], keep_last=s["last"], scores=s["scores"], ke=s["ke"])
        elif s["op"] == "dense":
            return s["attention"](s["q"], s["batch"], out=s["out"])
        else:
            return s["attention"](s["q"], s["batch"], blocks=s["list"], out=s["out"])
        return s["k"], s["v"], s["k_scale"], s["v_scale"], s["bounds"]
    return {"write": _write, "read": _read, "scores": _scores, "dense": _dense, "sparse": _sparse}[s["op"]](s)


def _tokens(s, T):
    """Sequence and position of each of the T new tokens."""
    t = torch.arange(T, device=s["kv_len"].device)
    seq = torch.searchsorted(s["q_start"][1:].long(), t, right=True)
    return seq, (s["kv_len"] - s["q_start"][1:])[seq].long() + t


def _quantise(x, page, off, start, codes, scale):
    """x [T, H, D] into the codes of their pages; `start` is the first offset written in each page (a page's size where none is)."""
    P = codes.shape[2]
    a = x.float().abs()
    a = torch.where(a.isfinite(), a, 0).amax(-1)
    top = torch.zeros_like(scale).index_reduce_(0, page, a, "amax")
    m, e = torch.frexp(top / 448)
    need = torch.exp2((e - (m == 0.5).int()).clamp(LOW, HIGH).float())
    need = torch.where(top > 0, need, 2.0 ** LOW)
    kept = (start > 0) & (start < P)
    after = torch.where(start[:, None] == 0, need, torch.where(kept[:, None], torch.maximum(need, scale), scale))
    # what the page held is brought to its new scale; then the new tokens are put in
    held = (codes.float() * (scale / after)[:, :, None, None]).to(FP8)
    below = torch.arange(P, device=x.device)[None] < torch.where(kept, start, 0)[:, None]
    codes.copy_(torch.where(below[:, None, :, None], held.float(), codes.float()).to(FP8))
    y = x.float() / after[page][:, :, None]
    y = torch.where(y.isfinite(), y.clamp(-448, 448), math.nan).to(FP8)
    codes.view(torch.uint8)[page, :, off] = y.view(torch.uint8)
    scale.copy_(after)


def _write(s):
    T, P = s["new_k"].shape[0], s["page"]
    seq, pos = _tokens(s, T)
    page, off = s["table"][seq, pos // P].long(), pos % P
    start = torch.full((s["k"].shape[0],), P, device=page.device).index_reduce_(0, page, off, "amin")
    _quantise(s["new_k"], page, off, start, s["k"], s["k_scale"])
    _quantise(s["new_v"], page, off, start, s["v"], s["v_scale"])
    most = torch.finfo(s["bounds"].dtype).max
    x = torch.where(s["new_k"].isnan(), 0, s["new_k"]).float().clamp(-most, most)
    fresh = (start == 0)[:, None, None]
    old = s["bounds"].float()
    hi = torch.where(fresh, -math.inf, old[:, :, 0]).index_reduce_(0, page, x, "amax")
    lo = torch.where(fresh, math.inf, old[:, :, 1]).index_reduce_(0, page, x, "amin")
    s["bounds"].copy_(torch.stack([hi, lo], 2))
    return s["k"], s["v"], s["k_scale"], s["v_scale"], s["bounds"]


def _read(s):
    T, P = s["out_k"].shape[0], s["page"]
    seq, pos = _tokens(s, T)
    page, off = s["table"][seq, pos // P].long(), pos % P
    for name in ("k", "v"):
        x = s[name].view(torch.uint8)[page, :, off].view(FP8).float() * s[name + "_scale"][page][:, :, None]
        s["out_" + name].copy_(x)
    return s["out_k"], s["out_v"]


def _scores(s):
    T, H, G, P, D = s["q"].shape[0], s["heads"], s["group"], s["page"], s["dim"]
    B, width = s["table"].shape
    seq, pos = _tokens(s, T)
    q = s["q"].float().reshape(T, H, G, D)
    both = torch.cat([q.clamp(min=0), q.clamp(max=0)], -1)
    ends = s["bounds"].float().reshape(-1, H, 2 * D)[s["table"].long()]  # [B, width, H, 2D]
    most = s["most"]
    if B == 1:
        got = torch.einsum("thgd,whd->thgw", both, ends[0]).amax(2)
    else:  # each sequence's tokens side by side, short ones padded
        padded = torch.zeros(B, most, H, G, 2 * D, device=q.device)
        i = torch.arange(T, device=q.device) - s["q_start"][seq]
        padded[seq, i] = both
        got = torch.einsum("bthgd,bwhd->bthgw", padded, ends).amax(3)[seq, i]
    page, newest = torch.arange(width, device=q.device), (pos // P)[:, None, None]
    got = got.masked_fill((page < s["first"]) | (page > newest - s["last"]), math.inf)
    s["scores"].copy_(torch.where(page <= newest, got, s["scores"].reshape(T, H, width)).reshape(T * H, width))
    s["ke"].copy_((pos // P + 1)[:, None].expand(T, H).reshape(-1))
    return s["scores"], s["ke"]


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
        x = s[name].view(torch.uint8)[at].view(FP8).float()  # [B, width, H, P, D]
        x = x.mul_(s[name + "_scale"][at][..., None, None])
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
        x = s[name].view(torch.uint8)[at, head].view(FP8).float()  # [T, H, K, P, D]
        return x.mul_(s[name + "_scale"][at, head][..., None, None]).reshape(T, H, K * P, D)

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
    seen = [[t - n + i + 1 for i in range(n)] for t, n in zip(total, new)]  # tokens that each new token sees
    if c["op"] == "write":
        reached = sum(_pages(c))
        return {"bytes": T * H * D * (2 + 1) * 2 + reached * H * (2 * 2 * D + 8), "flops": T * H * D * 8}
    if c["op"] == "read":
        return {"bytes": T * H * D * (2 + 1) * 2 + sum(_pages(c)) * H * 8, "flops": T * H * D * 2}
    if c["op"] == "scores":
        pairs = sum(-(-x // P) for v in seen for x in v)
        return {"bytes": sum(_pages(c)) * H * D * 4 + T * H * G * D * 2 + pairs * H * 4, "flops": 2 * pairs * H * G * 2 * D}
    if c["op"] == "dense":
        pairs = sum(sum(v) for v in seen)
        return {"bytes": sum(total) * H * D * 2 + sum(_pages(c)) * H * 8 + T * H * G * D * 4, "flops": 4 * pairs * H * G * D}
    pairs = sum(min(x, c["blocks"] * P) for v in seen for x in v)
    # the cached bytes of a list's pages: those of one token alone are its own, a longer run's are at most the whole cache
    held = sum(min(t, sum(min(x, c["blocks"] * P) for x in v)) for t, v in zip(total, seen))
    return {"bytes": held * H * D * 2 + T * H * (c["blocks"] * 4 + G * D * 4), "flops": 4 * pairs * H * G * D}


def _e4m3(y):
    """The e4m3 value nearest to each y in [-448, 448], ties to the even one."""
    a = y.abs()
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -6)))
    e = torch.where(torch.exp2(e) > a.clamp(min=2.0 ** -6), e - 1, e)
    step = torch.exp2(e - 3)
    return torch.copysign(torch.round(a / step) * step, y)


def _scale_of(top):
    e = LOW
    while e < HIGH and top > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def exact(c, seed):
    s = prepare(c, seed)
    total, new = _lengths(c)
    D, P, H, G, T = c["dim"], c["page"], c["heads"], c["group"], sum(new)
    width = s["table"].shape[1]
    first = [sum(new[:b]) for b in range(len(new))]
    if c["op"] == "write":
        if T * H * D > 2e8 or sum(_pages(c)) * H > 20000:
            return None
        out = {}
        for name in ("k", "v"):
            x, codes, scale = s["new_" + name].double().cpu(), s[name].double().cpu(), s[name + "_scale"].double().cpu()
            ends = s["bounds"].double().cpu()
            for b, (t, n) in enumerate(zip(total, new)):
                at = t - n
                while at < t:
                    p, o = int(s["table"][b, at // P]), at % P
                    m = min(P - o, t - at)
                    y = x[first[b] + at - (t - n):][:m].transpose(0, 1)  # [H, m, D]
                    for h in range(H):
                        was = float(scale[p, h])
                        now = _scale_of(float(y[h].abs().max()))
                        if o:
                            now = max(now, was)
                            codes[p, h, :o] = _e4m3(codes[p, h, :o] * (was / now))
                        codes[p, h, o:o + m] = _e4m3(y[h] / now)
                        scale[p, h] = now
                    hi, lo = y.amax(1), y.amin(1)
                    ends[p, :, 0] = torch.maximum(hi, ends[p, :, 0]) if o else hi
                    ends[p, :, 1] = torch.minimum(lo, ends[p, :, 1]) if o else lo
                    at += m
            out[name] = codes, scale
            if name == "k":
                out["bounds"] = ends
        return out["k"][0], out["v"][0], out["k"][1], out["v"][1], out["bounds"]
    rows = {n: s[n] for n in ("k", "v")}

    def stored(name, b, h, at):  # pages `at` of sequence b in 64 bits, one token a row
        p = s["table"][b].long()[at]
        return (rows[name][:, h].view(torch.uint8)[p].view(FP8).double() * s[name + "_scale"][p, h].double()[:, None, None]).reshape(-1, D)

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
    if c["op"] == "scores":
        if T * H * G * width * D > 2e11:
            return None
        got = s["scores"].double().reshape(T, H, width)
        for b, (t, n) in enumerate(zip(total, new)):
            ends = s["bounds"][s["table"][b].long()].double()  # [width, H, 2, D]
            for i in range(0, n, 64):
                for h in range(H):
                    u = q[first[b] + i:first[b] + min(n, i + 64), h * G:(h + 1) * G]
                    m = u.shape[0]
                    x = (u.clamp(min=0).reshape(-1, D) @ ends[:, h, 0].T + u.clamp(max=0).reshape(-1, D) @ ends[:, h, 1].T).reshape(m, G, width).amax(1)
                    for j in range(m):
                        newest = (t - n + i + j) // P
                        row = x[j, :newest + 1].clone()
                        row[:c["first"]] = math.inf
                        row[max(0, newest + 1 - c["last"]):] = math.inf
                        got[first[b] + i + j, h, :newest + 1] = row
        return got.reshape(T * H, width), None
    pairs = work(c)["flops"] / 4 / D
    if pairs > 3e8 or T > 4096:
        return None
    got = torch.zeros(T, H * G, D, dtype=torch.float64, device="cuda")
    for b, (t, n) in enumerate(zip(total, new)):
        every = torch.arange(-(-t // P), device="cuda")
        for h in range(H):
            if c["op"] == "dense":
                k, v = stored("k", b, h, every), stored("v", b, h, every)
            for i in range(n):
                r, end = first[b] + i, t - n + i + 1
                if c["op"] == "sparse":
                    want = sorted({x for x in s["list"][r * H + h].tolist() if 0 <= x <= (end - 1) // P})
                    if not want:
                        continue
                    at = torch.tensor(want, device="cuda")
                    k, v = stored("k", b, h, at), stored("v", b, h, at)
                    place = (at[:, None] * P + torch.arange(P, device="cuda")).reshape(-1)
                    k, v = k[place < end], v[place < end]
                    end = k.shape[0]
                p = torch.softmax(q[r, h * G:(h + 1) * G] @ k[:end].T / math.sqrt(D), -1)
                got[r, h * G:(h + 1) * G] = p @ v[:end]
    return got
