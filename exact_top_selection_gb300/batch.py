"""Python binding of the operators on a batch's rows and tables (include/exact_topk_cache.h).

What comes before the cache in a serving step: page tables, lengths and row ranges that live on the
GPU, and queries and keys turned by their positions::

    tables = PageTables.allocate(num_pages, num_seqs, table_width, page_size, max_tokens, device="cuda")
    rotary = Rotary(head_dim, base=500000.0)
    tables.update(new_tokens)                              # int32 [num_seqs]: more tokens, or fewer
    q, k = rotary(q, k, batch=tables.batch)
    cache_write(cache, tables.batch, k, v)

Argument checks and marshalling only, as in ``cache.py``: every step runs in the CUDA kernels of
``libexact_topk.so``.  Calls are enqueued on ``stream`` (default: the current stream of the tensors'
device), allocate nothing when their outputs are given, and can be captured in a CUDA graph after one
call outside the capture.
"""

from __future__ import annotations

import ctypes
import math
from collections import namedtuple
from fractions import Fraction

import exact_top_selection_gb300 as _etk

from . import cache as _cache

__all__ = ["Rotary", "PageTables"]

_PI = Fraction("3.14159265358979323846264338327950288419716939937510")
_RowsOf = namedtuple("_RowsOf", "device dtype head_dim")  # what rows are checked against
_bound = None


class _Spec(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("amplitude", ctypes.c_float), ("head_dim", ctypes.c_int32),
                ("rotary_dim", ctypes.c_int32), ("neighbours", ctypes.c_int32), ("type", ctypes.c_int32),
                ("page_size", ctypes.c_int32)]


class _Tables(ctypes.Structure):
    _fields_ = [(name, ctypes.c_void_p) for name in ("page_table", "kv_len", "q_start", "applied", "slots",
                                                     "positions", "free_pages", "free_range", "counters")] + [
        ("counter_bytes", ctypes.c_size_t), ("table_pitch", ctypes.c_int64), ("max_tokens", ctypes.c_int64),
        ("num_seqs", ctypes.c_int32), ("table_width", ctypes.c_int32), ("num_pages", ctypes.c_int32),
        ("page_size", ctypes.c_int32)]


def _lib():
    global _bound
    if _bound is None:
        lib = _cache._lib()
        p, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        batch, rows, tables = (ctypes.POINTER(t) for t in (_cache._Batch, _cache._Rows, _Tables))
        lib.exact_topk_rotary.argtypes = [ctypes.POINTER(_Spec), batch, p, i64, i32, rows, rows, i32, rows, rows,
                                          i32, p]
        lib.exact_topk_update_tables.argtypes = [tables, p, i32, p]
        _bound = lib
    return _bound


def _apart(a, b, name):
    """Rows a and b share no memory. Both may be slices of one wider tensor of tokens, or of one wider tensor of heads.

    By residues: modulo p, dimensions whose stride is a multiple of p fall together, and an array's bytes lie in one run,
    as long as its other dimensions span. Runs that are apart are apart in memory too. Each stride is tried as p;
    those of dimensions of one element mean nothing."""
    if a.is_contiguous() and b.is_contiguous():
        a0, b0 = a.data_ptr(), b.data_ptr()
        if a0 >= b0 + b.nbytes or b0 >= a0 + a.nbytes:
            return
    (a0, a1), (b0, b1) = _cache._span(a), _cache._span(b)
    if a0 >= b1 or b0 >= a1 or a.numel() == 0 or b.numel() == 0:
        return
    size = a.element_size()
    steps = [[(n - 1, s * size) for n, s in zip(t.shape[:2], t.stride()[:2]) if n > 1] for t in (a, b)]
    for p in {s for step in steps for _, s in step if s > 0}:
        run, other = (t.shape[2] * size + sum(n * s for n, s in step if s % p) for t, step in zip((a, b), steps))
        at = (b0 - a0) % p  # of b's run behind the start of one of a's
        if at >= run and at + other <= p:
            return
    raise ValueError(f"{name} must not share memory with another row argument")


def _rows_like(t, name, like, x, xr):
    """As _cache._rows, of an output with the shape of the rows x that are described already."""
    if t.shape == x.shape and t.dtype is x.dtype and t.device == x.device and t.is_contiguous():
        return _cache._Rows(t.data_ptr(), x.shape[1] * x.shape[2], x.shape[2])
    return _cache._rows(t, name, like, x.shape[1], x.shape[0])


def _check_places(x, xr, y, yr):
    """Outputs y are the rows x themselves, or apart from them; no two of their rows overlap."""
    if not y.is_contiguous():
        _cache._written(y, "out", y[:0])
    if xr.data != yr.data or xr.token_stride != yr.token_stride or xr.head_stride != yr.head_stride:
        _apart(y, x, "out")


class Rotary:
    """Rotary positions: pairs of a head's channels turned by angles in proportion to their token's position.

    The first rotary_dim channels (default: all of head_dim) turn, in pairs (i, i + rotary_dim / 2), or with
    neighbours=True (2 i, 2 i + 1); pair i by base^(-2 i / rotary_dim) radians a position.  For contexts
    longer than trained on: factor divides the frequencies.  With original_length it does so by parts: a pair
    that turns more than `fast` times within original_length is kept, one that turns less than `slow` times is
    divided by the factor, with a ramp between, and the result is scaled by `amplitude`, 0.1 ln(factor) + 1
    unless given (1 without original_length).  ("YaRN: Efficient Context Window Extension of Large Language
    Models", section 3.)  Other schemes: `frequencies`, rotary_dim / 2 numbers in radians a position, which
    base and factor do not change.  Angles are exact at every position."""

    def __init__(self, head_dim, rotary_dim=None, base=10000.0, neighbours=False, factor=1.0, original_length=None,
                 slow=1.0, fast=32.0, amplitude=None, frequencies=None, device=None):
        torch = _cache._need_torch()
        rotary_dim = head_dim if rotary_dim is None else rotary_dim
        if head_dim < 8 or head_dim > 1024 or head_dim % 8:
            raise ValueError(f"head_dim must be a multiple of 8 up to 1024, got {head_dim}")
        if rotary_dim < 2 or rotary_dim % 2 or rotary_dim > min(head_dim, 512):
            raise ValueError(f"rotary_dim must be even and 2 to {min(head_dim, 512)}, got {rotary_dim}")
        if frequencies is None:
            if not (base > 0 and factor > 0 and math.isfinite(base) and math.isfinite(factor)):
                raise ValueError("base and factor must be positive and finite")
            if original_length is not None and not (original_length > 0 and slow < fast):
                raise ValueError("need original_length > 0 and slow < fast")
            frequencies = []
            for i in range(rotary_dim // 2):
                f = base ** (-2 * i / rotary_dim)
                keep = 0.0
                if original_length is not None:
                    keep = (original_length * f / (2 * math.pi) - slow) / (fast - slow)
                    keep = min(1.0, max(0.0, keep))
                frequencies.append(f if factor == 1.0 else f * keep + f / factor * (1 - keep))
        frequencies = [float(f) for f in frequencies]
        if len(frequencies) != rotary_dim // 2 or not all(map(math.isfinite, frequencies)):
            raise ValueError(f"frequencies must be {rotary_dim // 2} finite numbers")
        if amplitude is None:
            amplitude = 1.0 if original_length is None or factor <= 1.0 else 0.1 * math.log(factor) + 1.0
        if not math.isfinite(amplitude) or abs(amplitude) > 3e38:
            raise ValueError(f"amplitude must be finite, got {amplitude}")
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        if dev.type != "cuda":
            raise ValueError(f"rotary positions need a CUDA device, got {dev}")
        if dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.head_dim, self.rotary_dim, self.neighbours = head_dim, rotary_dim, bool(neighbours)
        self.frequencies, self.amplitude, self.device, self._index = frequencies, float(amplitude), dev, dev.index
        # radians as turns in 64 bits: the angle of a position is an integer product
        turns = [int(Fraction(f) / (2 * _PI) * 2 ** 64) % 2 ** 64 for f in frequencies]
        self.turns = torch.tensor([t - 2 ** 64 if t >= 2 ** 63 else t for t in turns], dtype=torch.int64, device=dev)
        with torch.cuda.device(dev):
            _cache._wait_for_buffers()
        self._specs = {}
        for i, dtype in enumerate((torch.bfloat16, torch.float16)):
            specs = {page or None: _Spec(self.turns.data_ptr(), self.amplitude, head_dim, rotary_dim, int(self.neighbours), i, page)
                     for page in (0, *_cache.PAGE_SIZES)}
            self._specs[dtype] = specs, _RowsOf(dev, dtype, head_dim)

    def __call__(self, q, k=None, batch=None, positions=None, out=None, inverse=False, stream=None, page_size=None):
        """q [num_tokens, q_heads, head_dim] turned, and with k [num_tokens, k_heads, head_dim] the pair of both.

        batch: rows have the positions of their tokens in it; rows of no sequence are left as they are in
        ``out`` (zeros where it is not given).  positions, int32 [num_tokens], instead: any numbers.  out: rows to write into (a
        pair with k); q and k themselves are turned in place, other rows must not overlap them.  inverse: turns
        by the negative angles, with the same amplitude: the gradient of q and k by that of the outputs, and the way back
        where the amplitude is 1 (else it ends at amplitude^2 times the rows).  page_size: of the batch's tables; a length beyond
        table_width * page_size is clamped to it, as by the cache's operators (without, lengths are taken as they are)."""
        torch = _cache.torch
        if q.dtype not in self._specs:
            raise TypeError(f"q must be bfloat16 or float16, got {q.dtype}")
        specs, like = self._specs[q.dtype]
        spec = specs.get(page_size)
        if spec is None:
            raise ValueError(f"page_size must be None or in {_cache.PAGE_SIZES}, got {page_size}")
        heads = q.shape[1] if q.dim() == 3 else 0
        qr = _cache._rows(q, "q", like, heads)
        if heads < 1:
            raise ValueError("q must have at least one head")
        T = q.shape[0]
        if (batch is None) == (positions is None):
            raise ValueError("either batch or positions is needed")
        if batch is not None:
            batch._check(self, T)
        else:
            _etk._check_tensor(positions, "positions", torch.int32, self.device, 1)
            if positions.shape[0] != T or not positions.is_contiguous():
                raise ValueError(f"positions must be contiguous [{T}]")
        pair = k is not None
        if pair:
            k_heads = k.shape[1] if k.dim() == 3 else 0
            kr = _cache._rows(k, "k", like, k_heads, T)
            if k_heads < 1:
                raise ValueError("k must have at least one head")
        if out is None:
            with torch.cuda.stream(stream):
                q_out = torch.zeros(q.shape, dtype=q.dtype, device=q.device)
                k_out = torch.zeros(k.shape, dtype=k.dtype, device=k.device) if pair else None
            qo = _cache._rows(q_out, "out", like, heads, T)
            ko = _cache._rows(k_out, "out", like, k_heads, T) if pair else None
        else:
            q_out, k_out = out if pair else (out, None)
            qo = _rows_like(q_out, "out" if not pair else "out[0]", like, q, qr)
            ko = _rows_like(k_out, "out[1]", like, k, kr) if pair else None
            _check_places(q, qr, q_out, qo)
            if pair:
                _check_places(k, kr, k_out, ko)
                _apart(q_out, k_out, "out[0]")
                if ko.data != kr.data:  # in place, k is what the line above looked at
                    _apart(q_out, k, "out[0]")
                if qo.data != qr.data:
                    _apart(k_out, q, "out[1]")
        _cache._call(self, stream, _lib().exact_topk_rotary, ctypes.byref(spec), None if batch is None else batch._ref,
                     None if positions is None else positions.data_ptr(), T, heads, qr, qo, k_heads if pair else 0,
                     kr if pair else None, ko if pair else None, int(bool(inverse)))
        return (q_out, k_out) if pair else q_out


class PageTables:
    """Page tables, lengths and row ranges of sequences that grow and shrink on the GPU, with the pages
    that no sequence has.

    page_table int32 [num_seqs, table_width] (rows may be strided); kv_len int32 [num_seqs]; free_pages int32
    [num_pages], a ring of page ids, of which free_range, int32 [2], gives the first free one's place and
    how many there are.  Each page's id stands once, in the ring or in a table.  Written by each call: q_start
    int32 [num_seqs + 1], slots and positions int32 [max_tokens] (made here where not given), and
    `applied`, int32 [num_seqs].  ``batch`` is the SequenceBatch of these tensors.  Everything stays on the GPU: a
    captured step can grow its sequences by itself.  Calls of one object must not overlap on the GPU."""

    def __init__(self, page_table, kv_len, free_pages, free_range, page_size, max_tokens, q_start=None, slots=None,
                 positions=None):
        torch = _cache._need_torch()
        if page_size not in _cache.PAGE_SIZES:
            raise ValueError(f"page_size must be in {_cache.PAGE_SIZES}, got {page_size}")
        if not 0 <= max_tokens <= 1 << 24:
            raise ValueError(f"max_tokens must be 0 to 2^24, got {max_tokens}")
        dev = page_table.device
        if dev.type != "cuda":
            raise ValueError(f"the tables must be on a CUDA device, got {dev}")
        B = page_table.shape[0]
        with torch.cuda.device(dev):
            if q_start is None:
                q_start = torch.zeros(B + 1, dtype=torch.int32, device=dev)
            slots, positions = (torch.zeros(max_tokens, dtype=torch.int32, device=dev) if t is None else t
                                for t in (slots, positions))
            self.applied = torch.zeros(B, dtype=torch.int32, device=dev)
            self.counters = torch.zeros(16, dtype=torch.uint8, device=dev)
            _cache._wait_for_buffers()
        self.batch = _cache.SequenceBatch(page_table, kv_len, q_start)
        for t, name, size in ((free_pages, "free_pages", None), (free_range, "free_range", 2),
                              (slots, "slots", max_tokens), (positions, "positions", max_tokens)):
            _etk._check_tensor(t, name, torch.int32, dev, 1)
            if not t.is_contiguous() or t.shape[0] < 1 and size is None or size is not None and t.shape[0] != size:
                raise ValueError(f"{name} must be contiguous [{'num_pages' if size is None else size}]")
        pages = free_pages.shape[0]
        if pages * page_size >= 1 << 31:
            raise ValueError(f"num_pages * page_size must be below 2^31, got {pages} * {page_size}")
        self.page_table, self.kv_len, self.q_start = page_table, kv_len, q_start
        self.free_pages, self.free_range, self.slots, self.positions = free_pages, free_range, slots, positions
        self.page_size, self.max_tokens, self.num_pages, self.num_seqs = page_size, max_tokens, pages, B
        self.device, self._index = dev, dev.index
        self._c = _Tables(page_table.data_ptr(), kv_len.data_ptr(), q_start.data_ptr(), self.applied.data_ptr(),
                          slots.data_ptr(), positions.data_ptr(), free_pages.data_ptr(), free_range.data_ptr(),
                          self.counters.data_ptr(), self.counters.numel(), self.batch._c.table_pitch, max_tokens,
                          B, self.batch.table_width, pages, page_size)
        self._ref = ctypes.byref(self._c)

    @classmethod
    def allocate(cls, num_pages, num_seqs, table_width, page_size, max_tokens, device=None):
        """Empty sequences, every page free, in ascending order; ready for any stream."""
        torch = _cache._need_torch()
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        table = torch.full((num_seqs, table_width), -1, dtype=torch.int32, device=dev)
        kv_len = torch.zeros(num_seqs, dtype=torch.int32, device=dev)
        free = torch.arange(num_pages, dtype=torch.int32, device=dev)
        return cls(table, kv_len, free, torch.tensor([0, num_pages], dtype=torch.int32, device=dev), page_size, max_tokens)

    def update(self, change, stream=None):
        """Sequence b gets change[b] more tokens (int32 [num_seqs]), or loses its last -change[b] (all, where it has
        fewer).  Pages no longer reached become free, in the sequences' order, and are used in this call last.  A
        sequence gets all its tokens or none: none where they do not fit its table, where the pages that it and
        those before it ask for are more than there are, or their tokens more than max_tokens.  ``applied`` is
        the change that was made; q_start, slots (page * page_size + offset) and positions are those of the new
        tokens' rows.  Returns the batch."""
        return self._update(change, 0, stream)

    def drop(self, counts, stream=None):
        """As update with -counts: sequence b loses its last counts[b] tokens, as after some were not accepted."""
        return self._update(counts, 1, stream)

    def _update(self, change, negate, stream):
        _etk._check_tensor(change, "change", _cache.torch.int32, self.device, 1)
        if change.shape[0] != self.num_seqs or not change.is_contiguous():
            raise ValueError(f"change must be contiguous [{self.num_seqs}]")
        _cache._call(self, stream, _lib().exact_topk_update_tables, self._ref, change.data_ptr(), negate)
        return self.batch
