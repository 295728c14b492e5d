"""Python binding of the cache operators (include/exact_topk_cache.h).

The steps of sparse attention around the exact Top-K: a paged key/value cache in
8 bits, the page scores that the selection reads, and the attention over the pages it
selected (or over the whole cache)::

    cache = KVCache.allocate(num_pages, kv_heads, page_size, head_dim, device="cuda")
    batch = SequenceBatch(page_table, kv_len, q_start)     # q_start=None: one row per sequence
    cache_write(cache, batch, k, v)                        # [num_tokens, kv_heads, head_dim]
    scores, ke = block_scores(cache, batch, q)             # [num_tokens * kv_heads, table_width]
    pages = ExactTopK(num_tokens * kv_heads, table_width, 32)(scores, ke)
    out = CacheAttention(cache, num_seqs, num_tokens, q_heads, table_width,
                         num_blocks=32)(q, batch, blocks=pages)

``SparseAttention`` runs these as one object with its own buffers.

Argument checks and marshalling only: every step runs in the CUDA kernels of
``libexact_topk.so``, and there is no fallback.  Calls are enqueued on ``stream`` (default: the
current stream of the tensors' device), allocate nothing when their outputs are
given, and can be captured in a CUDA graph after one call outside the capture.
"""

from __future__ import annotations

import ctypes
import math

import exact_top_selection_gb300 as _etk

__all__ = ["KVCache", "SequenceBatch", "AttentionPlan", "CacheAttention", "SparseAttention", "cache_write",
           "cache_read", "block_scores", "make_attention_plan", "CACHE_SYMBOLS", "PAGE_SIZES", "HEAD_DIMS"]

PAGE_SIZES = (16, 32, 64, 128)
HEAD_DIMS = (64, 128)
CACHE_SYMBOLS = ("exact_topk_cache_write", "exact_topk_cache_read", "exact_topk_block_scores",
                 "exact_topk_make_attention_plan", "exact_topk_attention_run", "exact_topk_set_wait_limit")


class _Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("key_bounds", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("type", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class _Batch(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                ("q_start", ctypes.c_void_p), ("num_seqs", ctypes.c_int32),
                ("table_width", ctypes.c_int32), ("table_pitch", ctypes.c_int64)]


class _Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class AttentionPlan(ctypes.Structure):
    """Launch plan of the attention (exact_topk_attention_plan)."""
    _fields_ = [("num_tokens", ctypes.c_int64), ("num_seqs", ctypes.c_int32),
                ("q_heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("table_width", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
                ("columns", ctypes.c_int32), ("tile_tokens", ctypes.c_int32),
                ("tile_heads", ctypes.c_int32), ("workers", ctypes.c_int32),
                ("min_units", ctypes.c_int32), ("prompt_tokens", ctypes.c_int32),
                ("prompt_heads", ctypes.c_int32), ("counter_bytes", ctypes.c_uint64),
                ("workspace_bytes", ctypes.c_uint64)]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}

    def __repr__(self):
        return f"AttentionPlan({self.as_dict()})"


_bound = None
torch = None  # imported with the first tensor that arrives here


def _need_torch():
    global torch
    if torch is None:
        import torch as module
        torch = module
    return torch


def _lib():
    global _bound
    if _bound is None:
        lib = _etk.library()
        p, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
        cache, batch, rows = (ctypes.POINTER(t) for t in (_Cache, _Batch, _Rows))
        lib.exact_topk_cache_write.argtypes = [cache, batch, i64, rows, rows, p]
        lib.exact_topk_cache_read.argtypes = [cache, batch, i64, rows, rows, p]
        lib.exact_topk_block_scores.argtypes = [cache, batch, i64, i32, rows, i32, i32, p, i64, p, p, p]
        lib.exact_topk_make_attention_plan.argtypes = [i64] + [i32] * 9 + [
            ctypes.POINTER(_etk.DeviceInfo), ctypes.POINTER(AttentionPlan)]
        lib.exact_topk_attention_run.argtypes = [ctypes.POINTER(AttentionPlan), cache, batch, rows, rows,
                                                 p, ctypes.c_float, p, sz, p, sz, p]
        lib.exact_topk_set_wait_limit.argtypes = [i64]
        for name in CACHE_SYMBOLS:
            getattr(lib, name).restype = ctypes.c_int
        _bound = lib
    return _bound


def _call(cache, stream, fn, *args):
    """fn(*args, stream handle) with the cache's device current; raises on an error status."""
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(cache._index)  # current_stream(...).cuda_stream
    elif stream.device != cache.device:
        raise ValueError(f"stream must be of {cache.device}, got {stream.device}")
    else:
        handle = stream.cuda_stream
    if torch.cuda.current_device() == cache._index:
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(cache._index):
            rc = fn(*args, handle)
    if rc != 0:
        raise _etk.ExactTopKError(rc, fn.__name__)


def _wait_for_buffers():
    """Lets the current stream fill an object's buffers: its first call may be on another stream."""
    if not torch.cuda.is_current_stream_capturing():
        torch.cuda.current_stream().synchronize()


def _rows(t, name, cache, heads, tokens=None):
    """Checks rows [num_tokens, heads, head_dim] and describes them."""
    dim = cache.head_dim
    if t.dtype is not cache.dtype:
        raise TypeError(f"{name} must be {cache.dtype}, got {t.dtype}")
    if t.device != cache.device:
        raise ValueError(f"{name} must be on {cache.device}, got {t.device}")
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim or (tokens is not None and shape[0] != tokens):
        raise ValueError(f"{name} must be [{'num_tokens' if tokens is None else tokens}, {heads}, {dim}], "
                         f"got {list(shape)}")
    if t.is_contiguous():
        return _Rows(t.data_ptr(), heads * dim, dim)
    token, head, channel = t.stride()
    if channel != 1:
        raise ValueError(f"{name} must have contiguous channels")
    # strides of dimensions of one element carry no meaning
    return _Rows(t.data_ptr(), token if shape[0] > 1 else 0, head if heads > 1 else 0)


def _span(t):
    """Addresses of the first element of rows and behind the last one."""
    at = t.data_ptr()
    if t.is_contiguous():
        return at, at + t.nbytes
    ends = [(n - 1) * s * t.element_size() for n, s in zip(t.shape, t.stride())]
    return at + sum(e for e in ends if e < 0), at + sum(e for e in ends if e > 0) + t.element_size()


def _written(t, name, other):
    """An output's rows must share no memory with one another, nor with the rows `other`."""
    if t.is_contiguous() and other.is_contiguous():
        a, c = t.data_ptr(), other.data_ptr()
        if a < c + other.nbytes and c < a + t.nbytes:
            raise ValueError(f"{name} must not share memory with another row argument")
        return
    if t.numel() == 0:
        return
    if not t.is_contiguous():
        need = t.shape[2]  # elements that the dimensions so far span
        for n, s in sorted(zip(t.shape[:2], map(abs, t.stride()[:2])), key=lambda x: x[1]):
            if n > 1:
                if s < need:
                    raise ValueError(f"the rows of {name} must not overlap")
                need += (n - 1) * s
    a, b = _span(t)
    c, d = _span(other)
    if a < d and c < b:
        raise ValueError(f"{name} must not share memory with another row argument")


class KVCache:
    """A paged cache of e4m3 codes with one scale for each page and key head.

    k, v: float8_e4m3fn [num_pages, kv_heads, page_size, head_dim]; k_scale, v_scale: float32
    [num_pages, kv_heads]; key_bounds: bfloat16 or float16 [num_pages, kv_heads, 2, head_dim],
    each channel's largest and smallest key.  All contiguous and on one device; the bounds'
    type is that of the rows written, read and asked with.  The tensors stay the caller's: they
    are used in place and kept alive by this object.
    """

    def __init__(self, k, v, k_scale, v_scale, key_bounds):
        _need_torch()
        if k.dim() != 4 or k.shape != v.shape:
            raise ValueError("k and v must be [num_pages, kv_heads, page_size, head_dim]")
        pages, heads, page, dim = k.shape
        if pages < 1 or heads < 1 or page not in PAGE_SIZES or dim not in HEAD_DIMS:
            raise ValueError(f"need pages, kv_heads >= 1, page_size in {PAGE_SIZES}, head_dim in {HEAD_DIMS}; "
                             f"got {list(k.shape)}")
        if key_bounds.dtype not in (torch.bfloat16, torch.float16):
            raise TypeError(f"key_bounds must be bfloat16 or float16, got {key_bounds.dtype}")
        self.device, self._index = k.device, k.device.index
        if self.device.type != "cuda":
            raise ValueError(f"the cache must be on a CUDA device, got {self.device}")
        fp8 = torch.float8_e4m3fn
        for t, name, dtype, shape in ((k, "k", fp8, k.shape), (v, "v", fp8, k.shape),
                                      (k_scale, "k_scale", torch.float32, (pages, heads)),
                                      (v_scale, "v_scale", torch.float32, (pages, heads)),
                                      (key_bounds, "key_bounds", key_bounds.dtype, (pages, heads, 2, dim))):
            if t.dtype != dtype:
                raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
            if t.device != self.device:
                raise ValueError(f"{name} must be on {self.device}, got {t.device}")
            if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous {list(shape)}, got {list(t.shape)}")
        self.k, self.v, self.k_scale, self.v_scale, self.key_bounds = k, v, k_scale, v_scale, key_bounds
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = pages, heads, page, dim
        self.dtype = key_bounds.dtype
        self._c = _Cache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                         key_bounds.data_ptr(), pages, heads, page, dim,
                         0 if self.dtype == torch.bfloat16 else 1, 0)
        self._ref = ctypes.byref(self._c)

    @classmethod
    def allocate(cls, num_pages, kv_heads, page_size, head_dim, dtype=None, device=None):
        """A new cache with every page empty (codes 0, scales 1, bounds 0), ready for any stream."""
        _need_torch()
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        shape = (num_pages, kv_heads, page_size, head_dim)
        k, v = (torch.zeros(shape, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn) for _ in range(2))
        ks, vs = (torch.ones(shape[:2], dtype=torch.float32, device=dev) for _ in range(2))
        bounds = torch.zeros(num_pages, kv_heads, 2, head_dim, dtype=dtype or torch.bfloat16, device=dev)
        cache = cls(k, v, ks, vs, bounds)
        with torch.cuda.device(cache.device):
            _wait_for_buffers()  # tokens written on another stream must not meet the fills
        return cache


class SequenceBatch:
    """The sequences of a call: page_table int32 [num_seqs, table_width] (rows may be strided),
    kv_len int32 [num_seqs] with the call's own tokens counted in, and q_start int32 [num_seqs + 1],
    ascending: rows q_start[b] to q_start[b + 1] - 1 are the LAST tokens of sequence b.  Without
    q_start each sequence has one row.  Contents are read on the device when a call runs: they
    may change between calls and between the replays of a captured graph."""

    def __init__(self, page_table, kv_len, q_start=None):
        _need_torch()
        dev = page_table.device
        for t, name, ndim in ((page_table, "page_table", 2), (kv_len, "kv_len", 1), (q_start, "q_start", 1)):
            if t is not None:
                _etk._check_tensor(t, name, torch.int32, dev, ndim)
        B, width = page_table.shape
        if B < 1 or width < 1 or page_table.stride(1) != 1 and width > 1:
            raise ValueError("page_table must be [num_seqs, table_width] with contiguous rows")
        pitch = page_table.stride(0) if B > 1 else width
        if pitch < width:
            raise ValueError("page_table's rows must not overlap")
        if tuple(kv_len.shape) != (B,) or not kv_len.is_contiguous():
            raise ValueError(f"kv_len must be contiguous [{B}]")
        if q_start is not None and (tuple(q_start.shape) != (B + 1,) or not q_start.is_contiguous()):
            raise ValueError(f"q_start must be contiguous [{B + 1}]")
        self.page_table, self.kv_len, self.q_start = page_table, kv_len, q_start
        self.num_seqs, self.table_width, self.device = B, width, dev
        self._c = _Batch(page_table.data_ptr(), kv_len.data_ptr(), None if q_start is None else q_start.data_ptr(),
                         B, width, pitch)
        self._ref = ctypes.byref(self._c)

    def _check(self, cache, tokens):
        if self.device != cache.device:
            raise ValueError(f"the batch must be on {cache.device}, got {self.device}")
        if self.q_start is None and tokens != self.num_seqs:
            raise ValueError(f"without q_start there is one row for each of {self.num_seqs} sequences, got {tokens}")


def cache_write(cache, batch, k, v, stream=None):
    """Quantises rows k, v [num_tokens, kv_heads, head_dim] into the pages of their positions.

    A page's scale is the power of two that brings its largest magnitude within e4m3's 448; a page
    continued by larger rows has its earlier codes rescaled, one written from its first offset starts
    anew.  The key bounds follow.  Infinities and NaN are stored as NaN."""
    kr = _rows(k, "k", cache, cache.kv_heads)
    vr = _rows(v, "v", cache, cache.kv_heads, k.shape[0])
    batch._check(cache, k.shape[0])
    _call(cache, stream, _lib().exact_topk_cache_write, cache._ref, batch._ref, k.shape[0], kr, vr)


def cache_read(cache, batch, num_tokens=None, out=None, stream=None):
    """The stored rows of the batch's tokens, (k, v) [num_tokens, kv_heads, head_dim] of the cache's
    type.  ``out``: a pair of tensors to write into; rows of no sequence are left as they are there."""
    if out is None:
        if num_tokens is None:
            num_tokens = batch.num_seqs if batch.q_start is None else None
        if num_tokens is None:
            raise ValueError("num_tokens or out is needed with q_start")
        with torch.cuda.stream(stream):
            out = tuple(torch.zeros(num_tokens, cache.kv_heads, cache.head_dim, dtype=cache.dtype,
                                    device=cache.device) for _ in range(2))
    k, v = out
    kr = _rows(k, "out[0]", cache, cache.kv_heads, num_tokens)
    vr = _rows(v, "out[1]", cache, cache.kv_heads, k.shape[0])
    _written(k, "out[0]", v)
    if not v.is_contiguous():
        _written(v, "out[1]", k)
    batch._check(cache, k.shape[0])
    _call(cache, stream, _lib().exact_topk_cache_read, cache._ref, batch._ref, k.shape[0], kr, vr)
    return k, v


def block_scores(cache, batch, q, keep_first=0, keep_last=0, scores=None, ke=None, num_valid_rows=None,
                 stream=None):
    """Page scores of q [num_tokens, q_heads, head_dim] as the exact Top-K reads them: (scores, ke).

    scores float32 [num_tokens * kv_heads, table_width]: row token * kv_heads + head holds, for each page
    the token sees, the largest over the key head's query heads of an upper bound of q . k over the page's
    keys as they were written (from the key bounds); the first keep_first pages and the newest keep_last get +inf.  ke int32
    [num_tokens * kv_heads] is the number of pages seen.  Entries beyond it, and rows of no sequence, are
    left as they were.  num_valid_rows, an int32 tensor of one element, gets the number of live rows."""
    heads = q.shape[1] if q.dim() == 3 else 0
    qr = _rows(q, "q", cache, heads)
    if heads < 1 or heads % cache.kv_heads:
        raise ValueError(f"q must have a multiple of {cache.kv_heads} heads, got {heads}")
    T = q.shape[0]
    batch._check(cache, T)
    rows = T * cache.kv_heads
    if scores is None or ke is None:
        with torch.cuda.stream(stream):
            if scores is None:
                scores = torch.empty(rows, batch.table_width, dtype=torch.float32, device=cache.device)
            if ke is None:
                ke = torch.zeros(rows, dtype=torch.int32, device=cache.device)
    _etk._check_tensor(scores, "scores", torch.float32, cache.device, 2)
    _etk._check_tensor(ke, "ke", torch.int32, cache.device, 1)
    if scores.shape[0] != rows or scores.shape[1] != batch.table_width or \
            (scores.shape[1] > 1 and scores.stride(1) != 1):
        raise ValueError(f"scores must be [{rows}, {batch.table_width}] with contiguous rows")
    pitch = scores.stride(0) if rows > 1 else batch.table_width
    if pitch < batch.table_width:
        raise ValueError("the rows of scores must not overlap")
    if ke.shape[0] != rows or not ke.is_contiguous():
        raise ValueError(f"ke must be contiguous [{rows}]")
    if num_valid_rows is not None:
        _etk._check_tensor(num_valid_rows, "num_valid_rows", torch.int32, cache.device)
        if num_valid_rows.numel() != 1:
            raise ValueError("num_valid_rows must have one element")
    if keep_first < 0 or keep_last < 0:
        raise ValueError("keep_first and keep_last must not be negative")
    most = batch.table_width
    _call(cache, stream, _lib().exact_topk_block_scores, cache._ref, batch._ref, T, heads, qr,
          min(int(keep_first), most), min(int(keep_last), most), scores.data_ptr(), pitch, ke.data_ptr(),
          None if num_valid_rows is None else num_valid_rows.data_ptr())
    return scores, ke


def make_attention_plan(num_tokens, num_seqs, q_heads, kv_heads, head_dim, page_size, table_width, num_blocks=0,
                        single_rows=False, device_info=None, prompt=-1) -> AttentionPlan:
    """The attention's launch plan (pure host logic; needs a DeviceInfo, queried when omitted).
    prompt: whether the kernel for prompts runs: -1 the planner's choice, 0 no, 1 yes."""
    if device_info is None:
        device_info = _etk.query_device()
    plan = AttentionPlan()
    _etk._check(_lib().exact_topk_make_attention_plan(
        int(num_tokens), int(num_seqs), int(bool(single_rows)), int(q_heads), int(kv_heads), int(head_dim),
        int(page_size), int(table_width), int(num_blocks), int(prompt), ctypes.byref(device_info), ctypes.byref(plan)),
        "exact_topk_make_attention_plan")
    return plan


class CacheAttention:
    """Attention of a batch's rows over their cached tokens, for one captured shape; owns its
    plan, counters and workspace.

    num_blocks=0 attends to every cached token up to the row's own; num_blocks=K to those of the pages
    listed for each token and key head (``blocks`` int32 [num_tokens * kv_heads, K], as ExactTopK selects
    them: a set in any order, -1 and anything outside the pages that the token sees ignored, repeats counted
    once).  A row that sees nothing gives zeros.  Calls of one object must not overlap on the GPU: graphs
    that may run at the same time each need an object of their own.  Keep the object until its last call has run."""

    def __init__(self, cache, num_seqs, num_tokens, q_heads, table_width, num_blocks=0, **overrides):
        self.cache = cache
        with torch.cuda.device(cache.device):
            self.plan = make_attention_plan(num_tokens, num_seqs, q_heads, cache.kv_heads, cache.head_dim,
                                            cache.page_size, table_width, num_blocks,
                                            single_rows=num_tokens == num_seqs, **overrides)
            self.counters = torch.zeros(max(16, self.plan.counter_bytes), dtype=torch.uint8, device=cache.device)
            self.workspace = torch.empty(max(16, self.plan.workspace_bytes), dtype=torch.uint8,
                                         device=cache.device)
            _wait_for_buffers()
        self._plan = ctypes.byref(self.plan)
        self._buffers = (self.counters.data_ptr(), self.counters.numel(), self.workspace.data_ptr(),
                         self.workspace.numel())

    def __call__(self, q, batch, blocks=None, out=None, scale=None, stream=None):
        """out [num_tokens, q_heads, head_dim]; scale defaults to 1 / sqrt(head_dim)."""
        cache, plan = self.cache, self.plan
        qr = _rows(q, "q", cache, plan.q_heads, plan.num_tokens)
        batch._check(cache, plan.num_tokens)
        if batch.num_seqs != plan.num_seqs or batch.table_width != plan.table_width:
            raise ValueError(f"the batch must have {plan.num_seqs} sequences and a table of {plan.table_width} pages")
        if out is None:
            with torch.cuda.stream(stream):
                out = torch.zeros(q.shape, dtype=q.dtype, device=q.device)
        outr = _rows(out, "out", cache, plan.q_heads, plan.num_tokens)
        _written(out, "out", q)
        if (blocks is None) != (plan.num_blocks == 0):
            raise ValueError(f"this object's rows have {plan.num_blocks} listed pages each")
        if blocks is not None:
            _etk._check_tensor(blocks, "blocks", torch.int32, cache.device, 2)
            if tuple(blocks.shape) != (plan.num_tokens * plan.kv_heads, plan.num_blocks) or \
                    not blocks.is_contiguous():
                raise ValueError(f"blocks must be contiguous [{plan.num_tokens * plan.kv_heads}, {plan.num_blocks}]")
        if scale is None:
            scale = 1.0 / math.sqrt(cache.head_dim)
        _call(cache, stream, _lib().exact_topk_attention_run, self._plan, cache._ref, batch._ref, qr, outr,
              None if blocks is None else blocks.data_ptr(), scale, *self._buffers)
        return out


class SparseAttention:
    """A sparse-attention step for one captured shape: page scores, the exact Top-K of them, and the
    attention over the pages selected for each token and key head.  Owns every buffer between.

    keep_first and keep_last pages (the sequence's first and newest) are always among the num_blocks
    selected, which must be at least as many.  As of CacheAttention, calls of one object must not overlap
    on the GPU, and the object is kept until its last call has run."""

    def __init__(self, cache, num_seqs, num_tokens, q_heads, table_width, num_blocks, keep_first=0, keep_last=1):
        if keep_first < 0 or keep_last < 0 or keep_first + keep_last > num_blocks:
            raise ValueError("need 0 <= keep_first + keep_last <= num_blocks")
        if num_tokens < 1 or num_blocks < 1:
            raise ValueError("need num_tokens, num_blocks >= 1")
        self.cache, self.keep = cache, (keep_first, keep_last)
        rows = num_tokens * cache.kv_heads
        self.attention = CacheAttention(cache, num_seqs, num_tokens, q_heads, table_width, num_blocks)
        self.select = _etk.ExactTopK(rows, table_width, num_blocks, device=cache.device)
        dev = cache.device
        self.scores = torch.empty(rows, table_width, dtype=torch.float32, device=dev)
        self.ke = torch.zeros(rows, dtype=torch.int32, device=dev)
        self.live = torch.zeros(1, dtype=torch.int32, device=dev)
        self.blocks = torch.full((rows, num_blocks), -1, dtype=torch.int32, device=dev)
        with torch.cuda.device(dev):
            _wait_for_buffers()

    def __call__(self, q, batch, k=None, v=None, out=None, scale=None, stream=None):
        """Attends with q [num_tokens, q_heads, head_dim]; rows k, v of the same tokens, where given, are
        written to the cache first.  self.blocks holds the pages selected."""
        if (k is None) != (v is None):
            raise ValueError("k and v go together")
        if stream is None:
            stream = torch.cuda.current_stream(self.cache.device)
        if k is not None:
            if k.shape[0] != q.shape[0]:
                raise ValueError("k, v and q must have the same tokens")
            cache_write(self.cache, batch, k, v, stream=stream)
        block_scores(self.cache, batch, q, *self.keep, scores=self.scores, ke=self.ke,
                     num_valid_rows=self.live, stream=stream)
        self.select(self.scores, self.ke, num_valid_rows=self.live, out=self.blocks, stream=stream)
        return self.attention(q, batch, blocks=self.blocks, out=out, scale=scale, stream=stream)
