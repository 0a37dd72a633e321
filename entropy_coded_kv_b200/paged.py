"""Paged compressed KV cache: rotary positions, append, attention of new tokens,
page copies and compaction (include/ecco.h, "Paged compressed cache").

A pool holds the 64-byte blocks of one layer's keys (or values) in pages,
uint8 [n_pages, kv_heads, page_size, 64]; a sequence is a row of page numbers
and a length.  The functions below are the thin binding: they check shapes,
types and devices and pass device pointers and the current stream on.
`PageAllocator` keeps the book of pages on the host, and `PagedCache` joins it
with the pools and the calls."""
from __future__ import annotations

import ctypes
import heapq
import math
from array import array

import torch

from . import _lib

GROUP, BLOCK_BYTES = 128, 64
_DTYPES = {torch.bfloat16: _lib.BF16, torch.float16: _lib.F16, torch.float32: _lib.F32}
_BF16, _F32, _U8, _I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
_CONTIGUOUS = torch.contiguous_format
# (a torch without CUDA lacks these two; it can import the package, and has no tensor to call with)
_get_device, _get_stream = (getattr(torch._C, f, None) for f in ("_cuda_getDevice", "_cuda_getCurrentRawStream"))

# A single token's call lasts a few microseconds on the GPU, so the checks come
# twice: one expression that holds for every valid call, and, where it does not,
# the checks one by one, which say what is wrong.


def _on(t, dtype, dim, name, device=None):
    """A `dim`-dimensional CUDA tensor of the type, on the device (an index) if one is given; its device's index."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype:
        raise TypeError(f"{name} must be a {dtype} tensor")
    at = t.get_device()
    if at < 0 or (device is not None and at != device):
        raise ValueError(f"{name} is on {t.device}" + (f", expected cuda:{device}" if device is not None else ""))
    if t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions")
    return at


def _dense(t, dtype, dim, name, device=None):
    """The same, contiguous."""
    at = _on(t, dtype, dim, name, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return at


def _strides(t, shape, name):
    """Token and head strides of [tokens, heads, dim]; those of a dimension of size one say nothing."""
    n, h, d = shape
    if t.is_contiguous():
        return h * d, d
    st, sh, sd = t.stride()
    if sd != 1 and d > 1 and n and h:
        raise ValueError(f"{name}: the values of a head must be contiguous")
    if h <= 1:
        sh = (d + 7) // 8 * 8
    return (st if n > 1 else h * sh), sh


def _call(fn, device, *args):
    """The library call on the device's current stream, with that device current."""
    f = getattr(_lib._lib or _lib.load(), fn)
    if _get_device() == device:
        rc = f(*args, _get_stream(device))
    else:
        with torch.cuda.device(device):
            rc = f(*args, _get_stream(device))
    if rc:  # _lib.ECCO_OK is 0
        _lib.check(rc, fn)


_2_31 = 1 << 31


def _int32(v, name):
    """v as an int that the C call takes whole (ctypes would keep its low 32 bits)."""
    v = int(v)
    if not -_2_31 <= v < _2_31:
        raise ValueError(f"{name} = {v} does not fit 32 bits")
    return v


def _ptr(t):
    return None if t is None else t.data_ptr()


def _tables_on(k_tables, v_tables):
    dev = k_tables.device.index
    if v_tables.device.index != dev:
        raise ValueError(f"v_tables are on {v_tables.device}, k_tables on {k_tables.device}")
    return _get_device() if dev is None else dev


# ------------------------------------------------------------------ rotary positions
def rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: dict | None = None):
    """(inv_freq, magnitude): angle of pair i per position, base ** (-2 i /
    rotary_dim), and the factor on cos and sin.  `scaling` stretches them for
    long contexts by its "factor" s, by "kind":
      "linear"  every frequency / s;
      "ntk"     base * s ** (rotary_dim / (rotary_dim - 2)): the slowest pair is
                stretched by s, the fastest hardly;
      "bands"   pairs that turn fewer than `low` times (1) over the `original`
                context are stretched by s, those above `high` (4) are kept, and
                between them the two are mixed linearly in the number of turns;
      "yarn"    the same with a ramp linear in the pair's index between the
                pairs that turn `high` (32) and `low` (1) times, and cos and sin
                times 0.1 ln s + 1 (arXiv 2309.00071)."""
    half = rotary_dim // 2
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even")
    if not base > 1 or not math.isfinite(base):
        raise ValueError("base must be above 1")
    freq = [base ** (-2.0 * i / rotary_dim) for i in range(half)]
    if scaling is None:
        return freq, 1.0
    kind, s = scaling["kind"], float(scaling["factor"])
    if not s >= 1 or not math.isfinite(s):
        raise ValueError("factor must be at least 1")
    if kind == "linear":
        return [f / s for f in freq], 1.0
    if kind == "ntk":
        if rotary_dim == 2:
            return freq, 1.0
        return rope_frequencies(rotary_dim, base * s ** (rotary_dim / (rotary_dim - 2.0)))
    if kind not in ("bands", "yarn"):
        raise ValueError(f"unknown scaling kind {kind!r}")
    original = float(scaling["original"])
    low, high = float(scaling.get("low", 1)), float(scaling.get("high", 4 if kind == "bands" else 32))
    if not (original > 0 and 0 < low < high):
        raise ValueError("scaling wants original > 0 and 0 < low < high")
    if kind == "bands":
        keep = [min(1.0, max(0.0, (original * f / (2 * math.pi) - low) / (high - low))) for f in freq]
        return [f * k + f / s * (1 - k) for f, k in zip(freq, keep)], 1.0
    at = [rotary_dim * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (high, low)]
    first, last = max(0, math.floor(at[0])), min(rotary_dim - 1, math.ceil(at[1]))
    width = max(last - first, 1e-3)
    keep = [1 - min(1.0, max(0.0, (i - first) / width)) for i in range(half)]
    return [f * k + f / s * (1 - k) for f, k in zip(freq, keep)], (0.1 * math.log(s) + 1.0 if s > 1 else 1.0)


def rope_table(n_positions: int, rotary_dim: int, base: float = 10000.0, scaling: dict | None = None,
               device=None) -> torch.Tensor:
    """fp32 [n_positions, rotary_dim / 2, 2]: cos and sin of every position's
    angles, from fp64 angles (rope_frequencies gives the arguments)."""
    freq, magnitude = rope_frequencies(rotary_dim, base, scaling)
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    if dev.type != "cuda":
        raise ValueError("the table lives on a CUDA device")
    table = torch.empty((int(n_positions), rotary_dim // 2, 2), dtype=_F32, device=dev)
    arr = (ctypes.c_double * len(freq))(*freq)
    _call("ecco_rope_table", table.get_device(), arr, len(freq), magnitude, int(n_positions), table.data_ptr())
    return table


def _table(rope, device):
    _dense(rope, _F32, 3, "table", device)
    n, half, two = rope.shape
    if two != 2:
        raise ValueError("table must be [n_positions, rotary_dim / 2, 2]")
    return n, 2 * half


_FLAGS = ((0, _lib.ROPE_INVERSE), (_lib.ROPE_INTERLEAVED, _lib.ROPE_INTERLEAVED | _lib.ROPE_INVERSE))


def rope(x: torch.Tensor, table: torch.Tensor, positions: torch.Tensor, interleaved: bool = False,
         inverse: bool = False, out: torch.Tensor | None = None) -> torch.Tensor:
    """x [tokens, heads, dim] (bf16, fp16 or fp32) with the first rotary_dim
    values of each head turned by the angles of its row's position (int32
    [tokens]; one outside the table takes its nearest row): pairs (i, i +
    rotary_dim / 2), or (2 i, 2 i + 1) if interleaved.
    inverse takes the angles' negatives, which is the gradient of x from that of
    the result; it undoes a turn by a table of magnitude 1, one of magnitude m
    (yarn) it returns times m * m.  `out` may be x.  The result of an x that
    requires a gradient has one (not with `out`: torch would not know of the
    write)."""
    if isinstance(x, torch.Tensor) and x.requires_grad and torch.is_grad_enabled():
        if out is not None:
            raise ValueError("x requires a gradient: no `out`, or under torch.no_grad()")
        return _Rope.apply(x, table, positions, bool(interleaved), bool(inverse))
    if not isinstance(x, torch.Tensor) or x.dtype not in _DTYPES:
        raise TypeError("x must be a bf16, fp16 or fp32 tensor")
    dev, shape = x.get_device(), x.shape
    if not (isinstance(table, torch.Tensor) and isinstance(positions, torch.Tensor) and dev >= 0 and len(shape) == 3
            and table.dtype is _F32 and positions.dtype is _I32 and table.get_device() == positions.get_device() == dev
            and table.dim() == 3 and positions.dim() == 1 and table.is_contiguous() and positions.is_contiguous()):
        _on(x, x.dtype, 3, "x")
        _table(table, dev)
        _dense(positions, _I32, 1, "positions", dev)
    tokens, heads, dim = shape
    n, half, two = table.shape
    if two != 2:
        raise ValueError("table must be [n_positions, rotary_dim / 2, 2]")
    rotary = 2 * half
    if positions.shape[0] != tokens:
        raise ValueError("positions must have an entry for each row of x")
    if out is None:
        out = torch.empty_like(x, memory_format=_CONTIGUOUS)
    else:
        _on(out, x.dtype, 3, "out", dev)
        if out.shape != shape:
            raise ValueError("out must have x's shape")
    _call("ecco_rope", dev, x.data_ptr(), *_strides(x, shape, "x"), out.data_ptr(), *_strides(out, shape, "out"), _DTYPES[x.dtype],
          tokens, heads, dim, table.data_ptr(), n, rotary, positions.data_ptr(), _FLAGS[bool(interleaved)][bool(inverse)])
    return out


class _Rope(torch.autograd.Function):
    """rope where autograd records: a linear map, its gradient is the transposed one."""

    @staticmethod
    def forward(ctx, x, table, positions, interleaved, inverse):
        ctx.save_for_backward(table, positions)
        ctx.flags = interleaved, inverse
        return rope(x, table, positions, interleaved, inverse)

    @staticmethod
    def backward(ctx, dy):
        table, positions = ctx.saved_tensors
        interleaved, inverse = ctx.flags
        dy = dy.contiguous()  # of a sum, say, it has no strides
        if dy.data_ptr() % 16:
            dy = dy.clone()
        return rope(dy, table, positions, interleaved, not inverse), None, None, None, None


# ------------------------------------------------------------------ the paged cache
def _paged(k_pages, v_pages, page_table, kv_lens, cu_q, device):
    if not (isinstance(k_pages, torch.Tensor) and isinstance(v_pages, torch.Tensor)
            and isinstance(page_table, torch.Tensor) and isinstance(kv_lens, torch.Tensor)
            and k_pages.dtype is v_pages.dtype is _U8 and page_table.dtype is kv_lens.dtype is _I32
            and k_pages.get_device() == v_pages.get_device() == page_table.get_device() == kv_lens.get_device() == device
            and k_pages.dim() == 4 and page_table.dim() == 2 and kv_lens.dim() == 1
            and k_pages.is_contiguous() and v_pages.is_contiguous() and kv_lens.is_contiguous()):
        _dense(k_pages, _U8, 4, "k_pages", device)
        _dense(v_pages, _U8, 4, "v_pages", device)
        _on(page_table, _I32, 2, "page_table", device)
        _dense(kv_lens, _I32, 1, "kv_lens", device)
    shape = k_pages.shape
    n_pages, heads, page_size, block = shape
    if v_pages.shape != shape or block != BLOCK_BYTES:
        raise ValueError("k_pages / v_pages must be [n_pages, kv_heads, page_size, 64] of the same shape")
    batch, max_pages = page_table.shape
    stride, one = page_table.stride()
    if one != 1 and max_pages > 1 and batch:
        raise ValueError("the entries of a page_table row must be contiguous")
    if kv_lens.shape[0] != batch:
        raise ValueError("kv_lens must have an entry for each row of page_table")
    cu = None
    if cu_q is not None:
        if not (isinstance(cu_q, torch.Tensor) and cu_q.dtype is _I32 and cu_q.get_device() == device and cu_q.dim() == 1
                and cu_q.is_contiguous()):
            _dense(cu_q, _I32, 1, "cu_q", device)
        if cu_q.shape[0] != batch + 1:
            raise ValueError("cu_q must have one entry more than page_table has rows")
        cu = cu_q.data_ptr()
    return _lib.Paged(n_pages, page_size, heads, batch, max_pages, stride if batch > 1 else max_pages,
                      page_table.data_ptr(), kv_lens.data_ptr(), cu)


def paged_append(k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, k_tables, v_tables,
                 page_table: torch.Tensor, kv_lens: torch.Tensor, cu_q: torch.Tensor,
                 rope: torch.Tensor | None = None, positions: torch.Tensor | None = None, interleaved: bool = False,
                 inverse: bool = False, stats: torch.Tensor | None = None) -> None:
    """Encodes the new tokens' keys and values (bf16 [tokens, kv_heads, 128])
    into their pages: row cu_q[b] + i goes to position kv_lens[b] - (cu_q[b + 1]
    - cu_q[b]) + i of sequence b (kv_lens counts the new tokens).  With `rope`
    (a rope_table of at most 128 values) the keys are turned first, by their own
    positions or by `positions` (int32 [tokens]); one outside the table takes its
    nearest row."""
    dev = _tables_on(k_tables, v_tables)
    _on(k, _BF16, 3, "k", dev)
    _on(v, _BF16, 3, "v", dev)
    p = _paged(k_pages, v_pages, page_table, kv_lens, cu_q, dev)
    shape = k.shape
    tokens, heads, dim = shape
    if v.shape != shape or heads != p.kv_heads or dim != GROUP:
        raise ValueError("k and v must be [tokens, kv_heads, 128]")
    n, rotary = (0, 0) if rope is None else _table(rope, dev)
    if positions is not None:
        _dense(positions, _I32, 1, "positions", dev)
        if positions.shape[0] != tokens:
            raise ValueError("positions must have an entry for each row of k")
    if stats is not None:
        _dense(stats, torch.int64, 1, "stats", dev)
        if stats.numel() < len(_lib.STATS_FIELDS):
            raise ValueError("stats must be a buffer of new_stats")
    _call("ecco_paged_append", dev, k_tables.handle, v_tables.handle, p, k.data_ptr(), *_strides(k, shape, "k"), v.data_ptr(),
          *_strides(v, shape, "v"), tokens, k_pages.data_ptr(), v_pages.data_ptr(), _ptr(rope), n, rotary,
          _ptr(positions), _FLAGS[bool(interleaved)][bool(inverse)], _ptr(stats))


_BOUNDS = ("batch up to 1024, 1 to 1024 KV heads, group 1 to 16, max_q up to 2^26, max_kv up to 2^30, "
           "batch * ceil(max_kv / 128) up to 2^24")


def paged_attention_workspace_bytes(batch: int, kv_heads: int, group: int, max_q: int, max_kv: int) -> int:
    """Bytes of workspace of a paged_attention call; 0 for bounds that the call
    refuses.  It never shrinks when an argument grows: a workspace of the largest
    bounds serves every smaller call."""
    return int(_lib.load().ecco_paged_attention_workspace_bytes(
        _int32(batch, "batch"), _int32(kv_heads, "kv_heads"), _int32(group, "group"), _int32(max_q, "max_q"),
        _int32(max_kv, "max_kv")))


def paged_attention(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, k_tables, v_tables,
                    page_table: torch.Tensor, kv_lens: torch.Tensor, cu_q: torch.Tensor, scale: float,
                    max_q: int | None = None, max_kv: int | None = None, window: int = 0,
                    out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Causal attention of new tokens, already appended, over the paged cache (no
    gradient).

    q: bf16 [tokens, kv_heads * group, 128], rows cu_q[b] .. cu_q[b + 1] - 1 the
    last tokens of sequence b.  Returns bf16 of q's shape; `lse` (fp32 [tokens,
    kv_heads * group]) takes the log-sums of the scores.  window > 0: a token
    sees the last `window` keys up to its own.  max_q and max_kv bound the new
    tokens and the keys of one sequence (by default all rows, and what a
    page_table row holds); they size the workspace
    (paged_attention_workspace_bytes), which may be passed to reuse it, and they
    choose kernels: the same call gives the same bits, other bounds or another
    batch values within the same roundings.  Rows of no sequence (before cu_q[0],
    behind cu_q[-1]) and new tokens past max_q are not written: in `out` and `lse`
    they stay as they were, in a result of the call's own they are whatever its
    memory held."""
    dev = _tables_on(k_tables, v_tables)
    _on(q, _BF16, 3, "q", dev)
    p = _paged(k_pages, v_pages, page_table, kv_lens, cu_q, dev)
    shape = q.shape
    tokens, heads, dim = shape
    kv_heads = p.kv_heads
    if dim != GROUP or not kv_heads or heads % kv_heads:
        raise ValueError("q must be [tokens, kv_heads * group, 128]")
    group = heads // kv_heads
    if out is None:
        out = torch.empty_like(q, memory_format=_CONTIGUOUS)
    else:
        _on(out, _BF16, 3, "out", dev)
        if out.shape != shape:
            raise ValueError("out must have q's shape")
    if lse is not None:
        _dense(lse, _F32, 2, "lse", dev)
        if lse.shape != (tokens, heads):
            raise ValueError("lse must be [tokens, kv_heads * group]")
    max_q = tokens if max_q is None else int(max_q)
    max_kv = p.max_pages * p.page_size if max_kv is None else int(max_kv)
    window = int(window)
    if not (-_2_31 <= max_q < _2_31 and -_2_31 <= max_kv < _2_31 and -_2_31 <= window < _2_31):
        _int32(max_q, "max_q"), _int32(max_kv, "max_kv"), _int32(window, "window")
    if workspace is None:
        workspace = torch.empty(max(1, paged_attention_workspace_bytes(p.batch, kv_heads, group, max_q, max_kv)),
                                dtype=_U8, device=q.device)
    else:
        _dense(workspace, _U8, 1, "workspace", dev)
    try:
        _call("ecco_paged_attention", dev, k_tables.handle, v_tables.handle, p, k_pages.data_ptr(), v_pages.data_ptr(),
              q.data_ptr(), *_strides(q, shape, "q"), group, tokens, max_q, max_kv, window, float(scale), out.data_ptr(),
              *_strides(out, shape, "out"), _ptr(lse), workspace.data_ptr(), workspace.numel())
    except _lib.EccoError as e:
        if e.code == _lib.ECCO_ERR_ARG:  # the two refusals that say too little
            need = paged_attention_workspace_bytes(p.batch, kv_heads, group, max_q, max_kv)
            if not need:
                raise _lib.EccoError(e.code, f"ecco_paged_attention ({_BOUNDS})") from None
            if workspace.numel() < need:
                raise _lib.EccoError(e.code, f"ecco_paged_attention (a workspace of {workspace.numel()} bytes for {need})") from None
        raise
    return out


def _host_ids(ids, name):
    """Page numbers on the host as an int32 tensor; none is rounded or cut to 32 bits."""
    if str(getattr(ids, "dtype", None)) == "int32":  # a numpy array: as it is
        ids = torch.as_tensor(ids)
    if isinstance(ids, torch.Tensor):
        if ids.dtype is not _I32 or ids.get_device() >= 0 or ids.dim() != 1:
            raise TypeError(f"{name} must be a list or a one-dimensional int32 CPU tensor")
        return ids if ids.is_contiguous() else ids.contiguous()
    try:
        flat = array("i", ids)
    except OverflowError:
        raise ValueError(f"{name} holds a number past 32 bits") from None
    return torch.frombuffer(flat, dtype=_I32) if flat else torch.empty(0, dtype=_I32)


def copy_pages(k_pages: torch.Tensor, v_pages: torch.Tensor, src, dst) -> None:
    """Copies page src[i] to page dst[i] of both pools.  src and dst are page
    numbers on the host (lists or int32 CPU tensors); no destination may appear
    twice or be a source."""
    if not (isinstance(k_pages, torch.Tensor) and isinstance(v_pages, torch.Tensor) and k_pages.dtype is v_pages.dtype is _U8
            and (dev := k_pages.get_device()) == v_pages.get_device() >= 0 and k_pages.dim() == 4
            and k_pages.is_contiguous() and v_pages.is_contiguous()):
        dev = _dense(k_pages, _U8, 4, "k_pages")
        _dense(v_pages, _U8, 4, "v_pages", dev)
    n_pages, heads, page_size, block = k_pages.shape
    if v_pages.shape != k_pages.shape or block != BLOCK_BYTES:
        raise ValueError("k_pages / v_pages must be [n_pages, kv_heads, page_size, 64] of the same shape")
    src, dst = _host_ids(src, "src"), _host_ids(dst, "dst")
    if src.numel() != dst.numel():
        raise ValueError("src and dst must be of the same length")
    _call("ecco_copy_pages", dev, k_pages.data_ptr(), v_pages.data_ptr(), n_pages, heads * page_size * BLOCK_BYTES,
          src.data_ptr(), dst.data_ptr(), src.numel())


def compact_pages(k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor, kv_lens: torch.Tensor,
                  keep: torch.Tensor, dst_table: torch.Tensor, out_lens: torch.Tensor | None = None) -> torch.Tensor:
    """Moves the kept tokens of each sequence (keep: bool or uint8 [batch, at
    least the longest length]) to the front of the pages dst_table (int32
    [batch, dst_pages]), in their order, and returns the new lengths (int32
    [batch]; `out_lens` may not be kv_lens).  The blocks move as they are:
    nothing is encoded again.  The destination pages may not be among the pages
    read."""
    dev = _on(k_pages, _U8, 4, "k_pages")
    p = _paged(k_pages, v_pages, page_table, kv_lens, None, dev)
    _on(keep, keep.dtype if isinstance(keep, torch.Tensor) and keep.dtype in (torch.bool, _U8) else torch.bool,
        2, "keep", dev)
    if not keep.is_contiguous():
        raise ValueError("keep must be contiguous")
    _on(dst_table, _I32, 2, "dst_table", dev)
    if dst_table.shape[1] > 1 and dst_table.stride(1) != 1 and p.batch:
        raise ValueError("the entries of a dst_table row must be contiguous")
    if keep.shape[0] != p.batch or dst_table.shape[0] != p.batch:
        raise ValueError("keep and dst_table must have a row for each of page_table")
    if out_lens is None:
        out_lens = torch.empty_like(kv_lens)
    _dense(out_lens, _I32, 1, "out_lens", dev)
    if out_lens.shape[0] != p.batch:
        raise ValueError("out_lens must have an entry for each row of page_table")
    _call("ecco_compact_pages", dev, p, k_pages.data_ptr(), v_pages.data_ptr(), keep.data_ptr(), keep.shape[1],
          dst_table.data_ptr(), dst_table.stride(0) if p.batch > 1 else dst_table.shape[1], dst_table.shape[1],
          out_lens.data_ptr())
    return out_lens


# ------------------------------------------------------------------ the book of pages
class OutOfPages(RuntimeError):
    """The pool has fewer free pages than a request needs; nothing was changed."""


class PageAllocator:
    """Host-side book of a pool's pages: which sequence holds which pages, how
    many sequences share a page, which are free.  Sequences are numbered; the
    lowest free page is handed out first.  A shared page is never written: the
    partly filled last page of a forked sequence is copied when it grows."""

    def __init__(self, n_pages: int, page_size: int):
        if n_pages < 0 or page_size < 1:
            raise ValueError("n_pages >= 0 and page_size >= 1")
        self.n_pages, self.page_size = int(n_pages), int(page_size)
        self._free = list(range(self.n_pages))
        self._users = [0] * self.n_pages
        self._pages: dict[int, list[int]] = {}
        self._len: dict[int, int] = {}
        self._next = 0

    @property
    def free_pages(self) -> int:
        return len(self._free)

    def pages(self, seq: int) -> list[int]:
        return list(self._pages[seq])

    def length(self, seq: int) -> int:
        return self._len[seq]

    def _take(self) -> int:
        p = heapq.heappop(self._free)
        self._users[p] = 1
        return p

    def _drop(self, page: int) -> None:
        self._users[page] -= 1
        if self._users[page] == 0:
            heapq.heappush(self._free, page)

    def add(self) -> int:
        """A new, empty sequence."""
        s = self._next
        self._next += 1
        self._pages[s], self._len[s] = [], 0
        return s

    def fork(self, seq: int) -> int:
        """A sequence with the same tokens, on the same pages."""
        pages, n = self._pages[seq], self._len[seq]
        s = self.add()
        for p in pages:
            self._users[p] += 1
        self._pages[s], self._len[s] = list(pages), n
        return s

    def free(self, seq: int) -> None:
        for p in self._pages.pop(seq):
            self._drop(p)
        del self._len[seq]

    def extend(self, seqs: list[int], new: list[int]) -> list[tuple[int, int]]:
        """Room for new[i] more tokens of each sequence.  Returns the (source,
        destination) pages to copy before they are written."""
        if len(seqs) != len(new) or len(set(seqs)) != len(seqs):
            raise ValueError("one count for each sequence, and no sequence twice")
        if any(n < 0 for n in new):
            raise ValueError("counts must not be negative")
        ps = self.page_size
        # users: the sharers left once the earlier sequences of this call have their own copy
        shared, need, split = {}, 0, []
        for s, n in zip(seqs, new):
            pages, have = self._pages[s], self._len[s]
            need += max(0, -(-(have + n) // ps) - len(pages))
            if n and have % ps:
                last = pages[have // ps]
                if shared.setdefault(last, self._users[last]) > 1:
                    shared[last] -= 1
                    need += 1
                    split.append(s)
        if need > len(self._free):
            raise OutOfPages(f"{need} pages needed, {len(self._free)} free")
        copies = []
        for s in split:
            at = self._len[s] // ps
            old, own = self._pages[s][at], self._take()
            self._pages[s][at] = own
            self._drop(old)
            copies.append((old, own))
        for s, n in zip(seqs, new):
            self._len[s] += n
            while len(self._pages[s]) * ps < self._len[s]:
                self._pages[s].append(self._take())
        return copies

    def shrink(self, seq: int, length: int) -> None:
        """Drops the tokens from `length` on, and the pages that only they used."""
        if not 0 <= length <= self._len[seq]:
            raise ValueError("length must be between 0 and the sequence's")
        keep = -(-length // self.page_size)
        for p in self._pages[seq][keep:]:
            self._drop(p)
        del self._pages[seq][keep:]
        self._len[seq] = length

    def replace(self, seqs: list[int]) -> list[list[int]]:
        """As many fresh pages as each sequence has; the caller moves the tokens
        to them and then calls `settle`, or gives them back with `cancel`."""
        need = sum(len(self._pages[s]) for s in seqs)
        if len(set(seqs)) != len(seqs):
            raise ValueError("no sequence twice")
        if need > len(self._free):
            raise OutOfPages(f"{need} pages needed, {len(self._free)} free")
        return [[self._take() for _ in self._pages[s]] for s in seqs]

    def settle(self, seqs: list[int], fresh: list[list[int]], lengths: list[int]) -> None:
        for s, pages, n in zip(seqs, fresh, lengths):
            for p in self._pages[s]:
                self._drop(p)
            self._pages[s] = pages
            self._len[s] = len(pages) * self.page_size
            self.shrink(s, n)

    def cancel(self, fresh: list[list[int]]) -> None:
        for pages in fresh:
            for p in pages:
                self._drop(p)


class Step:
    """One batch's view of the cache, on the device: page_table, kv_lens (the
    new tokens among them), cu_q, positions; and on the host the number of new
    tokens, the bounds max_q and max_kv, and the largest position (-1: none)."""

    def __init__(self, page_table, kv_lens, cu_q, positions, tokens, max_q, max_kv, max_position=-1):
        self.page_table, self.kv_lens, self.cu_q, self.positions = page_table, kv_lens, cu_q, positions
        self.tokens, self.max_q, self.max_kv, self.max_position = tokens, max_q, max_kv, max_position


class PagedCache:
    """A paged compressed cache of several layers: pools, allocator and calls.

        cache = PagedCache(n_pages, page_size, kv_heads, k_tables, v_tables)   # one pair of tables a layer
        s = cache.add()
        step = cache.extend([s], [len(prompt)])          # pages, lengths and positions of the new tokens
        for layer in range(cache.layers):
            cache.append(step, layer, k, v, rope=table)  # keys turned, keys and values encoded
            out = cache.attend(step, layer, q, scale)    # q turned by rope(q, table, step.positions)
        t = cache.fork(s)                                # shares the pages
        cache.shrink(s, n)                               # drops the tokens from n on (a rejected draft)
        cache.compact([s], keep)                         # drops tokens
        cache.free(t)

    All calls of a cache belong on one stream: a freed page is handed out again
    at once, and only the stream's order keeps its readers before its writers.
    Dropped tokens leave the others' turned keys as they are, so after `compact`
    a sequence's next position is no longer its length: `extend` continues from
    the last position given."""

    def __init__(self, n_pages: int, page_size: int, kv_heads: int, k_tables, v_tables):
        self.k_tables = list(k_tables) if isinstance(k_tables, (list, tuple)) else [k_tables]
        self.v_tables = list(v_tables) if isinstance(v_tables, (list, tuple)) else [v_tables]
        if not self.k_tables or len(self.k_tables) != len(self.v_tables):
            raise ValueError("one pair of tables for each layer")
        self.device = self.k_tables[0].device
        if any(t.device != self.device for t in self.k_tables + self.v_tables):
            raise ValueError("all tables must be on one device")
        self.layers, self.kv_heads, self.page_size = len(self.k_tables), int(kv_heads), int(page_size)
        self.book = PageAllocator(n_pages, page_size)
        shape = (self.layers, n_pages, kv_heads, page_size, BLOCK_BYTES)
        self.k_pages = torch.empty(shape, dtype=_U8, device=self.device)
        self.v_pages = torch.empty(shape, dtype=_U8, device=self.device)
        # per sequence: its length after the last compaction, and the position of the token after it
        self._base: dict[int, tuple[int, int]] = {}

    def _next_position(self, seq: int) -> int:
        """The position of the sequence's next token, from its length, whoever changed that."""
        n, position = self._base[seq]
        have = self.book.length(seq)
        if have < n:  # shrunk into what was compacted: those positions are not known any more, and none is given twice
            n = have
            self._base[seq] = n, position
        return position + have - n

    def _on_device(self, *lists):
        """Each list of ints as int32 on the device, in one copy that nothing waits
        for: from pinned memory, which torch keeps until the copy has run."""
        flat = array("i")
        for v in lists:
            flat.extend(v)
        host = torch.empty(len(flat), dtype=_I32, pin_memory=True)
        host.copy_(torch.frombuffer(flat, dtype=_I32))
        return host.to(self.device, non_blocking=True).split([len(v) for v in lists])

    @staticmethod
    def _table_of(pages):
        """Page lists as the rows of a table, -1 behind their ends: (entries, width)."""
        width = max((len(p) for p in pages), default=0)
        return [e for p in pages for e in p + [-1] * (width - len(p))], width

    def add(self) -> int:
        s = self.book.add()
        self._base[s] = 0, 0
        return s

    def fork(self, seq: int) -> int:
        s = self.book.fork(seq)
        self._base[s] = self._base[seq]
        return s

    def free(self, seq: int) -> None:
        self.book.free(seq)
        del self._base[seq]

    def length(self, seq: int) -> int:
        return self.book.length(seq)

    def shrink(self, seq: int, length: int) -> None:
        """Drops the tokens from `length` on, and the pages that only they used.
        The next `extend` gives their positions again."""
        self.book.shrink(seq, length)
        self._next_position(seq)

    def extend(self, seqs: list[int], new: list[int]) -> Step:
        """Pages for new[i] more tokens of each sequence (OutOfPages if there are
        too few, with nothing changed), and the batch's view for the layers'
        calls.  Pages that are shared and about to be written are copied.  Waits
        for nothing on the device; the view is new memory each step, written by a
        copy from the host, so it cannot be captured into a graph (a captured step
        takes its own arrays, into which the view is copied).  The table is laid
        out on the host each time: 0.05 ms at 8 sequences of 64 pages, 2.5 ms at
        128 of 512."""
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("extend copies from the host: not while a graph is captured")
        if len(seqs) > _lib.MAX_BATCH:
            raise ValueError(f"at most {_lib.MAX_BATCH} sequences a step")
        first = [self._next_position(s) for s in seqs]
        copies = self.book.extend(seqs, new)
        if copies:
            n = self.book.n_pages
            src = [a + l * n for l in range(self.layers) for a, _ in copies]
            dst = [b + l * n for l in range(self.layers) for _, b in copies]
            copy_pages(self.k_pages.flatten(0, 1), self.v_pages.flatten(0, 1), src, dst)
        lens, cu = [self.book.length(s) for s in seqs], [0]
        for n in new:
            cu.append(cu[-1] + n)
        positions = [p + i for p, n in zip(first, new) for i in range(n)]
        entries, width = self._table_of([self.book.pages(s) for s in seqs])
        table, kv_lens, cu_q, pos = self._on_device(entries, lens, cu, positions)
        return Step(table.view(len(seqs), width), kv_lens, cu_q, pos, cu[-1], max(new, default=0),
                    max(lens, default=0), max(positions, default=-1))

    def append(self, step: Step, layer: int, k: torch.Tensor, v: torch.Tensor, rope: torch.Tensor | None = None,
               interleaved: bool = False, stats: torch.Tensor | None = None) -> None:
        """Encodes the step's keys and values (bf16 [tokens, kv_heads, 128]) into
        the layer's pages.  A rope_table that ends before the step's positions is
        refused (by `rope` it is not: it gets the positions on the device)."""
        if k.shape[0] != step.tokens:
            raise ValueError("k and v must have a row for each new token of the step")
        if rope is not None and step.max_position >= rope.shape[0]:
            raise ValueError(f"position {step.max_position} is past the {rope.shape[0]} of the rope_table")
        paged_append(k, v, self.k_pages[layer], self.v_pages[layer], self.k_tables[layer], self.v_tables[layer],
                     step.page_table, step.kv_lens, step.cu_q, rope=rope,
                     positions=step.positions if rope is not None else None, interleaved=interleaved, stats=stats)

    def attend(self, step: Step, layer: int, q: torch.Tensor, scale: float, window: int = 0,
               out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None) -> torch.Tensor:
        """Attention of the step's tokens (bf16 [tokens, kv_heads * group, 128]) over the layer's pages."""
        if q.shape[0] != step.tokens:
            raise ValueError("q must have a row for each new token of the step")
        return paged_attention(q, self.k_pages[layer], self.v_pages[layer], self.k_tables[layer],
                               self.v_tables[layer], step.page_table, step.kv_lens, step.cu_q, scale,
                               max_q=step.max_q, max_kv=step.max_kv, window=window, out=out, lse=lse,
                               workspace=workspace)

    def compact(self, seqs: list[int], keep: torch.Tensor) -> list[int]:
        """Keeps the tokens of each sequence whose entry of `keep` (bool or uint8
        [len(seqs), at least the longest length]) is not zero, in every layer,
        and frees the pages that are left over.  Takes as many free pages as the
        sequences hold while it runs.  Blocks until the new lengths are known;
        returns them."""
        if len(seqs) > _lib.MAX_BATCH:
            raise ValueError(f"at most {_lib.MAX_BATCH} sequences a call")
        lens, after = [self.book.length(s) for s in seqs], [self._next_position(s) for s in seqs]
        if keep.dim() != 2 or keep.shape[0] != len(seqs) or keep.shape[1] < max(lens, default=0):
            raise ValueError("keep must be [len(seqs), at least the longest length]")
        if not seqs:
            return []
        fresh = self.book.replace(seqs)
        try:
            entries, width = self._table_of([self.book.pages(s) for s in seqs])
            table, dst, kv_lens = self._on_device(entries, self._table_of(fresh)[0], lens)
            table, dst = table.view(len(seqs), width), dst.view(len(seqs), width)
            for layer in range(self.layers):
                new = compact_pages(self.k_pages[layer], self.v_pages[layer], table, kv_lens, keep, dst)
            lengths = new.tolist()
        except BaseException:
            self.book.cancel(fresh)
            raise
        self.book.settle(seqs, fresh, lengths)
        self._base.update(zip(seqs, zip(lengths, after)))
        return lengths
