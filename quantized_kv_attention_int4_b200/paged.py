"""Paged INT4 key-value cache of many requests: ctypes binding of include/flashloop_paged.h
(same names) and ``PagedCache``, the tables, pools and workspace of one model.

Argument marshalling only, as in ``abi``: every wrapper checks placement, dtype, shape and
strides, passes raw device pointers and the current CUDA stream of the tensors' device, and
raises FlashLoopError on a non-OK status.
"""
from __future__ import annotations

import ctypes

import torch

from . import abi
from .abi import FlashLoopError, GROUP_RECORD, HEAD_DIM, lib

PAGE = 64
MAX_BATCH = 8192
MAX_SLOTS = 131072
MAX_BLOCKS = 16384
MAX_KEEP = 16384
WS_HEAD = 8192

# device error codes beside abi's (include/flashloop_paged.h)
(FL_DEV_SLOT_RANGE, FL_DEV_SLOT_TWICE, FL_DEV_NO_PAGE, FL_DEV_TOO_LONG, FL_DEV_COUNT, FL_DEV_PAGE_RANGE,
 FL_DEV_SEL_BLOCK) = range(16, 23)
EXPORTED = ("fl_paged_index_init", "fl_paged_extend", "fl_paged_release", "fl_paged_slot_map", "fl_paged_append",
            "fl_paged_read", "fl_paged_workspace_bytes", "fl_paged_workspace_init", "fl_paged_select",
            "fl_paged_attn_decode")

_P, _I, _L, _Z = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t


class fl_paged_index(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("table", "length", "free_pages", "n_free", "status")] + [
        (n, _I) for n in ("slots", "max_pages", "pages")]


class fl_paged_pool(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("rec", "tail_k", "tail_v")] + [
        (n, _I) for n in ("kv_heads", "head_dim", "page_tokens")]


_XP, _PP = ctypes.POINTER(fl_paged_index), ctypes.POINTER(fl_paged_pool)
_c_index_init = abi._sig("fl_paged_index_init", _I, _XP, _P)
_c_extend = abi._sig("fl_paged_extend", _I, _XP, _I, _P, _P, _P, _P, _P)
_c_release = abi._sig("fl_paged_release", _I, _XP, _I, _P, _P)
_c_slot_map = abi._sig("fl_paged_slot_map", _I, _XP, _I, _P, _P, _P, _I, _P, _P, _P)
_c_append = abi._sig("fl_paged_append", _I, _XP, _PP, _I, _P, _P, _P, _I, _P, _P, _L, _L, _P)
_c_read = abi._sig("fl_paged_read", _I, _XP, _PP, _I, _P, _P, _P, _L, _L, _P)
_c_ws_bytes = abi._sig("fl_paged_workspace_bytes", _Z, _XP, _PP, _I, _I)
_c_ws_init = abi._sig("fl_paged_workspace_init", _I, _P, _Z, _P)
_c_select = abi._sig("fl_paged_select", _I, _XP, _PP, _I, _P, _I, _P, _L, _L, _I, _P, _P, _Z, _P)
_c_attn = abi._sig("fl_paged_attn_decode", _I, _XP, _PP, _I, _P, _I, _P, _L, _L, _P, _I, _P, _L, _L, _P, _P, _Z, _P)


_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _flat(t, dtype, dev, name, numel=-1):
    """Data pointer of a contiguous tensor of `dtype` on device number `dev` (None stays None)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev or dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor on device {dev}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel >= 0 and t.numel() != numel:
        raise ValueError(f"{name} must hold {numel} entries, got {t.numel()}")
    return t.data_ptr()


def _rows(t, dtype, dev, name, heads):
    """(rows, pointer, row stride, head stride) of [n][heads][128] with contiguous channels;
    heads = 0: any number."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev or dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor on device {dev}, got {t.device}")
    shape = t.shape
    if len(shape) != 3 or (heads and shape[1] != heads) or shape[2] != HEAD_DIM:
        raise ValueError(f"{name} must be [n][{heads or 'heads'}][{HEAD_DIM}], got {list(shape)}")
    n, h = shape[0], shape[1]
    rs, hs, cs = t.stride()
    if cs != 1:
        raise ValueError(f"{name} must have contiguous channels")
    return n, t.data_ptr(), rs if n > 1 else h * HEAD_DIM, hs if h > 1 else HEAD_DIM


def _call(where, dev, stream, fn, *args):
    """fn(*args, stream) with device number `dev` current; raises FlashLoopError unless FL_OK."""
    if stream is None:
        stream = _raw_stream(dev)
    elif isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    if _current_device() == dev:
        st = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, stream)
    if st:
        raise FlashLoopError(where, st)


class PagedIndex:
    """Block tables of many requests: ``table`` int32 [slots][max_pages], ``length`` int32
    [slots], ``free_pages`` int32 [pages] (a stack, its top at n_free - 1), ``n_free`` int32
    [1], ``status`` int32 [3] or None.  The tensors stay the caller's."""

    def __init__(self, table, length, free_pages, n_free, status=None):
        if not isinstance(table, torch.Tensor) or table.dim() != 2:
            raise ValueError("table must be [slots][max_pages]")
        self.device, self.dev = table.device, table.get_device()
        i32, dev = torch.int32, self.dev
        self.slots, self.max_pages, self.pages = table.shape[0], table.shape[1], free_pages.numel()
        self.table, self.length, self.free_pages, self.n_free, self.status = table, length, free_pages, n_free, status
        self.c = fl_paged_index(
            _flat(table, i32, dev, "table"), _flat(length, i32, dev, "length", self.slots),
            _flat(free_pages, i32, dev, "free_pages"), _flat(n_free, i32, dev, "n_free", 1),
            _flat(status, i32, dev, "status", 3), self.slots, self.max_pages, self.pages)
        self.ref = ctypes.byref(self.c)

    @classmethod
    def empty(cls, slots: int, max_pages: int, pages: int, device="cuda", stream=None):
        """An index of `slots` empty requests of up to 64 max_pages tokens over `pages` free pages."""
        new = lambda *shape: torch.empty(shape, dtype=torch.int32, device=device)  # noqa: E731
        x = cls(new(slots, max_pages), new(slots), new(pages), new(1), new(3))
        fl_paged_index_init(x, stream)
        return x


class PagedPool:
    """One layer's keys and values: ``rec`` uint8 [pages][kv_heads][9216], ``tail_k`` and
    ``tail_v`` BF16 [slots][kv_heads][64][128].  The tensors stay the caller's."""

    def __init__(self, rec, tail_k, tail_v):
        if not isinstance(rec, torch.Tensor) or rec.dim() != 3 or rec.shape[2] != GROUP_RECORD:
            raise ValueError(f"rec must be [pages][kv_heads][{GROUP_RECORD}]")
        self.device, self.dev = rec.device, rec.get_device()
        self.pages, self.kv_heads = rec.shape[0], rec.shape[1]
        for t, name in ((tail_k, "tail_k"), (tail_v, "tail_v")):
            if not isinstance(t, torch.Tensor) or t.dim() != 4 or tuple(t.shape[1:]) != (self.kv_heads, PAGE, HEAD_DIM):
                raise ValueError(f"{name} must be [slots][{self.kv_heads}][{PAGE}][{HEAD_DIM}]")
        if tail_k.shape != tail_v.shape:
            raise ValueError("tail_k and tail_v must have the same shape")
        self.slots = tail_k.shape[0]
        self.rec, self.tail_k, self.tail_v = rec, tail_k, tail_v
        bf16, dev = torch.bfloat16, self.dev
        self.c = fl_paged_pool(
            _flat(rec, torch.uint8, dev, "rec"), _flat(tail_k, bf16, dev, "tail_k"),
            _flat(tail_v, bf16, dev, "tail_v"), self.kv_heads, HEAD_DIM, PAGE)
        self.ref = ctypes.byref(self.c)

    @classmethod
    def empty(cls, index: PagedIndex, kv_heads: int):
        """An uninitialised pool for `index` (a token's bytes are written before they are read)."""
        tails = lambda: torch.empty(index.slots, kv_heads, PAGE, HEAD_DIM, dtype=torch.bfloat16,  # noqa: E731
                                    device=index.device)
        return cls(torch.empty(index.pages, kv_heads, GROUP_RECORD, dtype=torch.uint8, device=index.device), tails(),
                   tails())


def _fit(index, pool):
    if pool.pages < index.pages or pool.slots < index.slots:
        raise ValueError("the pool must hold the index's pages and slots")
    if pool.dev != index.dev:
        raise ValueError("index and pool must be on one device")


def _named(index, slots, batch=None):
    """(batch, pointer) of the named slots; None names rows 0 .. batch - 1 (all by default)."""
    if slots is None:
        return index.slots if batch is None else batch, None
    p = _flat(slots, torch.int32, index.dev, "slots")
    n = slots.numel()
    if batch is not None and n != batch:
        raise ValueError(f"slots must hold one entry per batch row ({batch}), got {n}")
    return n, p


def fl_paged_index_init(index, stream=None):
    _call("fl_paged_index_init", index.dev, stream, _c_index_init, index.ref)


def fl_paged_extend(index, slots, n_new, start, cu, stream=None):
    """Lengths += n_new (int32 [batch]); start (int32 [batch]) and cu (int32 [batch + 1]) are
    written: where the new tokens begin (-1: padded or refused) and their input rows."""
    dev, i32 = index.dev, torch.int32
    np = _flat(n_new, i32, dev, "n_new")
    n, sp = _named(index, slots, n_new.numel())
    _call("fl_paged_extend", dev, stream, _c_extend, index.ref, n, sp, np, _flat(start, i32, dev, "start", n),
          _flat(cu, i32, dev, "cu", n + 1))


def fl_paged_release(index, slots, stream=None):
    n, sp = _named(index, slots)
    _call("fl_paged_release", index.dev, stream, _c_release, index.ref, n, sp)


def fl_paged_slot_map(index, slots, start, cu, place, pos, stream=None):
    """Place and position (int32 [n_tokens], either may be None) of tokens start[i] .. of the
    entries' rows cu[i] .. cu[i + 1] - 1."""
    dev, i32 = index.dev, torch.int32
    tp = _flat(start, i32, dev, "start")
    n, sp = _named(index, slots, start.numel())
    out = place if place is not None else pos
    t = 0 if out is None else out.numel()
    _call("fl_paged_slot_map", dev, stream, _c_slot_map, index.ref, n, sp, tp, _flat(cu, i32, dev, "cu", n + 1), t,
          _flat(place, i32, dev, "place", t), _flat(pos, i32, dev, "pos", t))


def _pair(k, v, dev, heads):
    """(rows, k, v, row stride, head stride) of keys and values that are laid out alike."""
    n, kp, ts, hs = _rows(k, torch.bfloat16, dev, "k", heads)
    m, vp, vts, vhs = _rows(v, torch.bfloat16, dev, "v", heads)
    if n != m or ts != vts or hs != vhs:
        raise ValueError("k and v must have the same shape and strides")
    return n, kp, vp, ts, hs


def fl_paged_append(index, pool, slots, start, cu, k, v, stream=None):
    """k, v: BF16 [n_tokens][kv_heads][128] (contiguous channels, the same strides): rows
    cu[i] .. cu[i + 1] - 1 are tokens start[i] .. of request i (fl_paged_extend's)."""
    _fit(index, pool)
    dev, i32 = index.dev, torch.int32
    tp = _flat(start, i32, dev, "start")
    n, sp = _named(index, slots, start.numel())
    rows, kp, vp, ts, hs = _pair(k, v, dev, pool.kv_heads)
    _call("fl_paged_append", dev, stream, _c_append, index.ref, pool.ref, n, sp, tp, _flat(cu, i32, dev, "cu", n + 1),
          rows, kp, vp, ts, hs)


def fl_paged_read(index, pool, place, k, v, stream=None):
    """k, v: BF16 [n_tokens][kv_heads][128], row t receives the token at place[t] (int32; -1:
    left as it was)."""
    _fit(index, pool)
    dev = index.dev
    rows, kp, vp, ts, hs = _pair(k, v, dev, pool.kv_heads)
    _call("fl_paged_read", dev, stream, _c_read, index.ref, pool.ref, rows, _flat(place, torch.int32, dev, "place", rows),
          kp, vp, ts, hs)


def fl_paged_workspace_bytes(index, pool, batch: int, q_heads: int) -> int:
    return int(_c_ws_bytes(index.ref, pool.ref, batch, q_heads))


def fl_paged_workspace_init(ws, stream=None):
    dev = ws.get_device()
    _call("fl_paged_workspace_init", dev, stream, _c_ws_init, _flat(ws, torch.uint8, dev, "ws"), ws.numel())


def workspace(index, pool, batch: int, q_heads: int, stream=None) -> torch.Tensor:
    """An initialised workspace of fl_paged_select and fl_paged_attn_decode for up to `batch`
    entries and `q_heads` query heads."""
    _fit(index, pool)
    n = fl_paged_workspace_bytes(index, pool, batch, q_heads)
    if n == 0:
        raise FlashLoopError("fl_paged_workspace_bytes", abi.FL_ERR_INVALID)
    ws = torch.empty(n, dtype=torch.uint8, device=index.device)
    fl_paged_workspace_init(ws, stream)
    return ws


def _selection(sel, dev, n, kv_heads):
    """(keep, pointer) of a selection [n][kv_heads][keep]."""
    p = _flat(sel, torch.int32, dev, "sel")
    if sel.dim() != 3 or sel.shape[0] != n or sel.shape[1] != kv_heads:
        raise ValueError(f"sel must be [{n}][{kv_heads}][keep]")
    return sel.shape[2], p


def fl_paged_select(index, pool, slots, q, sel, ws, stream=None):
    """q: BF16 [batch][q_heads][128]; sel: int32 [batch][kv_heads][keep] receives the blocks of
    the highest score, ascending, -1 behind the last."""
    _fit(index, pool)
    dev = index.dev
    n, qp, qb, qh = _rows(q, torch.bfloat16, dev, "q", 0)
    _, sp = _named(index, slots, n)
    keep, selp = _selection(sel, dev, n, pool.kv_heads)
    _call("fl_paged_select", dev, stream, _c_select, index.ref, pool.ref, n, sp, q.shape[1], qp, qb, qh, keep, selp,
          _flat(ws, torch.uint8, dev, "ws"), ws.numel())


def fl_paged_attn_decode(index, pool, slots, q, o, ws, lse=None, sel=None, stream=None):
    """o (fp32 [batch][q_heads][128]) = attention of q (BF16, same shape) over each request's
    cache, or over the blocks of sel (int32 [batch][kv_heads][keep]) and the tail; lse: None or
    fp32 [batch][q_heads] (base 2)."""
    _fit(index, pool)
    dev = index.dev
    n, qp, qb, qh = _rows(q, torch.bfloat16, dev, "q", 0)
    heads = q.shape[1]
    m, op, ob, oh = _rows(o, torch.float32, dev, "o", heads)
    if m != n:
        raise ValueError("o must have q's shape")
    _, sp = _named(index, slots, n)
    keep, selp = (0, None) if sel is None else _selection(sel, dev, n, pool.kv_heads)
    _call("fl_paged_attn_decode", dev, stream, _c_attn, index.ref, pool.ref, n, sp, heads, qp, qb, qh, selp, keep, op, ob,
          oh, _flat(lse, torch.float32, dev, "lse", n * heads), _flat(ws, torch.uint8, dev, "ws"), ws.numel())


class PagedCache:
    """One index, a pool per plane (a layer, or a (layer, loop) of a looped model) and a
    workspace; every call works on the current stream.

    ``slots`` requests of up to ``max_tokens`` tokens share ``pages`` pages of 64 tokens;
    calls take up to ``max_batch`` entries and ``q_heads`` query heads."""

    def __init__(self, planes: int, kv_heads: int, slots: int, max_tokens: int, pages: int, q_heads: int | None = None,
                 max_batch: int | None = None, device="cuda"):
        self.kv_heads, self.q_heads = kv_heads, q_heads or kv_heads
        if self.q_heads % kv_heads:
            raise ValueError("q_heads must be a multiple of kv_heads")
        if torch.device(device).index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        self.index = PagedIndex.empty(slots, -(-max_tokens // PAGE), pages, device)
        self.pools = [PagedPool.empty(self.index, kv_heads) for _ in range(planes)]
        self.max_batch = max_batch or min(slots, MAX_BATCH)
        self.ws = workspace(self.index, self.pools[0], self.max_batch, self.q_heads)
        self.device = self.index.device

    def extend(self, slots, n_new):
        """(start, cu) of the step's new tokens; takes pages (fl_paged_extend)."""
        n = n_new.numel()
        start = torch.empty(n, dtype=torch.int32, device=self.device)
        cu = torch.empty(n + 1, dtype=torch.int32, device=self.device)
        fl_paged_extend(self.index, slots, n_new, start, cu)
        return start, cu

    def places(self, slots, start, cu, n_tokens: int):
        """(place, pos) of the tokens start[i] .. in rows cu[i] ..; -1 behind the last row."""
        place = torch.full((n_tokens,), -1, dtype=torch.int32, device=self.device)
        pos = torch.full((n_tokens,), -1, dtype=torch.int32, device=self.device)
        fl_paged_slot_map(self.index, slots, start, cu, place, pos)
        return place, pos

    def append(self, plane: int, slots, start, cu, k, v):
        fl_paged_append(self.index, self.pools[plane], slots, start, cu, k, v)

    def read(self, plane: int, place):
        """BF16 (k, v) [len(place)][kv_heads][128] of the tokens at `place` (zero where -1)."""
        shape = (place.numel(), self.kv_heads, HEAD_DIM)
        k = torch.zeros(shape, dtype=torch.bfloat16, device=self.device)
        v = torch.zeros(shape, dtype=torch.bfloat16, device=self.device)
        fl_paged_read(self.index, self.pools[plane], place, k, v)
        return k, v

    def select(self, plane: int, slots, q, keep: int):
        """int32 [batch][kv_heads][keep] blocks of the highest score (-1: none)."""
        sel = torch.full((q.shape[0], self.kv_heads, keep), -1, dtype=torch.int32, device=self.device)
        fl_paged_select(self.index, self.pools[plane], slots, q, sel, self.ws)
        return sel

    def attend(self, plane: int, slots, q, o=None, lse=None, keep: int | None = None):
        """Attention of q over each request's cache, or over its `keep` best blocks and tail."""
        if o is None:
            o = torch.zeros(q.shape, dtype=torch.float32, device=self.device)
        sel = None if keep is None else self.select(plane, slots, q, keep)
        fl_paged_attn_decode(self.index, self.pools[plane], slots, q, o, self.ws, lse=lse, sel=sel)
        return o

    def release(self, slots):
        fl_paged_release(self.index, slots)

    def status(self, clear: bool = True):
        """[first error code, detail, count]; synchronises the device."""
        out = self.index.status.tolist()
        if clear:
            self.index.status.zero_()
        return out
