"""Serving operators of libattn: rotary positions, the paged key/value cache, and exact
attention of new (drafted) tokens over it.

Argument marshalling only, as in the package's other entry points: every step runs in the
CUDA library through the C ABI of ``include/attn_cache.h``.

One step of speculative decoding, for sequences ``slots`` whose drafted trees are packed by
``cu_q``::

    cache.alloc(slots, lens_with_drafts)                      # pages for the drafted tokens
    q = rope_append(cache, q, k, v, cu_q, plan=rope, positions=depths, slots=slots)
    o, lse = tree_fwd(cache, q, cu_q, mask=tree, slots=slots)
    cache.compact(cu_q, path, accepted, slots=slots)          # what verification kept

With one token per sequence and no mask this is ordinary decoding.
"""
from __future__ import annotations

import ctypes
import math
import struct
from typing import Optional, Tuple

import torch

_lib_of = None  # set by the package: loads the library
_check = None   # set by the package: raises AttnError

_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


class RopePlan(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("dim", ctypes.c_int),
                ("interleaved", ctypes.c_int), ("amplitude", ctypes.c_float)]


class Rows(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("heads", ctypes.c_int),
                ("src_batch", ctypes.c_int64), ("src_token", ctypes.c_int64),
                ("src_head", ctypes.c_int64), ("dst_batch", ctypes.c_int64),
                ("dst_token", ctypes.c_int64), ("dst_head", ctypes.c_int64)]


class CacheView(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("lens", ctypes.c_void_p), ("refs", ctypes.c_void_p), ("layers", ctypes.c_int),
                ("pages", ctypes.c_int), ("page_size", ctypes.c_int), ("heads", ctypes.c_int),
                ("d", ctypes.c_int), ("slots", ctypes.c_int), ("max_pages", ctypes.c_int),
                ("e4m3", ctypes.c_int), ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


# `Rows` structs, passed as bytes written in one step: two addresses, the heads, six strides.
_one_row = "PPi4x6q"
assert struct.calcsize(_one_row) == ctypes.sizeof(Rows)
_row, _two_rows = struct.Struct(_one_row).pack, struct.Struct(2 * _one_row).pack
_no_row = (0, 0, 0, 0, 0, 0, 0, 0, 0)
_Tensor, _int32, _bf16 = torch.Tensor, torch.int32, torch.bfloat16


def declare(lib) -> None:
    """Argument types of the entry points of include/attn_cache.h."""
    vp, ci, cf, cs = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    for name, args in {
            "attn_rope": [vp, ci, ci, vp, ci, ci, ci, ci, vp, vp, vp],
            "attn_rope_append": [vp, ci, vp, vp, vp, vp, ci, ci, vp, vp, vp, vp],
            "attn_cache_alloc": [vp, vp, vp, ci, vp, vp],
            "attn_cache_free": [vp, vp, ci, vp],
            "attn_cache_fork": [vp, vp, vp, ci, vp, vp, cs, vp],
            "attn_cache_copy": [vp, vp, vp, ci, vp],
            "attn_cache_compact": [vp, vp, vp, ci, vp, vp, ci, vp],
            "attn_tree_fwd": [vp, ci, vp, vp, vp, ci, ci, ci, vp, vp, vp, ci, cf, vp, cs, vp],
    }.items():
        f = getattr(lib, name)
        f.argtypes, f.restype = args, ci
    lib.attn_cache_fork_workspace_size.argtypes = [ci]
    lib.attn_cache_fork_workspace_size.restype = cs
    lib.attn_tree_workspace_size.argtypes = [ci]
    lib.attn_tree_workspace_size.restype = cs


_current_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _stream(dev: torch.device, stream: Optional[torch.cuda.Stream]) -> int:
    """The raw stream of a call."""
    return _current_stream(dev.index) if stream is None else stream.cuda_stream


def made_for(stream: Optional[torch.cuda.Stream], make, *args, **kw) -> torch.Tensor:
    """A tensor that a call on `stream` (None: the current one) writes first.  Its memory is that
    stream's: a block of the caller's stream may still be in use there by work queued before.  It is kept
    for the caller's stream too, where the result is read when that stream has waited for the other."""
    if stream is None:
        return make(*args, **kw)
    caller = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        t = make(*args, **kw)
    if caller != stream:
        t.record_stream(caller)
    return t


def _like(stream: Optional[torch.cuda.Stream], x: torch.Tensor) -> torch.Tensor:
    if stream is None:
        return torch.empty_like(x, memory_format=torch.contiguous_format)
    return made_for(stream, torch.empty_like, x, memory_format=torch.contiguous_format)


def _on(dev: torch.device, f, *args) -> None:
    """Calls the library with `dev` current; raises on an error status."""
    if _current_device() == dev.index:
        st = f(*args)
    else:
        with torch.cuda.device(dev):
            st = f(*args)
    if st:
        _check(st)


def _list(t, name: str, dev: torch.device, n: Optional[int] = None) -> int:
    """The address of a contiguous int32 list on `dev`."""
    if not isinstance(t, _Tensor) or t.dtype is not _int32:
        raise ValueError(f"{name} must be an int32 tensor")
    if t.get_device() != dev.index:
        raise ValueError(f"{name} must be on {dev}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if n is not None and t.numel() != n:
        raise ValueError(f"{name} must hold {n} values")
    return t.data_ptr()


def _cuda(t, name: str):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")


def _used(shape, b: int, n: int, h: int):
    """The strides of batch, token and head.  That of a dimension of one element is never used, and may be
    anything: it is left out, so that the library's check of the others' alignment holds."""
    return b if shape[0] > 1 else 0, n if shape[-3] > 1 else 0, h if shape[-2] > 1 else 0


def _rows(x, y, name: str, dtype, dev: torch.device, shape, batch: bool):
    """One entry of the library's row descriptions, checked: tensor, result (None: it has
    none), heads and the six strides of [*lead, H, d] with contiguous heads."""
    if x.dtype is not dtype or x.get_device() != dev.index:
        raise ValueError(f"{name} must be {dtype} on {dev}")
    sx = x.stride()
    if sx[-1] != 1 and x.numel():
        raise ValueError(f"the values of a head of {name} must be contiguous")
    bx, tx, hx = sx[0] if batch else 0, sx[-3], sx[-2]
    if (bx | tx | hx) & 7:
        bx, tx, hx = _used(shape, bx, tx, hx)
    if y is None:
        return x.data_ptr(), 0, shape[-2], bx, tx, hx, bx, tx, hx
    if y is x:
        at = x.data_ptr()
        return at, at, shape[-2], bx, tx, hx, bx, tx, hx
    if y.dtype is not dtype or y.get_device() != dev.index:
        raise ValueError(f"out of {name} must be {dtype} on {dev}")
    if y.shape != shape:
        raise ValueError(f"out of {name} has the wrong shape")
    sy = y.stride()
    if sy[-1] != 1 and y.numel():
        raise ValueError(f"the values of a head of out of {name} must be contiguous")
    by, ty, hy = sy[0] if batch else 0, sy[-3], sy[-2]
    if (by | ty | hy) & 7:
        by, ty, hy = _used(shape, by, ty, hy)
    return x.data_ptr(), y.data_ptr(), shape[-2], bx, tx, hx, by, ty, hy


class Rope:
    """Rotary positions of one kind: which values of a head turn, and how fast.

    Pair i of the first ``dim`` values turns by ``position * base**(-2i/dim)``.  The pairs
    are values (i, i + dim/2), or (2i, 2i+1) with ``interleaved``.  ``scaling`` stretches
    them for contexts ``factor`` times longer than those of training:

    * ``"linear"``: every frequency divided by ``factor`` (position interpolation);
    * ``"ntk"``: ``base`` multiplied by ``factor**(dim/(dim-2))``;
    * ``"yarn"``: frequencies that turn more than ``beta_fast`` times over the
      ``original_len`` tokens of training stay, those below ``beta_slow`` turns are divided
      by ``factor``, with a linear ramp over the index between; the rotated values are
      multiplied by ``1 + 0.1 ln(factor)``.

    ``amplitude`` overrides that multiplier (1 for the other kinds).  The frequencies are
    kept on ``device`` as exact 64-bit fractions of a turn, so positions may be any int32.
    """

    def __init__(self, dim: int, base: float = 10000.0, interleaved: bool = False,
                 scaling: Optional[str] = None, factor: float = 1.0,
                 original_len: Optional[int] = None, beta_fast: float = 32.0,
                 beta_slow: float = 1.0, amplitude: Optional[float] = None, device="cuda"):
        if dim <= 0 or dim % 16:
            raise ValueError("dim must be a positive multiple of 16")
        if not (math.isfinite(base) and base > 1.0):
            raise ValueError("base must be finite and > 1")
        if not (math.isfinite(factor) and factor >= 1.0):
            raise ValueError("factor must be finite and >= 1")
        if scaling not in (None, "linear", "ntk", "yarn"):
            raise ValueError("scaling must be None, 'linear', 'ntk' or 'yarn'")
        self.dim, self.interleaved = dim, bool(interleaved)
        amp = 1.0
        if scaling == "ntk":
            base = base * factor ** (dim / (dim - 2))
        freqs = [base ** (-2.0 * i / dim) for i in range(dim // 2)]
        if scaling == "linear":
            freqs = [f / factor for f in freqs]
        if scaling == "yarn":
            if original_len is None or original_len <= 0 or not beta_fast > beta_slow > 0:
                raise ValueError("yarn needs original_len > 0 and beta_fast > beta_slow > 0")

            def index(turns):
                return dim * math.log(original_len / (turns * 2 * math.pi)) / (2 * math.log(base))
            lo = max(math.floor(index(beta_fast)), 0)
            hi = min(math.ceil(index(beta_slow)), dim - 1)  # may lie behind the last pair
            for i, f in enumerate(freqs):
                ramp = min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
                freqs[i] = f * (1 - ramp) + f / factor * ramp
            amp = 0.1 * math.log(factor) + 1.0
        self.amplitude = amp if amplitude is None else float(amplitude)
        if not (math.isfinite(self.amplitude) and self.amplitude > 0):
            raise ValueError("amplitude must be finite and > 0")
        # f < 1, so a fraction of a turn is below 2^62 and fits int64
        self.turns = torch.tensor([round(f / (2 * math.pi) * 2.0 ** 64) for f in freqs],
                                  dtype=torch.int64).to(device)
        self._view = RopePlan(self.turns.data_ptr(), dim, int(self.interleaved), self.amplitude)
        self._ref = ctypes.byref(self._view)


def _rope(plan: Rope, inverse: int, q, k, positions, cu_seqlens, out, stream):
    lib = _lib_of()
    _cuda(q, "q")
    dev, dtype, shape = q.device, q.dtype, q.shape
    kind = _TYPES.get(dtype)
    if kind is None:
        raise ValueError("q must be bfloat16, float16 or float32")
    if plan.turns.device != dev:
        raise ValueError(f"the plan must be on {dev}")
    packed = cu_seqlens is not None
    if len(shape) != (3 if packed else 4):
        raise ValueError("packed q must be [T, H, d]" if packed else "dense q must be [B, N, H, d]")
    if k is not None:
        _cuda(k, "k")
        k_shape = k.shape
        if len(k_shape) != len(shape) or k_shape[:-2] != shape[:-2] or k_shape[-1] != shape[-1]:
            raise ValueError("q and k must hold the same tokens and head dim")
    if out is None:
        q_out = _like(stream, q)
        k_out = None if k is None else _like(stream, k)
    else:
        q_out, k_out = (out, None) if isinstance(out, torch.Tensor) else out
        _cuda(q_out, "out of q")
        if k is not None:
            _cuda(k_out, "out of k")
    batch = not packed
    rows = _two_rows(*_rows(q, q_out, "q", dtype, dev, shape, batch),
                     *(_no_row if k is None else _rows(k, k_out, "k", dtype, dev, k_shape, batch)))
    if packed:
        cu = _list(cu_seqlens, "cu_seqlens", dev)
        B, tokens = cu_seqlens.numel() - 1, shape[0]
        N = tokens
    else:
        cu, B, N = None, shape[0], shape[1]
        tokens = B * N
    pos = None if positions is None else _list(positions, "positions", dev, tokens)
    _on(dev, lib.attn_rope, plan._ref, inverse, kind, rows, 1 if k is None else 2, shape[-1], B, N,
        cu, pos, _stream(dev, stream))
    return q_out if k is None else (q_out, k_out)


def rope_fwd(plan: Rope, q: torch.Tensor, k: Optional[torch.Tensor] = None,
             positions: Optional[torch.Tensor] = None,
             cu_seqlens: Optional[torch.Tensor] = None, out=None,
             stream: Optional[torch.cuda.Stream] = None):
    """Rotates q, and k with it, by their tokens' positions, in one launch.

    Dense ``[B, N, H, d]`` or, with ``cu_seqlens`` (int32 ``[B+1]``), packed ``[T, H, d]``;
    bf16, fp16 or fp32.  Token and head strides may be anything that keeps rows 16-byte
    aligned (slices of a joint projection); the head counts of q and k may differ.
    ``positions`` is int32, one per token (default: its index in its sequence; packed rows
    that belong to no sequence are then left unwritten).  ``out=(q_out, k_out)`` receives the
    results; the inputs themselves are allowed (in place).  Returns (q', k'), or q' alone
    without k."""
    return _rope(plan, 0, q, k, positions, cu_seqlens, out, stream)


def rope_bwd(plan: Rope, dq: torch.Tensor, dk: Optional[torch.Tensor] = None,
             positions: Optional[torch.Tensor] = None,
             cu_seqlens: Optional[torch.Tensor] = None, out=None,
             stream: Optional[torch.cuda.Stream] = None):
    """The gradients of ``rope_fwd`` with respect to its q and k, from those of its results:
    the rotation by the negative angles.  Arguments as there."""
    return _rope(plan, 1, dq, dk, positions, cu_seqlens, out, stream)


class KVCache:
    """A paged key/value cache on one GPU.

    ``k``, ``v``: ``[layers, pages, page_size, heads, d]`` (a 4-D tensor is one layer), bf16, or
    float8_e4m3fn holding the real values divided by ``k_scale`` / ``v_scale``.
    ``page_table``: int32 ``[slots, max_pages]``; ``lens``: int32 ``[slots]``, the tokens of each
    slot; ``refs``: int32 ``[pages]``, how many slots hold a page (0: free).  All contiguous, on
    one device; the cache works on these tensors and keeps nothing else.  Page sizes are
    powers of two from 16 to 1024, d is 64 or 128.

    The methods change the state on the device and synchronise nothing.  What only the
    device sees (a bad slot or page number, an inconsistent length) leaves that
    sequence alone and is reported by ``get_device_status``.  Calls that change
    one cache must be ordered, e.g. issued on one stream."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor,
                 lens: torch.Tensor, refs: torch.Tensor, k_scale: float = 1.0,
                 v_scale: float = 1.0):
        for t, name in ((k, "k"), (v, "v")):
            _cuda(t, name)
            if t.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
                raise ValueError(f"{name} must be bfloat16 or float8_e4m3fn")
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
        if k.shape != v.shape or k.dtype != v.dtype or k.device != v.device:
            raise ValueError("k and v must share shape, type and device")
        if k.dim() not in (4, 5):
            raise ValueError("k must be [layers, pages, page_size, heads, d]")
        layers, pages, page_size, heads, d = (1, *k.shape) if k.dim() == 4 else k.shape
        dev = k.device
        if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
            raise ValueError("page_table must be [slots, max_pages]")
        slots, max_pages = page_table.shape
        e4m3 = k.dtype == torch.float8_e4m3fn
        if not e4m3 and (k_scale != 1.0 or v_scale != 1.0):
            raise ValueError("scales belong to an E4M3 cache")
        self._k, self._v, self._table, self._lens, self._refs = k, v, page_table, lens, refs
        self.device, self.dtype, self.d, self.heads = dev, k.dtype, d, heads
        self.layers, self.pages, self.page_size = layers, pages, page_size
        self.slots, self.max_pages = slots, max_pages
        self.k_scale, self.v_scale = float(k_scale), float(v_scale)
        self._view = CacheView(k.data_ptr(), v.data_ptr(), _list(page_table, "page_table", dev),
                               _list(lens, "lens", dev, slots), _list(refs, "refs", dev, pages),
                               layers, pages, page_size, heads, d, slots, max_pages, int(e4m3),
                               self.k_scale, self.v_scale)
        self._ref = ctypes.byref(self._view)
        self._ws = max(_lib_of().attn_tree_workspace_size(d), 256)

    @classmethod
    def empty(cls, layers: int, pages: int, page_size: int, heads: int, d: int, slots: int,
              max_pages: int, dtype=torch.bfloat16, device="cuda", k_scale: float = 1.0,
              v_scale: float = 1.0) -> "KVCache":
        """A cache with every page free and every slot empty."""
        shape = (layers, pages, page_size, heads, d)
        i32 = dict(dtype=torch.int32, device=device)
        return cls(torch.empty(shape, dtype=dtype, device=device),
                   torch.empty(shape, dtype=dtype, device=device),
                   torch.full((slots, max_pages), -1, **i32), torch.zeros(slots, **i32),
                   torch.zeros(pages, **i32), k_scale, v_scale)

    # The tensors are fixed for the cache's life: the library is given their addresses.
    k = property(lambda self: self._k)
    v = property(lambda self: self._v)
    page_table = property(lambda self: self._table)
    lens = property(lambda self: self._lens)
    refs = property(lambda self: self._refs)

    def alloc(self, slots: torch.Tensor, new_lens: torch.Tensor,
              stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """Grows slot ``slots[i]`` to ``new_lens[i]`` tokens.  Pages are handed out in order
        of i, lowest number first; returns int32 ``granted[i]``: 1 iff request i needs no page
        or requests 0..i need no more than are free.  One not granted changes nothing.  A slot that
        grows inside a page which another slot holds too (``compact`` may leave one) gets a page of its
        own in its place, its tokens copied."""
        lib, dev, n = _lib_of(), self.device, slots.numel()
        granted = made_for(stream, torch.empty, n, dtype=torch.int32, device=dev)
        _on(dev, lib.attn_cache_alloc, self._ref, _list(slots, "slots", dev),
            _list(new_lens, "new_lens", dev, n), n, granted.data_ptr(),
            _stream(dev, stream))
        return granted

    def free(self, slots: torch.Tensor, stream: Optional[torch.cuda.Stream] = None) -> None:
        """Empties the slots; pages that no other slot holds become free."""
        dev = self.device
        _on(dev, _lib_of().attn_cache_free, self._ref, _list(slots, "slots", dev), slots.numel(),
            _stream(dev, stream))

    def fork(self, src: torch.Tensor, dst: torch.Tensor,
             stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """Forks slot ``src[i]`` into the empty slot ``dst[i]``: full pages are shared, the
        tokens of a last page that is not full are copied to a new one, in every layer.
        Returns ``granted`` as ``alloc`` does."""
        lib, dev, n = _lib_of(), self.device, src.numel()
        granted = made_for(stream, torch.empty, n, dtype=torch.int32, device=dev)
        ws = made_for(stream, torch.empty, max(lib.attn_cache_fork_workspace_size(n), 16),
                      dtype=torch.uint8, device=dev)
        _on(dev, lib.attn_cache_fork, self._ref, _list(src, "src", dev),
            _list(dst, "dst", dev, n), n, granted.data_ptr(), ws.data_ptr(), ws.numel(),
            _stream(dev, stream))
        return granted

    def copy(self, src: torch.Tensor, dst: torch.Tensor,
             stream: Optional[torch.cuda.Stream] = None) -> None:
        """Copies page ``src[i]`` to page ``dst[i]`` in every layer (the tables stay as they
        are).  Of a destination named twice the last copy counts; a source that is also a
        destination is refused."""
        dev, n = self.device, src.numel()
        _on(dev, _lib_of().attn_cache_copy, self._ref, _list(src, "src", dev),
            _list(dst, "dst", dev, n), n, _stream(dev, stream))

    def compact(self, cu_q: torch.Tensor, path: torch.Tensor, accepted: torch.Tensor,
                slots: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None) -> None:
        """Keeps the accepted path of each sequence's drafted tokens (its last ``cu_q[b+1] -
        cu_q[b]`` tokens): ``path[b, :accepted[b]]``, strictly increasing, names which of them
        stay; they move together behind the context in every layer, and surplus pages are
        released.  ``path`` is int32 ``[B, width]``; ``slots`` defaults to 0..B-1."""
        dev, B = self.device, cu_q.numel() - 1
        if path.dim() != 2 or path.shape[0] != B:
            raise ValueError("path must be [B, width]")
        _on(dev, _lib_of().attn_cache_compact, self._ref, _list(cu_q, "cu_q", dev),
            _list(path, "path", dev), path.shape[1], _list(accepted, "accepted", dev, B),
            None if slots is None else _list(slots, "slots", dev, B), B, _stream(dev, stream))


def rope_append(cache: KVCache, q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor,
                cu_q: torch.Tensor, plan: Optional[Rope] = None,
                positions: Optional[torch.Tensor] = None, slots: Optional[torch.Tensor] = None,
                layer: int = 0, out: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None) -> Optional[torch.Tensor]:
    """Writes new tokens into a layer of the cache and rotates their queries, in one launch.

    q ``[T, Hq, d]`` and k, v ``[T, heads, d]`` (bf16; strides as in ``rope_fwd``) are packed by
    ``cu_q`` (int32 ``[B+1]``); sequence b is slot ``slots[b]`` (default b), and its tokens are the
    last ones of that slot: ``alloc`` first.  q and k turn by ``plan`` (None: not at all) at
    ``positions`` (int32 ``[T]``; default: the token's place in the cache).  Returns the rotated q
    (``out``; q itself is allowed), or None without q."""
    lib = _lib_of()
    dev = cache.device
    _cuda(k, "k")
    _cuda(v, "v")
    T, _, d = shape = k.shape if k.dim() == 3 else (0, 0, 0)
    if d != cache.d or v.shape != shape:
        raise ValueError(f"k and v must be [T, heads, {cache.d}]")
    q_row = None
    if q is not None:
        _cuda(q, "q")
        q_shape = q.shape
        if len(q_shape) != 3 or q_shape[0] != T or q_shape[2] != d:
            raise ValueError(f"q must be [T, Hq, {cache.d}]")
        if out is None:
            out = _like(stream, q)
        else:
            _cuda(out, "out")
        q_row = _row(*_rows(q, out, "q", _bf16, dev, q_shape, False))
    k_row = _row(*_rows(k, None, "k", _bf16, dev, shape, False))
    v_row = _row(*_rows(v, None, "v", _bf16, dev, shape, False))
    if plan is not None and plan.turns.device != dev:
        raise ValueError(f"the plan must be on {dev}")
    cu = _list(cu_q, "cu_q", dev)
    B = cu_q.numel() - 1
    _on(dev, lib.attn_rope_append, cache._ref, layer, None if plan is None else plan._ref,
        q_row, k_row, v_row, B, T, cu,
        None if slots is None else _list(slots, "slots", dev, B),
        None if positions is None else _list(positions, "positions", dev, T),
        _stream(dev, stream))
    return None if q is None else out


def tree_fwd(cache: KVCache, q: torch.Tensor, cu_q: torch.Tensor,
             mask: Optional[torch.Tensor] = None, slots: Optional[torch.Tensor] = None,
             layer: int = 0, scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
             lse: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None
             ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Exact attention of each sequence's newest tokens over its slot of the cache.

    q ``[T, Hq, d]`` (bf16, contiguous, rotated) is packed by ``cu_q`` (int32 ``[B+1]``); the
    tokens of sequence b are the last ones of slot ``slots[b]`` (default b), already in the cache.
    Query heads share the cache's heads in groups of ``Hq / heads``.  Every token sees the
    context before them; among them, token t sees token j iff ``mask[t, j]`` (bool or uint8
    ``[T, width]``, j within the sequence, at most 256 drafted tokens each), or iff j <= t
    without a mask.  Returns (O ``[T, Hq, d]`` bf16, LSE ``[Hq, T]`` fp32, natural log); a token
    that sees nothing gets 0 and -inf.  The workspace is allocated with torch."""
    lib = _lib_of()
    dev, d = cache.device, cache.d
    _cuda(q, "q")
    if q.dtype is not _bf16 or q.get_device() != dev.index or not q.is_contiguous():
        raise ValueError(f"q must be a contiguous bfloat16 tensor on {dev}")
    shape = q.shape
    if len(shape) != 3 or shape[2] != d:
        raise ValueError(f"q must be [T, Hq, {d}]")
    T, Hq, _ = shape
    cu = _list(cu_q, "cu_q", dev)
    B = cu_q.numel() - 1
    if out is None:
        out = made_for(stream, torch.empty_like, q)
    elif not (out.is_cuda and out.device == dev and out.dtype is torch.bfloat16
              and out.shape == shape and out.is_contiguous()):
        raise ValueError("out must be like q")
    if lse is None:
        lse = made_for(stream, torch.empty, Hq, T, dtype=torch.float32, device=dev)
    elif not (lse.is_cuda and lse.device == dev and lse.dtype is torch.float32
              and tuple(lse.shape) == (Hq, T) and lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 [Hq, T]")
    m, width = None, 0
    if mask is not None:
        _cuda(mask, "mask")
        if mask.dtype not in (torch.bool, torch.uint8) or mask.device != dev:
            raise ValueError(f"mask must be bool or uint8 on {dev}")
        if mask.dim() != 2 or mask.shape[0] != T or not mask.is_contiguous():
            raise ValueError("mask must be a contiguous [T, width]")
        m, width = mask.data_ptr(), mask.shape[1]
    ws = made_for(stream, torch.empty, cache._ws, dtype=torch.uint8, device=dev)
    _on(dev, lib.attn_tree_fwd, cache._ref, layer, q.data_ptr(), out.data_ptr(), lse.data_ptr(),
        Hq, B, T, cu, None if slots is None else _list(slots, "slots", dev, B), m, width,
        1.0 / math.sqrt(d) if scale is None else float(scale), ws.data_ptr(), cache._ws,
        _stream(dev, stream))
    return out, lse
