"""Paged compressed cache and its operators (PyTorch binding of the ``octo_paged_*`` and ``octo_rope`` C ABI).

* :class:`RopeTable`, :func:`rope` - rotary positions with up to four axes (``octo_rope_freqs``, ``octo_rope``)
* :class:`PagedCache`              - a pool of pages of compressed keys and bf16 values (``octo_pages``)
* :func:`paged_write`              - codes staged by ``encode`` and new values into pages (``octo_paged_write``)
* :func:`paged_append`             - ``encode`` of new keys, then :func:`paged_write`
* :func:`paged_attn`               - attention of a chunk of new tokens over the pages (``octo_paged_attn``)
* :func:`paged_mass`               - attention weight gathered per cached token (``octo_paged_mass``)
* :func:`paged_evict`              - cut sequences back to the tokens of the largest weight (``octo_paged_evict``)

Page tables are int32 [B][pages] tensors, lengths int32 [B], both on the cache's device: sequence i's slot s is in page
``page_table[i, s // page_size]``. Entries behind a sequence's last page are not read. The kernels see these values, the
host does not: what they find wrong goes to the cache's status word (:meth:`PagedCache.check`).

As the whole binding, this module only marshals arguments; shapes, types and devices that plain pointers hide from the C
ABI are refused with ValueError. Calls run on the tensors' device, on ``stream`` or torch's current stream there; tensors
used on a stream other than the one they were made on need ``record_stream`` as in any torch program. What a call with
``stream`` allocates (outputs, scratch) is made on that stream.
"""

from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass

import numpy as np
import torch

from . import _lib, api

_F32, _BF16, _I32 = torch.float32, torch.bfloat16, torch.int32
_DTYPES = {_F32: _lib.F32, _BF16: _lib.BF16}
_byref = ctypes.byref
_on, _on_its_stream = api._on, api._on_its_stream


def _same_device(index: int, *tensors):
    """All tensors are on CUDA device ``index``."""
    for t in tensors:
        if t is not None and (index < 0 or t.get_device() != index):
            dev = {str(x.device) for x in tensors if x is not None}
            raise ValueError(f"the tensors must be on one CUDA device, they are on device {', '.join(sorted(dev))} "
                             f"and {index if index >= 0 else 'none'}")


def _vector(t: torch.Tensor, what: str, n: int):
    if t.dtype is not _I32 or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous int32 [{n}], got {t.dtype} {tuple(t.shape)}")


def _dense(t: torch.Tensor, what: str, dtype, shape):
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} {list(shape)} tensor, got {t.dtype} {tuple(t.shape)}")


# ------------------------------------------------------------------ rotary positions
class RopeTable:
    """Frequencies of :func:`rope`: ``sections[k]`` consecutive frequencies turn with axis k's position. One frequency
    scale theta^(-i / F) runs over all F = sum(sections) of them, or one per axis, theta^(-j / sections[k])."""

    def __init__(self, sections, theta: float = 10000.0, per_axis: bool = False, device="cuda"):
        self._sections = tuple(int(s) for s in sections)
        sec = np.asarray(self._sections, np.int32)
        f = np.zeros(max(1, int(sum(self.sections))), np.uint64)
        _lib.check(_lib.lib().octo_rope_freqs(float(theta), len(sec), sec.ctypes.data, int(bool(per_axis)), f.ctypes.data),
                   "octo_rope_freqs")
        self._theta, self._per_axis = float(theta), bool(per_axis)
        self.c_sections, self._count = sec, len(f)
        self.freqs = torch.from_numpy(f.view(np.int64)).to(device)
        self.sections_ptr = sec.ctypes.data

    # of the frequencies as computed: not to be assigned
    sections = property(lambda self: self._sections)
    theta = property(lambda self: self._theta)
    per_axis = property(lambda self: self._per_axis)
    freqs_ptr = property(lambda self: self.freqs.data_ptr())


def _end(t: torch.Tensor) -> int:
    return t.data_ptr() + t.element_size() * (1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride())))


def _meet(x: torch.Tensor, y: torch.Tensor) -> bool:
    """Whether two [tokens][heads][d] tensors of one type may share memory. Strided views that lie between one another's
    rows, as those of a fused projection, do not: their rows repeat at a distance at which they stay apart."""
    if not x.numel() or not y.numel() or x.data_ptr() >= _end(y) or y.data_ptr() >= _end(x):
        return False
    gap = (y.data_ptr() - x.data_ptr()) // x.element_size()
    for dims in (1, 2):  # tokens repeat, with a token's heads as one run; or tokens and heads repeat
        m = math.gcd(*(t.stride(k) for t in (x, y) for k in range(dims) if t.shape[k] > 1))
        runs = [t.shape[2] + ((t.shape[1] - 1) * t.stride(1) if dims == 1 else 0) for t in (x, y)]
        if m and (y.data_ptr() - x.data_ptr()) % x.element_size() == 0 and gap % m >= runs[0] and gap % m + runs[1] <= m:
            return False
    return True


def _rope_pair(x: torch.Tensor, y: torch.Tensor | None, what: str):
    """(output, octo_rope_tensor) of one of rope's tensors."""
    sx = x.stride()
    if y is None:
        y = torch.empty_like(x)
        sy = y.stride()
    else:
        sy = y.stride()
        if y.shape != x.shape or y.dtype is not x.dtype:
            raise ValueError(f"{what} must have its input's shape and type")
        if any(s == 0 and n > 1 for n, s in zip(y.shape, sy)):
            raise ValueError(f"{what} must not be an expanded view")
        same = y.data_ptr() == x.data_ptr() and all(n == 1 or a == b for n, a, b in zip(x.shape, sx, sy))
        if not same and _meet(x, y):
            raise ValueError(f"{what} must be the input itself or not overlap it")
    if (sx[2] != 1 or sy[2] != 1) and x.shape[2] > 1:
        raise ValueError("rope's tensors must be contiguous in their last dimension")
    return y, _lib.OctoRopeTensor(x.data_ptr(), y.data_ptr(), x.shape[1], sx[0], sx[1], sy[0], sy[1])


@_on_its_stream
def rope(q: torch.Tensor, positions: torch.Tensor, table: RopeTable, k: torch.Tensor | None = None,
         interleaved: bool = False, inverse: bool = False, out: torch.Tensor | None = None,
         k_out: torch.Tensor | None = None, stream=None):
    """Rotary positions on q [tokens][heads][d] and, in the same launch, k [tokens][heads][d] (float32 or bfloat16, any
    token and head strides): the pairs (x_i, x_{i+F}), or neighbours when ``interleaved``, turn by
    positions[axis(i)][token] * f_i; coordinates from 2F on are copied. positions is int32 [axes][tokens].

    ``inverse`` turns back; as the rotation is orthogonal this is also the gradient: grad_q = rope(grad_out, ...,
    inverse=True). out / k_out may be their own inputs (in place), and must not overlap anything else of the call.
    Returns the rotated q, or (q, k).
    """
    dt = _DTYPES.get(q.dtype)
    if dt is None or q.dim() != 3:
        raise ValueError(f"q must be float32 or bfloat16 [tokens][heads][d], got {q.dtype} {tuple(q.shape)}")
    n, _, d = q.shape
    axes, freqs = len(table._sections), table.freqs
    if freqs.dtype is not torch.int64 or freqs.numel() < table._count or not freqs.is_contiguous():
        raise ValueError(f"the table's freqs must be contiguous int64 [{table._count}], got {freqs.dtype} {tuple(freqs.shape)}")
    if positions.dtype is not _I32 or positions.shape != (axes, n) or (n > 1 and positions.stride(1) != 1):
        raise ValueError(f"positions must be int32 [{axes}][{n}], contiguous in its last dimension, got "
                         f"{positions.dtype} {tuple(positions.shape)}")
    if axes > 1 and positions.stride(0) < n:
        raise ValueError("positions must not be an expanded view: its rows overlap")
    out_given = out is not None
    out, a = _rope_pair(q, out, "out")
    b = None
    if k is not None:
        if k.dtype is not q.dtype or k.dim() != 3 or k.shape[0] != n or k.shape[2] != d:
            raise ValueError(f"k must be {q.dtype} [{n}][heads][{d}], got {k.dtype} {tuple(k.shape)}")
        given = out_given or k_out is not None
        k_out, c = _rope_pair(k, k_out, "k_out")
        if given and (_meet(out, k) or _meet(k_out, q) or _meet(out, k_out)):
            raise ValueError("out and k_out must not overlap one another, nor the other's input")
        b = _byref(c)
    index = q.get_device()
    _same_device(index, k, positions, freqs, out, k_out)
    stride = positions.stride(0)
    st = _on(index, stream, lambda s: _lib.lib().octo_rope(
        _byref(a), b, dt, n, d, positions.data_ptr(), stride if stride > n else n, axes, table.sections_ptr,
        freqs.data_ptr(), interleaved, inverse, s))
    if st:
        _lib.check(st, "octo_rope")
    return out if k is None else (out, k_out)


# ------------------------------------------------------------------ the paged cache
@dataclass
class PagedCache:
    """A pool of pages of ``page_size`` slots, each holding every KV head: packed codes int32 (uint32 words)
    [pages][heads][W][page_size], norms float32 [pages][heads][page_size], values bfloat16
    [pages][heads][page_size][d] (None: a pool of keys only)."""
    packed: torch.Tensor
    gamma: torch.Tensor
    V: torch.Tensor | None = None
    status: torch.Tensor | None = None  # int32 [1], bits PAGED_* that the kernels found

    def __post_init__(self):
        p, g, v = self.packed, self.gamma, self.V
        if p.dtype != torch.int32 or p.dim() != 4 or not p.is_contiguous():
            raise ValueError("packed must be a contiguous int32 [pages][heads][words][page_size] tensor")
        n, h, _, s = p.shape
        if g.dtype != torch.float32 or tuple(g.shape) != (n, h, s) or not g.is_contiguous():
            raise ValueError(f"gamma must be a contiguous float32 {(n, h, s)} tensor")
        if v is not None and (v.dtype != torch.bfloat16 or v.dim() != 4 or tuple(v.shape[:3]) != (n, h, s) or
                              not v.is_contiguous()):
            raise ValueError(f"V must be a contiguous bfloat16 [{n}][{h}][{s}][d] tensor")
        if s % 16 != 0 or s < 16 or n < 1 or h < 1:
            raise ValueError("page_size must be a positive multiple of 16, with at least one page and head")
        if self.status is None:
            self.status = torch.zeros(1, dtype=torch.int32, device=p.device)
        elif self.status.dtype != torch.int32 or self.status.numel() != 1:
            raise ValueError(f"status must be int32 [1], got {self.status.dtype} {tuple(self.status.shape)}")
        if any(t is not None and t.device != p.device for t in (g, v, self.status)):
            raise ValueError("the cache's tensors must be on one device")
        self.shape = (n, h, p.shape[2], s, None if v is None else v.shape[3])  # pages, heads, words, page size, d
        self.index = p.get_device()
        self._held = (p, g, v, self.status)
        self._at = (p.data_ptr(), g.data_ptr(), None if v is None else v.data_ptr(), self.status.data_ptr())
        self._ref = _byref(_lib.OctoPages(*self._at[:3], n, h, s, self._at[3]))

    def current(self) -> PagedCache:
        """The pool, described anew (and checked) if a field was assigned or a tensor's memory moved since: calls use the
        tensors that it holds now."""
        p, g, v, s = self._held
        if (p is not self.packed or g is not self.gamma or v is not self.V or s is not self.status or
                self._at != (p.data_ptr(), g.data_ptr(), None if v is None else v.data_ptr(), s.data_ptr())):
            self.__post_init__()
        return self

    @property
    def ref(self):
        """The ``octo_pages`` of the tensors held now, for the C ABI."""
        return self.current()._ref

    @property
    def c(self) -> _lib.OctoPages:
        return self.ref._obj

    @classmethod
    def empty(cls, layout: api.Layout, n_pages: int, n_heads: int, page_size: int, values: bool = True, device="cuda"):
        """A zeroed pool."""
        packed = torch.zeros((n_pages, n_heads, layout.words, page_size), dtype=torch.int32, device=device)
        gamma = torch.zeros((n_pages, n_heads, page_size), dtype=torch.float32, device=device)
        V = torch.zeros((n_pages, n_heads, page_size, layout.d), dtype=torch.bfloat16, device=device) if values else None
        return cls(packed, gamma, V)

    @classmethod
    def from_cache(cls, cache: api.Cache, V: torch.Tensor | None, n_heads: int):
        """A contiguous cache of B * n_heads heads (and its V [B * n_heads][cap][d]) seen as a pool of B pages of cap
        slots, sharing its memory; the capacity must be a multiple of 16. Page i is sequence i's whole cache."""
        if n_heads < 1 or cache.n_heads % n_heads != 0 or cache.cap % 16 != 0:
            raise ValueError(f"{cache.n_heads} cache heads of {cache.cap} slots are no pages of {n_heads} heads and a "
                             "multiple of 16 slots")
        B, cap = cache.n_heads // n_heads, cache.cap
        return cls(cache.packed.view(B, n_heads, -1, cap), cache.gamma.view(B, n_heads, cap),
                   None if V is None else V.view(B, n_heads, cap, -1))

    @property
    def n_pages(self) -> int:
        return int(self.packed.shape[0])

    @property
    def n_heads(self) -> int:
        return int(self.packed.shape[1])

    @property
    def page_size(self) -> int:
        return int(self.packed.shape[3])

    def check(self) -> None:
        """Raises if a kernel found a page id outside the pool, a length that the tables do not hold, or gave up a
        bounded wait (waits for the device's calls, on whatever stream; clears the word)."""
        if self.status.is_cuda:
            torch.cuda.synchronize(self.status.device)
        bits = int(self.status.item())
        if bits:
            self.status.zero_()
            if self.status.is_cuda:  # cleared before a call on another stream can set it again
                torch.cuda.synchronize(self.status.device)
            names = [n for b, n in ((_lib.PAGED_TIMEOUT, "a wait expired"), (_lib.PAGED_BAD_PAGE, "a page id outside the pool"),
                                    (_lib.PAGED_BAD_LENGTH, "a length or offset that the tables do not hold")) if bits & b]
            raise RuntimeError("paged cache: " + ", ".join(names))


def _check_pool(layout: api.Layout, cache: PagedCache, values: bool):
    """The pool fits the layout. Comes before any other look at the pool's shape."""
    c = layout.c
    cache.current()
    if cache.shape[2] != c.words:
        raise ValueError(f"the cache holds {cache.shape[2]} words per key, {layout!r} has {c.words}")
    if cache.shape[4] is None:
        if values:
            raise ValueError("the cache holds no values")
    elif cache.shape[4] != c.d:
        raise ValueError(f"the cache's V rows have {cache.shape[4]} elements, {layout!r} has d={c.d}")


def _table(page_table: torch.Tensor, B: int, what: str = "page_table"):
    if page_table.dtype is not _I32 or page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError(f"{what} must be int32 [{B}][pages], got {page_table.dtype} {tuple(page_table.shape)}")
    n = page_table.shape[1]
    s0, s1 = page_table.stride()
    if s1 != 1 and n > 1:
        raise ValueError(f"{what} must be contiguous in its last dimension")
    if B > 1 and s0 < n:
        raise ValueError(f"{what} must not be an expanded view: its rows overlap")
    return _lib.OctoPageTable(page_table.data_ptr(), s0 if s0 > n else n, B, n)


def paged_write(layout: api.Layout, staged: api.Cache, V: torch.Tensor | None, cache: PagedCache,
                page_table: torch.Tensor, starts: torch.Tensor, cu: torch.Tensor, stream=None) -> PagedCache:
    """New tokens into pages: packed row r = cu[i] + t of sequence i goes to slot starts[i] + t.

    staged: a contiguous :class:`api.Cache` whose ``cache.n_heads`` heads hold the rows' codes from token 0 (``encode``
    of the packed keys); V [rows][heads][d] bfloat16, any row and head strides that are multiples of 8 elements, or None
    for a cache without values; starts int32 [B], cu int32 [B + 1]. No two tokens may go to one slot. Rows
    from cu[B] on (a batch padded to a fixed size) are left alone.
    """
    _check_pool(layout, cache, False)
    B, H, W, d = starts.numel(), cache.shape[1], cache.shape[2], layout.c.d
    _vector(starts, "starts", B)
    _vector(cu, "cu", B + 1)
    if (V is None) != (cache.V is None):
        raise ValueError("the cache holds values: V is needed" if V is None else "the cache holds no values")
    if V is None:
        rows, sr, sh, pv = staged.length, 0, 0, None
    else:
        if V.dtype is not _BF16 or V.dim() != 3 or V.shape[1] != H or V.shape[2] != d or V.stride(2) != 1:
            raise ValueError(f"V must be bfloat16 [rows][{H}][{d}], contiguous in its last dimension")
        rows, sr, sh, pv = V.shape[0], V.stride(0), V.stride(1), V.data_ptr()
        if sr % 8 or sh % 8 or pv % 16:
            raise ValueError("V rows must start on 16-byte boundaries")
    p, g = staged.packed, staged.gamma
    cap = p.shape[-1]
    if p.dtype is not _I32 or p.shape != (H, W, cap) or cap < rows or not p.is_contiguous():
        raise ValueError(f"staged must hold {H} heads of {layout!r} with at least {rows} tokens")
    _dense(g, "staged.gamma", _F32, (H, cap))
    t = _table(page_table, B)
    index = cache.index
    _same_device(index, p, g, V, page_table, starts, cu)
    st = _on(index, stream, lambda s: _lib.lib().octo_paged_write(
        layout.ref, cache._ref, _byref(t), p.data_ptr(), g.data_ptr(), cap, pv, sr, sh, rows, starts.data_ptr(),
        cu.data_ptr(), s))
    if st:
        _lib.check(st, "octo_paged_write")
    return cache


@_on_its_stream
def paged_append(layout: api.Layout, tables: api.DeviceTables, keys: torch.Tensor, V: torch.Tensor | None,
                 cache: PagedCache, page_table: torch.Tensor, starts: torch.Tensor, cu: torch.Tensor,
                 staged: api.Cache | None = None, stream=None) -> PagedCache:
    """``encode`` of packed new keys [rows][heads][d], then :func:`paged_write` of their codes and V. ``staged`` may be
    given to reuse a staging cache of at least ``rows`` tokens."""
    if keys.dim() != 3 or keys.shape[1] != cache.n_heads:
        raise ValueError(f"keys must be [rows][{cache.n_heads}][{layout.d}], got {tuple(keys.shape)}")
    rows = int(keys.shape[0])
    if V is not None and V.shape[0] != rows:
        raise ValueError(f"V holds {V.shape[0]} rows, keys {rows}")
    if staged is None:
        staged = api.Cache.empty(layout, cache.n_heads, max(rows, 1), device=keys.device)
    rows_of = keys.transpose(0, 1)
    _on(keys.get_device(), stream, lambda s: api.encode(layout, tables, rows_of, staged, 0, stream=stream))
    staged.length = rows
    return paged_write(layout, staged, V, cache, page_table, starts, cu, stream=stream)


def _chunk(layout, tables, q, cache, page_table, seq_lens, cu_q):
    """Checks of the calls that take a chunk of queries; returns (dtype, rows, Hq, B, cu_q, octo_page_table)."""
    d, H = layout.c.d, cache.shape[1]
    dt = _DTYPES.get(q.dtype)
    if dt is None:
        raise ValueError(f"unsupported query dtype {q.dtype}")
    if q.dim() != 3 or q.shape[2] != d or q.stride(2) != 1:
        raise ValueError(f"q must be [rows][heads][{d}], contiguous in its last dimension, got {tuple(q.shape)}")
    rows, Hq, _ = q.shape
    if Hq < H or Hq % H:
        raise ValueError(f"{Hq} query heads over {H} cache heads")
    B = seq_lens.numel()
    _vector(seq_lens, "seq_lens", B)
    if cu_q is None:
        if B == 0 or rows % B:
            raise ValueError(f"{rows} query rows over {B} sequences: cu_q is needed")
        cu_q = torch.arange(B + 1, dtype=_I32, device=q.device) * (rows // B)
    _vector(cu_q, "cu_q", B + 1)
    t = _table(page_table, B)
    tables.check(layout)
    _same_device(cache.index, q, page_table, seq_lens, cu_q, tables.dir_c, tables.signs)
    return dt, rows, Hq, B, cu_q, t


def paged_attn_workspace_bytes(layout: api.Layout, rows: int, B: int, Hq: int, Hkv: int) -> int:
    return int(_lib.lib().octo_paged_attn_workspace(layout.ref, rows, B, Hq, Hkv))


def paged_mass_workspace_bytes(layout: api.Layout, rows: int, B: int, Hq: int, Hkv: int) -> int:
    return int(_lib.lib().octo_paged_mass_workspace(layout.ref, rows, B, Hq, Hkv))


def _scratch(workspace, need: int, cache: PagedCache):
    """A device buffer of ``need`` bytes: the workspace's, or one for this call."""
    if workspace is None:
        return torch.empty((need + 255) // 256 * 64, dtype=_I32, device=cache.packed.device)
    if workspace.buf.get_device() != cache.index:
        raise ValueError(f"the workspace is on {workspace.buf.device}, the cache on {cache.packed.device}")
    return workspace.ensure(need).buf


@_on_its_stream
def paged_attn(layout: api.Layout, tables: api.DeviceTables, q: torch.Tensor, cache: PagedCache, page_table: torch.Tensor,
               seq_lens: torch.Tensor, cu_q: torch.Tensor | None = None, causal: bool = True, scale: float | None = None,
               dtype=None, out: torch.Tensor | None = None, lse=None, workspace: api.Workspace | None = None, stream=None):
    """Attention of a chunk of new tokens over a paged cache that already holds them.

    q [rows][Hq][d] (float32 or bfloat16): rows cu_q[i] .. cu_q[i+1] - 1 (cu_q int32 [B + 1]; None: the same number for
    each) are the last tokens of sequence i, whose cache holds seq_lens[i] slots. With ``causal`` each new token sees the
    slots up to its own, else all of its sequence. A row that sees nothing gives 0 (lse -inf). Values of slots that one row
    of a sequence sees must be finite for its other rows too, and sum to less than 2^60 in magnitude. Returns out [rows][Hq][d]
    (``dtype`` float32 or bfloat16, by default q's), and with ``lse`` (True, or a float32 [rows][Hq] tensor) the pair
    (out, lse) with lse = ln sum exp(scale * logits).

    Queries enter the tensor cores as one fp16 value each, weights as bf16: a float32 output carries no more than that
    (errors of about 1e-3 relative). Rows of no sequence are left as they were (an ``out`` made here: uninitialised).

    A workspace serves one call at a time, whichever (``decode_attn``'s too): calls that may overlap on the GPU (streams,
    graphs) need one each. None allocates it for this call.
    """
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype if dtype is None else dtype, device=q.device)
    elif out.shape != q.shape or not out.is_contiguous() or dtype not in (None, out.dtype):
        raise ValueError(f"out must be a contiguous {tuple(q.shape)} tensor")
    elif q.numel() and out.data_ptr() < _end(q) and q.data_ptr() < _end(out):
        raise ValueError("out must not overlap q")
    odt = _DTYPES.get(out.dtype)
    if odt is None:
        raise ValueError(f"unsupported output dtype {out.dtype}")
    if lse is True:
        lse = torch.empty(q.shape[:2], dtype=_F32, device=q.device)
    elif lse is False:
        lse = None
    elif lse is not None:
        _dense(lse, "lse", _F32, q.shape[:2])
    _check_pool(layout, cache, True)
    dt, rows, Hq, B, cu_q, t = _chunk(layout, tables, q, cache, page_table, seq_lens, cu_q)
    index, lib = cache.index, _lib.lib()
    _same_device(index, out, lse)

    def call(s):
        ws = _scratch(workspace, lib.octo_paged_attn_workspace(layout.ref, rows, B, Hq, cache.shape[1]), cache)
        return lib.octo_paged_attn(
            layout.ref, tables.ref, cache._ref, _byref(t), seq_lens.data_ptr(), q.data_ptr(), dt, q.stride(0), q.stride(1),
            rows, Hq, cu_q.data_ptr(), causal, layout.c.d ** -0.5 if scale is None else scale, out.data_ptr(), odt,
            None if lse is None else lse.data_ptr(), ws.data_ptr(), ws.numel() * 4, s)

    st = _on(index, stream, call)
    if st:
        _lib.check(st, "octo_paged_attn")
    return out if lse is None else (out, lse)


@_on_its_stream
def paged_mass(layout: api.Layout, tables: api.DeviceTables, q: torch.Tensor, lse: torch.Tensor, cache: PagedCache,
               page_table: torch.Tensor, seq_lens: torch.Tensor, mass: torch.Tensor, cu_q: torch.Tensor | None = None,
               causal: bool = True, scale: float | None = None, decay: float = 1.0, out: torch.Tensor | None = None,
               workspace: api.Workspace | None = None, stream=None) -> torch.Tensor:
    """Adds the attention weight that each cached token gathers from a chunk: out[i][h][j] = decay * mass[i][h][j] + the
    sum over the chunk's rows and the cache head's query heads of exp(scale * logit_j - lse), for slots j < seq_lens[i];
    later slots of out are left as they were. Sequences without new rows, and a chunk without any, decay alone. q, masks and lse (float32 [rows][Hq]) as in :func:`paged_attn`; mass
    float32 [B][heads][slots]; out is mass itself (in place) by default."""
    _check_pool(layout, cache, False)
    B, H = seq_lens.numel(), cache.shape[1]
    slots = mass.shape[-1]
    _dense(mass, "mass", _F32, (B, H, slots))
    if out is None:
        out = mass
    elif out is not mass:
        _dense(out, "out", _F32, (B, H, slots))
        if out.data_ptr() != mass.data_ptr() and abs(out.data_ptr() - mass.data_ptr()) < 4 * mass.numel():
            raise ValueError("out must be mass itself or not overlap it")
    _dense(lse, "lse", _F32, q.shape[:2])
    dt, rows, Hq, B, cu_q, t = _chunk(layout, tables, q, cache, page_table, seq_lens, cu_q)
    index, lib = cache.index, _lib.lib()
    _same_device(index, lse, mass, out)

    def call(s):
        ws = _scratch(workspace, lib.octo_paged_mass_workspace(layout.ref, rows, B, Hq, H), cache)
        return lib.octo_paged_mass(
            layout.ref, tables.ref, cache._ref, _byref(t), seq_lens.data_ptr(), q.data_ptr(), dt, q.stride(0), q.stride(1),
            rows, Hq, cu_q.data_ptr(), causal, layout.c.d ** -0.5 if scale is None else scale, lse.data_ptr(), decay,
            mass.data_ptr(), out.data_ptr(), slots, ws.data_ptr(), ws.numel() * 4, s)

    st = _on(index, stream, call)
    if st:
        _lib.check(st, "octo_paged_mass")
    return out


@_on_its_stream
def paged_evict(layout: api.Layout, cache: PagedCache, page_table: torch.Tensor, seq_lens: torch.Tensor,
                mass: torch.Tensor, keep: int, dst_table: torch.Tensor, sink: int = 0, recent: int = 0,
                dst: PagedCache | None = None, kept: torch.Tensor | None = None, new_lens: torch.Tensor | None = None,
                new_mass: torch.Tensor | None = None, stream=None):
    """Cuts every (sequence, head) back to ``keep`` slots: the first ``sink``, the last ``recent`` and those of the
    largest mass between them (ties: the lower slot), in their order, copied to the pages of dst_table [B][pages] (in
    ``dst``, by default the same pool; pages written must not hold tokens that the call reads). Sequences of at most
    ``keep`` slots move whole. mass float32 [B][heads][slots].

    Returns (new_lens int32 [B], which may be given as seq_lens itself; kept int32 [B][heads][keep]: the slots kept, -1 behind the last; new_mass float32
    [B][heads][keep], 0 behind the last). Kept tokens keep the positions that their keys were rotated by.
    """
    _check_pool(layout, cache, False)
    if dst is None:
        dst = cache
    else:
        _check_pool(layout, dst, False)
    B, H, slots = seq_lens.numel(), cache.shape[1], mass.shape[-1]
    _vector(seq_lens, "seq_lens", B)
    _dense(mass, "mass", _F32, (B, H, slots))
    if keep < 1:
        raise ValueError(f"keep must be at least 1, got {keep}")
    dev, index = mass.device, cache.index
    if kept is None:
        kept = torch.empty((B, H, keep), dtype=_I32, device=dev)
    else:
        _dense(kept, "kept", _I32, (B, H, keep))
    if new_lens is None:
        new_lens = torch.empty((B,), dtype=_I32, device=dev)
    else:
        _vector(new_lens, "new_lens", B)
        if new_lens.data_ptr() != seq_lens.data_ptr() and abs(new_lens.data_ptr() - seq_lens.data_ptr()) < 4 * B:
            raise ValueError("new_lens must be seq_lens itself or not overlap it")
    if new_mass is None:
        new_mass = torch.empty((B, H, keep), dtype=_F32, device=dev)
    else:
        _dense(new_mass, "new_mass", _F32, (B, H, keep))
        if mass.numel() and new_mass.data_ptr() < _end(mass) and mass.data_ptr() < _end(new_mass):
            raise ValueError("new_mass must not overlap mass")
    t, z = _table(page_table, B), _table(dst_table, B, "dst_table")
    _same_device(index, page_table, seq_lens, mass, dst_table, dst.packed, kept, new_lens, new_mass)
    st = _on(index, stream, lambda s: _lib.lib().octo_paged_evict(
        layout.ref, cache._ref, _byref(t), seq_lens.data_ptr(), mass.data_ptr(), slots, keep, sink, recent, dst._ref,
        _byref(z), kept.data_ptr(), new_lens.data_ptr(), new_mass.data_ptr(), s))
    if st:
        _lib.check(st, "octo_paged_evict")
    return new_lens, kept, new_mass
