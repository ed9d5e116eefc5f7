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
used on a stream other than the one they were made on need ``record_stream`` as in any torch program.
"""

from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass

import numpy as np
import torch

from . import _lib, api

_DTYPES = {torch.float32: _lib.F32, torch.bfloat16: _lib.BF16}


class _On:
    """Makes the tensors' device current for a call (and nothing else when it already is), and finds the stream."""

    def __init__(self, device: torch.device, stream):
        self.guard = None
        if device.type == "cuda" and device.index != torch.cuda.current_device():
            self.guard = torch.cuda.device(device)
        self.device, self.given = device, stream

    def __enter__(self) -> int:
        if self.guard is not None:
            self.guard.__enter__()
        s = self.given
        if s is None:
            if self.device.type != "cuda":
                raise ValueError(f"the tensors are on {self.device}: a CUDA device is needed")
            s = torch.cuda.current_stream()
        elif s.device != self.device:
            raise ValueError(f"the stream is on {s.device}, the tensors on {self.device}")
        return int(s.cuda_stream)

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _same_device(device, *tensors):
    for t in tensors:
        if t is not None and t.device != device:
            raise ValueError(f"a tensor is on device {t.device}, others on device {device}")


def _ints(t: torch.Tensor, what: str, shape) -> torch.Tensor:
    if t.dtype != torch.int32 or t.dim() != len(shape) or any(w is not None and w != n for w, n in zip(shape, t.shape)):
        raise ValueError(f"{what} must be int32 {['n' if w is None else w for w in shape]}, got {t.dtype} {tuple(t.shape)}")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{what} must be contiguous in its last dimension")
    return t


# ------------------------------------------------------------------ rotary positions
class RopeTable:
    """Frequencies of :func:`rope`: ``sections[k]`` consecutive frequencies turn with axis k's position. One frequency
    scale theta^(-i / F) runs over all F = sum(sections) of them, or one per axis, theta^(-j / sections[k])."""

    def __init__(self, sections, theta: float = 10000.0, per_axis: bool = False, device="cuda"):
        self.sections = tuple(int(s) for s in sections)
        sec = np.asarray(self.sections, np.int32)
        f = np.zeros(max(1, int(sum(self.sections))), np.uint64)
        _lib.check(_lib.lib().octo_rope_freqs(float(theta), len(sec), sec.ctypes.data, int(bool(per_axis)), f.ctypes.data),
                   "octo_rope_freqs")
        self.theta, self.per_axis = float(theta), bool(per_axis)
        self.c_sections = sec
        self.freqs = torch.from_numpy(f.view(np.int64)).to(device)


def _rope_tensor(x: torch.Tensor, y: torch.Tensor):
    return _lib.OctoRopeTensor(x.data_ptr(), y.data_ptr(), x.shape[1], x.stride(0), x.stride(1), y.stride(0), y.stride(1))


def _rope_out(x, out, what):
    if out is None:
        return torch.empty(x.shape, dtype=x.dtype, device=x.device)
    if out.shape != x.shape or out.dtype != x.dtype or (out.stride(-1) != 1 and out.shape[-1] > 1):
        raise ValueError(f"{what} must have its input's shape and type, contiguous in the last dimension")
    if out.data_ptr() != x.data_ptr() or out.stride() != x.stride():
        # the input itself (turned in place) or memory apart from it
        end = lambda t: t.data_ptr() + t.element_size() * (1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride())))  # noqa: E731
        if x.numel() and out.data_ptr() < end(x) and x.data_ptr() < end(out):
            raise ValueError(f"{what} must be the input itself or not overlap it")
    return out


def rope(q: torch.Tensor, positions: torch.Tensor, table: RopeTable, k: torch.Tensor | None = None,
         interleaved: bool = False, inverse: bool = False, out: torch.Tensor | None = None,
         k_out: torch.Tensor | None = None, stream=None):
    """Rotary positions on q [tokens][heads][d] and, in the same launch, k [tokens][heads][d] (float32 or bfloat16, any
    token and head strides): the pairs (x_i, x_{i+F}), or neighbours when ``interleaved``, turn by
    positions[axis(i)][token] * f_i; coordinates from 2F on are copied. positions is int32 [axes][tokens].

    ``inverse`` turns back; as the rotation is orthogonal this is also the gradient: grad_q = rope(grad_out, ...,
    inverse=True). out / k_out may be the inputs (in place). Returns the rotated q, or (q, k).
    """
    d = q.shape[-1] if q.dim() == 3 else -1
    dt = _DTYPES.get(q.dtype)
    if d < 0 or dt is None or (q.stride(-1) != 1 and d > 1):
        raise ValueError(f"q must be float32 or bfloat16 [tokens][heads][d], contiguous in d, got {q.dtype} {tuple(q.shape)}")
    n = q.shape[0]
    if k is not None and (k.dim() != 3 or k.shape[0] != n or k.shape[2] != d or k.dtype != q.dtype or
                          (k.stride(-1) != 1 and d > 1)):
        raise ValueError(f"k must be {q.dtype} [{n}][heads][{d}], contiguous in d, got {k.dtype} {tuple(k.shape)}")
    _ints(positions, "positions", (len(table.sections), n))
    out = _rope_out(q, out, "out")
    pair = None
    if k is not None:
        k_out = _rope_out(k, k_out, "k_out")
        pair = ctypes.byref(_rope_tensor(k, k_out))
    _same_device(q.device, k, positions, table.freqs, out, k_out)
    with _On(q.device, stream) as st:
        _lib.check(_lib.lib().octo_rope(ctypes.byref(_rope_tensor(q, out)), pair, dt, n, d, positions.data_ptr(),
                                        max(positions.stride(0), n), len(table.sections), table.c_sections.ctypes.data,
                                        table.freqs.data_ptr(), int(interleaved), int(inverse), st), "octo_rope")
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
        _same_device(p.device, g, v, self.status)
        self.c = _lib.OctoPages(p.data_ptr(), g.data_ptr(), None if v is None else v.data_ptr(), n, h, s,
                                self.status.data_ptr())

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
        bounded wait (synchronises; clears the word)."""
        bits = int(self.status.item())
        if bits:
            self.status.zero_()
            names = [n for b, n in ((_lib.PAGED_TIMEOUT, "a wait expired"), (_lib.PAGED_BAD_PAGE, "a page id outside the pool"),
                                    (_lib.PAGED_BAD_LENGTH, "a length or offset that the tables do not hold")) if bits & b]
            raise RuntimeError("paged cache: " + ", ".join(names))


def _check_pool(layout: api.Layout, cache: PagedCache, values: bool):
    if cache.packed.shape[2] != layout.words:
        raise ValueError(f"the cache holds {cache.packed.shape[2]} words per key, {layout!r} has {layout.words}")
    if cache.V is None:
        if values:
            raise ValueError("the cache holds no values")
    elif cache.V.shape[3] != layout.d:
        raise ValueError(f"the cache's V rows have {cache.V.shape[3]} elements, {layout!r} has d={layout.d}")


def _table(page_table: torch.Tensor, B: int):
    _ints(page_table, "page_table", (B, None))
    return _lib.OctoPageTable(page_table.data_ptr(), max(page_table.stride(0), page_table.shape[1]), B, page_table.shape[1])


def paged_write(layout: api.Layout, staged: api.Cache, V: torch.Tensor | None, cache: PagedCache,
                page_table: torch.Tensor, starts: torch.Tensor, cu: torch.Tensor, stream=None) -> PagedCache:
    """New tokens into pages: packed row r = cu[i] + t of sequence i goes to slot starts[i] + t.

    staged: a contiguous :class:`api.Cache` whose ``cache.n_heads`` heads hold the rows' codes from token 0 (``encode``
    of the packed keys); V [rows][heads][d] bfloat16, any row and head strides that are multiples of 8 elements, or None
    for a cache without values; starts int32 [B], cu int32 [B + 1]. No two tokens may go to one slot.
    """
    _check_pool(layout, cache, False)
    B = int(starts.shape[0])
    _ints(starts, "starts", (B,))
    _ints(cu, "cu", (B + 1,))
    H = cache.n_heads
    if V is None:
        if cache.V is not None:
            raise ValueError("the cache holds values: V is needed")
        rows = staged.length
        vs = (0, 0)
    else:
        if cache.V is None:
            raise ValueError("the cache holds no values")
        if V.dtype != torch.bfloat16 or V.dim() != 3 or V.shape[1] != H or V.shape[2] != layout.d or V.stride(2) != 1:
            raise ValueError(f"V must be bfloat16 [rows][{H}][{layout.d}], contiguous in its last dimension")
        rows, vs = int(V.shape[0]), (V.stride(0), V.stride(1))
        if vs[0] % 8 or vs[1] % 8 or V.data_ptr() % 16:
            raise ValueError("V rows must start on 16-byte boundaries")
    p = staged.packed
    if (p.dtype != torch.int32 or p.dim() != 3 or p.shape[0] != H or p.shape[1] != layout.words or p.shape[2] < rows or
            not p.is_contiguous() or staged.gamma.dtype != torch.float32 or
            tuple(staged.gamma.shape) != (H, p.shape[2]) or not staged.gamma.is_contiguous()):
        raise ValueError(f"staged must hold {H} heads of {layout!r} with at least {rows} tokens")
    _same_device(cache.packed.device, p, staged.gamma, V, page_table, starts, cu)
    with _On(cache.packed.device, stream) as st:
        _lib.check(_lib.lib().octo_paged_write(layout.ref, ctypes.byref(cache.c), ctypes.byref(_table(page_table, B)),
                                               p.data_ptr(), staged.gamma.data_ptr(), p.shape[2],
                                               None if V is None else V.data_ptr(), vs[0], vs[1], rows, starts.data_ptr(),
                                               cu.data_ptr(), st), "octo_paged_write")
    return cache


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
    with _On(keys.device, stream):
        api.encode(layout, tables, keys.transpose(0, 1), staged, 0, stream=stream)
    staged.length = rows
    return paged_write(layout, staged, V, cache, page_table, starts, cu, stream=stream)


def _chunk(layout, tables, q, cache, page_table, seq_lens, cu_q, extra):
    """Checks of the calls that take a chunk of queries; returns (dtype, rows, Hq, B, cu_q)."""
    if q.dim() != 3 or q.shape[2] != layout.d or (q.stride(2) != 1 and layout.d > 1):
        raise ValueError(f"q must be [rows][heads][{layout.d}], contiguous in its last dimension, got {tuple(q.shape)}")
    dt = _DTYPES.get(q.dtype)
    if dt is None:
        raise ValueError(f"unsupported query dtype {q.dtype}")
    rows, Hq, H = int(q.shape[0]), int(q.shape[1]), cache.n_heads
    if Hq < H or Hq % H:
        raise ValueError(f"{Hq} query heads over {H} cache heads")
    B = int(seq_lens.shape[0])
    _ints(seq_lens, "seq_lens", (B,))
    if cu_q is None:
        if B == 0 or rows % B:
            raise ValueError(f"{rows} query rows over {B} sequences: cu_q is needed")
        cu_q = torch.arange(B + 1, dtype=torch.int32, device=q.device) * (rows // B)
    _ints(cu_q, "cu_q", (B + 1,))
    _same_device(cache.packed.device, q, page_table, seq_lens, cu_q, tables.dir_c, tables.rho_c, tables.signs, *extra)
    return dt, rows, Hq, B, cu_q


def paged_attn_workspace_bytes(layout: api.Layout, rows: int, B: int, Hq: int, Hkv: int) -> int:
    return int(_lib.lib().octo_paged_attn_workspace(layout.ref, rows, B, Hq, Hkv))


def paged_mass_workspace_bytes(layout: api.Layout, rows: int, B: int, Hq: int, Hkv: int) -> int:
    return int(_lib.lib().octo_paged_mass_workspace(layout.ref, rows, B, Hq, Hkv))


def _workspace(workspace, need, device):
    if workspace is None:
        workspace = torch.empty((need + 255) // 256 * 64, dtype=torch.int32, device=device)
        return workspace, workspace.data_ptr(), workspace.numel() * 4
    if workspace.buf.device != device:
        raise ValueError(f"the workspace is on {workspace.buf.device}, the cache on {device}")
    workspace.ensure(need)
    return workspace, workspace.buf.data_ptr(), workspace.nbytes


def paged_attn(layout: api.Layout, tables: api.DeviceTables, q: torch.Tensor, cache: PagedCache, page_table: torch.Tensor,
               seq_lens: torch.Tensor, cu_q: torch.Tensor | None = None, causal: bool = True, scale: float | None = None,
               dtype=None, out: torch.Tensor | None = None, lse=None, workspace: api.Workspace | None = None, stream=None):
    """Attention of a chunk of new tokens over a paged cache that already holds them.

    q [rows][Hq][d] (float32 or bfloat16): rows cu_q[i] .. cu_q[i+1] - 1 (cu_q int32 [B + 1]; None: the same number for
    each) are the last tokens of sequence i, whose cache holds seq_lens[i] slots. With ``causal`` each new token sees the
    slots up to its own, else all of its sequence. A row that sees nothing gives 0 (lse -inf). Returns out [rows][Hq][d]
    (``dtype`` float32 or bfloat16, by default q's), and with ``lse`` (True, or a float32 [rows][Hq] tensor) the pair
    (out, lse) with lse = ln sum exp(scale * logits).

    A workspace serves one call at a time: calls that may overlap on the GPU (streams, graphs) need one each. None
    allocates it for this call.
    """
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype if dtype is None else dtype, device=q.device)
    elif out.shape != q.shape or not out.is_contiguous() or dtype not in (None, out.dtype):
        raise ValueError(f"out must be a contiguous {tuple(q.shape)} tensor")
    odt = _DTYPES.get(out.dtype)
    if odt is None:
        raise ValueError(f"unsupported output dtype {out.dtype}")
    if lse is True:
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    elif lse is False:
        lse = None
    elif lse is not None and (lse.dtype != torch.float32 or lse.shape != q.shape[:2] or not lse.is_contiguous()):
        raise ValueError(f"lse must be a contiguous float32 {tuple(q.shape[:2])} tensor")
    _check_pool(layout, cache, True)
    dt, rows, Hq, B, cu_q = _chunk(layout, tables, q, cache, page_table, seq_lens, cu_q, (out, lse))
    lib = _lib.lib()
    with _On(q.device, stream) as st:
        need = lib.octo_paged_attn_workspace(layout.ref, rows, B, Hq, cache.n_heads)
        hold, ws, nbytes = _workspace(workspace, need, q.device)
        _lib.check(lib.octo_paged_attn(layout.ref, tables.ref, ctypes.byref(cache.c), ctypes.byref(_table(page_table, B)),
                                       seq_lens.data_ptr(), q.data_ptr(), dt, q.stride(0), q.stride(1), rows, Hq,
                                       cu_q.data_ptr(), int(causal), 1.0 / math.sqrt(layout.d) if scale is None else scale,
                                       out.data_ptr(), odt, None if lse is None else lse.data_ptr(), ws, nbytes, st),
                   "octo_paged_attn")
    return out if lse is None else (out, lse)


def paged_mass(layout: api.Layout, tables: api.DeviceTables, q: torch.Tensor, lse: torch.Tensor, cache: PagedCache,
               page_table: torch.Tensor, seq_lens: torch.Tensor, mass: torch.Tensor, cu_q: torch.Tensor | None = None,
               causal: bool = True, scale: float | None = None, decay: float = 1.0, out: torch.Tensor | None = None,
               workspace: api.Workspace | None = None, stream=None) -> torch.Tensor:
    """Adds the attention weight that each cached token gathers from a chunk: out[i][h][j] = decay * mass[i][h][j] + the
    sum over the chunk's rows and the cache head's query heads of exp(scale * logit_j - lse), for slots j < seq_lens[i];
    later slots of out are left as they were. q, masks and lse (float32 [rows][Hq]) as in :func:`paged_attn`; mass
    float32 [B][heads][slots]; out is mass itself (in place) by default."""
    H = cache.n_heads
    if out is None:
        out = mass
    for t, what in ((mass, "mass"), (out, "out")):
        if t.dtype != torch.float32 or t.dim() != 3 or tuple(t.shape[:2]) != (seq_lens.shape[0], H) or not t.is_contiguous():
            raise ValueError(f"{what} must be a contiguous float32 [{seq_lens.shape[0]}][{H}][slots] tensor")
    if out.shape != mass.shape:
        raise ValueError(f"out must be {tuple(mass.shape)} as mass is")
    if out.data_ptr() != mass.data_ptr() and abs(out.data_ptr() - mass.data_ptr()) < 4 * mass.numel():
        raise ValueError("out must be mass itself or not overlap it")
    if lse.dtype != torch.float32 or tuple(lse.shape) != tuple(q.shape[:2]) or not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous float32 {tuple(q.shape[:2])} tensor")
    _check_pool(layout, cache, False)
    dt, rows, Hq, B, cu_q = _chunk(layout, tables, q, cache, page_table, seq_lens, cu_q, (lse, mass, out))
    lib = _lib.lib()
    with _On(q.device, stream) as st:
        need = lib.octo_paged_mass_workspace(layout.ref, rows, B, Hq, H)
        hold, ws, nbytes = _workspace(workspace, need, q.device)
        _lib.check(lib.octo_paged_mass(layout.ref, tables.ref, ctypes.byref(cache.c), ctypes.byref(_table(page_table, B)),
                                       seq_lens.data_ptr(), q.data_ptr(), dt, q.stride(0), q.stride(1), rows, Hq,
                                       cu_q.data_ptr(), int(causal), 1.0 / math.sqrt(layout.d) if scale is None else scale,
                                       lse.data_ptr(), decay, mass.data_ptr(), out.data_ptr(), mass.shape[2], ws, nbytes,
                                       st), "octo_paged_mass")
    return out


def paged_evict(layout: api.Layout, cache: PagedCache, page_table: torch.Tensor, seq_lens: torch.Tensor,
                mass: torch.Tensor, keep: int, dst_table: torch.Tensor, sink: int = 0, recent: int = 0,
                dst: PagedCache | None = None, kept: torch.Tensor | None = None, new_lens: torch.Tensor | None = None,
                new_mass: torch.Tensor | None = None, stream=None):
    """Cuts every (sequence, head) back to ``keep`` slots: the first ``sink``, the last ``recent`` and those of the
    largest mass between them (ties: the lower slot), in their order, copied to the pages of dst_table [B][pages] (in
    ``dst``, by default the same pool; pages written must not hold tokens that the call reads). Sequences of at most
    ``keep`` slots move whole. mass float32 [B][heads][slots].

    Returns (new_lens int32 [B], kept int32 [B][heads][keep]: the slots kept, -1 behind the last; new_mass float32
    [B][heads][keep], 0 behind the last). Kept tokens keep the positions that their keys were rotated by.
    """
    dst = cache if dst is None else dst
    _check_pool(layout, cache, False)
    _check_pool(layout, dst, False)
    B, H, keep = int(seq_lens.shape[0]), cache.n_heads, int(keep)
    _ints(seq_lens, "seq_lens", (B,))
    if mass.dtype != torch.float32 or mass.dim() != 3 or tuple(mass.shape[:2]) != (B, H) or not mass.is_contiguous():
        raise ValueError(f"mass must be a contiguous float32 [{B}][{H}][slots] tensor")
    if keep < 1:
        raise ValueError(f"keep must be at least 1, got {keep}")
    dev = cache.packed.device
    if kept is None:
        kept = torch.empty((B, H, keep), dtype=torch.int32, device=dev)
    if new_lens is None:
        new_lens = torch.empty((B,), dtype=torch.int32, device=dev)
    if new_mass is None:
        new_mass = torch.empty((B, H, keep), dtype=torch.float32, device=dev)
    for t, what, shape, ty in ((kept, "kept", (B, H, keep), torch.int32), (new_lens, "new_lens", (B,), torch.int32),
                               (new_mass, "new_mass", (B, H, keep), torch.float32)):
        if t.dtype != ty or tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError(f"{what} must be a contiguous {ty} {shape} tensor")
    _same_device(dev, page_table, seq_lens, mass, dst_table, dst.packed, kept, new_lens, new_mass)
    with _On(dev, stream) as st:
        _lib.check(_lib.lib().octo_paged_evict(layout.ref, ctypes.byref(cache.c), ctypes.byref(_table(page_table, B)),
                                               seq_lens.data_ptr(), mass.data_ptr(), mass.shape[2], keep, int(sink),
                                               int(recent), ctypes.byref(dst.c), ctypes.byref(_table(dst_table, B)),
                                               kept.data_ptr(), new_lens.data_ptr(), new_mass.data_ptr(), st),
                   "octo_paged_evict")
    return new_lens, kept, new_mass
