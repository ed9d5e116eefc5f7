"""CPU tests of the paged operators' refusals: the C ABI returns a status before anything is launched, and the binding
raises ValueError for what plain pointers hide. Nothing here reaches CUDA."""

import ctypes

import numpy as np
import pytest
import torch

from rotation_preconditioned_quantization_b200 import _lib, api, paged

EINVAL, EUNS, EWS, OK = _lib.OCTO_EINVAL, _lib.OCTO_EUNSUPPORTED, _lib.OCTO_EWORKSPACE, _lib.OCTO_OK
TABS = _lib.OctoTables(256, 256, 256, 256, 256, None, 1)


def _pages(**k):
    f = dict(packed=256, gamma=256, V=256, n_pages=4, n_heads=2, page_size=16, status=None)
    f.update(k)
    return _lib.OctoPages(*f.values())


def _table(**k):
    f = dict(pages=256, stride=4, n_seqs=2, max_pages=4)
    f.update(k)
    return _lib.OctoPageTable(*f.values())


BAD_POOLS = [({"packed": None}, EINVAL), ({"gamma": None}, EINVAL), ({"n_pages": 0}, EINVAL), ({"n_heads": 0}, EINVAL),
             ({"page_size": 8}, EINVAL), ({"page_size": 24}, EINVAL), ({"V": 264}, EINVAL), ({"n_pages": 1 << 40}, EINVAL),
             ({"n_pages": 1 << 30, "n_heads": 64}, EUNS)]
BAD_TABLES = [({"pages": None}, EINVAL), ({"stride": 3}, EINVAL), ({"n_seqs": -1}, EINVAL), ({"max_pages": -1}, EINVAL),
              ({"max_pages": 1 << 28, "stride": 1 << 28}, EUNS)]


def _write(lay=None, pages=None, table=None, packed=256, gamma=256, cap=8, V=256, vr=128, vh=64, rows=4, starts=256, cu=256):
    lay = lay or api.Layout(64, 2)
    return _lib.lib().octo_paged_write(lay.ref, ctypes.byref(pages or _pages()), ctypes.byref(table or _table()), packed,
                                       gamma, cap, V, vr, vh, rows, starts, cu, None)


def _attn(lay=None, pages=None, table=None, tabs=TABS, lens=256, q=256, qd=0, qr=512, qh=64, rows=4, Hq=8, cu=256, scale=0.1,
          out=256, od=0, ws=256, wsn=1 << 40):
    lay = lay or api.Layout(64, 2)
    return _lib.lib().octo_paged_attn(lay.ref, ctypes.byref(tabs), ctypes.byref(pages or _pages()),
                                      ctypes.byref(table or _table()), lens, q, qd, qr, qh, rows, Hq, cu, 1, scale, out, od,
                                      None, ws, wsn, None)


def _mass(lay=None, pages=None, table=None, tabs=TABS, lens=256, q=256, qd=0, rows=4, Hq=8, cu=256, scale=0.1, lse=256,
          decay=1.0, m=256, out=256, stride=64, ws=256, wsn=1 << 40):
    lay = lay or api.Layout(64, 2)
    return _lib.lib().octo_paged_mass(lay.ref, ctypes.byref(tabs), ctypes.byref(pages or _pages()),
                                      ctypes.byref(table or _table()), lens, q, qd, 512, 64, rows, Hq, cu, 1, scale, lse, decay,
                                      m, out, stride, ws, wsn, None)


def _evict(lay=None, src=None, st=None, lens=256, m=256, stride=64, keep=16, sink=0, recent=0, dst=None, dt=None, kept=256,
           nl=256):
    lay = lay or api.Layout(64, 2)
    return _lib.lib().octo_paged_evict(lay.ref, ctypes.byref(src or _pages()), ctypes.byref(st or _table()), lens, m, stride,
                                       keep, sink, recent, ctypes.byref(dst or _pages()), ctypes.byref(dt or _table()), kept,
                                       nl, None, None)


@pytest.mark.parametrize("call", [_write, _attn, _mass])
def test_pools_tables_and_layouts_are_checked(call):
    for k, want in BAD_POOLS:
        assert call(pages=_pages(**k)) == want, k
    for k, want in BAD_TABLES:
        assert call(table=_table(**k)) == want, k
    assert call(lay=api.Layout(128, 4, qjl=True)) == EUNS          # the sketch has no paged form
    assert call(lay=api.Layout(128, 3, delta=0)) == EUNS           # nor have the sweep's splits
    bad = api.Layout(64, 2)
    bad.c.words += 1
    assert call(lay=bad) == EINVAL


def test_write_arguments():
    assert _write(rows=-1) == EINVAL and _write(cap=3) == EINVAL and _write(vr=-8) == EINVAL
    assert _write(vr=12) == EINVAL and _write(vh=4) == EINVAL and _write(V=264) == EINVAL   # V rows off 16 bytes
    assert _write(V=None) == EINVAL                                                         # the pool holds values
    assert _write(pages=_pages(V=None)) == EINVAL                                           # the pool holds none
    for k in ("packed", "gamma", "starts", "cu"):
        assert _write(**{k: None}) == EINVAL, k
    assert _write(rows=0, packed=None, gamma=None, starts=None, cu=None) == OK
    assert _write(table=_table(n_seqs=0)) == OK


@pytest.mark.parametrize("call", [_attn, _mass])
def test_chunk_arguments(call):
    assert call(lay=api.Layout(256, 2)) == EUNS
    assert call(tabs=_lib.OctoTables()) == EINVAL
    assert call(qd=3) == EINVAL and call(rows=-1) == EINVAL and call(Hq=7) == EINVAL and call(Hq=1) == EINVAL
    assert call(Hq=1024) == EUNS                                                            # 512 query heads per cache head
    for x in (float("nan"), float("inf")):
        assert call(scale=x) == EINVAL
    for k in ("q", "out", "lens", "cu"):
        assert call(**{k: None}) == EINVAL, k
    assert call(ws=None) == EINVAL and call(ws=264) == EINVAL and call(wsn=100) == EWS
    assert call(rows=1 << 31) == EUNS
    assert call(rows=0, q=None, out=None, lens=None, cu=None, ws=None) == OK
    assert call(table=_table(n_seqs=0)) == OK


def test_attn_and_mass_arguments():
    assert _attn(pages=_pages(V=None)) == EINVAL and _attn(od=5) == EINVAL and _attn(out=264) == EINVAL
    assert _attn(qr=-1) == EINVAL
    assert _mass(lse=None) == EINVAL and _mass(decay=float("nan")) == EINVAL and _mass(stride=-1) == EINVAL
    lay = api.Layout(64, 2)
    lib = _lib.lib()
    for f in (lib.octo_paged_attn_workspace, lib.octo_paged_mass_workspace):
        assert f(lay.ref, 4, 2, 8, 2) > 0
        assert f(api.Layout(256, 2).ref, 4, 2, 8, 2) == 0 and f(lay.ref, 4, 2, 7, 2) == 0 and f(lay.ref, -1, 2, 8, 2) == 0


def test_evict_arguments():
    for k, want in BAD_POOLS:
        assert _evict(src=_pages(**k)) == want and _evict(dst=_pages(**k)) == want, k
    for k, want in BAD_TABLES:
        assert _evict(st=_table(**k)) == want and _evict(dt=_table(**k)) == want, k
    assert _evict(keep=0) == EINVAL and _evict(sink=-1) == EINVAL and _evict(recent=-1) == EINVAL
    assert _evict(keep=10, sink=6, recent=5) == EINVAL and _evict(stride=-1) == EINVAL
    assert _evict(keep=65) == EINVAL                                                        # the destination holds 64 slots
    assert _evict(dst=_pages(n_heads=1)) == EINVAL and _evict(dst=_pages(page_size=32)) == EINVAL
    assert _evict(dst=_pages(V=None)) == EINVAL and _evict(dt=_table(n_seqs=1)) == EINVAL
    assert _evict(st=_table(n_seqs=40000), dt=_table(n_seqs=40000)) == EUNS
    for k in ("lens", "m", "kept", "nl"):
        assert _evict(**{k: None}) == EINVAL, k
    assert _evict(st=_table(n_seqs=0), dt=_table(n_seqs=0)) == OK


def test_rope_arguments():
    lib = _lib.lib()
    sec = np.array([8, 8], np.int32)

    def rope(a=None, b=None, dt=0, n=4, d=32, pos=256, ps=4, axes=2, s=sec, freqs=256):
        a = a or _lib.OctoRopeTensor(256, 256, 2, 64, 32, 64, 32)
        return lib.octo_rope(ctypes.byref(a), b, dt, n, d, pos, ps, axes, s.ctypes.data, freqs, 0, 0, None)
    assert rope(dt=4) == EINVAL and rope(n=-1) == EINVAL and rope(d=31) == EINVAL and rope(ps=3) == EINVAL
    assert rope(axes=0) == EUNS and rope(axes=5) == EUNS and rope(d=2048) == EUNS
    assert rope(d=30) == EINVAL                                    # 16 frequencies over 30 coordinates
    assert rope(s=np.array([-1, 8], np.int32)) == EINVAL
    assert rope(pos=None) == EINVAL and rope(freqs=None) == EINVAL
    assert rope(a=_lib.OctoRopeTensor(None, 256, 2, 64, 32, 64, 32)) == EINVAL
    assert rope(a=_lib.OctoRopeTensor(256, 256, -1, 64, 32, 64, 32)) == EINVAL
    assert rope(a=_lib.OctoRopeTensor(256, 256, 2, -64, 32, 64, 32)) == EINVAL
    assert rope(n=0, pos=None, freqs=None) == OK
    assert rope(a=_lib.OctoRopeTensor(None, None, 0, 0, 0, 0, 0), pos=None, freqs=None) == OK
    f = np.zeros(16, np.uint64)
    g = lib.octo_rope_freqs
    assert g(10000.0, 2, sec.ctypes.data, 0, None) == EINVAL and g(10000.0, 2, None, 0, f.ctypes.data) == EINVAL
    assert g(0.5, 2, sec.ctypes.data, 0, f.ctypes.data) == EINVAL and g(float("nan"), 2, sec.ctypes.data, 0, f.ctypes.data) == EINVAL
    assert g(10000.0, 5, sec.ctypes.data, 0, f.ctypes.data) == EUNS


@pytest.mark.parametrize("per_axis", [False, True])
@pytest.mark.parametrize("sections,theta", [((32,), 10000.0), ((12, 10, 10), 500.0), ((1,), 1.0), ((0, 5), 1e6)])
def test_rope_frequencies(sections, theta, per_axis):
    """theta^(-e) / (2 pi) in 2^-64 turns: to the rounding of 64 bits in long double, checked here to 2^-58 of a turn."""
    t = paged.RopeTable(sections, theta, per_axis, device="cpu")
    F, i, want = sum(sections), 0, []
    for s in sections:
        for j in range(s):
            e = np.longdouble(j) / s if per_axis else np.longdouble(i) / F
            want.append(np.longdouble(theta) ** -e / (2 * np.pi * np.longdouble(1)))
            i += 1
    got = t.freqs.numpy().view(np.uint64)[:F].astype(np.longdouble) / np.longdouble(2) ** 64
    assert np.all(np.abs(got - np.array(want)) <= np.longdouble(2) ** -52)  # (numpy's pi is a double)


# ---------------------------------------------------------------- the binding, on CPU tensors: refused before the call
def _cpu(H=2, d=64, b=2, page=16, pages=4, values=True):
    lay = api.Layout(d, b)
    tabs = api.DeviceTables.build(lay, 0, H, device="cpu")
    return lay, tabs, paged.PagedCache.empty(lay, pages, H, page, values=values, device="cpu")


def _i32(v):
    return torch.tensor(v, dtype=torch.int32)


def test_cache_construction():
    lay, _, c = _cpu()
    for k in ({"packed": c.packed.float()}, {"gamma": c.gamma[:1]}, {"V": c.V.float()}, {"V": c.V[:, :1]},
              {"packed": c.packed.transpose(0, 1)}):
        f = dict(packed=c.packed, gamma=c.gamma, V=c.V)
        f.update(k)
        with pytest.raises(ValueError):
            paged.PagedCache(**f)
    with pytest.raises(ValueError, match="multiple of 16"):
        paged.PagedCache.empty(lay, 2, 1, 24, device="cpu")
    with pytest.raises(ValueError, match="device"):
        paged.PagedCache(c.packed, c.gamma.to("meta"))
    flat = api.Cache.empty(lay, 4, 32, device="cpu")
    p = paged.PagedCache.from_cache(flat, None, 2)
    assert (p.n_pages, p.n_heads, p.page_size) == (2, 2, 32) and p.packed.data_ptr() == flat.packed.data_ptr()
    with pytest.raises(ValueError, match="pages of"):
        paged.PagedCache.from_cache(flat, None, 3)
    with pytest.raises(ValueError, match="pages of"):
        paged.PagedCache.from_cache(api.Cache.empty(lay, 4, 20, device="cpu"), None, 2)


def test_binding_refuses_shapes_types_and_devices():
    lay, tabs, c = _cpu()
    q, lens, table = torch.zeros(4, 4, 64), _i32([5, 6]), _i32([[0, 1], [2, 3]])
    attn = lambda q=q, lens=lens, table=table, lay=lay, c=c, **k: paged.paged_attn(lay, tabs, q, c, table, lens, **k)  # noqa: E731
    for bad, match in ((dict(q=q.half()), "dtype"), (dict(q=q[:, :3]), "heads"), (dict(q=q[..., :32]), "q must be"),
                       (dict(q=q.transpose(1, 2)), "q must be"), (dict(lens=lens.long()), "seq_lens"),
                       (dict(table=table[:1]), "page_table"), (dict(table=table.long()), "page_table"),
                       (dict(q=q[:3]), "cu_q"), (dict(cu_q=_i32([0, 4])), "cu_q"), (dict(lay=api.Layout(128, 2)), "words"),
                       (dict(out=torch.zeros(4, 4, 32)), "out"), (dict(out=torch.zeros(4, 4, 64), dtype=torch.bfloat16), "out"),
                       (dict(dtype=torch.float16), "dtype"), (dict(lse=torch.zeros(4)), "lse"), (dict(), "CUDA"),
                       (dict(c=_cpu(values=False)[2]), "no values")):
        with pytest.raises(ValueError, match=match):
            attn(**bad)
    lse, m = torch.zeros(4, 4), torch.zeros(2, 2, 32)
    mass = lambda lse=lse, m=m, **k: paged.paged_mass(lay, tabs, q, lse, c, table, lens, m, **k)  # noqa: E731
    buf = torch.zeros(200)
    for bad, match in ((dict(lse=lse[:3]), "lse"), (dict(m=m[:1]), "mass"), (dict(m=m.double()), "mass"),
                       (dict(out=torch.zeros(2, 2, 31)), "out"),
                       (dict(m=buf[:128].view(2, 2, 32), out=buf[8:136].view(2, 2, 32)), "overlap"), (dict(), "CUDA")):
        with pytest.raises(ValueError, match=match):
            mass(**bad)
    ev = lambda m=m, keep=16, dst=table, **k: paged.paged_evict(lay, c, table, lens, m, keep, dst, **k)  # noqa: E731
    for bad, match in ((dict(m=m[:, :1]), "mass"), (dict(keep=0), "keep"), (dict(dst=table[:1]), "dst_table"),
                       (dict(kept=torch.zeros(2, 2, 16)), "kept"), (dict(new_lens=_i32([1])), "new_lens"),
                       (dict(new_mass=torch.zeros(2, 2, 8)), "new_mass"), (dict(), "CUDA")):
        with pytest.raises(ValueError, match=match):
            ev(**bad)
    st, V = api.Cache.empty(lay, 2, 8, device="cpu"), torch.zeros(6, 2, 64, dtype=torch.bfloat16)
    wr = lambda st=st, V=V, starts=lens, cu=_i32([0, 3, 6]), **k: paged.paged_write(lay, st, V, c, table, starts, cu, **k)  # noqa: E731
    for bad, match in ((dict(V=V.float()), "V must"), (dict(V=V[:, :1]), "V must"), (dict(V=None), "V is needed"),
                       (dict(V=torch.zeros(6 * 2 * 66, dtype=torch.bfloat16).view(6, 2, 66)[..., :64]), "16-byte"),
                       (dict(V=torch.zeros(9, 2, 64, dtype=torch.bfloat16)), "staged"), (dict(cu=_i32([0, 6])), "cu"),
                       (dict(starts=lens.long()), "starts"), (dict(st=api.Cache.empty(lay, 1, 8, device="cpu")), "staged"),
                       (dict(), "CUDA")):
        with pytest.raises(ValueError, match=match):
            wr(**bad)
    with pytest.raises(ValueError, match="keys must"):
        paged.paged_append(lay, tabs, torch.zeros(6, 3, 64), V, c, table, lens, _i32([0, 3, 6]))


def test_rope_binding_refuses():
    t = paged.RopeTable((16,), device="cpu")
    q, p = torch.zeros(4, 2, 32), torch.zeros(1, 4, dtype=torch.int32)
    for bad, match in ((dict(q=q.half()), "q must"), (dict(q=q[0]), "q must"), (dict(p=p.long()), "positions"),
                       (dict(p=p[:, :3]), "positions"), (dict(k=torch.zeros(4, 1, 16)), "k must"),
                       (dict(k=torch.zeros(3, 1, 32)), "k must"), (dict(q=q.transpose(1, 2)), "contiguous"),
                       (dict(out=torch.zeros(4, 2, 16)), "out"), (dict(), "CUDA")):
        f = dict(q=q, p=p)
        f.update(bad)
        with pytest.raises(ValueError, match=match):
            paged.rope(f.pop("q"), f.pop("p"), t, **f)
    buf = torch.zeros(4 * 2 * 32 + 32)
    with pytest.raises(ValueError, match="overlap"):
        paged.rope(buf[:256].view(4, 2, 32), p, t, out=buf[32:].view(4, 2, 32))
    with pytest.raises(_lib.OctoError):
        paged.RopeTable((16,), theta=0.1, device="cpu")


def test_attn_refuses_an_output_over_its_queries():
    lay, tabs, c = _cpu()
    buf = torch.zeros(5 * 4 * 64)
    for at in (0, 64):
        with pytest.raises(ValueError, match="overlap"):
            paged.paged_attn(lay, tabs, buf[:1024].view(4, 4, 64), c, _i32([[0, 1], [2, 3]]), _i32([5, 6]),
                             out=buf[at:at + 1024].view(4, 4, 64))


def test_evict_refuses_a_new_mass_over_the_mass():
    lay, _, c = _cpu()
    buf = torch.zeros(2 * 2 * 32 + 16)
    with pytest.raises(ValueError, match="overlap"):
        paged.paged_evict(lay, c, _i32([[0, 1], [2, 3]]), _i32([5, 6]), buf[:128].view(2, 2, 32), 16,
                          _i32([[0, 1], [2, 3]]), new_mass=buf[64:128].view(2, 2, 16))


def test_expanded_views_are_refused():
    """One row read as many has no stride that the C ABI can take: it would be read beyond its end."""
    lay, tabs, c = _cpu()
    q, lens = torch.zeros(4, 4, 64), _i32([5, 6])
    with pytest.raises(ValueError, match="page_table must not be an expanded"):
        paged.paged_attn(lay, tabs, q, c, _i32([[0, 1]]).expand(2, 2), lens)
    with pytest.raises(ValueError, match="dst_table must not be an expanded"):
        paged.paged_evict(lay, c, _i32([[0, 1], [2, 3]]), lens, torch.zeros(2, 2, 32), 16, _i32([[0, 1]]).expand(2, 2))
    t = paged.RopeTable((4, 4), device="cpu")
    with pytest.raises(ValueError, match="positions must not be an expanded"):
        paged.rope(q, torch.zeros(1, 4, dtype=torch.int32).expand(2, 4), t)
    with pytest.raises(ValueError, match="out must not be an expanded"):
        paged.rope(q, torch.zeros(2, 4, dtype=torch.int32), t, out=torch.zeros(4, 1, 64).expand(4, 4, 64))
