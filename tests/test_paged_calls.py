"""CPU tests of the paged operators' calls: what is refused, and what is not, before anything reaches CUDA."""

import ctypes
import os
import re

import numpy as np
import pytest
import torch

from rotation_preconditioned_quantization_b200 import _lib, api, paged

EINVAL, EUNS, OK = _lib.OCTO_EINVAL, _lib.OCTO_EUNSUPPORTED, _lib.OCTO_OK


def _i32(v):
    return torch.tensor(v, dtype=torch.int32)


def _cpu(H=2, d=64, b=2, page=16, pages=4):
    lay = api.Layout(d, b)
    return lay, api.DeviceTables.build(lay, 0, H, device="cpu"), paged.PagedCache.empty(lay, pages, H, page, device="cpu")


def test_no_wait_of_the_paged_kernels_is_unbounded():
    """Roles that give up a bounded wait leave the others: within the roles nothing may wait without a limit, so no
    barrier of named threads, and every poll of an mbarrier is in the bounded loop."""
    src = os.path.join(os.path.dirname(paged.__file__), "csrc")
    for name in ("octo_paged.cuh", "octo_paged_attn.cu", "octo_paged_mass.cu"):
        text = open(os.path.join(src, name)).read()
        assert not re.search(r"\bbar(rier)?\.(sync|red)|named_sync", text), name
        assert len(re.findall(r"mbarrier\.(try|test)_wait", text)) == (1 if name == "octo_paged.cuh" else 0)
        roles = re.findall(r"__device__ __forceinline__ bool \w+_role\(.*?\n}\n", text, re.S)
        assert all("__syncthreads" not in r for r in roles)
    wait = open(os.path.join(src, "octo_paged.cuh")).read().split("bool bar_wait(")[1].split("\n}\n")[0]
    assert re.search(r"it < \(1 << \d+\)", wait) and "while" not in wait


@pytest.mark.parametrize("d", [64, 128])
def test_paged_scratch_lies_behind_the_words_that_decode_keeps(d):
    """octo_decode_attn's status word and the arrival counters of its at most 65535 cache heads come first."""
    lib, lay = _lib.lib(), api.Layout(d, 3)
    front = 256 + 4 * 65535
    assert lib.octo_paged_attn_workspace(lay.ref, 1, 1, 1, 1) >= front + 148 * 3 * 256 * d * 4
    assert lib.octo_paged_mass_workspace(lay.ref, 64, 1, 1, 1) >= front + 64 * d * 4


def _calls():
    """Each wrapped call with arguments that the device check refuses, up to `stream` by position and by keyword."""
    lay, tabs, c = _cpu()
    q, lens, table = torch.zeros(4, 4, 64), _i32([5, 6]), _i32([[0, 1], [2, 3]])
    m, lse = torch.zeros(2, 2, 32), torch.zeros(4, 4)
    V = torch.zeros(6, 2, 64, dtype=torch.bfloat16)
    return {
        "rope": (paged.rope, [q, torch.zeros(1, 4, dtype=torch.int32), paged.RopeTable((16,), device="cpu")], [None, False, False, None, None]),
        "paged_append": (paged.paged_append, [lay, tabs, torch.zeros(6, 2, 64), V, c, table, lens, _i32([0, 3, 6])], [None]),
        "paged_attn": (paged.paged_attn, [lay, tabs, q, c, table, lens], [None, True, None, None, None, None, None]),
        "paged_mass": (paged.paged_mass, [lay, tabs, q, lse, c, table, lens, m], [None, True, None, 1.0, None, None]),
        "paged_evict": (paged.paged_evict, [lay, c, table, lens, m, 16, table], [0, 0, None, None, None, None]),
    }


@pytest.mark.parametrize("name", ["rope", "paged_append", "paged_attn", "paged_mass", "paged_evict"])
def test_stream_is_current_within_the_call_however_it_is_passed(name, monkeypatch):
    class Entered(Exception):
        pass

    class Stream:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            raise Entered(self.s)

        def __exit__(self, *a):
            return False

    monkeypatch.setattr(torch.cuda, "stream", Stream)
    f, args, rest = _calls()[name]
    side = object()
    with pytest.raises(Entered) as e:
        f(*args, stream=side)
    assert e.value.args[0] is side
    with pytest.raises(Entered) as e:
        f(*args, *rest, side)
    assert e.value.args[0] is side
    for a, kw in ((args, {}), (args, {"stream": None}), (args + rest + [None], {})):
        with pytest.raises(ValueError, match="CUDA"):
            f(*a, **kw)


def test_writing_no_rows_needs_no_addresses():
    """torch gives an empty tensor the address 0: with no rows, V says nothing about the pool's values."""
    lay = api.Layout(64, 2)
    pages, table = _lib.OctoPages(256, 256, 256, 4, 2, 16, None), _lib.OctoPageTable(256, 4, 2, 4)
    f = _lib.lib().octo_paged_write
    assert f(lay.ref, ctypes.byref(pages), ctypes.byref(table), 256, 256, 8, None, 128, 64, 0, 256, 256, None) == OK
    assert f(lay.ref, ctypes.byref(pages), ctypes.byref(table), 256, 256, 8, None, 128, 64, 4, 256, 256, None) == EINVAL


def test_a_pool_describes_the_tensors_that_it_holds_now():
    lay, tabs, c = _cpu(pages=4)
    big = paged.PagedCache.empty(lay, 9, 2, 32, device="cpu")
    c.packed, c.gamma, c.V = big.packed, big.gamma, big.V
    now = c.ref._obj
    assert (now.packed, now.gamma, now.V, now.n_pages, now.page_size) == (big.packed.data_ptr(), big.gamma.data_ptr(),
                                                                          big.V.data_ptr(), 9, 32)
    assert (c.n_pages, c.n_heads, c.page_size) == (9, 2, 32)
    c.V = None
    assert c.ref._obj.V is None
    c.status = torch.zeros(1, dtype=torch.int32)
    assert c.ref._obj.status == c.status.data_ptr()
    c.gamma = c.gamma[:3]  # no pool's: refused where it is used
    with pytest.raises(ValueError, match="gamma"):
        paged.paged_attn(lay, tabs, torch.zeros(2, 2, 64), c, _i32([[0], [1]]), _i32([5, 6]))


@pytest.mark.parametrize("d,b", [(128, 2), (64, 3), (64, 4)])
def test_tables_of_another_layout_are_refused(d, b):
    """Codebooks and sign rows of another d or b would be read past their end."""
    lay, own, c = _cpu()
    tabs = api.DeviceTables.build(api.Layout(d, b), 0, 2, device="cpu")
    q, lens, table, V = torch.zeros(4, 4, 64), _i32([5, 6]), _i32([[0, 1], [2, 3]]), torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    flat = api.Cache.empty(lay, 2, 16, device="cpu")
    for t, match in ((tabs, "tables"), (own, "CUDA")):
        with pytest.raises(ValueError, match=match):
            paged.paged_attn(lay, t, q, c, table, lens)
        with pytest.raises(ValueError, match=match):
            paged.paged_mass(lay, t, q, torch.zeros(4, 4), c, table, lens, torch.zeros(2, 2, 32))
    for f in (lambda: api.encode(lay, tabs, torch.zeros(2, 4, 64), flat),
              lambda: api.dequant(lay, tabs, flat, 4),
              lambda: api.decode_attn(lay, tabs, torch.zeros(1, 4, 1, 64), flat, None, 2, kv_len=4, logits=True)):
        with pytest.raises(ValueError, match="tables"):
            f()


def test_sketch_matrices_of_other_heads_are_refused():
    lay = api.Layout(64, 3, qjl=True)
    tabs = api.DeviceTables.build(lay, 0, 4, device="cpu")
    tabs.qjl_S = tabs.qjl_S[:2]
    with pytest.raises(ValueError, match="tables"):
        api.encode(lay, tabs, torch.zeros(4, 4, 64), api.Cache.empty(lay, 4, 16, device="cpu"))
    lay = api.Layout(64, 3)
    for k in ("dir_t", "rho_t"):
        tabs = api.DeviceTables.build(lay, 0, 4, device="cpu")
        setattr(tabs, k, getattr(tabs, k)[:2])
        with pytest.raises(ValueError, match="tables"):
            api.encode(lay, tabs, torch.zeros(4, 4, 64), api.Cache.empty(lay, 4, 16, device="cpu"))


def test_rope_outputs_over_the_other_tensor_are_refused():
    """Both tensors turn in one launch: an output over the other's input, or over the other output, would race."""
    t, p = paged.RopeTable((16,), device="cpu"), torch.zeros(1, 4, dtype=torch.int32)
    buf = torch.zeros(4, 8, 32)
    a, b, c = buf[:, :2], buf[:, 2:4], buf[:, 4:6]
    for kw, match in ((dict(out=b), "overlap"), (dict(k_out=a), "overlap"), (dict(out=b, k_out=a), "overlap"),
                      (dict(out=c, k_out=c), "overlap"), (dict(out=c, k_out=buf[:, 5:7]), "overlap"),
                      (dict(out=buf[:, 1:3]), "overlap"),
                      (dict(out=a, k_out=b), "CUDA"), (dict(out=c, k_out=buf[:, 6:]), "CUDA"), (dict(out=c), "CUDA"),
                      (dict(), "CUDA")):
        with pytest.raises(ValueError, match=match):
            paged.rope(a, p, t, k=b, **kw)
    one = torch.zeros(4, 1, 32)
    with pytest.raises(ValueError, match="overlap"):
        paged.rope(buf[:, :2], p, t, out=buf.view(-1)[32:288].view(4, 2, 32))  # other strides over the same rows
    with pytest.raises(ValueError, match="CUDA"):
        paged.rope(one, p, t, k=one.clone(), out=one)
    with pytest.raises(ValueError, match="CUDA"):
        paged.rope(a, p, t, k=a)  # one input given twice is only read


def test_views_that_may_share_memory():
    """Views called apart share no element; and those of a fused buffer, by heads or between them, are called apart."""
    rng = np.random.default_rng(3)
    buf = torch.zeros(4000)
    apart = 0
    for _ in range(3000):
        v = []
        for _ in range(2):
            n, h, d = (int(rng.integers(1, k)) for k in (5, 4, 9))
            sh = int(rng.integers(d, 3 * d + 1))
            s = int(rng.integers(1, 4)) * sh * int(rng.integers(1, 5))
            v.append(buf.as_strided((n, h, d), (s, sh, 1), int(rng.integers(0, 200))))
        cells = [set((t.storage_offset() + np.add.outer(np.add.outer(np.arange(t.shape[0]) * t.stride(0),
                      np.arange(t.shape[1]) * t.stride(1)), np.arange(t.shape[2]))).ravel().tolist()) for t in v]
        if not paged._meet(*v):
            apart += 1
            assert not cells[0] & cells[1], [(t.shape, t.stride(), t.storage_offset()) for t in v]
    assert apart > 300
    x = torch.zeros(5, 12, 16)
    for a, b in ((x[:, :8], x[:, 8:]), (x[:, 0::2], x[:, 1::2]), (x[..., :8], x[..., 8:]), (x[:1, :8], x[:1, 8:]), (x[:2], x[2:])):
        assert not paged._meet(a, b) and not paged._meet(b, a) and paged._meet(a, a)


def test_a_status_word_is_one_int32():
    lay, _, c = _cpu()
    for s in (torch.zeros(0, dtype=torch.int32), torch.zeros(1), torch.zeros(1, dtype=torch.int64), torch.zeros(4, dtype=torch.uint8),
              torch.zeros((), dtype=torch.int16)):
        with pytest.raises(ValueError, match="status"):
            paged.PagedCache(c.packed, c.gamma, c.V, s)
    for s in (torch.zeros(1, dtype=torch.int32), torch.zeros((), dtype=torch.int32)):
        assert paged.PagedCache(c.packed, c.gamma, c.V, s).status is s


@pytest.mark.parametrize("page,slots,want", [(16, 2 ** 31 - 1 - 1024 - 15, EUNS), (16, 2 ** 31 - 65536, EUNS), (16, 2 ** 31 - 65552, OK),
                                             (1 << 20, 2 ** 31 - (1 << 20), OK)])
def test_slots_leave_room_for_rounded_up_tiles(page, slots, want):
    """Slot numbers are 32-bit, and the kernels round them up to the tiles and clusters that share them."""
    n = slots // page
    lay, pages, table = api.Layout(64, 2), _lib.OctoPages(256, 256, 256, 4, 2, page, None), _lib.OctoPageTable(256, n, 0, n)
    p, t = ctypes.byref(pages), ctypes.byref(table)
    lib = _lib.lib()
    assert lib.octo_paged_write(lay.ref, p, t, 256, 256, 8, 256, 128, 64, 4, 256, 256, None) == want
    assert lib.octo_paged_evict(lay.ref, p, t, 256, 256, 64, 16, 0, 0, p, t, 256, 256, None, None) == want


def test_lengths_that_may_be_replaced_in_place_are_not_read_as_read_only():
    """new_lens may be seq_lens: the launch that writes the one must not read the other through the read-only path."""
    text = open(os.path.join(os.path.dirname(paged.__file__), "csrc", "octo_paged_move.cu")).read()
    body = text[text.index("paged_gather_kernel("):]
    assert not re.search(r"(load_now|__ldg)\(a\.seq_lens", body[:body.index("\n}\n")])


def test_a_workspace_keeps_the_buffers_that_captured_calls_hold():
    ws = api.Workspace(1 << 12, device="cpu")
    first = ws.buf
    ws.ensure(1 << 13)
    assert ws.nbytes == 1 << 13 and not ws._replaced  # no call was captured: nothing is kept
    ws._captured = True
    held = ws.buf
    assert ws.ensure(1 << 12) is ws and ws.buf is held
    ws.ensure(1 << 14)
    assert ws._replaced == [held] and ws.buf is not held and ws.buf is not first and ws.nbytes == 1 << 14
    ws.ensure(1 << 15)
    assert ws._replaced == [held]


def test_new_lengths_over_a_part_of_the_old_are_refused():
    lay, _, c = _cpu()
    buf, table = torch.tensor([5, 6, 7], dtype=torch.int32), _i32([[0, 1], [2, 3]])
    ev = lambda a, b: paged.paged_evict(lay, c, table, a, torch.zeros(2, 2, 32), 16, table, new_lens=b)  # noqa: E731
    for a, b in ((buf[:2], buf[1:]), (buf[1:], buf[:2])):
        with pytest.raises(ValueError, match="overlap"):
            ev(a, b)
    for a, b in ((buf[:2], buf[:2]), (buf[:2], buf[:2].clone())):
        with pytest.raises(ValueError, match="CUDA"):
            ev(a, b)
    pages, tab = _lib.OctoPages(256, 256, 256, 4, 2, 16, None), _lib.OctoPageTable(256, 4, 2, 4)
    for lens, new in ((256, 260), (260, 256)):
        assert _lib.lib().octo_paged_evict(lay.ref, ctypes.byref(pages), ctypes.byref(tab), lens, 512, 64, 16, 0, 0,
                                           ctypes.byref(pages), ctypes.byref(tab), 1024, new, None, None) == EINVAL


@pytest.mark.parametrize("name", ["dequant", "decode_attn"])
def test_stream_is_current_within_the_contiguous_calls_too(name, monkeypatch):
    """Outputs and workspaces (zeroed) that they make belong to the stream that uses them."""
    class Entered(Exception):
        pass

    class Stream:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            raise Entered(self.s)

        def __exit__(self, *a):
            return False

    lay, tabs, _ = _cpu()
    flat = api.Cache.empty(lay, 2, 16, device="cpu")
    f, args, rest = {"dequant": (api.dequant, [lay, tabs, flat], [4, 0, None, torch.float32, None]),
                     "decode_attn": (api.decode_attn, [lay, tabs, torch.zeros(1, 4, 1, 64), flat, None, 2],
                                     [4, None, None, True, None])}[name]
    monkeypatch.setattr(torch.cuda, "stream", Stream)
    side = object()
    for a, kw in ((args, {"stream": side}), (args + rest + [side], {})):
        with pytest.raises(Entered) as e:
            f(*a, **kw)
        assert e.value.args[0] is side
    with pytest.raises(ValueError, match="CUDA"):
        f(*args, *rest)


def test_calls_run_on_the_tensors_device(monkeypatch):
    """With another device current, a call is made with the tensors' one current, on its stream."""
    now, seen = [0], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            now[0], self.index = self.index, now[0]

        def __exit__(self, *a):
            now[0], self.index = self.index, now[0]

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(api, "_current_device", lambda: now[0])
    monkeypatch.setattr(api, "_raw_stream", lambda index: 1000 + index)
    for index in (0, 3):
        api._on(index, None, lambda s: seen.append((now[0], s)))
    assert seen == [(0, 1000), (3, 1003)] and now == [0]
    with pytest.raises(ValueError, match="CUDA"):
        api._on(-1, None, None)
    lay, tabs, _ = _cpu()  # and all three calls of the contiguous cache go that way
    flat, asked = api.Cache.empty(lay, 2, 16, device="cpu"), []
    monkeypatch.setattr(api, "_on", lambda index, stream, call: asked.append(index) or _lib.OCTO_OK)
    api.encode(lay, tabs, torch.zeros(2, 4, 64), flat)
    api.dequant(lay, tabs, flat)
    api.decode_attn(lay, tabs, torch.zeros(1, 4, 1, 64), flat, None, 2, logits=True)
    assert asked == [-1] * 3
