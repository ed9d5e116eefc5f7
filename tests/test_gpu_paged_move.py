"""GPU tests of octo_paged_write and octo_paged_evict: values are moved, so everything is compared bit for bit."""

import numpy as np
import pytest
import torch

from rotation_preconditioned_quantization_b200 import api, inputs, paged

from . import paged_ref as pr

pytestmark = pytest.mark.gpu


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _bits(t):
    return t.view(torch.int16) if t.dtype == torch.bfloat16 else t.view(torch.int32)


def _snapshot(c):
    return [x.clone() if x is not None else None for x in (c.packed, c.gamma, c.V)]


def _same(c, want):
    for x, y in zip((c.packed, c.gamma, c.V), want):
        if x is not None:
            assert torch.equal(_bits(x), _bits(y))


@pytest.mark.parametrize("d,b", [(64, 2), (128, 3), (128, 4), (256, 3)])
@pytest.mark.parametrize("page,old,new", [(16, [0, 5, 16, 100], [3, 0, 33, 1]), (48, [47, 0], [2, 97]),
                                          (64, [63] * 20, [1] * 20), (256, [10], [1])])
def test_write_places_every_token(cuda_ok, d, b, page, old, new):
    lay, H = api.Layout(d, b), 3
    g = torch.Generator("cuda").manual_seed(1)
    counts = [-(-(a + z) // page) for a, z in zip(old, new)]
    n_pages = sum(counts) + 2
    cache = paged.PagedCache.empty(lay, n_pages, H, page)
    cache.packed.random_(-2 ** 31, 2 ** 31 - 1, generator=g)
    order = torch.randperm(n_pages, generator=g, device="cuda").tolist()
    table, at = np.full((len(old), max(counts)), -1, np.int32), 0
    for i, n in enumerate(counts):
        table[i, :n] = order[at:at + n]
        at += n
    rows = sum(new)
    staged = api.Cache.empty(lay, H, rows)
    staged.packed.random_(-2 ** 31, 2 ** 31 - 1, generator=g)
    staged.gamma.uniform_(generator=g)
    V = torch.randn(rows, 2, H, d, generator=g, device="cuda").to(torch.bfloat16)[:, 1]  # strided rows
    want = _snapshot(cache)
    cu = np.concatenate([[0], np.cumsum(new)])
    for i in range(len(old)):
        for t in range(new[i]):
            s, r = old[i] + t, cu[i] + t
            p, o = table[i, s // page], s % page
            want[0][p, :, :, o] = staged.packed[:, :, r]
            want[1][p, :, o] = staged.gamma[:, r]
            want[2][p, :, o] = V[r]
    paged.paged_write(lay, staged, V, cache, torch.from_numpy(table).cuda(), _i32(old), _i32(cu))
    torch.cuda.synchronize()
    cache.check()
    _same(cache, want)


def test_write_keys_only_and_no_rows(cuda_ok):
    lay = api.Layout(64, 2)
    cache = paged.PagedCache.empty(lay, 2, 2, 16, values=False)
    staged = api.Cache.empty(lay, 2, 8)
    staged.gamma.fill_(2.0)
    staged.length = 5
    paged.paged_write(lay, staged, None, cache, _i32([[1]]), _i32([3]), _i32([0, 5]))
    torch.cuda.synchronize()
    assert cache.gamma[1, :, 3:8].eq(2).all() and cache.gamma.sum() == 2 * 2 * 5
    staged.length = 0
    paged.paged_write(lay, staged, None, cache, _i32([[1]]), _i32([3]), _i32([0, 0]))
    cache.check()


def test_write_drops_and_reports_what_has_no_place(cuda_ok):
    lay = api.Layout(64, 2)
    cache = paged.PagedCache.empty(lay, 2, 1, 16)
    staged = api.Cache.empty(lay, 1, 8)
    staged.gamma.fill_(3.0)
    V = torch.ones(8, 1, 64, dtype=torch.bfloat16, device="cuda")
    # slots 12..19 of a sequence with one page: the last four have none
    paged.paged_write(lay, staged, V, cache, _i32([[0]]), _i32([12]), _i32([0, 8]))
    torch.cuda.synchronize()
    assert cache.gamma[0, 0, 12:].eq(3).all() and cache.gamma.sum() == 12
    with pytest.raises(RuntimeError, match="length"):
        cache.check()
    for page in (-1, 2, 1 << 30):
        paged.paged_write(lay, staged, V, cache, _i32([[page]]), _i32([0]), _i32([0, 8]))
        with pytest.raises(RuntimeError, match="page id"):
            cache.check()
    assert cache.gamma.sum() == 12
    # rows outside every sequence, and a negative start
    paged.paged_write(lay, staged, V, cache, _i32([[0]]), _i32([0]), _i32([6, 8]))
    with pytest.raises(RuntimeError, match="length"):
        cache.check()
    assert cache.gamma[0, 0, :2].eq(3).all() and cache.gamma.sum() == 18
    paged.paged_write(lay, staged, V, cache, _i32([[0]]), _i32([-9]), _i32([0, 8]))
    with pytest.raises(RuntimeError, match="length"):
        cache.check()
    assert cache.gamma.sum() == 18


def test_append_is_encode_and_write(cuda_ok):
    d, b, H, page = 128, 3, 2, 16
    lay = api.Layout(d, b)
    tabs = api.DeviceTables.build(lay, 1, H)
    new, old = [20, 1, 7], [3, 15, 0]
    keys = torch.from_numpy(inputs.llm_keys(1, 1, 28 * H, d)[0].reshape(28, H, d)).to(torch.bfloat16).cuda()
    V = torch.randn(28, H, d, device="cuda").to(torch.bfloat16)
    cache = paged.PagedCache.empty(lay, 6, H, page)
    table = _i32([[0, 1], [2, -1], [4, -1]])
    paged.paged_append(lay, tabs, keys, V, cache, table, _i32(old), _i32([0, 20, 21, 28]))
    torch.cuda.synchronize()
    cache.check()
    whole = api.Cache.empty(lay, H, 28)
    api.encode(lay, tabs, keys.transpose(0, 1), whole)
    r = 0
    for i in range(3):
        for t in range(new[i]):
            s = old[i] + t
            p, o = int(table[i, s // page]), s % page
            assert torch.equal(cache.packed[p, :, :, o], whole.packed[:, :, r])
            assert torch.equal(cache.gamma[p, :, o], whole.gamma[:, r]) and torch.equal(cache.V[p, :, o], V[r])
            r += 1


def _evict(seed, d, b, page, H, lens, keep, sink, recent, mass=None, slots=None, other=False, values=True):
    pool = pr.Pool(seed, d, b, page, H, lens, spare=2 + len(lens) * -(-keep // page), device=None, stale=0.5)
    if not values:
        pool.V = None
    slots = max(lens) + 3 if slots is None else slots
    rng = np.random.default_rng(seed)
    if mass is None:
        mass = rng.lognormal(-3, 2, (len(lens), H, slots)).astype(np.float32)
        mass[rng.random(mass.shape) < 0.3] = 0.0
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    cache = paged.PagedCache(t(pool.words.view(np.int32)), t(pool.gamma), None if not values else t(pool.V).to(torch.bfloat16))
    into = cache if not other else paged.PagedCache(torch.full_like(cache.packed, 7), torch.full_like(cache.gamma, 7),
                                                    torch.full_like(cache.V, 7) if values else None)
    per = -(-keep // page)
    dst = np.asarray(pool.free[:len(lens) * per], np.int32).reshape(len(lens), per)
    src, want = _snapshot(cache), _snapshot(into)
    new_lens, kept, new_mass = paged.paged_evict(pool.lay, cache, t(pool.table), _i32(lens), t(mass), keep, t(dst), sink=sink,
                                                 recent=recent, dst=into)
    torch.cuda.synchronize()
    cache.check()
    into.check()
    assert new_lens.tolist() == [min(n, keep) for n in lens]
    for i, n in enumerate(lens):
        for h in range(H):
            s = pr.select(mass[i, h], n, keep, sink, recent)
            k = kept[i, h].cpu().numpy()
            assert np.array_equal(k[:len(s)], s) and np.all(k[len(s):] == -1), (i, h)
            m = new_mass[i, h].cpu().numpy()
            assert np.array_equal(m[:len(s)], mass[i, h, s], equal_nan=True) and np.all(m[len(s):] == 0)
            z = np.arange(len(s))
            a, ao = torch.from_numpy(pool.table[i, s // page].astype(np.int64)).cuda(), torch.from_numpy(s % page).cuda()
            c, co = torch.from_numpy(dst[i, z // page].astype(np.int64)).cuda(), torch.from_numpy(z % page).cuda()
            want[0][c, h, :, co] = src[0][a, h, :, ao]
            want[1][c, h, co] = src[1][a, h, ao]
            if values:
                want[2][c, h, co] = src[2][a, h, ao]
    _same(into, want)


@pytest.mark.parametrize("d,b", [(64, 2), (64, 4), (128, 3), (256, 2)])
def test_evict_every_layout(cuda_ok, d, b):
    _evict(d + b, d, b, 32, 2, [300, 90], 64, 4, 16)


@pytest.mark.parametrize("lens,keep,sink,recent", [
    ([1], 1, 0, 0), ([2], 1, 0, 0), ([2], 1, 1, 0), ([2], 1, 0, 1), ([5, 0, 3], 3, 1, 1), ([33], 32, 0, 0), ([33], 32, 16, 16),
    ([1000], 999, 0, 0), ([1000], 1, 0, 0), ([1025, 1024, 1023], 100, 10, 20), ([5000], 77, 0, 77), ([5000], 77, 77, 0),
    ([40, 20, 64, 65], 64, 3, 7)])
@pytest.mark.parametrize("page", [16, 48])
def test_evict_sizes(cuda_ok, lens, keep, sink, recent, page):
    _evict(len(lens) + keep, 64, 2, page, 3, lens, keep, sink, recent)


def test_evict_long(cuda_ok):
    _evict(3, 64, 2, 256, 1, [100001], 30011, 4, 1000)


@pytest.mark.parametrize("slots", [4096, 4097, 139904, 139905])
def test_evict_at_the_bounds_of_its_variants(cuda_ok, slots):
    """One block or four per head, ordered bits held in shared memory or read again: the choice goes by the table's slots."""
    _evict(slots, 64, 2, 256, 1, [slots - 1, 300], 257, 3, 50, slots=slots, values=False)


def test_evict_into_another_pool_and_keys_only(cuda_ok):
    _evict(4, 128, 3, 64, 2, [500, 10], 200, 2, 30, other=True)
    _evict(5, 128, 3, 64, 2, [500, 10], 200, 2, 30, values=False)


@pytest.mark.parametrize("kind", ["equal", "signed", "extremes", "low_bits"])
def test_evict_ranks_every_float(cuda_ok, kind):
    rng = np.random.default_rng(6)
    n = 3001
    if kind == "equal":
        m = np.full((1, 2, n), 0.25, np.float32)
    elif kind == "signed":
        m = rng.standard_normal((1, 2, n)).astype(np.float32)
    elif kind == "extremes":  # NaN, infinities, zeros of both signs, subnormals
        m = rng.choice(np.array([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-42, -1e-42, 3.4e38, 1.0], np.float32), (1, 2, n))
    else:  # values that differ in the last bits only
        m = (np.float32(1.0).view(np.int32) + rng.integers(0, 4, (1, 2, n))).astype(np.int32).view(np.float32)
    for keep in (1, 500, 1500, 3000):
        _evict(7 + keep, 64, 2, 64, 2, [n], keep, 0, 0, mass=np.ascontiguousarray(m), slots=n)


def test_evict_reports_lengths_beyond_the_mass_and_bad_pages(cuda_ok):
    lay = api.Layout(64, 2)
    cache = paged.PagedCache.empty(lay, 8, 1, 16)
    cache.gamma.fill_(1.0)
    table, dst = _i32([[0, 1, 2]]), _i32([[4]])
    lens, kept, _ = paged.paged_evict(lay, cache, table, _i32([48]), torch.ones(1, 1, 20, device="cuda"), 16, dst)
    assert int(lens[0]) == 16 and kept[0, 0].tolist() == list(range(16))
    with pytest.raises(RuntimeError, match="length"):
        cache.check()
    bad = _i32([[0, 99, 2]])
    m = torch.zeros(1, 1, 48, device="cuda")
    m[..., 16:32] = 1.0
    paged.paged_evict(lay, cache, bad, _i32([48]), m, 16, dst)
    with pytest.raises(RuntimeError, match="page id"):
        cache.check()
    assert cache.gamma[4].eq(0).all()  # tokens without a source
    paged.paged_evict(lay, cache, table, _i32([48]), m, 16, _i32([[-5]]))
    with pytest.raises(RuntimeError, match="page id"):
        cache.check()


def test_evict_graph_replay(cuda_ok):
    lay = api.Layout(64, 2)
    cache = paged.PagedCache.empty(lay, 8, 2, 16)
    cache.gamma.uniform_()
    table, dst, lens = _i32([[0, 1, 2]]), _i32([[4, 5]]), _i32([40])
    mass = torch.rand(1, 2, 48, device="cuda")
    kept = torch.empty(1, 2, 20, dtype=torch.int32, device="cuda")
    nl, nm = _i32([0]), torch.empty(1, 2, 20, device="cuda")
    call = lambda: paged.paged_evict(lay, cache, table, lens, mass, 20, dst, sink=1, recent=2, kept=kept, new_lens=nl,  # noqa: E731
                                     new_mass=nm)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for n in (40, 48, 7):
        lens.fill_(n)
        mass.uniform_()
        graph.replay()
        torch.cuda.synchronize()
        for h in range(2):
            s = pr.select(mass[0, h].cpu().numpy(), n, 20, 1, 2)
            assert kept[0, h, :len(s)].cpu().numpy().tolist() == s.tolist() and int(nl[0]) == len(s)


@pytest.mark.parametrize("slots,heads", [(600, 24), (9000, 40)])
def test_evict_lengths_in_place(cuda_ok, slots, heads):
    """new_lens given as seq_lens: every head is cut by the lengths of before."""
    lay = api.Layout(64, 2)
    lens = [slots, slots - 77, 5, 0]
    per, keep = -(-slots // 16), 100
    cache = paged.PagedCache.empty(lay, 4 * (per + 7), heads, 16, values=False)
    cache.gamma.copy_(torch.rand(cache.gamma.shape, generator=torch.Generator().manual_seed(1)))
    table = torch.arange(4 * per, dtype=torch.int32, device="cuda").view(4, per)
    dst = (4 * per + torch.arange(28, dtype=torch.int32, device="cuda")).view(4, 7)
    mass = torch.rand(4, heads, slots, generator=torch.Generator().manual_seed(2)).cuda()
    want = paged.paged_evict(lay, cache, table, _i32(lens), mass, keep, dst, sink=2, recent=9)
    moved = cache.gamma[4 * per:].clone()
    for _ in range(5):
        cache.gamma[4 * per:] = -1.0
        now = _i32(lens)
        got = paged.paged_evict(lay, cache, table, now, mass, keep, dst, sink=2, recent=9, new_lens=now)
        assert got[0] is now and now.tolist() == [min(n, keep) for n in lens]
        assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
        for i, n in enumerate(lens):
            n = min(n, keep)
            rows = dst[i].long() - 4 * per
            a, b = (x[rows].transpose(0, 1).reshape(heads, -1)[:, :n] for x in (cache.gamma[4 * per:], moved))
            assert torch.equal(a, b)
    cache.check()
