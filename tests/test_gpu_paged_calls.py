"""GPU tests of calls that the paged operators' documentation allows beside their plain use: workspaces that serve other
calls too, chunks and batches without rows, pools whose tensors are replaced, other streams, values of any size."""

import numpy as np
import pytest
import torch

from rotation_preconditioned_quantization_b200 import api, inputs, paged

from . import paged_ref as pr

pytestmark = pytest.mark.gpu


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _queries(seed, rows, Hq, d):
    return torch.from_numpy(inputs.to_bf16(inputs.normal(seed, (rows, Hq, d)))).to(torch.bfloat16).cuda()


def test_one_workspace_serves_decode_and_the_paged_calls_in_turn(cuda_ok):
    """decode_attn's status word and arrival counters, which have to be zero before each of its calls, are not the paged
    calls' scratch: not for the heads that a call before had, nor for more."""
    d, H, n = 128, 2, 20000
    lay = api.Layout(d, 3)
    g = torch.Generator("cuda").manual_seed(1)
    cache = api.Cache.empty(lay, 4 * H, n)
    cache.packed.random_(-2 ** 31, 2 ** 31 - 1, generator=g)
    cache.gamma.uniform_(0.5, 2.0, generator=g)
    cache.length = n
    V = torch.randn(4 * H, n, d, device="cuda", generator=g).to(torch.bfloat16)
    q = torch.randn(4, 4 * H, 1, d, device="cuda", generator=g).to(torch.bfloat16)
    pool = pr.Pool(51, d, 3, 64, H, [900])
    pq = _queries(52, 200, 4 * H, d)
    lse = torch.full((200, 4 * H), 5.0, device="cuda")

    def decode(B, ws):
        return api.decode_attn(lay, pool.tables, q[:B], cache, V, H, workspace=ws)[0]

    want = {B: decode(B, None) for B in (1, 4)}
    ws = api.Workspace(0)
    assert torch.equal(decode(1, ws), want[1])
    args = (pq, pool.cache, pool.page_table, pool.seq_lens)
    for B in (1, 4, 1):
        paged.paged_mass(pool.lay, pool.tables, args[0], lse, *args[1:], torch.zeros(1, H, 900, device="cuda"), workspace=ws)
        assert torch.equal(decode(B, ws), want[B])
        paged.paged_attn(pool.lay, pool.tables, *args, lse=True, workspace=ws)
        assert torch.equal(decode(B, ws), want[B])
        assert ws.status() == 0 and not ws.counters(4 * H).any()
    pool.cache.check()


@pytest.mark.parametrize("cu", [None, [0, 0, 0, 0]])
@pytest.mark.parametrize("in_place", [False, True])
def test_mass_of_a_chunk_without_rows_decays(cuda_ok, cu, in_place):
    """A sequence without new rows decays its mass, whether or not another sequence of the batch has some."""
    pool = pr.Pool(61, 64, 2, 16, 2, [70, 0, 300])
    m = torch.rand(3, 2, 310, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    m0, out = m.clone(), m if in_place else torch.full_like(m, float("nan"))
    got = paged.paged_mass(pool.lay, pool.tables, torch.empty(0, 4, 64, device="cuda"), torch.empty(0, 4, device="cuda"),
                           pool.cache, pool.page_table, pool.seq_lens, m, cu_q=None if cu is None else _i32(cu), decay=0.75,
                           out=out)
    assert got is out
    pool.cache.check()
    for i, n in enumerate(pool.lens):
        assert torch.equal(out[i, :, :n], 0.75 * m0[i, :, :n])  # one product, rounded once
        assert torch.equal(out[i, :, n:], m0[i, :, n:]) if in_place else out[i, :, n:].isnan().all()


def test_mass_of_a_chunk_without_rows_reports_lengths(cuda_ok):
    pool = pr.Pool(62, 64, 2, 16, 1, [40], stale=0.0)
    m = torch.ones(1, 1, 48, device="cuda")
    call = lambda lens: paged.paged_mass(pool.lay, pool.tables, torch.empty(0, 1, 64, device="cuda"),  # noqa: E731
                                         torch.empty(0, 1, device="cuda"), pool.cache, pool.page_table, lens, m, decay=0.5)
    call(_i32([1000]))
    with pytest.raises(RuntimeError, match="length"):
        pool.cache.check()
    assert m.eq(0.5).all()


def test_check_waits_for_calls_on_other_streams(cuda_ok):
    """What a call on another stream than the current one finds is raised, and not lost to the clearing of the word."""
    pool = pr.Pool(71, 64, 2, 16, 1, [100], stale=0.0)
    q = _queries(72, 1, 1, 64)
    table = pool.page_table.clone()
    table[0, 3] = 1 << 20
    paged.paged_attn(pool.lay, pool.tables, q, pool.cache, pool.page_table, pool.seq_lens)
    pool.cache.check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)  # some twenty milliseconds
    paged.paged_attn(pool.lay, pool.tables, q, pool.cache, table, pool.seq_lens, stream=side)
    with pytest.raises(RuntimeError, match="page id"):
        pool.cache.check()
    torch.cuda.synchronize()
    assert int(pool.cache.status.item()) == 0


def test_stream_by_position_owns_what_the_call_allocates(cuda_ok):
    pool = pr.Pool(73, 128, 3, 64, 2, [3000, 64])
    q = _queries(74, 16, 8, 128)
    args = (pool.lay, pool.tables, q, pool.cache, pool.page_table, pool.seq_lens)
    want = paged.paged_attn(*args)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)  # the current stream is busy for some ten milliseconds
    out = paged.paged_attn(*args, None, True, None, None, None, None, None, side)
    junk = [torch.full((1 << k,), float("nan"), device="cuda") for k in range(10, 25)]
    side.synchronize()
    assert torch.equal(out, want)
    torch.cuda.synchronize()
    del junk


def test_no_tokens_into_a_pool_with_values(cuda_ok):
    lay = api.Layout(64, 2)
    tabs = api.DeviceTables.build(lay, 0, 2)
    cache = paged.PagedCache.empty(lay, 2, 2, 16)
    before = [x.clone() for x in (cache.packed, cache.gamma, cache.V)]
    V = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    paged.paged_write(lay, api.Cache.empty(lay, 2, 8), V, cache, _i32([[1]]), _i32([3]), _i32([0, 0]))
    for dt in (torch.bfloat16, torch.float32):
        paged.paged_append(lay, tabs, torch.empty(0, 2, 64, dtype=dt, device="cuda"), V, cache, _i32([[1]]), _i32([3]),
                           _i32([0, 0]))
    cache.check()
    assert all(torch.equal(a, b) for a, b in zip(before, (cache.packed, cache.gamma, cache.V)))


def test_a_pool_whose_tensors_are_replaced(cuda_ok):
    """A call uses the tensors that the pool holds then, as api.Cache's calls do: also more pages than before."""
    a, b = pr.Pool(81, 64, 2, 16, 2, [100]), pr.Pool(82, 64, 2, 16, 2, [400])
    b.tables = a.tables
    q = _queries(83, 5, 4, 64)
    call = lambda cache: paged.paged_attn(b.lay, b.tables, q, cache, b.page_table, b.seq_lens)  # noqa: E731
    want = call(b.cache)
    old = (a.cache.packed, a.cache.gamma, a.cache.V)  # (kept: the old addresses stay valid)
    a.cache.packed, a.cache.gamma, a.cache.V = b.cache.packed, b.cache.gamma, b.cache.V
    assert torch.equal(call(a.cache), want)
    a.cache.check()
    a.cache.V = torch.zeros_like(b.cache.V)
    assert not call(a.cache).any()
    assert old[0].shape[0] < b.cache.n_pages == a.cache.n_pages


def test_rope_frequencies_that_are_replaced(cuda_ok):
    q, pos = torch.randn(5, 2, 64, device="cuda"), torch.arange(5, dtype=torch.int32, device="cuda")[None] * 1000
    a, b = paged.RopeTable((32,), 10000.0), paged.RopeTable((32,), 500.0)
    old, a.freqs = a.freqs, b.freqs.clone()
    assert torch.equal(paged.rope(q, pos, a), paged.rope(q, pos, b)) and old.shape == b.freqs.shape


@pytest.mark.parametrize("d", [64, 128])
def test_large_values_behind_a_rise_of_the_logits(cuda_ok, d):
    """Whole key tiles whose logits pass the first tile's by far (2^87 in the weights by the first tile's reference),
    with values of 2^36: a row's output is as exact as bf16 weights say, and lies between the values that it averages.
    Enough equal rows that a CTA walks from an item's first tile into its next ones."""
    rows, n = 256 * 60, 1024
    pool = pr.Pool(91 + d, d, 3, 64, 1, [n])
    rng = np.random.default_rng(5)
    pool.words[:] = pool.words[:1, :, :, :1]  # one direction throughout
    p, o = pool.slots(0)
    pool.V[p, 0, o] = inputs.to_bf16((2.0 ** 36 * rng.uniform(1.0, 2.0, (n, d))).astype(np.float32))
    pool.gamma[p, 0, o] = np.where(np.arange(n) < 128, 0.01, 1.0).astype(np.float32)
    _, u, _ = pool.keys(0, 0)
    R = pr.codec.rotation_matrix(pool.signs[0])
    want = 88.0 * np.log(2.0)  # the logit of a slot behind the first tile
    q = (u[0] @ R / (u[0] @ u[0]) * want * np.sqrt(d))[None, None].astype(np.float32)
    pool.to("cuda")
    out, lse = paged.paged_attn(pool.lay, pool.tables, torch.from_numpy(q).cuda().expand(rows, 1, d), pool.cache,
                                pool.page_table, pool.seq_lens, causal=False, lse=True)
    pool.cache.check()
    ref, rl, mag, dmax = pr.attn(pool, q, [0, 1], False)
    assert abs(rl[0, 0] - want - np.log(n - 128.0)) < 1e-3 and dmax.max() < 0.5
    ref, mag, dmax = (np.broadcast_to(x, (rows,) + x.shape[1:]) for x in (ref, mag, dmax))
    pr.check_attn(out, ref, mag, dmax, False)
    assert np.all(np.abs(lse.cpu().numpy() - rl[0, 0]) <= dmax + 2.0 ** -20 * (1 + abs(rl[0, 0])))
    v, got = pool.V[p, 0, o], out.cpu().numpy()
    assert np.all(got >= v.min(0) * (1 - 2.0 ** -7)) and np.all(got <= v.max(0) * (1 + 2.0 ** -7))


def test_write_leaves_the_rows_behind_the_last_sequence(cuda_ok):
    """A batch padded to a fixed number of rows, as a captured call has it: the rows behind the last sequence are no
    tokens (the chunk calls leave theirs alone too). Those before the first sequence's are still reported."""
    lay = api.Layout(64, 2)
    cache = paged.PagedCache.empty(lay, 3, 1, 16)
    staged = api.Cache.empty(lay, 1, 40)
    staged.gamma.fill_(3.0)
    V = torch.ones(40, 1, 64, dtype=torch.bfloat16, device="cuda")
    for cu in ([0, 4, 7], [0, 7, 7], [0, 0, 7]):
        cache.gamma.zero_()
        paged.paged_write(lay, staged, V, cache, _i32([[0], [2]]), _i32([1, 2]), _i32(cu))
        cache.check()
        assert cache.gamma[0, 0, 1:1 + cu[1]].eq(3).all() and cache.gamma[2, 0, 2:2 + 7 - cu[1]].eq(3).all()
        assert cache.gamma.sum() == 21
    paged.paged_write(lay, staged, V, cache, _i32([[0], [2]]), _i32([1, 2]), _i32([0, 0, 0]))
    cache.check()
    assert cache.gamma.sum() == 21
    paged.paged_write(lay, staged, V, cache, _i32([[0], [2]]), _i32([1, 2]), _i32([1, 4, 7]))
    with pytest.raises(RuntimeError, match="length"):
        cache.check()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rope_into_another_part_of_a_fused_buffer(cuda_ok, dtype):
    """Outputs between the rows of their own inputs, and of the other tensor's, that meet none of them."""
    g = torch.Generator("cuda").manual_seed(7)
    x = torch.randn(33, 10, 64, device="cuda", generator=g).to(dtype)
    pos, table = torch.arange(33, dtype=torch.int32, device="cuda")[None] * 77, paged.RopeTable((32,))
    want = paged.rope(x[:, :4].clone(), pos, table, k=x[:, 4:5].clone())
    paged.rope(x[:, :4], pos, table, k=x[:, 4:5], out=x[:, 5:9], k_out=x[:, 9:])
    assert torch.equal(x[:, 5:9], want[0]) and torch.equal(x[:, 9:], want[1])


def test_a_workspace_that_grows_keeps_what_a_graph_holds(cuda_ok):
    """A captured call's scratch stays its own when a later call needs more than the workspace has."""
    pool = pr.Pool(101, 64, 2, 16, 2, [300])
    q, big = _queries(102, 4, 4, 64), _queries(103, 4000, 4, 64)
    lse, blse = torch.full((4, 4), 5.0, device="cuda"), torch.full((4000, 4), 5.0, device="cuda")
    m = torch.rand(1, 2, 300, device="cuda")
    ws = api.Workspace(paged.paged_mass_workspace_bytes(pool.lay, 4, 1, 4, 2))
    out = torch.empty_like(m)
    mass = lambda q, lse, out: paged.paged_mass(pool.lay, pool.tables, q, lse, pool.cache, pool.page_table, pool.seq_lens,  # noqa: E731
                                                m, out=out, workspace=ws)
    cu = _i32([0, 4])
    call = lambda out: paged.paged_mass(pool.lay, pool.tables, q, lse, pool.cache, pool.page_table, pool.seq_lens, m, cu_q=cu,  # noqa: E731
                                        out=out, workspace=ws)
    want = call(torch.empty_like(m))
    torch.cuda.synchronize()
    size = ws.nbytes
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out)
    mass(big, blse, torch.empty_like(m))
    assert ws.nbytes > size
    others = [torch.full((size // 4,), 7, dtype=torch.int32, device="cuda") for _ in range(8)]  # what took freed memory
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert all(x.eq(7).all() for x in others)


@pytest.mark.parametrize("slots", [4097, 24576, 24577, 34976, 34977])
@pytest.mark.parametrize("heads", [3, 32, 33])
def test_evict_at_the_bounds_of_its_choice(cuda_ok, slots, heads):
    """One block or four per head, by the slots and by how many (sequence, head) rows there are: the same slots stay."""
    lay, keep, sink, recent = api.Layout(64, 2), 300, 5, 70
    per = -(-slots // 256)
    cache = paged.PagedCache.empty(lay, per + 2, heads, 256, values=False)
    cache.gamma.copy_(torch.rand(cache.gamma.shape, generator=torch.Generator().manual_seed(1)))
    table, dst = torch.arange(per, dtype=torch.int32, device="cuda")[None], _i32([[per, per + 1]])
    g = torch.Generator("cuda").manual_seed(slots)
    m = torch.rand(1, heads, slots, generator=g, device="cuda")
    m[torch.rand(m.shape, generator=g, device="cuda") < 0.3] = 0.999  # ties at the border: the lower slots stay
    n = slots - 1
    lens, kept, mass = paged.paged_evict(lay, cache, table, _i32([n]), m, keep, dst, sink=sink, recent=recent)
    cache.check()
    w = m[0, :, :n].clone()
    w[:, :sink], w[:, n - recent:] = 2.0, 2.0
    want = torch.sort(w, descending=True, stable=True).indices[:, :keep].sort().values
    assert int(lens) == keep and torch.equal(kept[0].long(), want) and torch.equal(mass[0], m[0].gather(1, want))
    src = cache.gamma[:per].transpose(0, 1).reshape(heads, -1).gather(1, want)
    assert torch.equal(cache.gamma[per:].transpose(0, 1).reshape(heads, -1)[:, :keep], src)


def test_a_workspace_that_grows_behind_a_call_that_still_runs(cuda_ok):
    """Calls in order on a side stream, the second larger: the buffer that it replaces, made on the current stream, goes to
    nobody before the first call is done."""
    pool = pr.Pool(104, 64, 2, 16, 2, [300])
    q, big = _queries(105, 4, 4, 64), _queries(106, 4000, 4, 64)
    lse, blse = torch.full((4, 4), 5.0, device="cuda"), torch.full((4000, 4), 5.0, device="cuda")
    m = torch.rand(1, 2, 300, device="cuda")
    mass = lambda q, lse, out, **kw: paged.paged_mass(pool.lay, pool.tables, q, lse, pool.cache, pool.page_table, pool.seq_lens,  # noqa: E731
                                                      m, cu_q=_i32([0, len(q)]) if not kw else kw.pop("cu"), out=out, **kw)
    want = mass(q, lse, torch.empty_like(m)), mass(big, blse, torch.empty_like(m))
    outs, cus = [torch.empty_like(m) for _ in range(2)], [_i32([0, 4]), _i32([0, 4000])]
    ws = api.Workspace(paged.paged_mass_workspace_bytes(pool.lay, 4, 1, 4, 2))
    size, side = ws.nbytes, torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)  # some twenty milliseconds
    mass(q, lse, outs[0], cu=cus[0], workspace=ws, stream=side)
    mass(big, blse, outs[1], cu=cus[1], workspace=ws, stream=side)
    assert ws.nbytes > size
    others = [torch.full((size // 4,), 7, dtype=torch.int32, device="cuda") for _ in range(8)]  # what takes freed memory
    torch.cuda.synchronize()
    assert all(x.eq(7).all() for x in others)
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    pool.cache.check()


def test_a_decode_on_another_stream_owns_what_it_allocates(cuda_ok):
    """Workspace (zeroed) and output of a call with ``stream``, while the current stream is busy."""
    d, H, n = 128, 2, 20000
    lay = api.Layout(d, 3)
    tabs = api.DeviceTables.build(lay, 5, H)
    g = torch.Generator("cuda").manual_seed(1)
    cache = api.Cache.empty(lay, H, n)
    cache.packed.random_(-2 ** 31, 2 ** 31 - 1, generator=g)
    cache.gamma.uniform_(0.5, 2.0, generator=g)
    cache.length = n
    V = torch.randn(H, n, d, device="cuda", generator=g).to(torch.bfloat16)
    q = torch.randn(1, 4 * H, 1, d, device="cuda", generator=g).to(torch.bfloat16)
    want, keys = api.decode_attn(lay, tabs, q, cache, V, H)[0], api.dequant(lay, tabs, cache, 500)
    side = torch.cuda.Stream()
    junk = torch.full((1 << 22,), 7, dtype=torch.int32, device="cuda")
    del junk
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)  # the current stream is busy for some ten milliseconds
    out, _ = api.decode_attn(lay, tabs, q, cache, V, H, stream=side)
    got = api.dequant(lay, tabs, cache, 500, stream=side)
    junk = [torch.full((1 << k,), float("nan"), device="cuda") for k in range(10, 23)]
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(got, keys)
    torch.cuda.synchronize()
    del junk
