"""GPU tests of octo_paged_attn: chunk attention over the paged compressed cache against a float64 restatement, with the
error bounds derived in tests/paged_ref.py. Slots that no sequence holds carry NaN norms and values throughout."""

import numpy as np
import pytest
import torch

from rotation_preconditioned_quantization_b200 import api, inputs, paged

from . import paged_ref as pr

pytestmark = pytest.mark.gpu


def _queries(seed, rows, Hq, d, bf16=True):
    q = inputs.normal(seed, (rows, Hq, d))
    return inputs.to_bf16(q) if bf16 else q


def _run(pool, q, cu, bf16_in=True, **kw):
    t = torch.from_numpy(q).cuda()
    t = t.to(torch.bfloat16) if bf16_in else t
    r = paged.paged_attn(pool.lay, pool.tables, t, pool.cache, pool.page_table, pool.seq_lens,
                         cu_q=torch.tensor(cu, dtype=torch.int32, device="cuda"), **kw)
    torch.cuda.synchronize()
    pool.cache.check()
    return r


def _case(seed, d, b, page, Hkv, g, lens, fresh, causal=True, scale=None, bf16=True, table_heads=None):
    pool = pr.Pool(seed, d, b, page, Hkv, lens, table_heads=table_heads)
    cu = [0] + list(np.cumsum(fresh))
    q = _queries(seed + 1, cu[-1], g * Hkv, d, bf16)
    ref, lse, mag, dmax = pr.attn(pool, q, cu, causal, scale)
    out, got = _run(pool, q, cu, bf16, causal=causal, scale=scale, dtype=torch.bfloat16 if bf16 else torch.float32, lse=True)
    pr.check_attn(out, ref, mag, dmax, bf16)
    got = got.cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isneginf(got), np.isneginf(lse))
    ok = np.isfinite(lse)
    assert np.all(np.abs(got - np.where(ok, lse, 0))[ok] <= (dmax + 2.0 ** -20 * (1 + np.abs(np.where(ok, lse, 0))))[ok])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("b", [2, 3, 4])
def test_every_layout(cuda_ok, d, b):
    _case(10 * d + b, d, b, 64, 2, 4, [300, 129], [33, 5])


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 1000])
def test_single_token(cuda_ok, n):
    _case(n, 128, 3, 16, 2, 4, [n], [1])


@pytest.mark.parametrize("page", [16, 32, 48, 64, 80, 128, 240, 256, 1024])
def test_page_sizes(cuda_ok, page):
    _case(page, 64, 2, page, 1, 2, [517, 64], [40, 64])


@pytest.mark.parametrize("g,fresh", [(1, 1), (1, 128), (1, 129), (1, 300), (2, 64), (3, 86), (5, 51), (5, 52), (8, 33), (256, 2)])
@pytest.mark.parametrize("causal", [True, False])
def test_row_tiles(cuda_ok, g, fresh, causal):
    _case(g * 1000 + fresh, 64, 3, 32, 1, g, [fresh + 77], [fresh], causal=causal)


def test_whole_prompt_without_prefix(cuda_ok):
    _case(5, 128, 3, 64, 2, 2, [700, 1], [700, 1])


def test_ragged_batch_with_empty_sequences(cuda_ok):
    # no new tokens; no cache; both; rows before the cache's start see nothing
    _case(6, 128, 4, 16, 2, 3, [40, 0, 0, 500, 3, 1, 260], [0, 2, 0, 7, 5, 1, 260])


def test_many_sequences(cuda_ok):
    lens = [1 + (37 * i) % 200 for i in range(70)]
    _case(7, 64, 2, 16, 2, 2, lens, [1 + i % 3 if lens[i] > 3 else 1 for i in range(70)])


def test_long_context_splits_over_all_ctas(cuda_ok):
    _case(8, 128, 3, 64, 1, 4, [40000], [2])


@pytest.mark.parametrize("scale", [0.0, -0.05, 0.5])
def test_scales(cuda_ok, scale):
    _case(9, 64, 3, 32, 2, 2, [200], [50], scale=scale)


def test_fp32_queries_and_output_and_shared_sign_rows(cuda_ok):
    _case(11, 128, 3, 64, 4, 2, [333, 64], [70, 3], bf16=False, table_heads=2)


def test_strided_queries(cuda_ok):
    pool = pr.Pool(12, 64, 3, 32, 2, [150, 40])
    cu = [0, 10, 13]
    big = torch.randn(13, 12, 3, 64, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(torch.bfloat16)
    q = big[:, 2:6, 1]  # strides of a fused projection
    assert not q.is_contiguous()
    ref, _, mag, dmax = pr.attn(pool, q.float().cpu().numpy(), cu)
    out = paged.paged_attn(pool.lay, pool.tables, q, pool.cache, pool.page_table, pool.seq_lens,
                           cu_q=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    pr.check_attn(out, ref, mag, dmax, True)


def test_large_and_tiny_rows_and_norms(cuda_ok):
    """Queries and norms over many powers of two: logits that reach far beyond the reference raise it."""
    pool = pr.Pool(13, 128, 3, 64, 1, [900])
    pool.gamma *= np.where(np.random.default_rng(1).random(pool.gamma.shape) < 0.02, 20.0, 0.01).astype(np.float32)
    pool.to("cuda")
    q = _queries(14, 64, 2, 128)
    q *= (2.0 ** np.linspace(-20, 3, 64)).astype(np.float32)[:, None, None]
    q = inputs.to_bf16(q)
    ref, _, mag, dmax = pr.attn(pool, q, [0, 64])
    pr.check_attn(_run(pool, q, [0, 64]), ref, mag, dmax, True)
    z = np.zeros_like(q)
    ref, _, mag, dmax = pr.attn(pool, z, [0, 64])
    pr.check_attn(_run(pool, z, [0, 64]), ref, mag, dmax, True)


def test_rising_logits_move_the_reference(cuda_ok):
    """Norms that grow along the cache: later tiles, and the second half of a tile, pass the reference by far."""
    pool = pr.Pool(15, 64, 2, 64, 1, [1024])
    p, o = pool.slots(0)
    pool.gamma[p, 0, o] = (2.0 ** np.linspace(-3, 9, 1024)).astype(np.float32)
    pool.to("cuda")
    q = _queries(16, 70, 2, 64)
    ref, _, mag, dmax = pr.attn(pool, q, [0, 70], False)
    # logits of a few hundred: the bound on their error is a few units; compare where it is below one half
    out = _run(pool, q, [0, 70], causal=False).float().cpu().numpy()
    assert np.isfinite(out).all()
    ok = dmax < 0.5
    assert ok.any()
    tol = (np.expm1(2 * dmax)[..., None] + 2.0 ** -8 + 2.0 ** -16) * mag + 2.0 ** -8 * np.abs(ref)
    assert np.all((np.abs(out - ref) <= tol)[ok])


def test_contiguous_cache_as_pages(cuda_ok):
    """An encoded contiguous cache seen as pages gives decode_attn's result for one token."""
    d, b, B, H, n = 128, 3, 2, 2, 301
    lay = api.Layout(d, b)
    tabs = api.DeviceTables.build(lay, 3, H)
    cache = api.Cache.empty(lay, B * H, 304)
    keys = torch.from_numpy(inputs.llm_keys(1, B * H, n, d)).to(torch.bfloat16).cuda()
    V = torch.zeros((B * H, 304, d), dtype=torch.bfloat16, device="cuda")
    V[:, :n] = torch.from_numpy(inputs.normal(2, (B * H, n, d))).to(torch.bfloat16).cuda()
    api.encode(lay, tabs, keys, cache)
    q = torch.from_numpy(inputs.normal(3, (B, 4 * H, d))).to(torch.bfloat16).cuda()
    want, _ = api.decode_attn(lay, tabs, q.unsqueeze(2), cache, V, H)
    pool = paged.PagedCache.from_cache(cache, V, H)
    table = torch.arange(B, dtype=torch.int32, device="cuda").view(B, 1)
    got = paged.paged_attn(lay, tabs, q, pool, table, torch.full((B,), n, dtype=torch.int32, device="cuda"),
                           dtype=torch.float32)
    # both are within 2^-8 + 2 Dmax of the exact result; Dmax < 2^-8 for these keys' logits
    assert torch.all((got - want[:, :, 0]).abs() <= 2.0 ** -5 * V.float().abs().max())
    assert (got - want[:, :, 0]).norm() <= 2.0 ** -7 * want.norm()


def test_rows_of_no_sequence_are_left(cuda_ok):
    pool = pr.Pool(17, 64, 2, 16, 1, [30])
    q = _queries(18, 9, 1, 64)
    out = torch.full((9, 1, 64), 7.0, device="cuda")
    paged.paged_attn(pool.lay, pool.tables, torch.from_numpy(q).cuda(), pool.cache, pool.page_table, pool.seq_lens,
                     cu_q=torch.tensor([2, 6], dtype=torch.int32, device="cuda"), out=out)
    assert torch.all(out[:2] == 7.0) and torch.all(out[6:] == 7.0) and not torch.any(out[2:6] == 7.0)


def test_outputs_repeat_bit_for_bit(cuda_ok):
    pool = pr.Pool(19, 128, 3, 64, 2, [2000, 100])
    q = _queries(20, 80, 8, 128)
    a = _run(pool, q, [0, 60, 80])
    b = _run(pool, q, [0, 60, 80])
    assert torch.equal(a, b)


@pytest.mark.parametrize("page", [16, 64])
def test_ragged_tails_repeat_bit_for_bit(cuda_ok, page):
    """Pieces with many sequence ends, each in a tile that V's copies fill in part: the zeroing of V's rows behind an end
    meets neither the products of the tile that had the stage before nor a copy that is still landing. Row counts that
    leave lanes of a warp without rows: what those find in tensor memory must not move other rows' references."""
    lens = [1 + (613 * i) % 1500 for i in range(96)]
    fresh = [min(lens[i], 1 + (11 * i) % 40) for i in range(96)]
    pool = pr.Pool(41, 128, 3, page, 4, lens)
    cu = [0] + list(np.cumsum(fresh))
    q = _queries(42, cu[-1], 20, 128)
    q *= (2.0 ** np.linspace(-3, 3, cu[-1])).astype(np.float32)[:, None, None]
    q = inputs.to_bf16(q)
    ref, _, mag, dmax = pr.attn(pool, q, cu)
    first = _run(pool, q, cu)
    pr.check_attn(first, ref, mag, dmax, True)
    for _ in range(25):
        assert torch.equal(_run(pool, q, cu), first)


def test_bad_pages_and_lengths_are_reported(cuda_ok):
    """Page ids outside the pool and lengths beyond the table stay in bounds and are reported (the kernel's own checks)."""
    pool = pr.Pool(21, 64, 2, 16, 1, [100, 50], stale=0.0)
    q = torch.from_numpy(_queries(22, 4, 1, 64)).cuda()
    cu = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    table = pool.page_table.clone()
    table[0, 3] = 1 << 20
    ws = api.Workspace(0)
    good = paged.paged_attn(pool.lay, pool.tables, q, pool.cache, pool.page_table, pool.seq_lens, cu_q=cu, workspace=ws)
    out = paged.paged_attn(pool.lay, pool.tables, q, pool.cache, table, pool.seq_lens, cu_q=cu, workspace=ws)
    assert torch.equal(out[2:], good[2:])  # the other sequence is untouched
    with pytest.raises(RuntimeError, match="page id"):
        pool.cache.check()
    lens = torch.tensor([100000, 50], dtype=torch.int32, device="cuda")
    out = paged.paged_attn(pool.lay, pool.tables, q, pool.cache, pool.page_table, lens, cu_q=cu, workspace=ws)
    with pytest.raises(RuntimeError, match="length"):
        pool.cache.check()
    pool.cache.check()  # cleared


def test_graph_replay_with_new_lengths(cuda_ok):
    """A captured call replays on the lengths and pages that its tensors hold then; the workspace is reused."""
    pool = pr.Pool(23, 128, 2, 32, 2, [400, 90])
    q = torch.from_numpy(_queries(24, 6, 4, 128)).to(torch.bfloat16).cuda()
    cu = torch.tensor([0, 4, 6], dtype=torch.int32, device="cuda")
    out = torch.empty(6, 4, 128, dtype=torch.bfloat16, device="cuda")
    ws = api.Workspace(paged.paged_attn_workspace_bytes(pool.lay, 6, 2, 4, 2))
    call = lambda: paged.paged_attn(pool.lay, pool.tables, q, pool.cache, pool.page_table, pool.seq_lens, cu_q=cu,  # noqa: E731
                                    out=out, workspace=ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens in ([400, 90], [123, 2], [399, 0]):
        pool.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        pool.lens = lens
        out.fill_(float("nan"))
        # stale slots are those behind the lengths of now
        graph.replay()
        torch.cuda.synchronize()
        ref, _, mag, dmax = pr.attn(pool, q.float().cpu().numpy(), [0, 4, 6])
        pr.check_attn(out, ref, mag, dmax, True)
    pool.cache.check()


def test_two_streams_with_a_workspace_each(cuda_ok):
    pool = pr.Pool(25, 128, 3, 64, 2, [5000])
    q = torch.from_numpy(_queries(26, 32, 8, 128)).to(torch.bfloat16).cuda()
    args = (pool.lay, pool.tables, q, pool.cache, pool.page_table, pool.seq_lens)
    want = paged.paged_attn(*args)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [api.Workspace(paged.paged_attn_workspace_bytes(pool.lay, 32, 1, 8, 2)) for _ in range(2)]
    outs = [[torch.empty_like(want) for _ in range(8)] for _ in range(2)]
    torch.cuda.synchronize()
    for k in range(8):
        for s in range(2):
            paged.paged_attn(*args, out=outs[s][k], workspace=ws[s], stream=streams[s])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for s in outs for o in s)


def test_a_call_on_another_stream_owns_what_it_allocates(cuda_ok):
    """cu_q, scratch and outputs of a call with ``stream`` are made on that stream: neither a busy current stream nor one
    that reuses the memory at once reaches them. Appending tokens likewise."""
    pool = pr.Pool(27, 128, 3, 64, 2, [3000, 64])
    q = torch.from_numpy(_queries(28, 16, 8, 128)).to(torch.bfloat16).cuda()
    args = (pool.lay, pool.tables, q, pool.cache, pool.page_table, pool.seq_lens)
    want = paged.paged_attn(*args)
    keys = torch.randn(8, 2, 128, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    V = keys.to(torch.bfloat16)
    table = torch.arange(2, dtype=torch.int32, device="cuda").view(2, 1)
    starts, cu = torch.tensor([3, 9], dtype=torch.int32, device="cuda"), torch.tensor([0, 5, 8], dtype=torch.int32, device="cuda")
    pools = [paged.PagedCache.empty(pool.lay, 2, 2, 64) for _ in range(2)]
    paged.paged_append(pool.lay, pool.tables, keys, V, pools[0], table, starts, cu)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)  # the current stream is busy for some ten milliseconds
    out = paged.paged_attn(*args, stream=side)
    paged.paged_append(pool.lay, pool.tables, keys, V, pools[1], table, starts, cu, stream=side)
    junk = [torch.full((1 << k,), float("nan"), device="cuda") for k in range(10, 25)]
    side.synchronize()
    assert torch.equal(out, want)
    torch.cuda.synchronize()
    for a, b in ((pools[0].packed, pools[1].packed), (pools[0].gamma, pools[1].gamma), (pools[0].V, pools[1].V)):
        assert torch.equal(a, b)
    del junk
