"""GPU tests of octo_paged_mass (attention weight gathered per cached token) against a float64 restatement, with the error
bounds derived in tests/paged_ref.py; the lse handed in is the reference's own, rounded to fp32."""

import numpy as np
import pytest
import torch

from rotation_preconditioned_quantization_b200 import api, inputs, paged

from . import paged_ref as pr

pytestmark = pytest.mark.gpu


def _case(seed, d, b, page, Hkv, g, lens, fresh, causal=True, scale=None, decay=0.75, bf16=True, slots=None, table_heads=None):
    pool = pr.Pool(seed, d, b, page, Hkv, lens, table_heads=table_heads)
    cu = [0] + list(np.cumsum(fresh))
    q = inputs.normal(seed + 1, (cu[-1], g * Hkv, d))
    q = inputs.to_bf16(q) if bf16 else q
    lse = pr.attn(pool, q, cu, causal, scale)[1].astype(np.float32)
    slots = max(lens) + 5 if slots is None else slots
    prev = np.random.default_rng(seed).lognormal(-1, 1, (len(lens), Hkv, slots)).astype(np.float32)
    ref, tol = pr.mass(pool, q, lse, cu, prev, decay, causal, scale)
    t = torch.from_numpy(q).cuda()
    t = t.to(torch.bfloat16) if bf16 else t
    m = torch.from_numpy(prev).cuda()
    out = m.clone()
    args = (pool.lay, pool.tables, t, torch.from_numpy(lse).cuda(), pool.cache, pool.page_table, pool.seq_lens)
    kw = dict(cu_q=torch.tensor(cu, dtype=torch.int32, device="cuda"), causal=causal, scale=scale, decay=decay)
    paged.paged_mass(*args, m, out=out, **kw)
    paged.paged_mass(*args, m, **kw)  # in place
    torch.cuda.synchronize()
    pool.cache.check()
    assert torch.equal(m, out)
    got = out.cpu().numpy().astype(np.float64)
    for i, n in enumerate(lens):
        assert np.array_equal(got[i, :, n:], prev[i, :, n:])  # behind the sequence: as it was
    assert np.all(np.abs(got - ref) <= tol), f"worst {np.max(np.abs(got - ref) / np.maximum(tol, 1e-30)):.2f} x tolerance"
    return got, ref


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("b", [2, 3, 4])
def test_every_layout(cuda_ok, d, b):
    got, ref = _case(10 * d + b, d, b, 64, 2, 4, [300, 129], [33, 5], decay=0.0)
    assert np.linalg.norm(got - ref) <= 4e-6 * np.linalg.norm(ref)


@pytest.mark.parametrize("n", [1, 16, 127, 128, 129, 255, 256, 257, 513])
def test_single_token(cuda_ok, n):
    _case(n, 128, 3, 16, 2, 4, [n], [1])


@pytest.mark.parametrize("page", [16, 48, 80, 256, 1024])
def test_page_sizes(cuda_ok, page):
    _case(page, 64, 2, page, 1, 2, [517, 64], [40, 64])


@pytest.mark.parametrize("g,fresh", [(1, 1), (1, 64), (1, 65), (1, 300), (3, 86), (5, 13), (8, 33), (256, 2)])
@pytest.mark.parametrize("causal", [True, False])
def test_row_tiles(cuda_ok, g, fresh, causal):
    _case(g * 1000 + fresh, 64, 3, 32, 1, g, [fresh + 277], [fresh], causal=causal)


def test_whole_prompt_without_prefix(cuda_ok):
    _case(5, 128, 4, 64, 2, 2, [700, 1], [700, 1])


def test_ragged_batch_with_empty_sequences(cuda_ok):
    _case(6, 128, 4, 16, 2, 3, [40, 0, 0, 500, 3, 1, 260], [0, 2, 0, 7, 5, 1, 260])


def test_many_sequences(cuda_ok):
    lens = [1 + (37 * i) % 200 for i in range(70)]
    _case(7, 64, 2, 16, 2, 2, lens, [1 + i % 3 if lens[i] > 3 else 1 for i in range(70)])


def test_many_units(cuda_ok):
    _case(8, 64, 3, 64, 4, 1, [20000], [3])


@pytest.mark.parametrize("scale", [0.0, -0.05, 0.5])
def test_scales(cuda_ok, scale):
    _case(9, 64, 3, 32, 2, 2, [200], [50], scale=scale)


def test_fp32_queries_and_shared_sign_rows(cuda_ok):
    _case(11, 128, 3, 64, 4, 2, [333, 64], [70, 3], bf16=False, table_heads=2)


def test_weights_sum_to_the_rows(cuda_ok):
    """With paged_attn's own lse a chunk's weights sum to its rows, to the precision of that lse (Dmax)."""
    pool = pr.Pool(12, 128, 3, 64, 2, [1000])
    q = torch.from_numpy(inputs.to_bf16(inputs.normal(13, (50, 8, 128)))).to(torch.bfloat16).cuda()
    dmax = pr.attn(pool, q.float().cpu().numpy(), [0, 50])[3]
    out, lse = paged.paged_attn(pool.lay, pool.tables, q, pool.cache, pool.page_table, pool.seq_lens, lse=True)
    m = torch.zeros(1, 2, 1000, device="cuda")
    paged.paged_mass(pool.lay, pool.tables, q, lse, pool.cache, pool.page_table, pool.seq_lens, m)
    for h in range(2):
        assert abs(float(m[0, h].double().sum()) - 200) <= 200 * float(np.expm1(dmax.max()))


def test_slots_beyond_the_mass_are_reported(cuda_ok):
    pool = pr.Pool(14, 64, 2, 16, 1, [100])
    q = torch.from_numpy(inputs.normal(15, (2, 1, 64))).cuda()
    lse = torch.zeros(2, 1, device="cuda")
    m = torch.zeros(1, 1, 40, device="cuda")
    paged.paged_mass(pool.lay, pool.tables, q, lse, pool.cache, pool.page_table, pool.seq_lens, m)
    with pytest.raises(RuntimeError, match="length"):
        pool.cache.check()


def test_offsets_that_do_not_ascend_stay_in_bounds(cuda_ok):
    """cu_q values that give sequences the same rows exceed the row tiles that the workspace holds: the rest is left out."""
    pool = pr.Pool(16, 64, 2, 16, 1, [100, 100, 100, 100, 100], stale=0.0)
    q = torch.from_numpy(inputs.normal(17, (200, 1, 64))).cuda()
    lse = torch.zeros(200, 1, device="cuda")
    cu = torch.tensor([0, 200, 0, 200, 0, 200], dtype=torch.int32, device="cuda")
    m = torch.zeros(5, 1, 100, device="cuda")
    paged.paged_mass(pool.lay, pool.tables, q, lse, pool.cache, pool.page_table, pool.seq_lens, m, cu_q=cu)
    with pytest.raises(RuntimeError, match="length"):
        pool.cache.check()
    out = paged.paged_attn(pool.lay, pool.tables, q, pool.cache, pool.page_table, pool.seq_lens, cu_q=cu)
    assert out.shape == q.shape
    with pytest.raises(RuntimeError, match="length"):
        pool.cache.check()


def test_graph_replay(cuda_ok):
    pool = pr.Pool(18, 64, 3, 32, 2, [300])
    q = torch.from_numpy(inputs.to_bf16(inputs.normal(19, (9, 4, 64)))).to(torch.bfloat16).cuda()
    lse = torch.full((9, 4), 5.0, device="cuda")
    m, o = torch.rand(1, 2, 300, device="cuda"), torch.zeros(1, 2, 300, device="cuda")
    ws = api.Workspace(paged.paged_mass_workspace_bytes(pool.lay, 9, 1, 4, 2))
    call = lambda out: paged.paged_mass(pool.lay, pool.tables, q, lse, pool.cache, pool.page_table, pool.seq_lens, m,  # noqa: E731
                                        cu_q=cu, out=out, decay=0.5, workspace=ws)
    cu = torch.tensor([0, 9], dtype=torch.int32, device="cuda")
    want = call(torch.zeros_like(o)).clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(o)
    for _ in range(3):
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want)
