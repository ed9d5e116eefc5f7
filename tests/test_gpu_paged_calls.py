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
