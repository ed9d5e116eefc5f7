"""The paged operators as a streaming server runs them: chunk after chunk of two sequences, positions on queries and keys,
keys encoded into pages, the chunk's attention, the weight it gathers, and a cut back to a budget into fresh pages once a
sequence outgrows it. Every step is checked against float64 restatements over what the cache then holds."""

import numpy as np
import pytest
import torch

from oracle import codec, tables
from rotation_preconditioned_quantization_b200 import api, inputs, paged

from . import paged_ref as pr
from . import parity

pytestmark = pytest.mark.gpu


class _View(pr.Pool):
    """The reference's view of a cache on the GPU."""

    def __init__(self, lay, cache, table, lens, tb, signs):
        self.lay, self.olay, self.d, self.b = lay, codec.Layout(lay.d, lay.b), lay.d, lay.b
        self.page, self.Hkv, self.lens = cache.page_size, cache.n_heads, list(lens)
        self.words = cache.packed.cpu().numpy().view(np.uint32)
        self.gamma, self.V = cache.gamma.cpu().numpy(), cache.V.float().cpu().numpy()
        self.table, self.tb, self.signs = table.cpu().numpy(), tb, signs


@pytest.mark.parametrize("d,b,bf16", [(64, 2, True), (128, 3, True), (128, 4, False)])
def test_stream(cuda_ok, d, b, bf16):
    B, H, g, page, budget, sink, recent = 2, 2, 3, 16, 60, 4, 20
    dt = torch.bfloat16 if bf16 else torch.float32
    lay, tb, signs = api.Layout(d, b), parity.oracle_tables(d, b), tables.rotation_signs(5, d, H)
    tabs = api.DeviceTables(*tb, signs)
    cache = paged.PagedCache.empty(lay, 40, H, page)
    free, own = list(range(40)), [[], []]
    rope = paged.RopeTable((d // 2 - 2 * (d // 6), d // 6, d // 6), per_axis=True)
    ws = api.Workspace(0)
    rng = np.random.default_rng(d)
    lens, seen = [0, 0], [0, 0]
    mass = torch.zeros(B, H, 160, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    evicted = 0
    for step, new in enumerate([[33, 5], [40, 1], [1, 50], [17, 30], [1, 1]]):
        rows, cu = sum(new), np.concatenate([[0], np.cumsum(new)])
        x = lambda h: torch.from_numpy(inputs.normal(int(rng.integers(1 << 30)), (rows, h, d))).to(dt).cuda()  # noqa: E731
        q, k, V = x(H * g), x(H), x(H).to(torch.bfloat16)
        t = np.concatenate([seen[i] + np.arange(new[i]) for i in range(B)])
        pos = torch.from_numpy(np.stack([t // 12, t // 4 % 3, t % 4]).astype(np.int32)).cuda()  # frame, row, column
        q, k = paged.rope(q, pos, rope, k=k)
        for i in range(B):
            while len(own[i]) * page < lens[i] + new[i]:
                own[i].append(free.pop())
        width = max(len(o) for o in own)
        table = i32([o + [-1] * (width - len(o)) for o in own])
        paged.paged_append(lay, tabs, k, V, cache, table, i32(lens), i32(cu))
        for i in range(B):
            mass[i, :, lens[i]:lens[i] + new[i]] = 0.0
            lens[i] += new[i]
            seen[i] += new[i]
        n = i32(lens)
        out, lse = paged.paged_attn(lay, tabs, q, cache, table, n, cu_q=i32(cu), dtype=dt, lse=True, workspace=ws)
        before = mass.cpu().numpy()
        paged.paged_mass(lay, tabs, q, lse, cache, table, n, mass, cu_q=i32(cu), decay=0.5, workspace=ws)
        torch.cuda.synchronize()
        cache.check()
        view = _View(lay, cache, table, lens, tb, signs)
        qn = q.float().cpu().numpy()
        ref, _, mag, dmax = pr.attn(view, qn, cu)
        pr.check_attn(out, ref, mag, dmax, bf16)
        want, tol = pr.mass(view, qn, lse.cpu().numpy(), cu, before, 0.5)
        assert np.all(np.abs(mass.cpu().numpy() - want) <= tol)
        if max(lens) > budget:
            m = mass.cpu().numpy()
            pages = -(-budget // page)
            into = [[free.pop() for _ in range(pages)] for _ in range(B)]
            words, gam, val = cache.packed.clone(), cache.gamma.clone(), cache.V.clone()
            nl, kept, mass_kept = paged.paged_evict(lay, cache, table, n, mass, budget, i32(into), sink=sink, recent=recent)
            torch.cuda.synchronize()
            cache.check()
            for i in range(B):
                for h in range(H):
                    s = pr.select(m[i, h], lens[i], budget, sink, recent)
                    assert kept[i, h, :len(s)].cpu().numpy().tolist() == s.tolist()
                    z = np.arange(len(s))
                    a = [torch.from_numpy(v.astype(np.int64)).cuda() for v in (np.array(own[i])[s // page], s % page,
                                                                                np.array(into[i])[z // page], z % page)]
                    assert torch.equal(cache.packed[a[2], h, :, a[3]], words[a[0], h, :, a[1]])
                    assert torch.equal(cache.gamma[a[2], h, a[3]], gam[a[0], h, a[1]])
                    assert torch.equal(cache.V[a[2], h, a[3]], val[a[0], h, a[1]])
                free.extend(own[i])
                own[i] = into[i]
            lens = nl.tolist()
            mass.zero_()
            mass[:, :, :budget] = mass_kept
            evicted += 1
    assert evicted >= 2
