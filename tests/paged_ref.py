"""Plain float64 restatements of the paged operators for the tests (numpy and the oracle's codec; none of the kernels'
code), and the builder of small random pools.

Error bounds that the tests use, u = eps / 2 of a type (bf16 2^-8, fp16 2^-11, fp32 2^-24):

* a logit of ``paged_attn`` is off by at most D = |scale| * gamma * sum_d |q~_d| |u_d| * 3 * 2^-11 (one fp16 rounding
  of the rotated query, one of the decoded direction, or two where it is formed from a direction and a norm level) plus
  2^-24 * sqrt(d) * |scale| * gamma * max|q~| (fp16 subnormals below the row's power of two, |u| <= 1) plus the fp32
  accumulation, 4 d * 2^-24 of the sum of magnitudes. Weights are then off by a factor in exp(+-2 Dmax) (numerator and
  denominator), and by u(bf16) = 2^-8 from rounding the weight: |out - ref| <= (expm1(2 Dmax) + 2^-8 + 2^-16) * sum p |v|
  + u(out) |ref|; |lse - ref| <= Dmax + 2^-20 (1 + |ref|). The row sum is that of the rounded weights p (1 + e), |e| <=
  u / (1 + u) (half a step against a value that is at least one step above a power of two): out - ref = sum p e (v - ref)
  / (1 + sum p e), which is at most max|e| / (1 - max|e|) = u times sum p |v - ref|, with |v - ref| <= |v| + |ref| and
  |ref| <= sum p |v|. So the bound on the weights' rounding is 2^-8 * (sum p |v| + |ref|).
* a logit of ``paged_mass`` comes from hi + lo pairs, high parts on grids of 2^-11 (queries, scaled so that their row's
  largest is below 1 and at least 1/2: units of it cost a factor 2) and 2^-12 (keys): the dropped product is at most
  2^-12 * 2^-13 per term, d terms; the low parts round by 2^-23 and 2^-24, against sum |u| <= sqrt(d) and |q~|; the fp32
  accumulation of 2 d small terms and the sums round by less than 6 d * 2^-24 of the sum of magnitudes (the tensor core
  truncates: twice the rounding). D' = |scale| * gamma * (sum |q~| |u| * (3 * 2^-22 + 6 d * 2^-24) + (2^-24 d + 2^-22
  sqrt(d)) max|q~|) + 2^-22 (|logit| + |lse|). A mass is off by at most sum w * (expm1(D') + 2^-21 + rows * 2^-24) +
  2^-23 * |mass|.
"""

from __future__ import annotations

import numpy as np
import torch

from oracle import codec, tables
from rotation_preconditioned_quantization_b200 import api, inputs, paged

from . import parity


class Pool:
    """A random pool with sequences in it: torch tensors for the kernels, numpy arrays for the reference."""

    def __init__(self, seed, d, b, page, Hkv, lens, spare=2, table_heads=None, max_pages=None, device="cuda",
                 stale=float("nan")):
        rng = np.random.default_rng(seed)
        self.d, self.b, self.page, self.Hkv, self.lens = d, b, page, Hkv, list(lens)
        self.olay, self.lay = codec.Layout(d, b), api.Layout(d, b)
        W = self.lay.words
        counts = [-(-n // page) for n in lens]
        n_pages = max(1, sum(counts) + spare)
        self.words = rng.integers(0, 2 ** 32, (n_pages, Hkv, W, page), dtype=np.uint64).astype(np.uint32)
        self.gamma = (rng.lognormal(0.0, 0.5, (n_pages, Hkv, page)) * 1.5 * np.sqrt(d)).astype(np.float32)
        self.V = inputs.to_bf16(rng.standard_normal((n_pages, Hkv, page, d)).astype(np.float32))
        order = rng.permutation(n_pages)
        self.table = np.full((len(lens), max_pages or max(counts + [1])), -1, np.int32)
        at = 0
        used = np.zeros((n_pages, page), bool)
        for i, n in enumerate(counts):
            self.table[i, :n] = order[at:at + n]
            at += n
            for s in range(lens[i]):
                used[self.table[i, s // page], s % page] = True
        # slots that no sequence holds: whatever a page held before
        self.gamma[np.broadcast_to(~used[:, None], self.gamma.shape)] = stale
        self.V[np.broadcast_to(~used[:, None, :, None], self.V.shape)] = stale
        self.tb = parity.oracle_tables(d, b)
        self.signs = tables.rotation_signs(seed, d, table_heads or Hkv)
        self.free = order[at:]
        if device is not None:
            self.to(device)

    def to(self, device):
        t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(device)  # noqa: E731
        self.cache = paged.PagedCache(t(self.words.view(np.int32)), t(self.gamma), t(self.V).to(torch.bfloat16))
        self.page_table, self.seq_lens = t(self.table), t(np.asarray(self.lens, np.int32))
        self.tables = api.DeviceTables(*self.tb, self.signs, device=device)
        return self

    def slots(self, i, n=None):
        """(pages, offsets) of sequence i's first n slots."""
        s = np.arange(self.lens[i] if n is None else n)
        return self.table[i, s // self.page], s % self.page

    def keys(self, i, h):
        """(gamma [n], rotated unit directions [n][d], V [n][d]) of sequence i, head h in float64."""
        p, o = self.slots(i)
        ix, iy, ir = codec.unpack(self.words[p, h, :, o], self.olay)
        u = codec.decode_rotated(ix, iy, ir, tuple(np.asarray(x, np.float64) for x in self.tb), self.olay)
        return self.gamma[p, h, o].astype(np.float64), u[:, :self.d], self.V[p, h, o].astype(np.float64)


def rotated(pool, q, h):
    R = codec.rotation_matrix(pool.signs[h % len(pool.signs)])
    return q.astype(np.float64) @ R.T


def seen(n, fresh, g, causal):
    """[fresh * g][n] mask of rows (token, group head)."""
    t = np.repeat(np.arange(fresh), g)
    end = n - fresh + t + 1 if causal else np.full(fresh * g, n)
    return np.arange(n)[None] < end[:, None]


def attn(pool, q, cu, causal=True, scale=None):
    """Reference and bounds: out, lse, per-element tolerance factors (sum p |v|, Dmax)."""
    rows, Hq, d = q.shape
    g = Hq // pool.Hkv
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    out, lse = np.zeros((rows, Hq, d)), np.full((rows, Hq), -np.inf)
    mag, dmax = np.zeros((rows, Hq, d)), np.zeros((rows, Hq))
    for i, n in enumerate(pool.lens):
        a, z = cu[i], cu[i + 1]
        if z == a or n == 0:
            continue
        for h in range(pool.Hkv):
            gm, u, V = pool.keys(i, h)
            qr = rotated(pool, q[a:z, h * g:(h + 1) * g].reshape(-1, d), h)
            L = scale * (qr @ u.T) * gm
            ok = seen(n, z - a, g, causal)
            D = abs(scale) * gm * (np.abs(qr) @ np.abs(u).T * (3 * 2.0 ** -11 + 4 * d * 2.0 ** -24) +
                                   2.0 ** -24 * np.sqrt(d) * np.abs(qr).max(-1, keepdims=True))
            L = np.where(ok, L, -np.inf)
            some = ok.any(-1)
            m = np.where(some, L.max(-1, initial=-np.inf), 0.0)
            p = np.exp(L - m[:, None])
            l = p.sum(-1)
            p = p / np.where(l == 0, 1, l)[:, None]
            with np.errstate(divide="ignore"):
                ls = np.log(l) + m
            sl = (slice(a, z), slice(h * g, (h + 1) * g))
            out[sl] = (p @ V).reshape(z - a, g, d)
            mag[sl] = (p @ np.abs(V)).reshape(z - a, g, d)
            lse[sl] = np.where(some, ls, -np.inf).reshape(z - a, g)
            dmax[sl] = np.where(ok, D, 0).max(-1, initial=0).reshape(z - a, g)
    return out, lse, mag, dmax


def check_attn(out, ref, mag, dmax, bf16):
    got = out.float().cpu().numpy().astype(np.float64)
    tol = (np.expm1(2 * dmax)[..., None] + 2.0 ** -8 + 2.0 ** -16) * mag + 2.0 ** -8 * np.abs(ref) * (2 if bf16 else 1)
    err = np.abs(got - ref)
    assert np.isfinite(got).all(), "outputs are not finite"
    bad = err > tol
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside, worst {np.max(err / np.maximum(tol, 1e-30)):.2f} x tolerance"
    return float(np.linalg.norm(got - ref) / max(np.linalg.norm(ref), 1e-30))


def mass(pool, q, lse, cu, prev, decay, causal=True, scale=None):
    """Reference and tolerance of the gathered weight, [B][Hkv][slots] (slots behind a sequence: prev)."""
    rows, Hq, d = q.shape
    g = Hq // pool.Hkv
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    out = prev.astype(np.float64).copy()
    tol = np.zeros_like(out)
    for i, n in enumerate(pool.lens):
        a, z = cu[i], cu[i + 1]
        for h in range(pool.Hkv):
            if n == 0:
                continue
            gm, u, _ = pool.keys(i, h)
            base = float(np.float32(decay)) * prev[i, h, :n].astype(np.float64)
            w, tw = np.zeros(n), np.zeros(n)
            if z > a:
                qr = rotated(pool, q[a:z, h * g:(h + 1) * g].reshape(-1, d), h)
                L = scale * (qr @ u.T) * gm
                ls = lse[a:z, h * g:(h + 1) * g].reshape(-1, 1).astype(np.float64)
                ok = seen(n, z - a, g, causal) & np.isfinite(ls)
                ls = np.where(np.isfinite(ls), ls, 0)
                x = np.where(ok, np.exp(np.where(ok, L - ls, 0)), 0)
                D = abs(scale) * gm * (np.abs(qr) @ np.abs(u).T * (3 * 2.0 ** -22 + 6 * d * 2.0 ** -24) +
                                       (2.0 ** -24 * d + 2.0 ** -22 * np.sqrt(d)) * np.abs(qr).max(-1, keepdims=True))
                D = D + 2.0 ** -22 * (np.abs(L) + np.abs(ls))
                w = x.sum(0)
                tw = (x * (np.expm1(D) + 2.0 ** -21 + len(x) * 2.0 ** -24)).sum(0)
            out[i, h, :n] = base + w
            tol[i, h, :n] = tw + 2.0 ** -23 * np.abs(base + w)
    return out, tol


def select(m, n, keep, sink, recent):
    """Slots that stay of one (sequence, head)."""
    if n <= keep:
        return np.arange(n)
    mid = np.arange(sink, n - recent)
    v = m[mid].astype(np.float64)
    v = np.where(np.isnan(v), -np.inf, v)
    nan = np.isnan(m[mid])
    order = np.lexsort((mid, nan, -v))[:keep - sink - recent]
    return np.sort(np.concatenate([np.arange(sink), mid[order], np.arange(n - recent, n)]))
