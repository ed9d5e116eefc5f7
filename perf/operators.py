"""Cases and plain forms of the paged-cache operators: axis rotary positions, writing a chunk's codes and values into
pages, attention of a chunk of new tokens over the paged compressed cache, the attention weight that each cached token
gathers, and eviction by it.

With ``own`` false, ``run`` computes an operator from its formula with elementary torch operations; with ``own`` true it
calls the package's entry points on the same state.
"""

import math

import numpy as np
import torch

own = False

# Positive halves of the odd-symmetric direction codebooks (b + 1 bits), and the triplet norm codebooks for d = 64
# (b - 1 bits; for d = 128 they are about sqrt(2) smaller, and are given too).
_DIR = {
    2: [0.14300944, 0.38398433, 0.61601567, 0.85699058],
    3: [0.072156653, 0.20219183, 0.32377312, 0.44156352, 0.55843645, 0.67622685, 0.79780817, 0.92784333],
    4: [0.036160469, 0.10451804, 0.16968697, 0.23239897, 0.2933265, 0.35305834, 0.41207311, 0.4707267, 0.52927333,
        0.58792692, 0.64694166, 0.7066735, 0.76760101, 0.83031303, 0.89548194, 0.96383953],
}
_RHO = {
    (64, 2): [0.14256603, 0.27726799],
    (64, 3): [0.099079467, 0.17578395, 0.25094494, 0.34536657],
    (64, 4): [0.06753625, 0.11564261, 0.15666914, 0.19588847, 0.23605715, 0.27994666, 0.33219224, 0.40553474],
    (128, 2): [0.1007357, 0.19714524],
    (128, 3): [0.070077352, 0.12466352, 0.17862301, 0.24735287],
    (128, 4): [0.04780094, 0.081948116, 0.11117401, 0.13923694, 0.16813865, 0.19994155, 0.23816134, 0.29258722],
}


def listed():
    return [
        # one decode step's queries and keys of a few sequences, text positions, far into a long context
        {"name": "rope_step", "op": "rope", "tokens": 4, "hq": 32, "hk": 8, "d": 128, "axes": 1, "start": 131072,
         "bf16": True, "interleaved": False, "per_axis": False, "inverse": False},
        # a video chunk: time, height and width axes with their own frequencies
        {"name": "rope_video", "op": "rope", "tokens": 16384, "hq": 16, "hk": 16, "d": 64, "axes": 3, "start": 65536,
         "bf16": True, "interleaved": False, "per_axis": True, "inverse": False},
        # one token of each of 64 running sequences goes to its page
        {"name": "write_step", "op": "write", "B": 64, "hkv": 8, "d": 128, "b": 3, "page": 64, "ctx": 2048, "chunk": 1,
         "ragged": True},
        # prompt chunks of four sequences, lengths that end inside pages
        {"name": "write_chunk", "op": "write", "B": 4, "hkv": 8, "d": 128, "b": 4, "page": 64, "ctx": 4096,
         "chunk": 2047, "ragged": True},
        # one decode step of one sequence at a long context
        {"name": "attn_step", "op": "attn", "B": 1, "hq": 32, "hkv": 8, "d": 128, "b": 3, "page": 64, "ctx": 32767,
         "chunk": 1, "ragged": False, "causal": True, "bf16": True},
        # a mixed batch: short chunks and single tokens over small pages
        {"name": "attn_mixed", "op": "attn", "B": 7, "hq": 32, "hkv": 8, "d": 128, "b": 4, "page": 16, "ctx": 5000,
         "chunk": 37, "ragged": True, "causal": True, "bf16": True},
        # a prompt chunk over a long cached prefix
        {"name": "attn_chunk", "op": "attn", "B": 1, "hq": 32, "hkv": 8, "d": 128, "b": 3, "page": 64, "ctx": 32768,
         "chunk": 512, "ragged": False, "causal": True, "bf16": True},
        # a video chunk that sees itself whole and all frames before it
        {"name": "attn_video", "op": "attn", "B": 1, "hq": 16, "hkv": 16, "d": 64, "b": 2, "page": 128, "ctx": 65536,
         "chunk": 1024, "ragged": False, "causal": False, "bf16": True},
        # attention weight gathered in one decode step of four sequences
        {"name": "mass_step", "op": "mass", "B": 4, "hq": 32, "hkv": 8, "d": 128, "b": 3, "page": 64, "ctx": 32767,
         "chunk": 1, "ragged": True, "causal": True, "bf16": True},
        # attention weight gathered by a prompt chunk
        {"name": "mass_chunk", "op": "mass", "B": 1, "hq": 32, "hkv": 8, "d": 128, "b": 3, "page": 64, "ctx": 16384,
         "chunk": 512, "ragged": False, "causal": True, "bf16": True},
        # two short sequences cut back to a small budget
        {"name": "evict_small", "op": "evict", "B": 2, "hkv": 16, "d": 64, "b": 2, "page": 16, "len": 1500, "keep": 499,
         "sink": 4, "recent": 64, "ragged": True},
        # long sequences cut back to a quarter
        {"name": "evict_long", "op": "evict", "B": 4, "hkv": 8, "d": 128, "b": 3, "page": 64, "len": 32768, "keep": 8192,
         "sink": 4, "recent": 512, "ragged": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "write", "attn", "attn", "mass", "evict"])
    d, b, page = rng.choice([64, 128]), rng.choice([2, 3, 4]), rng.choice([16, 32, 48, 64, 128, 256])
    if op == "rope":
        hq, hk = rng.choice([1, 4, 16, 32]), rng.choice([0, 1, 4, 8, 16])
        d = rng.choice([64, 128, 256])
        bf16 = rng.random() < 0.7
        most = 16384 * 32 * 64 // ((hq + hk) * d) // (1 if bf16 else 2)
        return {"op": op, "tokens": _log_int(rng, 1, min(16384, most)), "hq": hq, "hk": hk, "d": d,
                "axes": rng.choice([1, 2, 3, 4]), "start": _log_int(rng, 1, 1 << 20), "bf16": bf16,
                "interleaved": rng.random() < 0.5, "per_axis": rng.random() < 0.5, "inverse": rng.random() < 0.5}
    hkv = rng.choice([1, 2, 4, 8, 16])
    if op == "write":
        B = _log_int(rng, 1, 64)
        return {"op": op, "B": B, "hkv": hkv, "d": d, "b": b, "page": page, "ctx": _log_int(rng, 1, 4096),
                "chunk": _log_int(rng, 1, max(1, 40000 // (B * hkv))), "ragged": rng.random() < 0.7}
    if op == "evict":
        B = rng.choice([1, 2, 3, 4])
        n = _log_int(rng, 2, 32768)
        keep = _log_int(rng, 1, n)
        if n * B * hkv > 1 << 20:
            hkv = max(1, (1 << 20) // (n * B))
        keep = min(keep, max(1, 8192 * 32 // (B * hkv)))
        sink = min(rng.choice([0, 4, 16]), keep)
        return {"op": op, "B": B, "hkv": hkv, "d": d, "b": b, "page": page, "len": n, "keep": keep, "sink": sink,
                "recent": min(rng.choice([0, 32, 256]), keep - sink), "ragged": rng.random() < 0.5}
    g = rng.choice([1, 2, 4, 5, 8])
    B = rng.choice([1, 1, 2, 3, 8])
    chunk = _log_int(rng, 1, 1024)
    ctx = _log_int(rng, 1, 65536)
    most = (16 * 1024 * 66560 * 64 if op == "attn" else 8 * 2048 * 16640 * 128) // (2 * d)  # (row, key) pairs
    while B * hkv * g * chunk * (ctx + chunk) > most or B * hkv * (ctx + chunk) > 1 << 20:
        if B > 1:
            B -= 1
        elif hkv > 1:
            hkv //= 2
        elif chunk > 64 and g > 1:
            g = 1
        else:
            ctx = max(1, ctx // 2)
    return {"op": op, "B": B, "hq": g * hkv, "hkv": hkv, "d": d, "b": b, "page": page, "ctx": ctx, "chunk": chunk,
            "ragged": rng.random() < 0.5, "causal": rng.random() < 0.7, "bf16": rng.random() < 0.8}


# ------------------------------------------------------------------ sizes that follow from a case
def _spread(most, B, ragged, mul, add, least):
    """One length per sequence, the first the largest."""
    if not ragged:
        return [most] * B
    return [most if i == 0 else least + (most - least) * ((i * mul + add) % 17) // 17 for i in range(B)]


def _lengths(c):
    """(new tokens, tokens cached before them) per sequence."""
    return _spread(c["chunk"], c["B"], c["ragged"], 7, 3, 1), _spread(c["ctx"], c["B"], c["ragged"], 5, 9, 0)


def _bits(c):
    C, T = 3 * c["b"] + 1, -(-c["d"] // 3)
    return C, T, -(-T * C // 32)


def _pairs(c):
    """(query token, key) pairs that the mask leaves, over one query head."""
    n = 0
    for new, old in zip(*_lengths(c)):
        n += new * old + (new * (new + 1) // 2 if c["causal"] else new * new)
    return n


def work(c):
    op = c["op"]
    if op == "rope":
        n = c["tokens"] * (c["hq"] + c["hk"]) * c["d"]
        return {"bytes": 2 * n * (2 if c["bf16"] else 4) + 4 * c["axes"] * c["tokens"], "flops": 3 * n}
    W = _bits(c)[2]
    if op == "write":
        n = sum(_lengths(c)[0]) * c["hkv"]
        return {"bytes": 2 * n * (4 * W + 4 + 2 * c["d"]), "flops": 0}
    if op == "evict":
        lens = _spread(c["len"], c["B"], c["ragged"], 5, 9, 1)
        kept = sum(min(n, c["keep"]) for n in lens) * c["hkv"]
        return {"bytes": 4 * sum(lens) * c["hkv"] + kept * (2 * (4 * W + 4 + 2 * c["d"]) + 8), "flops": sum(lens) * c["hkv"]}
    new, old = _lengths(c)
    units, rows = sum(a + b for a, b in zip(new, old)) * c["hkv"], sum(new) * c["hq"]
    q = rows * c["d"] * (2 if c["bf16"] else 4)
    if op == "attn":
        return {"bytes": units * (4 * W + 4 + 2 * c["d"]) + q + 2 * rows * c["d"], "flops": 4 * c["d"] * c["hq"] * _pairs(c)}
    return {"bytes": units * (4 * W + 4 + 8) + q + 4 * rows, "flops": 2 * c["d"] * c["hq"] * _pairs(c)}


# ------------------------------------------------------------------ inputs
def _normal(g, shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _pool(g, c, n_pages):
    """Pages as a running program holds them: every bit pattern is a valid code; norms as of keys with a few strong
    channels and a per-token factor."""
    W = _bits(c)[2]
    packed = torch.randint(-2 ** 31, 2 ** 31, (n_pages, c["hkv"], W, c["page"]), generator=g, device="cuda",
                           dtype=torch.int32)
    gamma = torch.empty((n_pages, c["hkv"], c["page"]), device="cuda").log_normal_(0.0, 0.5, generator=g)
    gamma *= 1.5 * math.sqrt(c["d"])
    return packed, gamma, _normal(g, (n_pages, c["hkv"], c["page"], c["d"]))


def _table(g, counts, n_pages):
    """Page table [B][most]: pages in no order, -1 behind a sequence's last."""
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    t = torch.full((len(counts), max(counts)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(counts):
        t[i, :n] = order[at:at + n]
        at += n
    return t


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _codec(s, c, g):
    half = np.array(_DIR[c["b"]], np.float32)
    s["dir_c"] = np.concatenate([-half[::-1], half])
    s["rho_c"] = np.array(_RHO[(c["d"], c["b"])], np.float32)
    s["signs"] = torch.randint(0, 2, (c["hkv"], c["d"]), generator=g, device="cuda").float().mul_(2).sub_(1).cpu().numpy()
    i = torch.arange(c["d"], device="cuda")
    par = i[:, None] & i[None, :]
    for sh in (4, 2, 1):
        par = par ^ (par >> sh)
    s["levels"] = torch.from_numpy(s["dir_c"]).cuda()
    s["norms"] = torch.from_numpy(s["rho_c"]).cuda()
    # rotation of head h: R[h] = H diag(signs[h]) / sqrt(d), H the Walsh-Hadamard matrix in Sylvester order
    s["R"] = (1 - 2 * (par & 1)).float()[None] * torch.from_numpy(s["signs"]).cuda()[:, None, :] / math.sqrt(c["d"])


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    op = c["op"]
    if op == "rope":
        dt = torch.bfloat16 if c["bf16"] else torch.float32
        s["q"] = _normal(g, (c["tokens"], c["hq"], c["d"]), dt)
        s["k"] = _normal(g, (c["tokens"], c["hk"], c["d"]), dt) if c["hk"] else None
        n, a = c["d"] // 2, c["axes"]
        s["sections"] = [n - (a - 1) * (n // a)] + [n // a] * (a - 1)
        t = torch.arange(c["tokens"], device="cuda")
        jitter = int(torch.randint(0, 64, (1,), generator=g, device="cuda"))
        axes = [c["start"] + jitter + (t if a == 1 else t // 1024), t // 32 % 32, t % 32, t % 7]  # frame, row, column, track
        s["positions"] = torch.stack(axes[:a]).to(torch.int32)
        return s
    P = c["page"]
    if op == "write":
        new, old = _lengths(c)
        total = sum(new)
        counts = [-(-(a + b) // P) for a, b in zip(new, old)]
        n_pages = sum(counts) + 3
        s["packed"], s["gamma"], s["V"] = _pool(g, c, n_pages)
        s["table"] = _table(g, counts, n_pages)
        cap = -(-total // 4) * 4
        s["new_packed"] = torch.randint(-2 ** 31, 2 ** 31, (c["hkv"], _bits(c)[2], cap), generator=g, device="cuda",
                                        dtype=torch.int32)
        s["new_gamma"] = torch.empty((c["hkv"], cap), device="cuda").log_normal_(2.0, 0.5, generator=g)
        s["new_V"] = _normal(g, (total, c["hkv"], c["d"]))
        s["total"], s["starts"] = total, _ints(old)
        s["cu"] = _ints([0] + list(np.cumsum(new)))
        return s
    if op == "evict":
        lens = _spread(c["len"], c["B"], c["ragged"], 5, 9, 1)
        kept = [min(n, c["keep"]) for n in lens]
        counts, into = [-(-n // P) for n in lens], [-(-n // P) for n in kept]
        n_pages = sum(counts) + sum(into)
        s["packed"], s["gamma"], s["V"] = _pool(g, c, n_pages)
        t = _table(g, counts + into, n_pages)
        s["table"] = t[:c["B"], :max(counts)].contiguous()
        s["into"] = t[c["B"]:, :max(into)].contiguous()
        s["lens"] = _ints(lens)
        # gathered weight: heavy-tailed, with tokens that nothing has looked at yet (exact zeros, so ties)
        m = torch.empty((c["B"], c["hkv"], max(lens)), device="cuda").log_normal_(-3.0, 2.0, generator=g)
        m[torch.rand(m.shape, generator=g, device="cuda") < 0.2] = 0.0
        s["mass"] = m
        return s
    new, old = _lengths(c)
    counts = [-(-(a + b) // P) for a, b in zip(new, old)]
    n_pages = sum(counts) + 2
    s["packed"], s["gamma"], s["V"] = _pool(g, c, n_pages)
    s["table"] = _table(g, counts, n_pages)
    s["lens"] = _ints([a + b for a, b in zip(new, old)])
    s["cu"] = _ints([0] + list(np.cumsum(new)))
    s["max_q"], s["max_kv"] = max(new), max(a + b for a, b in zip(new, old))
    _codec(s, c, g)
    s["q"] = _normal(g, (sum(new), c["hq"], c["d"]), torch.bfloat16 if c["bf16"] else torch.float32)
    if op == "mass":
        L, seen = _scores(s)
        lse = torch.logsumexp(L, -1)  # [B][hkv][max_q * g]
        del L
        B, g_ = c["B"], c["hq"] // c["hkv"]
        lse = lse.view(B, c["hkv"], s["max_q"], g_).permute(0, 2, 1, 3).reshape(B * s["max_q"], c["hq"])
        s["lse"] = lse[seen.reshape(-1)].contiguous()
        s["mass"] = torch.empty((B, c["hkv"], s["max_kv"]), device="cuda").log_normal_(-3.0, 2.0, generator=g)
        s["new_mass"] = torch.zeros_like(s["mass"])
    return s


# ------------------------------------------------------------------ plain forms
def _rope_plain(s):
    c = s["case"]
    n, dev = c["d"] // 2, "cuda"
    sec = s["sections"]
    axis = torch.repeat_interleave(torch.arange(len(sec), device=dev), torch.tensor(sec, device=dev))
    i = torch.arange(n, device=dev, dtype=torch.float64)
    if c["per_axis"]:
        first = torch.tensor([0] + list(np.cumsum(sec))[:-1], device=dev, dtype=torch.float64)
        share = (i - first[axis]) / torch.tensor(sec, device=dev, dtype=torch.float64)[axis]
    else:
        share = i / n
    angle = s["positions"].double().T[:, axis] * torch.pow(torch.tensor(10000.0, device=dev, dtype=torch.float64), -share)
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if c["inverse"]:
        sin = -sin

    def turn(x):
        y = x.float()
        a, b = (y[..., 0::2], y[..., 1::2]) if c["interleaved"] else (y[..., :n], y[..., n:])
        lo, hi = a * cos - b * sin, b * cos + a * sin
        y = torch.stack((lo, hi), -1).flatten(-2) if c["interleaved"] else torch.cat((lo, hi), -1)
        return y.to(x.dtype)

    return [turn(s["q"])] + ([turn(s["k"])] if s["k"] is not None else [])


def _write_plain(s):
    c = s["case"]
    cu, t = s["cu"].long(), torch.arange(s["total"], device="cuda")
    seq = torch.searchsorted(cu, t, right=True) - 1
    slot = s["starts"].long()[seq] + t - cu[seq]
    page, off = s["table"].long()[seq, slot // c["page"]], slot % c["page"]
    s["packed"][page, :, :, off] = s["new_packed"][:, :, :s["total"]].permute(2, 0, 1)
    s["gamma"][page, :, off] = s["new_gamma"][:, :s["total"]].T
    s["V"][page, :, off] = s["new_V"]
    return s["packed"], s["gamma"], s["V"]


def _gather(s, what):
    """A pool's pages in the sequences' order: [B][hkv][...][slots] with the page's last but `tail` axes kept."""
    x = s[what][s["table"].long().clamp(min=0)]
    if what == "packed":
        return x.permute(0, 2, 3, 1, 4).flatten(3)
    return x.transpose(1, 2).flatten(2, 3)


def _directions(s):
    """Decoded rotated unit directions [B][hkv][slots][d]."""
    c = s["case"]
    b, (C, T, W) = c["b"], _bits(c)
    words = _gather(s, "packed").long() & 0xFFFFFFFF
    at = torch.arange(T, device="cuda") * C
    first, sh = at // 32, (at % 32)[:, None]
    code = ((words[:, :, first] | (words[:, :, (first + 1).clamp(max=W - 1)] << 32)) >> sh) & ((1 << C) - 1)
    half = 1 << b
    mx, my = code & (half - 1), (code >> b) & (half - 1)
    sx, sy = (code >> (2 * b)) & 1, (code >> (2 * b + 1)) & 1
    x = s["levels"][torch.where(sx > 0, half - 1 - mx, half + mx)]
    y = s["levels"][torch.where(sy > 0, half - 1 - my, half + my)]
    z = 1 - x.abs() - y.abs()
    fx, fy = torch.copysign(1 - y.abs(), x), torch.copysign(1 - x.abs(), y)
    x, y = torch.where(z < 0, fx, x), torch.where(z < 0, fy, y)
    r = s["norms"][code >> (2 * b + 2)] / torch.sqrt(x * x + y * y + z * z)
    u = torch.stack((x * r, y * r, z * r), 3)  # [B][hkv][T][3][slots]
    return u.flatten(2, 3)[:, :, :c["d"]].transpose(2, 3)


def _scores(s):
    """Masked scaled logits [B][hkv][max_q * g][slots], and which query rows of the padded batch are there."""
    c = s["case"]
    B, g, most = c["B"], c["hq"] // c["hkv"], s["max_q"]
    cu, lens = s["cu"].long(), s["lens"].long()
    t = torch.arange(most, device="cuda")
    new = cu[1:] - cu[:-1]
    seen = t[None] < new[:, None]
    q = s["q"].float()[(cu[:-1, None] + t).clamp(max=s["q"].shape[0] - 1)]
    q = q.view(B, most, c["hkv"], g, c["d"]).permute(0, 2, 1, 3, 4).flatten(2, 3)
    q = q @ s["R"].transpose(1, 2)
    L = (q @ _directions(s).transpose(2, 3)) * (_gather(s, "gamma") / math.sqrt(c["d"]))[:, :, None]
    j = torch.arange(L.shape[-1], device="cuda")
    end = (lens - new)[:, None] + t + 1 if c["causal"] else lens[:, None].expand(B, most)
    ok = (j < end[..., None]) & seen[..., None]
    return L.masked_fill_(~ok.repeat_interleave(g, 1)[:, None], -math.inf), seen


def _attn_plain(s):
    c = s["case"]
    L, seen = _scores(s)
    m = L.amax(-1, keepdim=True)
    p = torch.exp_(L.sub_(torch.where(m.isinf(), 0.0, m)))
    l = p.sum(-1, keepdim=True)
    V = _gather(s, "V").float()
    V = V.masked_fill_((torch.arange(V.shape[2], device="cuda") >= s["lens"][:, None])[:, None, :, None], 0.0)
    o = (p @ V) / torch.where(l == 0, 1.0, l)
    o = o.view(c["B"], c["hkv"], s["max_q"], -1, c["d"]).permute(0, 2, 1, 3, 4).flatten(2, 3)
    return o[seen].to(torch.bfloat16)


def _mass_plain(s):
    c = s["case"]
    L, seen = _scores(s)
    lse = torch.full((c["B"], s["max_q"], c["hq"]), math.inf, device="cuda")
    lse[seen] = s["lse"]
    lse = lse.view(c["B"], s["max_q"], c["hkv"], -1).permute(0, 2, 1, 3).flatten(2, 3)
    w = torch.exp_(L.sub_(lse[..., None])).sum(2)[:, :, :s["max_kv"]]
    there = torch.arange(s["max_kv"], device="cuda") < s["lens"][:, None, None]
    s["new_mass"].copy_(torch.where(there, 0.9 * s["mass"] + w, s["new_mass"]))
    return s["new_mass"]


def _evict_plain(s):
    c = s["case"]
    B, H, P, keep = c["B"], c["hkv"], c["page"], c["keep"]
    n = s["lens"].long()[:, None, None]
    j = torch.arange(s["mass"].shape[-1], device="cuda")
    w = torch.where((j < c["sink"]) | (j >= n - c["recent"]), math.inf, s["mass"])
    w = torch.where(j < n, w, -math.inf)
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :keep]
    there = torch.arange(keep, device="cuda") < n
    kept = torch.sort(torch.where(there.expand(B, H, keep), order, j.numel()), -1).values
    seq = torch.arange(B, device="cuda")[:, None, None].expand(B, H, keep)[there.expand(B, H, keep)]
    head = torch.arange(H, device="cuda")[:, None].expand(B, H, keep)[there.expand(B, H, keep)]
    to = torch.arange(keep, device="cuda").expand(B, H, keep)[there.expand(B, H, keep)]
    src = kept[there.expand(B, H, keep)]
    a, ao = s["table"].long()[seq, src // P], src % P
    z, zo = s["into"].long()[seq, to // P], to % P
    s["packed"][z, head, :, zo] = s["packed"][a, head, :, ao]
    s["gamma"][z, head, zo] = s["gamma"][a, head, ao]
    s["V"][z, head, zo] = s["V"][a, head, ao]
    mass = torch.zeros((B, H, keep), device="cuda")
    mass[seq, head, to] = s["mass"][seq, head, src]
    kept = torch.where(there, kept, -1).to(torch.int32)
    return {"lens": s["lens"].clamp(max=keep), "kept": kept, "mass": mass, "packed": s["packed"], "gamma": s["gamma"],
            "V": s["V"]}


# ------------------------------------------------------------------ the package's calls
def _handle(s):
    """What a program makes once and keeps: layout, tables, the cache object over its pools, a workspace."""
    if "handle" not in s:
        import rotation_preconditioned_quantization_b200 as api

        c, h = s["case"], {"api": api}
        if c["op"] == "rope":
            h["table"] = api.RopeTable(s["sections"], theta=10000.0, per_axis=c["per_axis"])
        if c["op"] != "rope":
            h["layout"] = api.Layout(c["d"], c["b"])
            h["cache"] = api.PagedCache(s["packed"], s["gamma"], s["V"])
        if c["op"] == "write":
            h["staged"] = api.Cache(s["new_packed"], s["new_gamma"], length=s["total"])
        if "signs" in s:
            mid = lambda v: (v[1:] + v[:-1]) / 2  # noqa: E731
            h["tables"] = api.DeviceTables(s["dir_c"], mid(s["dir_c"]), s["rho_c"], mid(s["rho_c"]), s["signs"])
        h["workspace"] = api.Workspace(0)
        s["handle"] = h
    return s["handle"]


def _run_own(s):
    c, h = s["case"], _handle(s)
    api = h["api"]
    if c["op"] == "rope":
        out = api.rope(s["q"], s["positions"], h["table"], k=s["k"], interleaved=c["interleaved"], inverse=c["inverse"])
        return list(out) if s["k"] is not None else [out]
    if c["op"] == "write":
        api.paged_write(h["layout"], h["staged"], s["new_V"], h["cache"], s["table"], s["starts"], s["cu"])
        return s["packed"], s["gamma"], s["V"]
    if c["op"] == "attn":
        return api.paged_attn(h["layout"], h["tables"], s["q"], h["cache"], s["table"], s["lens"], cu_q=s["cu"],
                              causal=c["causal"], dtype=torch.bfloat16, workspace=h["workspace"])
    if c["op"] == "mass":
        return api.paged_mass(h["layout"], h["tables"], s["q"], s["lse"], h["cache"], s["table"], s["lens"], s["mass"],
                              cu_q=s["cu"], causal=c["causal"], decay=0.9, out=s["new_mass"], workspace=h["workspace"])
    lens, kept, mass = api.paged_evict(h["layout"], h["cache"], s["table"], s["lens"], s["mass"], c["keep"], s["into"],
                                       sink=c["sink"], recent=c["recent"])
    return {"lens": lens, "kept": kept, "mass": mass, "packed": s["packed"], "gamma": s["gamma"], "V": s["V"]}


def run(s):
    if own:
        return _run_own(s)
    op = s["case"]["op"]
    if op == "rope":
        return _rope_plain(s)
    if op == "write":
        return _write_plain(s)
    if op == "attn":
        return _attn_plain(s)
    if op == "mass":
        return _mass_plain(s)
    return _evict_plain(s)


# ------------------------------------------------------------------ the definition in 64 bits
def _decoded(s, i, n):
    """gamma * R^T-free decoded keys of sequence i in 64 bits: [hkv][n][d], by a table of every code."""
    c = s["case"]
    b, (C, T, W) = c["b"], _bits(c)
    codes = np.arange(1 << C)
    level = s["dir_c"].astype(np.float64)
    cell = lambda m, sign: np.where(sign == 1, (1 << b) - 1 - m, (1 << b) + m)  # noqa: E731
    lo = (1 << b) - 1
    xi, eta = level[cell(codes & lo, codes >> 2 * b & 1)], level[cell(codes >> b & lo, codes >> 2 * b + 1 & 1)]
    z = 1 - np.abs(xi) - np.abs(eta)
    x = np.where(z < 0, np.sign(xi) * (1 - np.abs(eta)), xi)
    y = np.where(z < 0, np.sign(eta) * (1 - np.abs(xi)), eta)
    v = np.stack((x, y, z), -1)
    v *= (s["rho_c"].astype(np.float64)[codes >> 2 * b + 2] / np.linalg.norm(v, axis=-1))[:, None]
    v = torch.from_numpy(v).cuda()
    pages = s["table"][i, :-(-n // c["page"])].long()
    words = s["packed"][pages].permute(1, 0, 3, 2).reshape(c["hkv"], -1, W)[:, :n].long() & 0xFFFFFFFF
    out = []
    for t in range(T):
        bit = t * C
        code = words[..., bit // 32] >> bit % 32
        if bit % 32 + C > 32:
            code = code | words[..., bit // 32 + 1] << (32 - bit % 32)
        out.append(v[code & ((1 << C) - 1)])
    k = torch.cat(out, -1)[..., :c["d"]]
    return k * s["gamma"][pages].permute(1, 0, 2).reshape(c["hkv"], -1)[:, :n, None].double(), pages


def _exact_scores(s, i, h, k):
    """Masked scaled logits of sequence i, cache head h: [new][g][n]."""
    c = s["case"]
    g = c["hq"] // c["hkv"]
    a, z = int(s["cu"][i]), int(s["cu"][i + 1])
    n = int(s["lens"][i])
    q = s["q"][a:z, h * g:(h + 1) * g].double() * torch.from_numpy(s["signs"][h]).cuda().double()
    m = q.shape
    w = 1
    while w < c["d"]:  # Walsh-Hadamard butterflies
        q = q.reshape(m[0], m[1], -1, 2, w)
        q = torch.stack((q[..., 0, :] + q[..., 1, :], q[..., 0, :] - q[..., 1, :]), -2)
        w *= 2
    q = q.reshape(m) / math.sqrt(c["d"])
    L = (q.reshape(-1, c["d"]) @ k.T).reshape(m[0], m[1], n) / math.sqrt(c["d"])
    if c["causal"]:
        last = n - m[0] + torch.arange(m[0], device="cuda")
        L[(torch.arange(n, device="cuda")[None] > last[:, None])[:, None].expand_as(L)] = -math.inf
    return L, a, z


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "rope":
        n = c["d"] // 2
        axis, freq = [], []
        for a, size in enumerate(s["sections"]):
            axis += [a] * size
            freq += [10000.0 ** -(f / size) for f in range(size)]
        if not c["per_axis"]:
            freq = [10000.0 ** -(f / n) for f in range(n)]
        ang = s["positions"].cpu().numpy().astype(np.float64)[axis].T * np.array(freq)
        e = torch.from_numpy(np.exp((-1j if c["inverse"] else 1j) * ang)).cuda()[:, None]
        res = []
        for x in (s["q"], s["k"]):
            if x is None:
                continue
            y = x.double()
            pair = torch.view_as_complex(y.reshape(*y.shape[:-1], n, 2)) if c["interleaved"] else torch.complex(y[..., :n], y[..., n:])
            pair = pair * e
            res.append(torch.view_as_real(pair).flatten(-2) if c["interleaved"] else torch.cat((pair.real, pair.imag), -1))
        return res
    if c["op"] in ("write", "evict"):
        return None  # values are moved, none is computed
    g = c["hq"] // c["hkv"]
    out = torch.zeros((s["q"].shape[0], c["hq"], c["d"]), dtype=torch.float64, device="cuda") if c["op"] == "attn" else s["new_mass"].double()
    for i in range(c["B"]):
        n = int(s["lens"][i])
        k, pages = _decoded(s, i, n)
        for h in range(c["hkv"]):
            L, a, z = _exact_scores(s, i, h, k[h])
            if c["op"] == "attn":
                V = s["V"][pages, h].reshape(-1, c["d"])[:n].double()
                out[a:z, h * g:(h + 1) * g] = torch.softmax(L, -1) @ V
            else:
                w = torch.exp(L - s["lse"][a:z, h * g:(h + 1) * g, None].double()).sum((0, 1))
                out[i, h, :n] = 0.9 * s["mass"][i, h, :n].double() + w
    return out
