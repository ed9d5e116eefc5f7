"""GPU tests of octo_rope against a float64 rotation.

Bounds: an output is a cos w -+ b sin w with the pair's magnitude r = hypot(a, b). Cosine and sine carry the angle's error
(fraction of a turn to 2^-32 plus its rounding to fp32, 2^-25 of a half turn: together below 2^-22.6 rad) and sincospif's
2 ulp (2^-23 each); two products and a sum round once each: below 2^-20 r in all, plus half a step of the output type."""

import numpy as np
import pytest
import torch

from rotation_preconditioned_quantization_b200 import inputs, paged

pytestmark = pytest.mark.gpu

ULP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def _angles(pos, sections, theta, per_axis):
    F = sum(sections)
    cols, i = [], 0
    for a, s in enumerate(sections):
        for j in range(s):
            e = j / s if per_axis else i / F
            cols.append(pos[a].astype(np.longdouble) * np.longdouble(theta) ** np.longdouble(-e))
            i += 1
    return np.stack(cols, -1).astype(np.longdouble) if cols else np.zeros((pos.shape[1], 0), np.longdouble)


def _ref(x, w, interleaved, inverse):
    """(rotated, magnitude of each element's pair)"""
    F = w.shape[1]
    c, s = np.cos(w)[:, None].astype(np.float64), np.sin(w)[:, None].astype(np.float64)
    if inverse:
        s = -s
    y, r = x.astype(np.float64).copy(), np.abs(x.astype(np.float64))
    ia, ib = (np.arange(F) * 2, np.arange(F) * 2 + 1) if interleaved else (np.arange(F), np.arange(F) + F)
    a, b = x[..., ia].astype(np.float64), x[..., ib].astype(np.float64)
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    r[..., ia] = r[..., ib] = np.hypot(a, b)
    return y, r


def _check(got, x, w, interleaved, inverse):
    ref, r = _ref(x.float().cpu().numpy(), w, interleaved, inverse)
    err = np.abs(got.float().cpu().numpy().astype(np.float64) - ref)
    tol = 2.0 ** -20 * r + ULP[got.dtype] * np.abs(ref)
    assert np.all(err <= tol), f"worst {np.max(err / np.maximum(tol, 1e-30)):.2f} x tolerance"


def _x(seed, shape, dtype):
    return torch.from_numpy(inputs.normal(seed, shape)).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("d,sections,per_axis", [(64, (32,), False), (64, (12, 10, 10), True), (128, (16, 24, 24), False),
                                                 (256, (32, 32, 32, 32), True), (64, (8, 8), False), (128, (64,), True),
                                                 (6, (1, 2), False), (2, (1,), False), (80, (3, 0, 30), True), (64, (0,), False)])
def test_every_form(cuda_ok, d, sections, per_axis, interleaved, inverse, dtype):
    T, rng = 37, np.random.default_rng(d)
    pos = rng.integers(-1000, 100000, (len(sections), T)).astype(np.int32)
    q, k = _x(1, (T, 5, d), dtype), _x(2, (T, 2, d), dtype)
    table = paged.RopeTable(sections, 10000.0, per_axis)
    qo, ko = paged.rope(q, torch.from_numpy(pos).cuda(), table, k=k, interleaved=interleaved, inverse=inverse)
    w = _angles(pos, sections, 10000.0, per_axis)
    _check(qo, q, w, interleaved, inverse)
    _check(ko, k, w, interleaved, inverse)
    F2 = 2 * sum(sections)
    assert torch.equal(qo[..., F2:], q[..., F2:])


@pytest.mark.parametrize("T", [1, 2, 3, 295, 296, 297, 2000, 9001])
def test_token_counts(cuda_ok, T):
    pos = np.stack([np.arange(T), np.arange(T) // 7, np.arange(T) % 7]).astype(np.int32)
    q = _x(T, (T, 3, 64), torch.bfloat16)
    out = paged.rope(q, torch.from_numpy(pos).cuda(), paged.RopeTable((12, 10, 10), 10000.0, True))
    _check(out, q, _angles(pos, (12, 10, 10), 10000.0, True), False, False)


def test_far_positions(cuda_ok):
    """Every 32-bit position: whole turns drop out exactly."""
    pos = np.array([[0, 1, -1, 2 ** 20, 10 ** 6 + 1, 2 ** 31 - 1, -2 ** 31, 123456789]], np.int32)
    for theta in (1.0, 10000.0, 5e8):
        q = _x(3, (8, 2, 128), torch.float32)
        out = paged.rope(q, torch.from_numpy(pos).cuda(), paged.RopeTable((64,), theta))
        # long double angles of 2^31 rad are right to 2^-33; the frequencies to 2^-64 of a turn, times 2^31
        _check(out, q, _angles(pos, (64,), theta, False), False, False)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_in_place_and_strided(cuda_ok, dtype):
    T, d = 50, 64
    pos = np.arange(T)[None].astype(np.int32) * 100
    table, p = paged.RopeTable((32,)), torch.from_numpy(pos).cuda()
    w = _angles(pos, (32,), 10000.0, False)
    fused = _x(4, (T, 3, 4, d), dtype)  # a fused projection: q, k, v
    q, k = fused[:, 0], fused[:, 1, :2]
    q0, k0, rest = q.clone(), k.clone(), fused[:, 2].clone()
    paged.rope(q, p, table, k=k, out=q, k_out=k)
    _check(q, q0, w, False, False)
    _check(k, k0, w, False, False)
    assert torch.equal(fused[:, 2], rest)
    odd = torch.zeros(T * 4 * 65 + 1, dtype=dtype, device="cuda")[1:].view(T, 4, 65)[..., :64]  # rows off 16 bytes
    odd.copy_(q0)
    _check(paged.rope(odd, p, table), q0, w, False, False)
    _check(paged.rope(odd, p, table, interleaved=True), q0, w, True, False)


def test_inverse_undoes_and_is_the_gradient(cuda_ok):
    T, d = 20, 32
    pos = torch.arange(T, dtype=torch.int32, device="cuda")[None] * 31
    table = paged.RopeTable((16,))
    q, g = _x(5, (T, 2, d), torch.float32), _x(6, (T, 2, d), torch.float32)
    y = paged.rope(q, pos, table)
    back = paged.rope(y, pos, table, inverse=True)
    r = torch.hypot(q[..., :16], q[..., 16:]).repeat(1, 1, 2)
    assert torch.all((back - q).abs() <= 2.0 ** -18 * r)
    # <rope(q), g> has gradient rope^T(g): against differences along random directions
    grad = paged.rope(g, pos, table, inverse=True).double()
    for s in range(4):
        e = _x(10 + s, (T, 2, d), torch.float32)
        step = 0.5  # the map is linear: any step gives the derivative
        diff = ((paged.rope(q + step * e, pos, table).double() - paged.rope(q - step * e, pos, table).double()) * g.double()).sum() / (2 * step)
        assert abs(float(diff - (grad * e.double()).sum())) <= 2.0 ** -17 * float((g.abs() * (q.abs() + e.abs())).sum())


def test_no_tokens_no_heads(cuda_ok):
    table = paged.RopeTable((32,))
    p = torch.zeros(1, 0, dtype=torch.int32, device="cuda")
    assert paged.rope(torch.zeros(0, 4, 64, device="cuda"), p, table).shape == (0, 4, 64)
    p = torch.zeros(1, 3, dtype=torch.int32, device="cuda")
    assert paged.rope(torch.zeros(3, 0, 64, device="cuda"), p, table).shape == (3, 0, 64)
    q = torch.ones(3, 2, 64, device="cuda")
    out, k = paged.rope(q, p, table, k=torch.zeros(3, 0, 64, device="cuda"))
    assert torch.equal(out, q) and k.shape == (3, 0, 64)


def test_graph_replay_follows_the_positions(cuda_ok):
    q = _x(7, (4, 2, 64), torch.bfloat16)
    pos = torch.zeros(1, 4, dtype=torch.int32, device="cuda")
    table, out = paged.RopeTable((32,)), torch.empty_like(q)
    paged.rope(q, pos, table, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        paged.rope(q, pos, table, out=out)
    pos.copy_(torch.tensor([[5, 6, 7, 8]], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    _check(out, q, _angles(np.array([[5, 6, 7, 8]], np.int32), (32,), 10000.0, False), False, False)
