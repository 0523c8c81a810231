"""GPU checks of mkv_rope against the rotation in float64.

Tolerance, element by element: the result is rounded to bf16 (2^-8 of it); before that the sine and
cosine are off by at most 2^-21 (an angle's fraction of a turn rounded to fp32, 2^-25 turns, and
two units in the last place of sincospi) and the two products and their sum by 2^-23 in all:
2^-20 (|a| + |b|) covers both."""
import numpy as np
import pytest
import torch

from mixed_format_paged_mkv_b200 import Pool

pytestmark = pytest.mark.gpu


def make(rows, Hq, Hkv, D, axes, R, far=100000, seed=0, base=10000.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, k = (torch.randn((rows, h, D), generator=g, device="cuda").to(torch.bfloat16) for h in (Hq, Hkv))
    pos = torch.randint(-3, far, (axes, rows), generator=g, device="cuda", dtype=torch.int32)
    inv = torch.tensor([base ** (-2.0 * i / R) for i in range(R // 2)], dtype=torch.float32, device="cuda")
    return q, k, pos, inv


def reference(x, pos, inv, axes, interleaved):
    half = inv.numel()
    ax = torch.as_tensor(axes if axes is not None else [0] * half, device="cuda")
    ang = pos.view(-1, x.shape[0])[ax].double().t() * inv.double()        # [rows, half]
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    x = x.double()
    y, tol = x.clone(), torch.zeros_like(x)
    a, b = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved
            else (slice(0, half), slice(half, 2 * half)))
    A, B = x[..., a], x[..., b]
    y[..., a], y[..., b] = A * c - B * s, B * c + A * s
    for part in (a, b):
        tol[..., part] = 2.0 ** -8 * y[..., part].abs() + 2.0 ** -20 * (A.abs() + B.abs())
    return y, tol


def check(out, x, pos, inv, axes, interleaved):
    ref, tol = reference(x, pos, inv, axes, interleaved)
    assert out.shape == x.shape and bool(((out.double() - ref).abs() <= tol).all())
    assert torch.equal(out[..., 2 * inv.numel():], x[..., 2 * inv.numel():])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rows,Hq,Hkv,D,R,n_axes", [
    (1, 1, 1, 64, 64, 1), (1, 8, 2, 128, 128, 3), (7, 6, 2, 128, 64, 2), (130, 32, 8, 128, 128, 1),
    (33, 24, 4, 256, 256, 3), (19, 3, 3, 256, 32, 2), (5, 128, 1, 256, 256, 4),
    (9, 4, 2, 64, 2, 1), (9, 4, 2, 64, 24, 3), (3, 5, 5, 128, 126, 3), (1000, 16, 4, 64, 16, 2),
])
def test_shapes(rows, Hq, Hkv, D, R, n_axes, interleaved):
    q, k, pos, inv = make(rows, Hq, Hkv, D, n_axes, R, seed=rows)
    axes = None if n_axes == 1 else [(i * 5 + i // 3) % n_axes for i in range(R // 2)]
    pool = Pool(Hkv, D, 1, 1, 1, 1)
    q0, k0 = q.clone(), k.clone()
    qo, ko = pool.rope(q, k, pos[0] if n_axes == 1 else pos, inv, axes=axes, interleaved=interleaved)
    assert torch.equal(q, q0) and torch.equal(k, k0)
    check(qo, q, pos, inv, axes, interleaved)
    check(ko, k, pos, inv, axes, interleaved)
    got = pool.rope(q, k, pos, inv, axes=axes, interleaved=interleaved, q_out=q, k_out=k)   # in place
    assert got[0] is q and torch.equal(q, qo) and torch.equal(k, ko)


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions_keep_their_phase(interleaved):
    q, k, pos, inv = make(64, 2, 1, 128, 1, 128, seed=3)
    pos[0, :8] = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1, 10 ** 9 + 7, 999999937])
    pool = Pool(1, 128, 1, 1, 1, 1)
    qo, ko = pool.rope(q, k, pos, inv, interleaved=interleaved)
    check(qo, q, pos, inv, None, interleaved)
    check(ko, k, pos, inv, None, interleaved)
    assert torch.equal(qo[0], q[0])            # position 0


@pytest.mark.parametrize("offset,pad", [(8, 16), (1, 3), (0, 2)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_parts_of_a_fused_array_in_place(offset, pad, interleaved):
    """q and k as parts of one row, rotated in place; the rest of the row stays; aligned rows and
    rows that rule out vectors give the same bits."""
    rows, Hq, Hkv, D = 21, 4, 2, 64
    q, k, pos, inv = make(rows, Hq, Hkv, D, 2, 64, seed=4)
    axes = [i % 2 for i in range(32)]
    pool = Pool(Hkv, D, 1, 1, 1, 1)
    want = pool.rope(q, k, pos, inv, axes=axes, interleaved=interleaved)
    fused = torch.full((rows, (Hq + Hkv) * D + offset + pad), 5.0, dtype=torch.bfloat16, device="cuda")
    a = offset + Hq * D
    fq, fk = fused[:, offset:a].unflatten(1, (Hq, D)), fused[:, a:a + Hkv * D].unflatten(1, (Hkv, D))
    fq.copy_(q)
    fk.copy_(k)
    pool.rope(fq, fk, pos, inv, axes=axes, interleaved=interleaved, q_out=fq, k_out=fk)
    assert torch.equal(fq, want[0]) and torch.equal(fk, want[1])
    assert bool((fused[:, :offset] == 5.0).all()) and bool((fused[:, a + Hkv * D:] == 5.0).all())


def test_nonfinite_channels_stay_in_their_pairs():
    q, k, pos, inv = make(5, 2, 1, 64, 1, 32, seed=6)
    pool = Pool(1, 64, 1, 1, 1, 1)
    want, _ = pool.rope(q, k, pos, inv)
    q[2, 1, 3], q[4, 0, 63] = float("nan"), float("inf")
    got, _ = pool.rope(q, k, pos, inv)
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[2, 1, [3, 19]] = True
    bad[4, 0, 63] = True
    assert torch.equal(~torch.isfinite(got), bad) and torch.equal(got[~bad], want[~bad])


def test_no_rows_captured_and_other_streams():
    pool = Pool(2, 128, 1, 1, 1, 1)
    q, k, pos, inv = make(0, 4, 2, 128, 1, 128)
    assert pool.rope(q, k, pos, inv)[0].shape == (0, 4, 128)
    a, b = make(40, 4, 2, 128, 1, 128, seed=7), make(40, 4, 2, 128, 1, 128, seed=8)
    wa, wb = pool.rope(*a), pool.rope(*b)
    static, out = [x.clone() for x in a], (torch.empty_like(wa[0]), torch.empty_like(wa[1]))
    s1 = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s1):
        pool.rope(*static, q_out=out[0], k_out=out[1])
    for x, y in zip(static, b):
        x.copy_(y)
    torch.cuda.synchronize()
    graph.replay()
    other = pool.rope(*a, stream=s1)
    torch.cuda.synchronize()
    assert torch.equal(out[0], wb[0]) and torch.equal(out[1], wb[1])
    assert torch.equal(other[0], wa[0]) and torch.equal(other[1], wa[1])


def test_more_than_2_to_the_31_elements():
    """q holds 2.3e9 elements: the first and the last rows come out as in calls of their own."""
    Hq, D, rows = 128, 256, 70001
    pool = Pool(1, D, 1, 1, 1, 1)
    _, _, pos, inv = make(rows, 1, 1, D, 1, D, seed=9)
    q = torch.empty((rows, Hq, D), dtype=torch.bfloat16, device="cuda")
    for a in range(0, rows, 10000):
        q[a:a + 10000] = torch.randn(q[a:a + 10000].shape, device="cuda")
    k = torch.randn((rows, 1, D), device="cuda").to(torch.bfloat16)
    qo, ko = pool.rope(q, k, pos, inv)
    assert qo.numel() > 2 ** 31
    for part in (slice(0, 5), slice(rows - 5, rows)):
        a, b = pool.rope(q[part], k[part], pos[:, part].contiguous(), inv)
        assert torch.equal(a, qo[part]) and torch.equal(b, ko[part])
        check(qo[part], q[part], pos[:, part], inv, None, False)
