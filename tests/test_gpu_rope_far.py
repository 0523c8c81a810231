"""GPU check of mkv_rope at far positions against angles without a rounding: position x frequency and its
remainder of 2 pi are formed with 60 decimal digits on the CPU.

Tolerance, element by element.  The kernel's angle in turns is fl(fl(position x frequency) x fl(1 / 2 pi)):
three roundings of 2^-53, so off by at most 3 2^-53 |angle| rad (second order: 1.01); the rest as for near
positions (see test_gpu_rope.py): 2^-8 of the result, and 2^-20 (|a| + |b|)."""
import decimal

import pytest
import torch

from mixed_format_paged_mkv_b200 import Pool

pytestmark = pytest.mark.gpu

PI = decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
POSITIONS = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 31 - 129, 2 ** 30 + 1, 2 ** 24 + 1, 10 ** 9 + 7, 999999937, -123456789,
             1 << 20, 77777777, 2147483629, 1800000011, -1999999973]


def reduced(pos, inv):
    """(angle mod 2 pi, |angle|) in float64, without rounding before the reduction."""
    with decimal.localcontext() as c:
        c.prec = 60
        a = decimal.Decimal(pos) * decimal.Decimal(inv)
        turns = a / (2 * PI)
        return float((turns - turns.to_integral_value()) * 2 * PI), abs(float(a))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("top", [1.0, 0.99, 7.5, 300.0])
def test_far_positions(top, interleaved):
    rows, D, half = len(POSITIONS), 128, 64
    g = torch.Generator(device="cuda").manual_seed(51)
    q, k = (torch.randn((rows, h, D), generator=g, device="cuda").to(torch.bfloat16) for h in (3, 1))
    pos = torch.tensor(POSITIONS, dtype=torch.int32, device="cuda")
    inv = torch.tensor([top * 10000.0 ** (-i / half) for i in range(half)], dtype=torch.float32, device="cuda")
    outs = Pool(1, D, 1, 1, 1, 1).rope(q, k, pos, inv, interleaved=interleaved)
    both = [[reduced(p, f) for f in inv.double().tolist()] for p in POSITIONS]
    ang, size = (torch.tensor([[x[i] for x in r] for r in both], dtype=torch.float64, device="cuda")[:, None] for i in (0, 1))
    a, b = ((slice(0, D, 2), slice(1, D, 2)) if interleaved else (slice(0, half), slice(half, D)))
    for x, y in ((q, outs[0]), (k, outs[1])):
        A, B = x.double()[..., a], x.double()[..., b]
        for part, want in ((a, A * ang.cos() - B * ang.sin()), (b, B * ang.cos() + A * ang.sin())):
            tol = 2.0 ** -8 * want.abs() + (2.0 ** -20 + 3.03 * 2.0 ** -53 * size) * (A.abs() + B.abs())
            err = (y.double()[..., part] - want).abs()
            assert bool((err <= tol).all()), float((err / tol).max())
