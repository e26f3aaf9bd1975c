"""The angle of paged_rope_write's rotation against position * frequency / 2 pi in whole numbers,
at the bound that the header states, where a result of fp16 shows it: pairs that the rotation
takes to (almost) 0.

The turn is off by position * (f 2^-52 + 2 pi 2^-64) radians (the frequency over 2 pi in 53 bits
after two roundings, then whole 2^-64 of a turn; for f below 0, 2^-54 of a turn for the latter: it
is one more rounding next to 1), and by 2^-32 of a turn and 2^-25 of pi as an fp32 number of half
turns: below 1.1e-7 more.  Sine and cosine by 2 ulp, 2^-22 at most; two products and their
difference by 2^-24 each.  All of it times |a| + |b|; the result by 2^-11 of itself or 2^-25."""
import math
from fractions import Fraction

import pytest
import torch

import paged_gqa_decode_03_gb300 as pgd

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def arctan_inverse(n, bits):
    """arctan(1 / n) in units of 2^-bits."""
    total, term, k = 0, (1 << bits) // n, 0
    while term:
        total += (-1) ** k * (term // (2 * k + 1))
        term //= n * n
        k += 1
    return total


BITS = 256
PI = Fraction(4 * (4 * arctan_inverse(5, BITS) - arctan_inverse(239, BITS)), 1 << BITS)


def angle_of(position, f):
    """position * f modulo 2 pi, between -pi and pi."""
    turns = Fraction(position) * Fraction(f) / (2 * PI)
    return float((turns - round(turns)) * 2 * PI)


@pytest.mark.parametrize("first", [0, 1000, (1 << 20) + 1, (1 << 31) - 40])
@pytest.mark.parametrize("sign", [1, -1])
def test_angles(first, sign):
    import __graft_entry__
    __graft_entry__.build()
    assert abs(float(PI) - math.pi) < 1e-15
    D, rows = 128, 40
    f, _ = pgd.rope_frequencies(D, base=500000.0)
    f = f * sign
    positions = [first + i for i in range(rows)]
    freq = [float(x) for x in f.cpu()]
    exact = torch.tensor([[angle_of(t, x) for x in freq] for t in positions], dtype=torch.float64)
    a, b = exact.sin().half(), exact.cos().half()
    q = torch.cat([a, b], 1)[:, None].contiguous().to(DEV)
    kc, vc = (torch.zeros((1, 1, 64, D), dtype=torch.float16, device=DEV) for _ in "kv")
    skip = torch.full((rows,), -1, dtype=torch.int32, device=DEV)
    out = torch.empty_like(q)
    pgd.paged_rope_write(kc, vc, out, q, q, q, skip, torch.tensor(positions, dtype=torch.int32, device=DEV), f)
    torch.cuda.synchronize()
    a, b, got = a.double(), b.double(), out.cpu().double()[:, 0]
    t, w = torch.tensor(positions, dtype=torch.float64)[:, None], torch.tensor(freq, dtype=torch.float64).abs()
    turn = t * (w * 2.0 ** -52 + 2 * math.pi * (2.0 ** -64 if sign > 0 else 2.0 ** -54)) + 1.1e-7
    near = (a.abs() + b.abs()) * (turn + 2.0 ** -22 + 3 * 2.0 ** -24)
    for have, want in ((got[:, :D // 2], a * exact.cos() - b * exact.sin()),
                       (got[:, D // 2:], b * exact.cos() + a * exact.sin())):
        tol = near + 2.0 ** -11 * (want.abs() + near) + 2.0 ** -25
        assert ((have - want).abs() <= tol).all(), float(((have - want).abs() / tol).max())
