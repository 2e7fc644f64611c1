"""The corrected quotients of sage_kv_append, in arithmetic: that they round as divisions do.

x / d is formed as n = x r, then n + r (x - n d) once (x of at most 11 bits) or twice (float32), r = fl32(1 / d),
every step one float32 rounding.  Signs and powers of two do not matter, so significands in [1, 2) are all there
is: for 11 bits every pair, 2^10 x 2^23, is tried; for float32 a sample of d for every x, and d = 127 and 448
for every x.

The steps are emulated in float64.  x r, n d, r e and their like are exact there (48 bits); fl32 of a float64
quotient is that of the quotient (53 >= 2 * 24 + 2 bits).  The sum n + r e can be rounded in float64 first: what it
lost is recovered exactly (Knuth's two-sum), and where the float64 sum lies half way between two floats its sign
says to which of them the sum rounds.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu


def f32(x):
    return x.float().double()


def fma32(a, b, c):
    """fl32(a b + c) of positive sums, a b exact in float64."""
    p = a * b
    s = c + p
    t = s - c
    lost = (c - (s - t)) + (p - t)
    bits = s.view(torch.int64)
    half_way = (bits & ((1 << 29) - 1)) == 1 << 28
    return f32((bits + half_way * lost.sign().long()).view(torch.float64))


def wrong(x, d, corrections):
    """Pairs whose corrected quotient is not fl32(x / d)."""
    r = f32(1.0 / d)
    n = f32(x * r)
    for _ in range(corrections):
        n = fma32(f32(x - n * d), r, n)
    return (n != f32(x / d)).sum()


def significands(lo, n):
    return 1.0 + torch.arange(lo, lo + n, device="cuda", dtype=torch.float64) * 2.0 ** -23


def test_eleven_bits_every_pair():
    x = 1.0 + torch.arange(1 << 10, device="cuda", dtype=torch.float64).view(-1, 1) * 2.0 ** -10
    step = 1 << 12
    assert sum(wrong(x, significands(lo, step), 1) for lo in range(0, 1 << 23, step)).item() == 0


def test_float32_quotients():
    d = torch.cat([significands(0, 8), significands((1 << 23) - 8, 8),
                   1.0 + torch.randint(0, 1 << 23, (48,), generator=torch.Generator().manual_seed(0)).double().cuda() * 2.0 ** -23])
    step = 1 << 20
    for lo in range(0, 1 << 23, step):
        x = significands(lo, step)
        assert wrong(x, d.view(-1, 1), 2).item() == 0
        for top in (127.0, 448.0):
            assert wrong(x, torch.full((), top, dtype=torch.float64, device="cuda"), 2).item() == 0
