"""Grouped products whose float32 sums are exact in any order, for the tests: where every product of
a result is a multiple of u and their magnitudes add up to at most 2^24 u, every partial sum is a
float32, so that the result has to be the exact one, and in bf16 its nearest value.  A dropped or
doubled product, and a sum held in fewer bits, then shows in the first element that it touches.

With e4m3 rows one thing more: the matrix core cuts the products of eight neighbours to multiples
of 2^(E - 13), 2^E at most the largest |a| times the largest |b|.  Where that is at most u, nothing
is cut."""
import numpy as np
import torch

from oracle import operators as O


def unit(v):
    """The largest power of two that every value of a row divides by ([R, K] -> [R])."""
    m, e = np.frexp(np.abs(v))
    bits = np.ldexp(m, 53).astype(np.int64)
    low = np.where(bits == 0, np.inf, np.ldexp((bits & -bits).astype(np.float64), e - 53))
    return low.min(1)


def exact(a, b, fmt):
    """(a @ b.T in float64, where a float32 sum of it is exact in any order), a [R, K], b [N, K]."""
    u = unit(a)[:, None] * unit(b)[None, :]
    ok = np.abs(a) @ np.abs(b).T <= 2.0**24 * u
    if fmt == "e4m3":
        ok &= np.abs(a).max(1)[:, None] * np.abs(b).max(1)[None, :] <= 2.0**13 * u
    return a @ b.T, ok


def nearest(want, dtype):
    """float64 values that are floats, rounded once to `dtype`."""
    return torch.from_numpy(want.astype(np.float32)).to(dtype).double().numpy()


def off(got, want, ok, dtype):
    """How many of the results that have to be exact are not."""
    return int(((got != nearest(want, dtype)) & ok).sum())


def operand(rng, rows, K, fmt, sign=False):
    """(codes, scales, values) of random elements with a product's worth of bits to spare: e2m1 of
    any magnitude, e4m3 of 1 to 3.75, two scales; above zero unless `sign`, so that sums grow."""
    if fmt == "e2m1":
        c = rng.integers(0, 8, (rows, K)).astype(np.uint8)
    else:
        c = rng.integers(7 << 3, 9 << 3, (rows, K)).astype(np.uint8)  # exponents 0 and 1
    if sign:
        c |= (rng.integers(0, 2, (rows, K)) << (3 if fmt == "e2m1" else 7)).astype(np.uint8)
    s = rng.integers(127, 129, (rows, K // 32)).astype(np.uint8)
    if fmt == "e2m1":
        p = O.pack4(c)
        return p, s, O.values_mx4(p, s)
    return c, s, O.values_mx8(c, s)
