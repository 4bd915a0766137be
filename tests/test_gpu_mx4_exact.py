"""The grouped product where its result is one number: sums that float32 holds exactly in any order
(both kernels, every form), operands and results past 2^32 bytes, the ends of the scales' range; and
the quantiser over every 16-bit value."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_mok_amd import _lib as L
from mixture_experts_layer_mok_amd import ops
from oracle import operators as O
from tests import mx4_exact as X
from tests.gpu_util import rel_fro, say
from tests.test_gpu_mx4 import quantised, values

pytestmark = pytest.mark.gpu
DEV = "cuda"
FMT = ["e2m1", "e4m3"]
OUT = [torch.bfloat16, torch.float32]
OUT_IDS = ["bf16", "fp32"]


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def f64(t):
    return t.detach().cpu().double().numpy()


def check(got, off, a, b, fmt, dtype, all_exact=True):
    """got [n, N] (-7 before the call) against the exact products of every expert's rows."""
    got = f64(got)
    rest = np.ones(got.shape[0], bool)
    for e in range(len(off) - 1):
        r = slice(int(off[e]), int(off[e + 1]))
        if r.stop > r.start:
            rest[r] = False
            want, ok = X.exact(a[r], b[e], fmt)
            assert ok.all() if all_exact else ok.mean() > 0.9
            assert X.off(got[r], want, ok, dtype) == 0, f"expert {e}"
    assert (got[rest] == -7).all()


KS = [32, 96, 512, 2080, 7168, 8448]
# few rows (16, 32 and 64 columns a workgroup); half tiles, whole ones, several a workgroup
SHAPES = [([1], 8, KS), ([3, 0, 21, 40], 72, KS), ([2] * 8, 2048, [32, 512, 2080]), ([33, 0, 5], 1032, KS),
          ([600, 1], 2056, [32, 544, 7168]), ([128] * 8, 4096, [512, 2080]),
          ([1100, 200, 0, 700], 2056, [96, 2080]), ([2000, 1500], 5128, [96, 512])]


@pytest.mark.parametrize("dtype", OUT, ids=OUT_IDS)
@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("counts,N,K", [(c, N, K) for c, N, ks in SHAPES for K in ks],
                         ids=[f"{sum(c)}x{N}x{K}" for c, N, ks in SHAPES for K in ks])
def test_exact_sums(counts, N, K, fmt, dtype):
    say(f"[mx4 exact] {counts} N={N} K={K} {fmt} {dtype}")
    rng = np.random.default_rng(N + K)
    E = len(counts)
    off = np.concatenate([[1], 1 + np.cumsum(counts)]).astype(np.int32)
    n = int(off[-1]) + 2
    for sign in (False, True):
        a, sa, va = X.operand(rng, n, K, fmt, sign)
        b, sb, vb = X.operand(rng, E * N, K, "e2m1", sign)
        out = torch.full((n, N), -7.0, dtype=dtype, device=DEV)
        ops.grouped_mx4(dev(a), dev(sa), dev(off), dev(b).view(E, N, -1), dev(sb).view(E, N, -1), out=out)
        check(out, off, va, vb.reshape(E, N, K), fmt, dtype)


@pytest.mark.parametrize("counts,N", [([21, 0, 40], 72), ([600, 90], 2056)])
@pytest.mark.parametrize("K", [288, 7168])
def test_quantised_normals_are_exact(counts, N, K):
    """MXFP4 rows and weights as the quantiser makes them of normal values."""
    rng = np.random.default_rng(K)
    E, off = len(counts), np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    n = int(off[-1])
    a, sa = quantised(rng, n, K, "e2m1")
    b, sb = quantised(rng, E * N, K, "e2m1", 0.1)
    for dtype in OUT:
        out = ops.grouped_mx4(a, sa, dev(off), b.view(E, N, -1), sb.view(E, N, -1), dtype=dtype)
        check(out, off, values(a, sa, "e2m1"), values(b, sb, "e2m1").reshape(E, N, K), "e2m1", dtype, False)


@pytest.mark.parametrize("rows,N", [(40, 264), (600, 2056)], ids=["few", "tiles"])
@pytest.mark.parametrize("K", [32, 2080, 7168])
def test_norm_of_the_error_of_eight_bit_rows(rows, N, K):
    """What the header states of normal values, 4e-6 of the norm, and half as much again for the
    draw; a sum in fp16 is off by 2^-11 of its last partial sums, 5e-4, a dropped block of 32 by
    (32 / K)^(1/2), 7e-2."""
    rng = np.random.default_rng(rows + K)
    a, sa = quantised(rng, rows, K, "e4m3")
    b, sb = quantised(rng, N, K, "e2m1", 0.1)
    off = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    out = ops.grouped_mx4(a, sa, off, b.view(1, N, -1), sb.view(1, N, -1), dtype=torch.float32)
    err = rel_fro(f64(out), values(a, sa, "e4m3") @ values(b, sb, "e2m1").T)
    say(f"[mx4 exact] MXFP8 rows K={K} rows={rows}: {err:.2e} of the norm")
    assert err <= 6e-6


# ----------------------------------------------------------------------------------------
# far offsets: only the rows that are used hold anything
# ----------------------------------------------------------------------------------------
def _far(n, first, counts, groups, N, K, fmt, ld_a, ld_as, ld_out):
    """The last rows of n, of the last experts of `groups`."""
    rng = np.random.default_rng(n)
    E, used = len(counts), sum(counts)
    assert first + used == n
    a, sa, va = X.operand(rng, used, K, fmt)
    b, sb, vb = X.operand(rng, E * N, K, "e2m1")
    wa = torch.empty(n, ld_a, dtype=torch.uint8, device=DEV)[:, :a.shape[1]]
    ws = torch.empty(n, ld_as, dtype=torch.uint8, device=DEV)[:, :K // 32]
    out = torch.empty(n, ld_out, dtype=torch.float32, device=DEV)[:, :N]
    wb = torch.empty(groups, N, K // 2, dtype=torch.uint8, device=DEV)
    wsb = torch.empty(groups, N, K // 32, dtype=torch.uint8, device=DEV)
    wa[first:], ws[first:] = dev(a), dev(sa)
    wb[groups - E:], wsb[groups - E:] = dev(b).view(E, N, -1), dev(sb).view(E, N, -1)
    out[:first] = -7
    off = np.full(groups + 1, first, np.int32)
    off[groups - E + 1:] = first + np.cumsum(counts)
    ops.grouped_mx4(wa, ws, dev(off), wb, wsb, out=out)
    assert (out[:first] == -7).all()
    got = f64(out[first:])
    at = 0
    for e, c in enumerate(counts):
        want, ok = X.exact(va[at:at + c], vb.reshape(E, N, K)[e], fmt)
        assert ok.all() and X.off(got[at:at + c], want, ok, torch.float32) == 0
        at += c
    return [t.stride(0) * (t.shape[0] - 1) * t.element_size() for t in (wa, ws, out, wb)]


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("first,counts,N", [(1090, [10], 72), (800, [300], 4104)], ids=["few", "tiles"])
def test_rows_past_32_bits(first, counts, N, fmt):
    say(f"[mx4 exact] far rows {first} {counts} {N} {fmt}")
    far = L.MOK_MX_MAX_LD
    assert min(_far(first + sum(counts), first, counts, 1, N, 288, fmt, far, far, 1 << 21)[:3]) > 2**32


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("n,counts,groups", [(5, [3, 1], 1024), (700, [300, 399], 1024)], ids=["few", "tiles"])
def test_experts_past_32_bits(n, counts, groups, fmt):
    say(f"[mx4 exact] far experts {counts} {groups} {fmt}")
    N, K = 2048, 8192
    ld = K if fmt == "e4m3" else K // 2
    assert _far(n, n - sum(counts), counts, groups, N, K, fmt, ld, K // 32, N)[3] > 2**32


# ----------------------------------------------------------------------------------------
# the ends of the scales' range
# ----------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", OUT, ids=OUT_IDS)
@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("rows,N", [(40, 72), (600, 2056)], ids=["few", "tiles"])
def test_scales_of_the_whole_range(rows, N, fmt, dtype):
    """Every pair of a row's scale and a column's, each the same along K: results from below
    float32's smallest to above its largest, of elements above zero.  A finite result is within the
    error of its sum, counting that a value below float32's smallest normal one may be taken as
    zero (2^-126 for each of K products); one past the largest is an infinity."""
    K = 64
    rng = np.random.default_rng(rows)
    a, b = X.operand(rng, rows, K, fmt)[0], X.operand(rng, N, K, "e2m1")[0]
    sa = rng.permutation(np.arange(rows) * 254 // (rows - 1)).astype(np.uint8)
    sb = rng.permutation(np.arange(N) * 254 // (N - 1)).astype(np.uint8)
    sa[:4], sb[:4] = [0, 254, 0, 254], [0, 254, 254, 0]
    s2a, s2b = np.repeat(sa[:, None], K // 32, 1), np.repeat(sb[:, None], K // 32, 1)
    va = O.values_mx4(a, s2a) if fmt == "e2m1" else O.values_mx8(a, s2a)
    vb = O.values_mx4(b, s2b)
    off = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    out = ops.grouped_mx4(dev(a), dev(s2a), off, dev(b)[None], dev(s2b)[None], dtype=dtype)
    want = va @ vb.T
    got = f64(out)
    half = 2.0**-8 if dtype == torch.bfloat16 else 2.0**-24
    err = K * 2.0**-23 * want + K * 2.0**-126
    most = float(torch.finfo(dtype).max)
    finite = want * (1 + half) + err < most
    inf = want - err > most * (1 + half)
    assert finite.any() and inf.any() and (want < 2.0**-140).any()
    assert np.isfinite(got[finite]).all()
    bad = np.abs(got - want)[finite] > (err + half * (want + err))[finite]
    assert not bad.any(), f"{bad.sum()} of {bad.size}"
    assert (got[inf] == np.inf).all()
    assert not np.isnan(got).any()


# ----------------------------------------------------------------------------------------
# ranges that overlap
# ----------------------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("n,N,K", [(40, 24, 96), (600, 2056, 256)], ids=["few", "tiles"])
def test_rows_outside_an_overlap(n, N, K, fmt):
    """Rows 5 and 6 lie in two ranges and get either result; every other row its own."""
    rng = np.random.default_rng(n)
    a, sa, va = X.operand(rng, n, K, fmt)
    b, sb, vb = X.operand(rng, 4 * N, K, "e2m1")
    vb = vb.reshape(4, N, K)
    for off in ([-2**31, -1, 7, 5, 2**31 - 1], [0, 0, 7, 5, n - 3]):
        out = torch.full((n, N), -7.0, device=DEV)
        ops.grouped_mx4(dev(a), dev(sa), dev(np.array(off, np.int32)), dev(b).view(4, N, -1),
                        dev(sb).view(4, N, -1), out=out)
        got = f64(out)
        one, three = va @ vb[1].T, va @ vb[3].T  # [0, 7) and [5, end)
        end = min(off[4], n)
        assert (got[:5] == one[:5]).all() and (got[7:end] == three[7:end]).all()
        assert (got[end:] == -7).all()
        assert ((got[5:7] == one[5:7]) | (got[5:7] == three[5:7])).all()


# ----------------------------------------------------------------------------------------
# the quantiser over every value
# ----------------------------------------------------------------------------------------
def _quantise(x):
    """Codes and scales of float64 rows x [R, 32], all rows at once: m 2^e with m in [1/2, 1) is at
    most 6 2^n = 3/4 2^(n + 3) for n = e - 3 where m is at most 3/4, else for n = e - 2."""
    amax = np.abs(x).max(1)
    m, e = np.frexp(amax)
    n = np.where(amax == 0, -127, np.maximum(e - 3 + (m > 0.75), -127))
    d = np.abs(np.abs(x)[:, :, None] * np.ldexp(1.0, -n)[:, None, None] - O.E2M1)
    # the nearest, of two at one distance the even one: even codes first in the order looked at
    order = np.array([0, 2, 4, 6, 1, 3, 5, 7])
    c = order[d[:, :, order].argmin(2)]
    return (c | np.signbit(x) * 8).astype(np.uint8), (n + 127).astype(np.uint8)[:, None]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
def test_quantise_all_16_bit_values(dtype):
    """Every finite value as the block's largest, and beside one 1, 2, 3 and 4 binades above it
    (where that is finite), with a third value between the two."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dtype)
    v = bits[torch.isfinite(bits)]
    some = torch.randperm(v.numel(), generator=torch.Generator().manual_seed(3))[:40]
    for up in range(5):
        x = torch.zeros(v.numel(), 32, dtype=dtype)
        x[:, 7] = v
        x[:, 20] = (v.float() * 2.0**up).to(dtype).nan_to_num(posinf=0.0, neginf=0.0)
        x[:, 31] = (v.float() * -(1.0 + up) / 2).to(dtype).nan_to_num(posinf=0.0, neginf=0.0)
        c, s = _quantise(f64(x))
        c1, s1 = O.quantize_mx4(f64(x[some]))
        np.testing.assert_array_equal(c[some], c1)
        np.testing.assert_array_equal(s[some], s1)
        codes, scales = ops.quantize_mx4(x.to(DEV))
        np.testing.assert_array_equal(scales.cpu().numpy(), s)
        np.testing.assert_array_equal(O.unpack4(codes.cpu().numpy()), c)
        back = torch.from_numpy(O.values_mx4(O.pack4(c), s)).to(dtype)
        np.testing.assert_array_equal(f64(ops.dequantize_mx4(codes, scales, dtype=dtype)), f64(back))
