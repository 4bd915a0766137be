"""MXFP4 operators on the GPU against their float64 forms: the quantiser bit for bit, its
inverse exactly, the grouped product within the error of its fp32 sums.

Tolerance of the product: the operands' values are exact, a sum of K products in fp32 is within
K 2^-23 S of the exact one in any order (one rounding an addition, to nearest or towards
zero), S the sum of the products' magnitudes; bf16 rounds by half a step, 2^-8 of the value."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_mok_amd import _lib as L
from mixture_experts_layer_mok_amd import gen, ops
from mixture_experts_layer_mok_amd.layer import MoKLayer
from oracle import operators as O
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.bfloat16, torch.float16, torch.float32]
IDS = ["bf16", "fp16", "fp32"]


def f64(t):
    return t.detach().cpu().double().numpy()


# ----------------------------------------------------------------------------------------
# quantiser
# ----------------------------------------------------------------------------------------
def check_quantise(src):
    """src: a device matrix; the codes and scales equal the float64 form's, and the values
    come back."""
    codes, scales = ops.quantize_mx4(src)
    c, s = O.quantize_mx4(f64(src))
    np.testing.assert_array_equal(scales.cpu().numpy(), s)
    got = O.unpack4(codes.cpu().numpy())
    np.testing.assert_array_equal(got, c)
    for dtype in TYPES:
        v = ops.dequantize_mx4(codes, scales, dtype=dtype)
        want = torch.from_numpy(O.values_mx4(codes.cpu().numpy(), s)).to(dtype)
        np.testing.assert_array_equal(f64(v), f64(want))
    return codes, scales


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (65, 160), (2, 2080), (1, 65536), (300, 32)])
def test_quantise(rows, cols, dtype):
    say(f"[mx4] quantise {rows} x {cols} {dtype}")
    rng = np.random.default_rng(rows + cols)
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-12, 8, (rows, cols)))
    x[rng.random((rows, cols)) < 0.05] = 0.0
    check_quantise(torch.from_numpy(x.astype(np.float32)).to(DEV, dtype))


@pytest.mark.parametrize("dtype", TYPES[:2], ids=IDS[:2])
def test_quantise_every_value(dtype):
    """Every finite 16-bit value as an element under every block maximum that matters: the
    value itself, and beside a larger one a few binades up (ties, subnormals, both ends)."""
    say(f"[mx4] every {dtype}")
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dtype)
    v = bits[torch.isfinite(bits)]
    rows = []
    for up in (0, 1, 2, 3, 4):
        b = torch.zeros(v.numel(), 32, dtype=dtype)
        b[:, 7] = v
        b[:, 20] = (v.float() * 2.0**up).to(dtype).nan_to_num(posinf=0.0, neginf=0.0)
        b[:, 31] = (v.float() * 1.5).to(dtype).nan_to_num(posinf=0.0, neginf=0.0)
        rows.append(b[torch.randperm(b.shape[0], generator=torch.Generator().manual_seed(up))[:3000]])
    rows.append(torch.stack([v, v.flip(0)], 1).reshape(-1, 1).expand(-1, 32)[::11])
    check_quantise(torch.cat([r.contiguous() for r in rows]).to(DEV))


def test_quantise_float32_ends():
    """Magnitudes at both ends of float32: subnormals, the smallest and the largest."""
    m = np.array([2.0**-149, 2.0**-140, 2.0**-127, 2.0**-126, 3 * 2.0**-126, 6 * 2.0**-127, 2.0**-125,
                  1.5 * 2.0**127, 3.4e38, 2.0**127, 1.0, 6.0, np.nextafter(np.float32(6), np.float32(7)),
                  np.nextafter(np.float32(6), np.float32(5))], np.float32)
    x = np.zeros((2 * len(m), 64), np.float32)
    for i, v in enumerate(m):
        x[2 * i, 3], x[2 * i, 40:44] = v, v * np.float32([0.25, -0.125, 0.5, 0.0625])
        x[2 * i + 1, 63], x[2 * i + 1, 5] = -v, v / np.float32(3)
    check_quantise(torch.from_numpy(x).to(DEV))


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_quantise_nan_and_infinity(dtype):
    x = torch.ones(4, 96, dtype=dtype)
    x[0, 40], x[1, 3], x[2, 95] = float("inf"), float("nan"), -float("inf")
    codes, scales = check_quantise(x.to(DEV))
    assert (scales.cpu() == 255).sum() == 3


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_quantise_strides(dtype):
    """Row strides of every operand; what lies between the rows stays."""
    rng = np.random.default_rng(3)
    rows, cols = 37, 96
    src = torch.from_numpy(rng.standard_normal((rows, cols + 40)).astype(np.float32)).to(DEV, dtype)[:, :cols]
    cb = torch.full((rows, 80), 0x5A, dtype=torch.uint8, device=DEV)
    sb = torch.full((rows, 7), 0x5A, dtype=torch.uint8, device=DEV)
    ops.quantize_mx4(src, codes=cb[:, :48], scales=sb[:, 2:5])
    c, s = ops.quantize_mx4(src.contiguous())
    assert torch.equal(cb[:, :48], c) and torch.equal(sb[:, 2:5], s)
    assert (cb[:, 48:] == 0x5A).all() and (sb[:, :2] == 0x5A).all() and (sb[:, 5:] == 0x5A).all()
    ob = torch.full((rows, cols + 16), -7.0, dtype=dtype, device=DEV)
    ops.dequantize_mx4(cb[:, :48], sb[:, 2:5], out=ob[:, :cols])
    assert torch.equal(ob[:, :cols], ops.dequantize_mx4(c, s, dtype=dtype))
    assert (ob[:, cols:] == -7).all()


def test_dequantise_every_code_and_scale():
    codes = torch.arange(256, dtype=torch.uint8).view(1, 1, 256).expand(256, 1, 256).contiguous()
    scales = torch.arange(256, dtype=torch.uint8).view(256, 1, 1).expand(256, 1, 16).contiguous()
    for dtype in TYPES:
        v = ops.dequantize_mx4(codes.to(DEV), scales.to(DEV), dtype=dtype)
        want = O.values_mx4(codes.numpy()[:, 0], scales.numpy()[:, 0])
        want = torch.from_numpy(want).float().to(dtype)  # exact in float32, bar overflow
        np.testing.assert_array_equal(f64(v)[:, 0], f64(want))
        assert torch.equal(torch.signbit(v).cpu()[:255, 0], torch.signbit(want)[:255])


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_quantise_more_than_the_cache(dtype):
    """A source past 256 MB: the rows at both ends and in between, and the same rows alone."""
    R, K = 70000, 2048
    src = torch.zeros(R, K, dtype=dtype, device=DEV)
    at = torch.tensor([0, 1, 35001, R - 2, R - 1], device=DEV)
    some = torch.randn(5, K, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
    src[at] = some.to(dtype)
    codes, scales = ops.quantize_mx4(src)
    c, s = check_quantise(src[at])
    assert torch.equal(codes[at], c) and torch.equal(scales[at], s)
    rest = torch.ones(R, dtype=torch.bool, device=DEV)
    rest[at] = False
    assert not codes[rest].any() and not scales[rest].any()
    back = ops.dequantize_mx4(codes, scales, dtype=dtype)
    assert torch.equal(back[at], ops.dequantize_mx4(c, s, dtype=dtype)) and not back[rest].any()


def test_empty():
    c, s = ops.quantize_mx4(torch.empty(0, 64, device=DEV))
    assert c.shape == (0, 32) and s.shape == (0, 2)
    assert ops.dequantize_mx4(c, s).shape == (0, 64)


# ----------------------------------------------------------------------------------------
# grouped product
# ----------------------------------------------------------------------------------------
def quantised(rng, rows, K, fmt, scale=1.0):
    x = torch.from_numpy((rng.standard_normal((rows, K)) * scale).astype(np.float32)).to(DEV, torch.bfloat16)
    if fmt == "e2m1":
        return ops.quantize_mx4(x)
    codes = torch.empty(rows, K, dtype=torch.uint8, device=DEV)
    scales = torch.empty(rows, K // 32, dtype=torch.uint8, device=DEV)
    L.mok_quantize_mx(x, rows, K, codes, scales)
    return codes, scales


def values(codes, scales, fmt):
    f = O.values_mx4 if fmt == "e2m1" else O.values_mx8
    return f(codes.cpu().numpy(), scales.cpu().numpy())


def scales8(fmt, sa, sb):
    return None if fmt == "e2m1" else (sa.cpu().numpy(), sb.cpu().numpy())


def check_product(got, want, e, what):
    got = f64(got)
    u = 2.0**-8 if what == torch.bfloat16 else 2.0**-24
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    ok = np.isnan(want) | (np.abs(got - want) <= e + u * (np.abs(want) + e) + 2.0**-133)
    assert ok.all(), f"{(~ok).sum()} of {ok.size} off, worst {np.nanmax(np.abs(got - want))}"


def run_product(counts, N, K, fmt, dtype, seed, slack=3, first=0, pad=0):
    rng = np.random.default_rng(seed)
    E = len(counts)
    off = np.concatenate([[first], first + np.cumsum(counts)]).astype(np.int32)
    n = int(off[-1]) + slack
    a, sa = quantised(rng, n, K, fmt)
    b, sb = quantised(rng, E * N, K, "e2m1", 0.1)
    if pad:
        wide = torch.full((n, a.shape[1] + 16 * pad), 0x77, dtype=torch.uint8, device=DEV)
        wide[:, :a.shape[1]] = a
        a = wide[:, :a.shape[1]]
        wide = torch.full((n, sa.shape[1] + pad), 255, dtype=torch.uint8, device=DEV)
        wide[:, :sa.shape[1]] = sa
        sa = wide[:, :sa.shape[1]]
    b, sb = b.view(E, N, K // 2), sb.view(E, N, K // 32)
    full = torch.full((n, N + 8 * pad), -7.0, dtype=dtype, device=DEV)
    out = full[:, :N]
    got = ops.grouped_mx4(a, sa, torch.from_numpy(off).to(DEV), b, sb, out=out)
    assert got is out
    want, e = O.grouped(values(a, sa, fmt), off, values(b, sb, "e2m1"), np.full((n, N), -7.0),
                        scales8(fmt, sa, sb))
    check_product(out, want, e, dtype)
    assert (full[:, N:] == -7).all()
    return out


FMT = ["e2m1", "e4m3"]


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("counts,N,K", [
    ([1], 8, 32), ([1], 16, 64), ([2, 0, 1], 24, 96), ([0, 0], 64, 128), ([17], 40, 160),
    ([16, 15, 1, 33], 72, 544), ([5, 0, 70, 31], 136, 1056), ([1, 1, 1, 1, 1], 264, 2048),
    ([130], 520, 288), ([64, 64], 256, 512),
])
def test_product(counts, N, K, fmt, dtype):
    say(f"[mx4] product {counts} N={N} K={K} {fmt} {dtype}")
    run_product(counts, N, K, fmt, dtype, seed=N + K)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("counts,N,K", [
    ([300], 264, 256), ([257, 1, 0, 511, 90], 520, 416), ([256, 256], 256, 7168),
    ([700, 3, 129], 1032, 1056), ([1025], 776, 160), ([513, 200], 512, 2080),
])
def test_product_many_rows(counts, N, K, fmt):
    say(f"[mx4] product {counts} N={N} K={K} {fmt}")
    run_product(counts, N, K, fmt, torch.bfloat16, seed=N + K + 1)
    run_product(counts, N, K, fmt, torch.float32, seed=N + K + 2)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("K", [64, 512, 544, 640])  # scales by single bytes, 16 and 4 bytes
@pytest.mark.parametrize("E,N", [(16, 2048), (16, 2040), (8, 2048), (8, 1024), (8, 1032), (3, 40)])
def test_product_few_rows_of_many_columns(E, N, K, fmt):
    """64, 32 and 16 columns a workgroup, whole and cut; an expert with several passes of rows
    among experts with a few or none."""
    say(f"[mx4] product few rows E={E} N={N} K={K} {fmt}")
    counts = np.random.default_rng(E + N + K).integers(0, 5, E)
    counts[1], counts[E - 1] = 0, 75
    run_product(list(counts), N, K, fmt, torch.bfloat16, seed=N + K + 3)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("N,counts", [
    (4104, [32] * 7), (4104, [32] * 8), (4104, [33] + [32] * 6), (4104, [224]), (4104, [225]), (4104, [1] * 7),
    (4104, [0, 1, 1, 1, 1, 1, 1, 1, 0, 1]), (72, [64, 65]), (72, [4096]), (72, [1] * 70 + [65] + [1] * 5),
    (4104, [160]), (4104, [192]), (2048, [32] * 16), (2048, [64] * 8), (2048, [256, 64, 32])])
@pytest.mark.parametrize("slack", [0, 300])
def test_product_around_the_choice_of_kernel(N, counts, slack, fmt):
    """Both sides of the passes of 32 rows times columns that the few-rows kernel takes, in
    matrices with and without rows behind the last expert's."""
    say(f"[mx4] product choice N={N} {counts} {slack} {fmt}")
    run_product(counts, N, 96, fmt, torch.bfloat16, seed=sum(counts), slack=slack)


@pytest.mark.parametrize("fmt", FMT)
def test_product_rows_of_a_capacity(fmt):
    """No rows, one and a few in a matrix for thousands; more than 4096."""
    for counts, slack in (([0, 0], 700), ([0, 1], 700), ([3, 5, 0, 2], 4086), ([3, 5, 0, 2], 4087),
                          ([2000, 1500], 900)):
        run_product(counts, 24, 96, fmt, torch.float32, seed=len(counts) + slack, slack=slack)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("K", [4096, 4128, 8448])  # one chunk a wave and more
def test_product_long_rows(K, fmt):
    say(f"[mx4] product long rows K={K} {fmt}")
    run_product([3, 0, 21, 40], 72, K, fmt, torch.float32, seed=K)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("N,K", [(5128, 288), (4096, 1024), (4360, 2432)])
def test_product_several_tiles_a_workgroup(N, K, dtype, fmt):
    """More tiles than the GPU has workgroups for, of 1 to 256 rows, one after the other."""
    say(f"[mx4] product tiles N={N} K={K} {dtype} {fmt}")
    run_product([700, 3, 0, 129, 65, 1000, 257, 12], N, K, fmt, dtype, seed=N + K + 4, pad=K == 288)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("K", [96, 512, 1056, 2080])
@pytest.mark.parametrize("counts,N", [([500, 70, 0, 129, 64, 1], 1000), ([128] * 8, 4096), ([128] * 8 + [1], 4096),
                                      ([1000], 520), ([64] * 16, 2040)])
def test_product_tiles_of_half_the_size(counts, N, K, dtype, fmt):
    """One of them a CU at most, on both sides of that."""
    say(f"[mx4] product halves {counts} N={N} K={K} {dtype} {fmt}")
    run_product(counts, N, K, fmt, dtype, seed=N + K + 5)


@pytest.mark.parametrize("fmt", FMT)
def test_product_tiles_of_many_groups(fmt):
    counts = np.random.default_rng(23).integers(0, 40, 130)
    counts[[0, 63, 64, 127]] = 0
    counts[65], counts[129] = 300, 260
    run_product(list(counts), 520, 96, fmt, torch.bfloat16, 24)
    run_product([0] * 1000 + [3] + [0] * 22 + [30], 264, 64, fmt, torch.float32, 25)


@pytest.mark.parametrize("fmt", FMT)
def test_product_strides_and_first_row(fmt):
    say(f"[mx4] product strides {fmt}")
    run_product([20, 0, 13], 48, 352, fmt, torch.bfloat16, 5, first=4, pad=3)
    run_product([300, 290], 272, 352, fmt, torch.float32, 6, first=2, pad=5)


@pytest.mark.parametrize("rows", [1, 200])
@pytest.mark.parametrize("sign", [1, -1])
def test_product_of_eight_bits_cuts_small_products(rows, sign):
    """Eight neighbours' products are cut, toward zero, to 2^-13 of the largest exponent: beside
    256 * 4 = 2^10 a product keeps its multiples of 2^-3.  Beside products of other eights, and
    with 4-bit rows, nothing is cut."""
    K = 128
    small = [0.0625, 0.125, 0.1875, 0.234375]
    b = torch.zeros(8, K)
    b[:, 0] = 4.0
    for j in range(4):  # column j: the neighbour small[j]; column 4 + j: one of the next eight
        b[j, 1 + j] = b[4 + j, 8 + j] = sign
    a = torch.zeros(rows, K)
    a[:, 0] = 256.0
    a[:, 1:5] = a[:, 8:12] = torch.tensor(small)
    off = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    ones = torch.full((max(rows, 8), K // 32), 127, dtype=torch.uint8, device=DEV)
    bc, bs = ops.quantize_mx4(b.to(DEV))
    ac = a.to(DEV).to(torch.float8_e4m3fn).view(torch.uint8)
    out = ops.grouped_mx4(ac, ones[:rows], off, bc.view(1, 8, -1), bs.view(1, 8, -1), dtype=torch.float32)
    want = [1024 + sign * v for v in (0.0, 0.125, 0.125, 0.125, *small)]
    assert out[rows - 1].tolist() == want and out[0].tolist() == want
    a4 = torch.zeros(rows, K)
    a4[:, 0] = 6.0
    a4[:, 1:5] = a4[:, 8:12] = 0.5
    a4, s4 = ops.quantize_mx4(a4.to(DEV))
    out = ops.grouped_mx4(a4, s4, off, bc.view(1, 8, -1), bs.view(1, 8, -1), dtype=torch.float32)
    assert (out == 24 + sign * 0.5).all()


@pytest.mark.parametrize("fmt", FMT)
def test_product_many_groups(fmt):
    rng = np.random.default_rng(17)
    counts = rng.integers(0, 6, 130)
    counts[40] = 200
    run_product(list(counts), 32, 64, fmt, torch.bfloat16, 18)
    run_product([0] * 1023 + [3], 8, 32, fmt, torch.float32, 19)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("big", [False, True])
def test_product_offsets_cut_to_the_rows(fmt, big):
    """Offsets outside the rows are cut; ranges that end before they begin are empty."""
    rng = np.random.default_rng(31)
    n, N, K = (600, 264, 256) if big else (40, 24, 96)
    a, sa = quantised(rng, n, K, fmt)
    b, sb = quantised(rng, 4 * N, K, "e2m1")
    for off in ([-5, 3, 3, n - 3, n + 9], [0, 0, n, 2**31 - 1, n], [-2**31, -1, 7, 5, 2**31 - 1],
                [n, n + 1, n + 2, n + 3, n + 4], [-9, -8, -7, -6, -5]):
        out = torch.full((n, N), -7.0, device=DEV)
        ops.grouped_mx4(a, sa, torch.tensor(off, dtype=torch.int32, device=DEV), b.view(4, N, -1),
                        sb.view(4, N, -1), out=out)
        if off == [-2**31, -1, 7, 5, 2**31 - 1]:
            continue  # rows 5 and 6 are in two ranges: either result, but no fault
        want, e = O.grouped(values(a, sa, fmt), off, values(b.view(4, N, -1), sb.view(4, N, -1), "e2m1"),
                            np.full((n, N), -7.0), scales8(fmt, sa, sb.view(4, N, -1)))
        check_product(out, want, e, torch.float32)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("counts,N,K", [([9, 5], 24, 288), ([300, 280], 264, 288)])
def test_product_nan_scales(fmt, counts, N, K):
    """A NaN scale of a row or of a weight column makes that row, that expert's column NaN, and
    nothing else; the last block of an odd K among them."""
    rng = np.random.default_rng(41)
    n, E = sum(counts), len(counts)
    a, sa = quantised(rng, n, K, fmt)
    b, sb = quantised(rng, E * N, K, "e2m1")
    sa[2, 0] = 255
    sa[n - 1, K // 32 - 1] = 255
    sb[3, 1] = 255
    sb[N + 5, K // 32 - 1] = 255
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    out = torch.full((n, N), -7.0, device=DEV)
    ops.grouped_mx4(a, sa, torch.from_numpy(off).to(DEV), b.view(E, N, -1), sb.view(E, N, -1), out=out)
    want, e = O.grouped(values(a, sa, fmt), off, values(b.view(E, N, -1), sb.view(E, N, -1), "e2m1"),
                        np.full((n, N), -7.0), scales8(fmt, sa, sb.view(E, N, -1)))
    check_product(out, want, np.nan_to_num(e), torch.float32)
    assert 0 < np.isnan(want).sum() < want.size


def test_product_unaligned_scales():
    """Scales at odd addresses."""
    rng = np.random.default_rng(43)
    for counts, N, K in (([9], 24, 256), ([300], 264, 256)):
        n = sum(counts)
        a, sa = quantised(rng, n, K, "e2m1")
        b, sb = quantised(rng, N, K, "e2m1")
        off = torch.tensor([0, n], dtype=torch.int32, device=DEV)
        ref = ops.grouped_mx4(a, sa, off, b.view(1, N, -1), sb.view(1, N, -1))
        ha = torch.zeros(sa.numel() + 1, dtype=torch.uint8, device=DEV)
        ha[1:] = sa.view(-1)
        hb = torch.zeros(sb.numel() + 3, dtype=torch.uint8, device=DEV)
        hb[3:] = sb.view(-1)
        got = ops.grouped_mx4(a, ha[1:].view_as(sa), off, b.view(1, N, -1),
                              hb[3:].view(1, N, -1))
        assert torch.equal(ref, got)


def test_product_repeatable_streams_and_graph():
    rng = np.random.default_rng(51)
    for counts, N, K in (([3, 0, 7], 72, 320), ([400, 3, 260], 520, 320)):
        n, E = sum(counts), len(counts)
        b, sb = quantised(rng, E * N, K, "e2m1")
        b, sb = b.view(E, N, -1), sb.view(E, N, -1)

        def inputs(counts):
            off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
            x = torch.from_numpy(rng.standard_normal((n, K)).astype(np.float32)).to(DEV)
            return x, torch.from_numpy(off).to(DEV)

        def step(v, stream=None):
            a, sa = ops.quantize_mx4(v[0], stream=stream)
            h = ops.grouped_mx4(a, sa, v[1], b, sb, dtype=torch.float32, stream=stream)
            return ops.dequantize_mx4(a, sa, dtype=torch.float32, stream=stream), h

        cases = [inputs(counts), inputs(counts[::-1])]
        refs = [step(v) for v in cases]
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        got = step(cases[0], stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(g, r) for g, r in zip(got, refs[0]))
        held = [t.clone() for t in cases[0]]
        step(held)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(held)
        for i in (1, 0, 1):
            for t, s in zip(held, cases[i]):
                t.copy_(s)
            for t in out:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            again = step(cases[i])
            torch.cuda.synchronize()
            assert all(torch.equal(g, r) for g, r in zip(out, refs[i]))
            assert all(torch.equal(g, r) for g, r in zip(again, refs[i]))


@pytest.mark.parametrize("T", [5, 300])
@pytest.mark.parametrize("fmt", FMT)
def test_experts_of_four_bits(T, fmt):
    """The operators together, as a layer with 4-bit experts: schedule, permute, quantise, the
    gate and up products, SwiGLU, quantise, the down product, unpermute; every product against
    float64 on the operands it got, and the end against float64 on the last rows."""
    cfg = gen.small_config("mx4", T=T, D=192, I=128, E=6, k=3, M=64, e0=1, E_loc=4)
    d = gen.make_inputs(cfg)
    d["ids"] = gen.mask_ids(d["ids"], 0.1, seed=3)
    say(f"[mx4] layer T={T} {fmt}")
    layer = MoKLayer(L.desc_from_config(cfg))
    layer.schedule(torch.from_numpy(d["ids"]).to(DEV))
    t = layer.tables()
    R, off, D, I, E = t["R"], t["offsets"], cfg.D, cfg.I, cfg.n_local
    n = cfg.T * cfg.k
    x = torch.from_numpy(d["x"]).to(DEV, torch.bfloat16)
    g = torch.from_numpy(d["gates"]).to(DEV)
    w1 = torch.from_numpy(np.concatenate([d["wg"], d["wu"]], 1)).to(DEV)
    w2 = torch.from_numpy(d["wd"]).to(DEV)
    q1, q2 = ops.quantize_mx4(w1), ops.quantize_mx4(w2)
    assert q1[0].shape == (E, 2 * I, D // 2) and q2[1].shape == (E, D, I // 32)

    def rows_mx(r):
        if fmt == "e2m1":
            return ops.quantize_mx4(r)
        return layer.quantize_weights(r.to(torch.bfloat16))

    def check(codes, scales, q, out):
        want, e = O.grouped(values(codes, scales, fmt), off, values(*q, "e2m1"), np.zeros(out.shape),
                            scales8(fmt, scales, q[1]))
        check_product(out[:R], want[:R], e[:R], out.dtype)

    rows = layer.permute(x, torch.zeros(n, D, dtype=torch.bfloat16, device=DEV))
    a, sa = rows_mx(rows)
    h = layer.grouped_mx4(a, sa, *q1, out=torch.zeros(n, 2 * I, device=DEV))
    check(a, sa, q1, h)
    h = torch.nn.functional.silu(h[:, :I]) * h[:, I:]
    a, sa = rows_mx(h)
    o = layer.grouped_mx4(a, sa, *q2)
    check(a, sa, q2, o)
    y = layer.unpermute(o, g)
    o0 = f64(o)
    o0[R:] = 0
    want, s = O.unpermute(o0, t["pos"].reshape(cfg.T, cfg.k), d["gates"])
    e = (cfg.k + 1) * 2.0**-24 * s
    assert (np.abs(f64(y) - want) <= e + 2.0**-8 * (np.abs(want) + e)).all()
    assert layer.status() == 0
