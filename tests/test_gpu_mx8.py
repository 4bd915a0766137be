"""Activations held in 8 bits, on a GPU, against float64: the quantiser and its inverse bit for bit,
SwiGLU and its backward pass within what their roundings allow.

Tolerances of SwiGLU.  16-bit results: the exponential and the reciprocal are the hardware's, a few
units of 2^-24, and the exponential's argument -a log2(e) is rounded to 2^-24 of itself, an absolute
error of at most 2^-24 |a| log2(e) in the exponent, so a relative one of 2^-24 |a| in e^-a; with six
more operations of half a unit, (16 + |a|) 2^-24 of the terms covers it.  fp32 results: expf and the
division are within two units, the rest half a unit each: 16 * 2^-24.  The final rounding adds eps / 2
of the value, or half the smallest subnormal.

Far from zero the 16-bit forms lose e^-|a| below 2^-126, which the hardware's exponential gives as 0: s
(or 1 - s) is then off by less than 2^-126, the activation by less than 2^-126 |a b|, the gradients by
less than 2^-126 |dh b| (1 + |a|) and 2^-126 |dh a|; with |a| up to 300 and |b|, |dh| up to 1 here that is
at most 301 * 2^-126 (`lost`).  fp32 keeps s itself as a float, whose grid below 2^-126 is 2^-149: the same
sums with 2^-149 for 2^-126."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_mok_amd import _lib as L
from mixture_experts_layer_mok_amd import ops
from oracle import operators as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, FP, F32, U8 = torch.bfloat16, torch.float16, torch.float32, torch.uint8
TYPES = pytest.mark.parametrize("dtype", [BF, FP, F32], ids=["bf16", "fp16", "fp32"])


def f64(t):
    return t.detach().cpu().double().numpy()


def spaced(t, ld, fill=0):
    """t on the device with rows ld elements apart."""
    mem = torch.full((max(t.shape[0], 1), ld), fill, dtype=t.dtype, device=DEV)
    mem[:t.shape[0], :t.shape[1]] = t
    return mem, mem[:t.shape[0], :t.shape[1]]


def values(rows, cols, dtype, seed):
    """Blocks of many magnitudes, whole powers of two and the borders of 448 2^n among them."""
    rng = np.random.default_rng(seed)
    v = rng.standard_normal((rows, cols))
    span = 12 if dtype is FP else 100
    v *= 2.0 ** np.repeat(rng.integers(-span, span // 2 if dtype is FP else span, (rows, cols // 32)), 32, axis=1)
    for r in range(rows):
        for b in range(0, cols // 32, 3):
            v[r, 32 * b] = rng.choice([448, 449, 447, 450, 1, 0]) * 2.0 ** rng.integers(-14, 6)
    v[rng.random(v.shape) < 0.05] = 0
    if rows > 2:
        v[1, :32] = 0
        v[2, -32:] = -0.0
    return torch.from_numpy(v).to(dtype).to(DEV)


SHAPES = [(1, 32), (1, 96), (3, 64), (7, 2080), (64, 512), (65, 7168), (33, 65536), (777, 1056)]


@TYPES
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_quantise_and_back(dtype, shape):
    R, K = shape
    print(f"[mx8] {dtype} {R} x {K}", flush=True)
    x = values(R, K, dtype, R)
    some = np.unique(np.linspace(0, R - 1, min(R, 1 + 60000 // K)).astype(int))
    want_c, want_s = O.quantize_mx8(f64(x[some]))
    c, s = ops.quantize_mx8(x)
    assert np.array_equal(s[some].cpu().numpy(), want_s)
    assert np.array_equal(c[some].cpu().numpy(), want_c)
    if dtype is BF:  # the layer's own quantiser
        c2, s2 = torch.empty_like(c), torch.empty_like(s)
        L.mok_quantize_mx(x, R, K, c2, s2)
        assert torch.equal(c, c2) and torch.equal(s, s2)
    for out in (BF, FP, F32):
        with np.errstate(over="ignore"):
            want = torch.from_numpy(O.values_mx8(want_c, want_s)).to(out)
        back = ops.dequantize_mx8(c, s, dtype=out)
        assert back.dtype is out and torch.equal(back[some].cpu(), want)
    # rows apart, written around nothing else
    mem_x, xs = spaced(x, K + 40)
    mem_c, cs = spaced(torch.zeros_like(c), K + 16, 9)
    mem_s, ss = spaced(torch.zeros_like(s), K // 32 + 3, 9)
    ops.quantize_mx8(xs, codes=cs, scales=ss)
    assert torch.equal(cs, c) and torch.equal(ss, s)
    assert (mem_c[:, K:] == 9).all() and (mem_s[:, K // 32:] == 9).all()
    mem_o, os_ = spaced(torch.zeros_like(x), K + 24, 9)
    ops.dequantize_mx8(cs, ss, out=os_)
    assert torch.equal(os_, ops.dequantize_mx8(c, s, dtype=dtype)) and (mem_o[:, K:] == 9).all()


@TYPES
def test_all_codes_of_a_type(dtype):
    """Every finite 16-bit value (fp32: as many spread over its range) in a block with another."""
    if dtype is F32:
        bits = torch.arange(0, 2**32, 66049, dtype=torch.int64)
        v = bits.to(torch.int32).view(F32)
    else:
        v = torch.arange(-2**15, 2**15, dtype=torch.int32).to(torch.int16).view(dtype)
    v = v[torch.isfinite(v)]
    v = v[:len(v) // 32 * 32].view(-1, 32)
    for order in (torch.arange(v.numel()), torch.randperm(v.numel(), generator=torch.Generator().manual_seed(1))):
        x = v.reshape(-1)[order].view(-1, 32)
        c, s = ops.quantize_mx8(x.to(DEV))
        want_c, want_s = O.quantize_mx8(x.double().numpy())
        assert np.array_equal(s.cpu().numpy(), want_s)
        assert np.array_equal(c.cpu().numpy(), want_c)


def test_every_code_and_scale_back():
    codes = torch.arange(256, device=DEV).to(U8).repeat(256, 1)
    scales = torch.arange(256, device=DEV).to(U8).view(256, 1).repeat(1, 8)
    for out in (BF, FP, F32):
        got = ops.dequantize_mx8(codes, scales, dtype=out).cpu()
        with np.errstate(over="ignore"):
            want = torch.from_numpy(O.values_mx8(codes.cpu().numpy(), scales.cpu().numpy())).to(F32).to(out)
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(got), nan)
        bad = (got[~nan] != want[~nan])
        assert not bad.any(), (out, got[~nan][bad][:4], want[~nan][bad][:4])


@TYPES
def test_blocks_that_are_not_finite(dtype):
    x = torch.ones(4, 160, dtype=dtype, device=DEV)
    x[1, 40], x[2, 159], x[3, 64] = float("nan"), float("inf"), float("-inf")
    c, s = ops.quantize_mx8(x)
    want = torch.full((4, 5), 119, dtype=U8)
    want[1, 1] = want[2, 4] = want[3, 2] = 255
    assert torch.equal(s.cpu(), want)
    back = ops.dequantize_mx8(c, s, dtype=dtype)
    nan = want.to(DEV).repeat_interleave(32, dim=1) == 255
    assert torch.isnan(back[nan]).all() and (back[~nan] == 1).all() and not c[nan].any()


def near(got, want, terms, extra, dtype, lost=0.0):
    fi = torch.finfo(dtype)
    tol = extra * 2.0**-24 * terms + lost * (2.0**-23 if dtype is F32 else 1.0)
    tol = tol + (fi.eps / 2) * (np.abs(want) + tol) + fi.smallest_normal * fi.eps / 2
    err = np.abs(f64(got) - want)
    assert (err <= tol).all(), (np.argwhere(~(err <= tol))[:4].tolist(), float(np.nanmax(err / tol)))


def extra(a, dtype):
    """Units of 2^-24 that the sigmoid and the operations after it may be off by."""
    return 16.0 if dtype is F32 else 16.0 + np.abs(a)


@TYPES
@pytest.mark.parametrize("shape", [(1, 32), (5, 96), (64, 256), (33, 1056), (200, 2048), (3, 32768)], ids=str)
@pytest.mark.parametrize("spread", [0.1, 1.0, 8.0])
def test_swiglu_and_its_gradient(dtype, shape, spread):
    R, I = shape
    print(f"[mx8] swiglu {dtype} {R} x {I} spread {spread}", flush=True)
    rng = np.random.default_rng(R + I)
    ab = torch.from_numpy(spread * rng.standard_normal((R, 2 * I))).to(dtype).to(DEV)
    dh = torch.from_numpy(rng.standard_normal((R, I))).to(dtype).to(DEV)
    h, c, s = ops.swiglu_mx8(ab)
    c2, s2 = ops.quantize_mx8(ab)
    assert torch.equal(c, c2) and torch.equal(s, s2)
    x = f64(ab)
    near(h, O.swiglu(x), np.abs(O.swiglu(x)), extra(x[:, :I], dtype), dtype)
    d, again = ops.swiglu_mx8_backward(dh, c, s)
    v = O.values_mx8(c.cpu().numpy(), s.cpu().numpy())
    e = extra(v[:, :I], dtype)
    near(again, O.swiglu(v), np.abs(O.swiglu(v)), e, dtype)
    want, terms = O.swiglu_backward(v, f64(dh))
    near(d, want, terms, e if dtype is F32 else np.concatenate([e, e], 1), dtype)
    d2, none = ops.swiglu_mx8_backward(dh, c, s, with_h=False)
    assert none is None and torch.equal(d, d2)


@TYPES
def test_swiglu_strides_and_rows_behind_the_last(dtype):
    R, I, routed = 37, 160, 23
    rng = np.random.default_rng(3)
    ab = torch.from_numpy(rng.standard_normal((R, 2 * I))).to(dtype).to(DEV)
    dh = torch.from_numpy(rng.standard_normal((R, I))).to(dtype).to(DEV)
    h, c, s = ops.swiglu_mx8(ab)
    d, again = ops.swiglu_mx8_backward(dh, c, s)
    ab[routed:] = float("nan")
    dh[routed:] = float("inf")
    for last, rows in ((routed, routed), (0, 0), (-4, 0), (R + 50, R)):
        off = torch.tensor([0, 5, 5, last], dtype=torch.int32, device=DEV)
        full = {}
        for name, t in (("h", h), ("c", c), ("s", s), ("d", d), ("again", again)):
            pad = 3 if name == "s" else 16 if name == "c" else 24
            full[name] = spaced(torch.full_like(t, 9), t.shape[1] + pad, 9)
        if rows > routed:
            continue_in = (ab.nan_to_num(), dh.nan_to_num(posinf=1))
        else:
            continue_in = (ab, dh)
        ops.swiglu_mx8(spaced(continue_in[0], 2 * I + 8)[1], off, h=full["h"][1], codes=full["c"][1],
                       scales=full["s"][1])
        for name, t in (("h", h), ("c", c), ("s", s)):
            n = min(rows, routed)
            assert torch.equal(full[name][1][:n], t[:n])
            assert (full[name][0][rows:] == 9).all() and (full[name][0][:, t.shape[1]:] == 9).all()
        ops.swiglu_mx8_backward(spaced(continue_in[1], I + 8)[1], c, s, off, d_ab=full["d"][1], h=full["again"][1])
        for name, t in (("d", d), ("again", again)):
            n = min(rows, routed)
            assert torch.equal(full[name][1][:n], t[:n])
            assert (full[name][0][rows:] == 9).all() and (full[name][0][:, t.shape[1]:] == 9).all()


@TYPES
def test_swiglu_far_from_zero(dtype):
    """Gates where e^-a overflows or vanishes, and values that are not finite."""
    a = torch.tensor([-300., -104, -90, -88, -87, -30, 0, 30, 87, 90, 104, 300] * 8).view(3, 32)
    ab = torch.cat([a, torch.full_like(a, 0.5)], 1).to(dtype).to(DEV)
    h, c, s = ops.swiglu_mx8(ab)
    x = f64(ab)
    with np.errstate(over="ignore"):
        want = O.swiglu(x)
    near(h, want, np.abs(want), extra(x[:, :32], dtype), dtype, lost=301 * 2.0**-126)
    dh = torch.ones(3, 32, dtype=dtype, device=DEV)
    d, again = ops.swiglu_mx8_backward(dh, c, s)
    assert torch.isfinite(d).all() and torch.isfinite(again).all()
    big = f64(a) > 80
    assert (f64(d)[:, :32][big] == 0.5).all()
    ab[1, 4], ab[2, 40] = float("nan"), float("inf")
    h, c, s = ops.swiglu_mx8(ab)
    bad = ~torch.isfinite(h)
    assert bad.nonzero().tolist() in ([[1, 4], [2, 8]], [[1, 4]])  # (silu may be 0 where b is infinite)
    assert s.cpu()[1, 0] == 255 and s.cpu()[2, 1] == 255
    d, again = ops.swiglu_mx8_backward(dh, c, s)
    assert torch.isnan(d[1]).all() and torch.isnan(d[2, :32]).all() and torch.isfinite(d[0]).all()


@TYPES
def test_far_rows(dtype):
    """Rows past 2^32 bytes from the first."""
    I, R = 64, 9
    ld = 1 << 29 if dtype is F32 else 1 << 28
    x = torch.randn(R, 2 * I, device=DEV).to(dtype)
    h, c, s = ops.swiglu_mx8(x)

    def far(cols, t, step):
        mem = torch.empty(R * step, dtype=t, device=DEV)
        return mem.view(R, step)[:, 32:32 + cols]

    xs = far(2 * I, dtype, ld)
    xs.copy_(x)
    cs, ss = far(2 * I, U8, 1 << 29), far(I // 16, U8, 1 << 29)
    h2, c2, s2 = ops.swiglu_mx8(xs, codes=cs, scales=ss)
    assert torch.equal(h2, h) and torch.equal(c2, c) and torch.equal(s2, s)
    del xs
    dh = torch.randn(R, I, device=DEV).to(dtype)
    d, _ = ops.swiglu_mx8_backward(dh, c, s)
    ds = far(2 * I, dtype, ld)
    ops.swiglu_mx8_backward(dh, cs, ss, d_ab=ds, with_h=False)
    assert torch.equal(ds, d)
    q, p = ops.quantize_mx8(x)
    assert torch.equal(q, c) and torch.equal(p, s)
    assert torch.equal(ops.dequantize_mx8(cs, ss, dtype=dtype), ops.dequantize_mx8(c, s, dtype=dtype))
    del cs, ss, ds
    torch.cuda.empty_cache()


@TYPES
def test_large_calls_give_what_their_slices_give(dtype):
    """A call of hundreds of MiB reads its values another way; each element comes of its own block
    (or pair) only, so a slice of rows, taken alone, has the same bits."""
    rows, cols = (9001, 8256) if dtype is F32 else (17000, 8256)
    torch.manual_seed(7)
    x = torch.randn(rows, cols, device=DEV, dtype=dtype)
    dh = torch.randn(rows, cols // 2, device=DEV, dtype=dtype)
    codes, scales = ops.quantize_mx8(x)
    h, held, held_scales = ops.swiglu_mx8(x)
    d_ab, again = ops.swiglu_mx8_backward(dh, held, held_scales)
    assert torch.equal(codes, held) and torch.equal(scales, held_scales)
    for a, b in ((0, 1), (4000, 4313), (rows - 65, rows)):
        part, part_scales = ops.quantize_mx8(x[a:b])
        assert torch.equal(part, codes[a:b]) and torch.equal(part_scales, scales[a:b])
        h_part, _, _ = ops.swiglu_mx8(x[a:b])
        assert torch.equal(h_part, h[a:b])
        d_part, again_part = ops.swiglu_mx8_backward(dh[a:b], held[a:b], held_scales[a:b])
        assert torch.equal(d_part, d_ab[a:b]) and torch.equal(again_part, again[a:b])
