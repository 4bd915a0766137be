"""The grouped product of 16-bit rows and its gradients, on a GPU, against float64.

Tolerances.  fp32 sums of K products: each of the K additions is off by at most 2^-23 of the sum of
the magnitudes (a truncating adder included), so K 2^-23 of it; then one rounding to the result's type,
eps / 2 of the value (and half the smallest subnormal).  Where the operands are small whole numbers,
every sum below 2^24 is exact in fp32 in any order, and the result must be the exact one, rounded."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_mok_amd import _lib as L
from mixture_experts_layer_mok_amd import ops
from oracle import operators as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
IDS = {BF: "bf16", FP: "fp16", F32: "fp32"}.get


def say(*a):
    print(*a, flush=True)


def f64(t):
    return t.detach().cpu().double().numpy()


def padded(t, ld):
    """t on the device, its rows ld elements apart, NaN between them (255 of bytes)."""
    if ld is None:
        return t.to(DEV)
    fill = 255 if t.dtype is torch.uint8 else float("nan")
    mem = torch.full((max(t.shape[0], 1), ld), fill, dtype=t.dtype, device=DEV)
    mem[:t.shape[0], :t.shape[1]] = t.to(DEV)
    return mem[:t.shape[0], :t.shape[1]]


class Case:
    """Operands of the three products: counts rows an expert, `gap` rows of no expert (NaN) before
    each expert's and `slack` after the last."""

    def __init__(self, counts, n, k, dtype, seed=0, whole=False, gap=0, slack=5, ld=None, held=False):
        rng = np.random.default_rng(seed)
        self.n, self.k, self.dtype, E = n, k, dtype, len(counts)
        # an expert's range ends where the next begins, so gaps are experts of their own, left out
        self.offsets, at = [], 0
        for c in counts:
            self.offsets.append(at)
            at += c
        self.offsets.append(at)
        self.rows = at + slack

        def make(*shape, scale=1.0):
            v = rng.integers(-4, 5, shape) if whole else rng.standard_normal(shape) * scale
            return torch.from_numpy(np.asarray(v, np.float64)).to(dtype)

        a, g = make(self.rows, k), make(self.rows, n)
        self.b = make(E, n, k, scale=0.1)
        self.live = np.zeros(self.rows, bool)
        self.live[:at] = True
        a[~torch.from_numpy(self.live)] = float("nan")
        g[~torch.from_numpy(self.live)] = float("inf")
        self.scales = None
        if held:
            codes, scales = O.quantize_mx8(np.nan_to_num(a.double().numpy()) * (1 if whole else 3))
            if not whole:
                moved = scales.astype(int) + rng.integers(-3, 4, scales.shape)
                scales = np.where(scales > 9, moved, scales).astype(np.uint8)
            a = torch.from_numpy(O.values_mx8(codes, scales))  # exact in either type
            assert torch.equal(a.to(dtype).double(), a)
            scales[~self.live] = 255
            self.codes = padded(torch.from_numpy(codes), None if ld is None else ld * 2)
            self.scales = padded(torch.from_numpy(scales), None if ld is None else ld // 32 + 3)
        self.a64, self.g64, self.b64 = (np.asarray(v.double().numpy()) for v in (a, g, self.b))
        self.a, self.g = padded(a.to(dtype), ld), padded(g, ld)
        self.off = torch.tensor(self.offsets, dtype=torch.int32, device=DEV)
        self.b = self.b.to(DEV)

    def out(self, rows, cols, dtype, ld=None):
        return padded(torch.full((rows, cols), 7.0, dtype=dtype), ld)


def near(got, want, mag, terms, dtype):
    """got (tensor) within what fp32 sums of `terms` products and one rounding allow."""
    got = f64(got)
    fi = torch.finfo(dtype)
    sums = terms * 2.0**-23 * mag
    tol = sums + (fi.eps / 2) * (np.abs(want) + sums) + fi.smallest_normal * fi.eps / 2
    err = np.abs(got - want)
    assert np.isfinite(got).all()
    assert (err <= tol).all(), (np.argwhere(err > tol)[:4].tolist(), float((err / tol).max()))


def check(c, kind, out_dtype, exact, ld_out=None):
    E = len(c.offsets) - 1
    if kind == "out":
        o = c.out(c.rows, c.n, out_dtype, ld_out)
        r = ops.grouped_mm(c.a, c.off, c.b, out=o)
        want, mag = O.grouped_mm(c.a64, c.offsets, c.b64, np.full((c.rows, c.n), 7.0))
        terms = c.k
    elif kind == "rows":
        o = c.out(c.rows, c.k, out_dtype, ld_out)
        r = ops.grouped_mm_backward_rows(c.g, c.off, c.b, out=o)
        want, mag = O.grouped_mm_backward_rows(c.g64, c.offsets, c.b64, np.full((c.rows, c.k), 7.0))
        terms = c.n
    else:
        o = torch.full((E, c.n, c.k), 7.0, dtype=out_dtype, device=DEV)
        add = kind == "weights+"
        a = c.a if c.scales is None else c.codes
        r = ops.grouped_mm_backward_weights(c.g, a, c.off, a_scales=c.scales, out=o, accumulate=add)
        want, mag = O.grouped_mm_backward_weights(c.g64, c.a64, c.offsets)
        if add:
            want, mag = want + 7.0, mag + 7.0
        terms = max([int(h - lo) for lo, h in zip(c.offsets, c.offsets[1:])] + [0]) + 1
    torch.cuda.synchronize()
    assert r is o
    if exact:
        assert np.abs(mag).max() < 2**24
        assert torch.equal(o.cpu().double(), torch.from_numpy(want).to(out_dtype).double())
    else:
        near(o, want, mag, terms, out_dtype)
    if o.dim() == 2:
        assert (o[torch.from_numpy(~c.live)] == 7).all()
    return o


KINDS = ["out", "rows", "weights", "weights+", "held"]
SHAPES = [  # rows an expert, n, k
    ([1], 8, 8),
    ([1], 136, 72),
    ([3, 0, 1, 17], 64, 520),
    ([16, 33, 0, 0, 5], 1000, 264),
    ([64, 65], 256, 64),
    ([130, 1, 255], 264, 192),
    ([256, 256], 512, 320),
    ([700, 0, 90], 328, 1048),
    ([0, 0, 513], 72, 2056),
    ([2] * 70, 40, 96),
    ([40] * 9 + [0] * 60, 128, 136),
    ([1500, 300], 776, 392),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{sum(s[0])}r{len(s[0])}e-{s[1]}x{s[2]}")
@pytest.mark.parametrize("dtype", [BF, FP], ids=IDS)
@pytest.mark.parametrize("kind", KINDS)
def test_against_float64(kind, dtype, shape):
    counts, n, k = shape
    held = kind == "held"
    if held:
        k = (k + 31) // 32 * 32
        kind = "weights"
    for out_dtype in ([F32] if kind == "weights+" else [dtype, F32]):
        say(f"[mm] {kind} {IDS(dtype)} -> {IDS(out_dtype)} {counts[:4]} n {n} k {k} held {held}")
        # whole numbers up to 4 (fp8 holds them): sums below 16 * 2056 + 7
        check(Case(counts, n, k, dtype, seed=1, whole=True, held=held), kind, out_dtype, True)
        ld = max(n, k) + 72
        ld += -ld % 32
        check(Case(counts, n, k, dtype, seed=2, ld=ld, held=held), kind, out_dtype, False,
              ld_out=max(n, k) + 24)


@pytest.mark.parametrize("rows", [0, 1, 2, 7, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 127, 128, 129, 191, 192,
                                  255, 256, 257, 320, 511, 512, 513])
@pytest.mark.parametrize("kind", ["out", "rows", "weights", "held"])
def test_row_counts(kind, rows):
    """Whole numbers, so that a row too many or too few shows in the exact result."""
    held = kind == "held"
    say(f"[mm] {kind} rows {rows}")
    check(Case([rows, 3], 264, 288, BF, seed=rows, whole=True, slack=300, held=held),
          "weights" if held else kind, F32, True)


@pytest.mark.parametrize("k", [8, 16, 24, 56, 64, 72, 120, 128, 136, 184, 192, 200, 256, 264, 320, 504, 512, 520,
                               1024, 1032, 4104])
@pytest.mark.parametrize("kind", ["out", "rows", "weights"])
def test_depths_and_columns(kind, k):
    """k is summed over forward and is the columns backward; n the same for the rows' gradient."""
    say(f"[mm] {kind} k {k}")
    for n in (k, 40):
        check(Case([90, 200], n, k, FP, seed=k, whole=True), kind, F32, True)
        check(Case([5, 9], n, k, BF, seed=k, whole=True), kind, BF, True)


def test_many_tiles():
    """More tiles than compute units, many a workgroup, the last ones ragged."""
    c = Case([1300, 0, 2100, 77, 640], 2088, 200, BF, seed=3, whole=True)
    for kind in ("out", "rows", "weights"):
        say("[mm] many tiles", kind)
        check(c, kind, BF, True)
    check(Case([1300, 0, 2100, 77, 640], 2088, 224, BF, seed=3, whole=True, held=True), "weights", F32, True)


@pytest.mark.parametrize("dtype", [BF, FP], ids=IDS)
@pytest.mark.parametrize("held", [False, True], ids=["16", "held"])
@pytest.mark.parametrize("counts,n,k", [([300], 4104, 4064), ([129, 0, 700], 2312, 2336), ([1] + [150] * 70, 520, 544)],
                         ids=["1e", "3e", "71e"])
def test_weights_gradient_in_whole_tiles(counts, n, k, held, dtype):
    """More than 128 rows an expert and 256 tiles of 256 x 256."""
    say(f"[mm] whole tiles {counts[:3]} n {n} k {k} held {held}")
    assert sum(counts) > 128 * len(counts) and len(counts) * (-(-n // 256)) * (-(-k // 256)) >= 256
    for kind, out_dtype in (("weights", dtype), ("weights+", F32)):
        check(Case(counts, n, k, dtype, seed=31, whole=True, held=held), kind, out_dtype, True)
    check(Case(counts, n, k, dtype, seed=32, held=held), "weights", F32, False)


def test_more_than_64_experts_of_tiles():
    c = Case([130 + (7 * i) % 150 for i in range(100)], 136, 72, BF, seed=4, whole=True)
    for kind in ("out", "rows", "weights"):
        check(c, kind, F32, True)


@pytest.mark.parametrize("kind", ["out", "rows", "weights"])
def test_offsets_past_the_rows(kind):
    """Ranges cut to the rows there are; ranges that end before they begin are empty."""
    c = Case([40, 30, 0, 60], 72, 136, BF, seed=5, whole=True)
    for off in ([-5, 20, 20, 90, 500], [0, 0, 0, 0, 0], [30, 10, 50, 50, 135], [200, 300, 400, 500, 600]):
        c.offsets = off
        c.off = torch.tensor(off, dtype=torch.int32, device=DEV)
        c.live[:] = False
        for lo, hi in zip(off, off[1:]):
            c.live[max(lo, 0):max(min(hi, c.rows), 0)] = True
        c.a64, c.g64 = np.nan_to_num(c.a64), np.nan_to_num(c.g64, posinf=0)
        c.a, c.g = torch.nan_to_num(c.a), torch.nan_to_num(c.g, posinf=0)
        say("[mm] offsets", off)
        check(c, kind, F32, True)


@pytest.mark.parametrize("kind", ["out", "rows", "weights", "held"])
def test_rows_that_repeat(kind):
    """A read operand whose rows are one row (stride 0); codes may not."""
    c = Case([30, 50], 136, 96, BF, seed=6, whole=True, slack=0, held=kind == "held")
    if kind != "held":
        c.a, c.a64 = c.a[:1].expand(80, 96), np.repeat(c.a64[:1], 80, 0)
    c.g, c.g64 = c.g[:1].expand(80, 136), np.repeat(c.g64[:1], 80, 0)
    check(c, "weights" if kind == "held" else kind, F32, True)


@pytest.mark.parametrize("dtype", [BF, FP], ids=IDS)
def test_values_that_are_not_finite(dtype):
    """A NaN or an infinity stays in the row, column or weight that it enters, and nothing else."""
    c = Case([20, 300], 72, 136, dtype, seed=7)
    c.a[5, 3], c.a[100, 9], c.g[6, 2], c.g[200, 71] = float("nan"), float("inf"), float("nan"), float("inf")
    y = ops.grouped_mm(c.a, c.off, c.b, dtype=F32)
    bad = ~torch.isfinite(y[:320]).all(1)
    assert bad.nonzero().flatten().tolist() == [5, 100]
    d = ops.grouped_mm_backward_rows(c.g, c.off, c.b, dtype=F32)
    assert (~torch.isfinite(d[:320]).all(1)).nonzero().flatten().tolist() == [6, 200]
    w = ops.grouped_mm_backward_weights(c.g, c.a, c.off)
    ok = torch.isfinite(w)
    want = torch.ones_like(ok)
    want[0, :, 3], want[1, :, 9], want[0, 2, :], want[1, 71, :] = False, False, False, False
    assert torch.equal(ok, want)


def test_subnormals_are_kept():
    """Products of subnormal 16-bit values, and results that are subnormal."""
    for dtype, small in ((BF, 2.0**-133), (FP, 2.0**-24)):
        c = Case([40], 40, 64, dtype, seed=8, whole=True, slack=0)
        c.a, c.a64 = c.a * small, c.a64 * small
        scale = 2.0**100 if dtype is BF else 1.0
        c.b, c.b64 = c.b * scale, c.b64 * scale
        y = ops.grouped_mm(c.a, c.off, c.b, dtype=F32)
        want, _ = O.grouped_mm(c.a64, c.offsets, c.b64, np.zeros((40, 40)))
        assert np.array_equal(f64(y), want)


def test_held_blocks_without_a_value():
    """A block of NaN scale makes its columns of its expert's gradient NaN, and nothing else."""
    c = Case([20, 90], 72, 128, BF, seed=9, held=True)
    c.scales[50, 2] = 255
    w = ops.grouped_mm_backward_weights(c.g, c.codes, c.off, a_scales=c.scales)
    nan = torch.isnan(w)
    want = torch.zeros_like(nan)
    want[1, :, 64:96] = True
    assert torch.equal(nan, want)


def test_held_values_past_fp16():
    """Scales whose values fp16 rounds, or cannot hold."""
    g = torch.eye(32, dtype=FP, device=DEV)
    codes = torch.arange(32 * 32, device=DEV).remainder(120).to(torch.uint8).view(32, 32)
    scales = torch.arange(32, device=DEV).add(127 - 16).to(torch.uint8).view(32, 1)
    with np.errstate(over="ignore"):
        want = torch.from_numpy(O.values_mx8(codes.cpu().numpy(), scales.cpu().numpy())).to(FP)
    for r in range(32):  # one row at a time: infinities times the others' zeros are NaN
        one = torch.tensor([r, r + 1], dtype=torch.int32, device=DEV)
        w = ops.grouped_mm_backward_weights(g, codes, one, a_scales=scales)[0]
        if torch.isfinite(want[r]).all():
            assert torch.equal(w[r].cpu(), want[r].float()), r
            assert not w[torch.arange(32) != r].any()


def test_scales_at_any_address():
    c = Case([70, 33], 72, 160, BF, seed=10, whole=True, held=True)
    want = check(c, "weights", F32, True)
    for pad, skip in ((7, 1), (8, 2), (9, 3), (12, 5)):
        mem = torch.full((c.rows, pad), 255, dtype=torch.uint8, device=DEV)
        mem[:, skip:skip + 5] = c.scales
        w = ops.grouped_mm_backward_weights(c.g, c.codes, c.off, a_scales=mem[:, skip:skip + 5])
        assert torch.equal(w, want), (pad, skip)


def test_far_rows():
    """Row strides at their largest: byte offsets of a tile's rows, and past 2^32 from the first."""
    k, n, ld = 72, 40, 1 << 21
    counts = [3, 600, 500]
    c = Case(counts, n, k, BF, seed=11, whole=True, slack=2)

    def far(t, dtype):
        mem = torch.empty(c.rows * ld, dtype=dtype, device=DEV)
        v = mem.view(c.rows, ld)[:, 4096:4096 + t.shape[1]]
        v.copy_(t)
        return v

    c.a, c.g = far(c.a, BF), far(c.g, BF)
    assert c.rows * ld * 2 > 2**32
    for kind in ("out", "rows", "weights"):
        say("[mm] far", kind)
        check(c, kind, F32, True)
    o = far(torch.full((c.rows, n), 7.0, dtype=F32), F32)
    ops.grouped_mm(c.a, c.off, c.b, out=o)
    want, _ = O.grouped_mm(c.a64, c.offsets, c.b64, np.full((c.rows, n), 7.0))
    assert np.array_equal(f64(o), want)


def test_weights_past_32_bits():
    """Experts whose weights and gradients lie past 2^32 bytes."""
    E, n, k = 3, 8192, 65536 * 2 // 4
    off = [0, 40, 40, 90]
    a = torch.randint(-3, 4, (90, k), device=DEV).to(BF)
    g = torch.randint(-3, 4, (90, n), device=DEV).to(BF)
    b = torch.zeros(E, n, k, dtype=BF, device=DEV)
    b[2, -8:, :].copy_(torch.randint(-3, 4, (8, k), device=DEV))
    b[0, :8, :].copy_(torch.randint(-3, 4, (8, k), device=DEV))
    dev = torch.tensor(off, dtype=torch.int32, device=DEV)
    y = ops.grouped_mm(a, dev, b, dtype=F32)
    assert torch.equal(y[40:, -8:].double(), a[40:].double() @ b[2, -8:].double().t().contiguous())
    assert torch.equal(y[:40, :8].double(), a[:40].double() @ b[0, :8].double().t().contiguous())
    assert not y[:, 8:-8].any()
    d = ops.grouped_mm_backward_rows(g, dev, b, dtype=F32)
    assert torch.equal(d[40:].double(), g[40:, -8:].double() @ b[2, -8:].double())
    w = ops.grouped_mm_backward_weights(g, a, dev)
    assert not w[1].any()
    assert torch.equal(w[2, -8:].double(), g[40:, -8:].double().t().contiguous() @ a[40:].double())
    assert torch.equal(w[0, :8].double(), g[:40, :8].double().t().contiguous() @ a[:40].double())


@pytest.mark.parametrize("kind", ["out", "rows", "weights", "weights+", "held"])
def test_again_the_same_bits(kind):
    c = Case([300, 20, 700], 520, 544, BF, seed=12, held=kind == "held")
    kind = "weights" if kind == "held" else kind
    first = check(c, kind, F32, False)
    for _ in range(3):
        assert torch.equal(check(c, kind, F32, False), first)


def test_the_two_directions_meet():
    """<grouped_mm(a), g> = <a, rows' gradient> = <b, weights' gradient>, in float64 of fp32 results."""
    c = Case([50, 0, 300], 264, 200, BF, seed=13, slack=0)
    y = f64(ops.grouped_mm(c.a, c.off, c.b, dtype=F32))
    da = f64(ops.grouped_mm_backward_rows(c.g, c.off, c.b, dtype=F32))
    db = f64(ops.grouped_mm_backward_weights(c.g, c.a, c.off))
    s = [(y * c.g64).sum(), (da * c.a64).sum(), (db * c.b64).sum()]
    size = sum((np.abs(c.g64[lo:hi]) @ np.abs(c.b64[e]) * np.abs(c.a64[lo:hi])).sum()
               for e, (lo, hi) in enumerate(zip(c.offsets, c.offsets[1:])))
    assert abs(s[0] - s[1]) <= 600 * 2.0**-23 * size and abs(s[0] - s[2]) <= 600 * 2.0**-23 * size


def c_call(kind, c, out, ws):
    """The C entry point with a workspace of the caller's, or none."""
    E = len(c.offsets) - 1
    ty = {BF: L.MOK_TYPE_BF16, FP: L.MOK_TYPE_FP16, F32: L.MOK_TYPE_FP32}
    w = (ws, 0 if ws is None else ws.numel())
    if kind == "out":
        L.mok_grouped_mm(ty[c.dtype], c.a, c.k, c.rows, c.off, E, c.b, c.n, c.k, ty[out.dtype], out, c.n, *w)
    elif kind == "rows":
        L.mok_grouped_mm_bwd_rows(ty[c.dtype], c.g, c.n, c.rows, c.off, E, c.b, c.n, c.k, ty[out.dtype], out, c.k, *w)
    else:
        held = c.scales is not None
        L.mok_grouped_mm_bwd_weights(ty[c.dtype], c.g, c.n, c.codes if held else c.a, c.k, c.scales,
                                     c.k // 32 if held else 0, c.rows, c.off, E, c.n, c.k, ty[out.dtype], out,
                                     kind == "weights+", *w)


SPLITS = [  # rows an expert, n, k: long sums of few results
    ("out", [300], 136, 4104), ("out", [1, 200, 0, 77], 72, 8200), ("out", [130], 264, 1544),
    ("rows", [300], 4104, 136), ("rows", [1, 200, 0, 77], 8200, 72), ("rows", [130], 1544, 264),
    ("weights", [5000], 136, 264), ("weights", [4000, 0, 1, 700], 72, 40), ("weights", [0, 2100], 264, 8),
    ("weights", [513, 1830, 64, 63], 136, 136), ("weights", [30] * 70, 40, 24), ("weights+", [3000, 0, 70], 136, 72),
    ("held", [5000], 136, 288), ("held", [4000, 0, 1, 700], 72, 32), ("held", [513, 1830, 64, 63], 264, 160),
    ("weights", [6000] + [8] * 255, 128, 128),
    # a last round of few whole tiles: short ones, of 108 and of 208 rows
    ("out", [2053, 2030, 2048, 2061, 1999, 2001, 2077, 2040], 1024, 4104), ("out", [8300], 2040, 4096),
    ("out", [8400], 2048, 4160), ("rows", [2053, 2030, 2048, 2061, 1999, 2001, 2077, 2040], 4104, 1024),
    ("rows", [8300], 4096, 2040), ("rows", [0, 8400], 4160, 2048),
]


@pytest.mark.parametrize("kind,counts,n,k", SPLITS, ids=lambda v: str(v)[:24].replace(" ", ""))
@pytest.mark.parametrize("dtype", [BF, FP], ids=IDS)
def test_sums_split_over_workgroups(kind, counts, n, k, dtype):
    say(f"[mm] split {kind} {counts[:4]} n {n} k {k}")
    held = kind == "held"
    kind = "weights" if held else kind
    which = dict(out=0, rows=1).get(kind, 2)
    c = Case(counts, n, k, dtype, seed=21, whole=True, held=held)
    assert L.mok_grouped_mm_workspace(which, c.rows, len(counts), n, k) == L.MOK_MM_WORKSPACE_BYTES
    out_types = [F32] if kind == "weights+" else [dtype, F32]
    for out_dtype in out_types:
        o = check(c, kind, out_dtype, True)
        check(Case(counts, n, k, dtype, seed=22, held=held), kind, out_dtype, False)
        for ws in (None, torch.full((L.MOK_MM_WORKSPACE_BYTES,), 255, dtype=torch.uint8, device=DEV)):
            again = torch.full_like(o, 7.0)
            c_call(kind, c, again, ws)
            assert torch.equal(again, o)


def test_a_split_product_again_the_same_bits():
    for kind, counts, n, k in (SPLITS[1], SPLITS[4], SPLITS[7]):
        c = Case(counts, n, k, BF, seed=23)
        first = check(c, kind, F32, False)
        for _ in range(3):
            assert torch.equal(check(c, kind, F32, False), first)
