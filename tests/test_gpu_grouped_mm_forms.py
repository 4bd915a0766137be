"""The grouped product of 16-bit rows in each of its forms, on a GPU.  The cases lie in mm_forms.py with
the form that each takes, which test_mm_forms.py holds against the code that chooses.

Operands are whole numbers of at most 4: every sum is below 2^24 and exact in fp32 in any order, so the result
must be the exact one (from products in float64, expert by expert), rounded to its type."""
import pytest
import torch

from mixture_experts_layer_mok_amd import ops
from tests.mm_forms import FAR_OFFSETS, FAR_ROWS, MOST, form_cases, offsets_of, short
from tests.test_gpu_grouped_mm import Case, check

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, FP, F32, F64 = torch.bfloat16, torch.float16, torch.float32, torch.float64
NAN = float("nan")


def say(*a):
    print("[mm forms]", *a, flush=True)


def whole(gen, dtype, *shape):
    return torch.randint(-4, 5, shape, generator=gen, device=DEV, dtype=torch.int8).to(dtype)


def apart(t, ld):
    """t's rows ld elements apart; between them NaN."""
    if ld is None:
        return t
    mem = torch.full((t.shape[0], ld), NAN, dtype=t.dtype, device=DEV)
    mem[:, 8:8 + t.shape[1]] = t
    return mem[:, 8:8 + t.shape[1]]


class Call:
    """Operands of a case: `slack` rows after the last, of NaN, as are the spaces between rows."""

    def __init__(self, kind, counts, n, k, dtype, ld=0, ld_out=0, slack=5):
        gen = torch.Generator(device=DEV).manual_seed(n + 7 * k + len(counts))
        self.kind, self.n, self.k, self.offsets = kind.rstrip("+"), n, k, offsets_of(counts)
        self.add, self.dtype, self.ld_out = kind.endswith("+"), dtype, ld_out
        self.end, self.rows = self.offsets[-1], self.offsets[-1] + slack
        self.off = torch.tensor(self.offsets, dtype=torch.int32, device=DEV)
        self.a = self.g = self.b = self.scales = None
        if self.kind != "rows":
            self.a = whole(gen, dtype, self.rows, k)
            self.a[self.end:] = NAN
            if self.kind == "held":
                codes, self.scales = ops.quantize_mx8(self.a)
                assert torch.equal(ops.dequantize_mx8(codes, self.scales, dtype=dtype)[:self.end], self.a[:self.end])
                self.codes = codes
            self.a = apart(self.a, ld or None)
        if self.kind != "out":
            self.g = whole(gen, dtype, self.rows, n)
            self.g[self.end:] = NAN
            self.g = apart(self.g, ld or None)
        if self.kind in ("out", "rows"):
            self.b = whole(gen, dtype, len(counts), n, k)

    def shape(self):
        return {"out": (self.rows, self.n), "rows": (self.rows, self.k)}.get(self.kind, (len(self.offsets) - 1, self.n, self.k))

    def run(self, out):
        if self.kind == "out":
            return ops.grouped_mm(self.a, self.off, self.b, out=out)
        if self.kind == "rows":
            return ops.grouped_mm_backward_rows(self.g, self.off, self.b, out=out)
        a = self.codes if self.kind == "held" else self.a
        return ops.grouped_mm_backward_weights(self.g, a, self.off, a_scales=self.scales, out=out, accumulate=self.add)

    def wanted(self, dtype):
        want = torch.full(self.shape(), 7.0, dtype=F64, device=DEV)
        for e, (lo, hi) in enumerate(zip(self.offsets, self.offsets[1:])):
            if self.kind == "out":
                want[lo:hi] = self.a[lo:hi].to(F64) @ self.b[e].to(F64).t().contiguous()
            elif self.kind == "rows":
                want[lo:hi] = self.g[lo:hi].to(F64) @ self.b[e].to(F64)
            else:
                d = self.g[lo:hi].to(F64).t().contiguous() @ self.a[lo:hi].to(F64)
                want[e] = want[e] + d if self.add else d
        assert want.abs().max() < 2**24
        return want.to(dtype)

    def check(self, out_dtype):
        out = torch.full(self.shape(), 7.0, dtype=out_dtype, device=DEV)
        if self.ld_out:
            out = apart(out, self.ld_out)
        assert self.run(out) is out
        assert torch.equal(out, self.wanted(out_dtype))
        return out


@pytest.mark.parametrize("kind,counts,n,k,form", form_cases(), ids=short)
def test_every_form(kind, counts, n, k, form):
    for dtype, out_dtype in ((BF, F32), (FP, F32 if kind.endswith("+") else FP)):
        say(kind, short(counts), n, k, form, dtype)
        Call(kind, counts, n, k, dtype).check(out_dtype)


@pytest.mark.parametrize("kind,counts,n,k,form", [c for c in form_cases() if c[0] in ("out", "rows")][::7], ids=short)
def test_rows_apart(kind, counts, n, k, form):
    say("apart", kind, short(counts), n, k, form)
    top = max(n, k) + 40
    top += -top % 8
    for out_dtype in (BF, F32):
        c = Call(kind, counts, n, k, BF, ld=top, ld_out=top + 24)
        out = c.check(out_dtype)
        mem = torch.as_strided(out, (c.rows, 8), out.stride(), out.storage_offset() - 8)
        assert torch.isnan(mem).all()
        mem = torch.as_strided(out, (c.rows, 8), out.stride(), out.storage_offset() + out.shape[1])
        assert torch.isnan(mem).all()


@pytest.mark.parametrize("kind,counts,n,k,form", [c for c in form_cases() if c[0] in ("out", "rows")][3::9], ids=short)
def test_values_that_are_not_finite_stay_in_their_rows(kind, counts, n, k, form):
    """A NaN makes its row NaN, an infinity no other row than its own infinite or NaN."""
    say("not finite", kind, short(counts), n, k, form)
    c = Call(kind, counts, n, k, BF)
    x = c.a if kind == "out" else c.g
    rows = torch.unique(torch.tensor([0, c.end // 3, c.end // 2, c.end - 1], device=DEV))
    good = c.wanted(F32)
    x[rows, x.shape[1] - 1] = NAN
    x[rows[1:2], 0] = float("inf")
    out = torch.full(c.shape(), 7.0, dtype=F32, device=DEV)
    c.run(out)
    assert torch.isnan(out[rows]).all()
    good[rows], out[rows] = 0, 0
    assert torch.equal(out, good)


@pytest.mark.parametrize("kind", ["out", "rows"])
def test_rows_that_repeat(kind):
    """A read operand whose rows are one row (stride 0), in whole tiles."""
    _, counts, n, k, form = next(c for c in form_cases() if c[0] == kind and "only_whole" in c[-1] and 72 in c[2:4])
    say("repeat", kind, short(counts), n, k, form)
    c = Call(kind, counts, n, k, BF, slack=5)
    if kind == "out":
        c.a = c.a[:1].expand(c.rows, k)
    else:
        c.g = c.g[:1].expand(c.rows, n)
    c.check(F32)


@pytest.mark.parametrize("kind,counts,n,k,form", FAR_ROWS, ids=short)
def test_rows_as_far_apart_as_they_may_be(kind, counts, n, k, form):
    """256 rows of 2^21 elements are 2^31 bytes in fp32, less one row: what a tile's offsets reach."""
    say("far", kind, short(counts), n, k, form)
    ld = 1 << 21
    c = Call(kind, counts, n, k, BF, ld=ld, ld_out=ld if kind != "weights" else 0)
    out = c.check(F32)
    if kind != "weights":
        assert out.stride(0) == ld
        assert torch.isnan(torch.as_strided(out, (c.rows, 8), out.stride(), out.storage_offset() + out.shape[1])).all()
    del c, out
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kind,offsets,n,k,form", FAR_OFFSETS, ids=short)
def test_offsets_far_apart(kind, offsets, n, k, form):
    say("far offsets", kind, offsets, n, k, form)
    top = max(o for o in offsets if o < MOST)
    c = Case([top] + [0] * (len(offsets) - 2), n, k, BF, seed=41, whole=True, held=kind == "held")
    c.offsets = offsets
    c.off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    check(c, "weights" if kind == "held" else kind, F32, True)
