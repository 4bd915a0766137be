"""CPU checks of the grouped product of 16-bit rows and of the activations held in 8 bits: pins of
their float64 forms (autograd, differences, hand-worked codes), and the refusals of the C ABI and of
the torch-facing functions, which come before any GPU work."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_mok_amd import _lib as L
from mixture_experts_layer_mok_amd import ops
from oracle import operators as O

FAKE = 0x100000  # never dereferenced


def test_product_gradients_against_autograd_and_differences():
    rng = np.random.default_rng(1)
    off = np.array([0, 3, 3, 7])  # the second expert has no rows; rows 7 and 8 belong to none
    a, b, g = rng.standard_normal((9, 8)), rng.standard_normal((3, 16, 8)), rng.standard_normal((9, 16))

    def loss(a, b):
        return float((O.grouped_mm(a, off, b, np.zeros((9, 16)))[0] * g)[:7].sum())

    da, _ = O.grouped_mm_backward_rows(g, off, b, np.zeros((9, 8)))
    db, _ = O.grouped_mm_backward_weights(g, a, off)
    at, bt = (torch.tensor(v, requires_grad=True) for v in (a, b))
    sum((at[lo:hi] @ bt[e].t() * torch.tensor(g[lo:hi])).sum()
        for e, (lo, hi) in enumerate(zip(off, off[1:]))).backward()
    np.testing.assert_allclose(da, at.grad.numpy(), rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(db, bt.grad.numpy(), rtol=1e-12, atol=1e-14)
    assert not da[7:].any() and not db[1].any()
    h = 1e-5
    for x, d, at in ((a, da, (2, 5)), (a, da, (6, 0)), (a, da, (8, 1)), (b, db, (0, 3, 7)), (b, db, (1, 0, 0))):
        up, down = (v.copy() for v in (x, x))
        up[at] += h
        down[at] -= h
        diff = (loss(*((up, b) if x is a else (a, up))) - loss(*((down, b) if x is a else (a, down)))) / (2 * h)
        assert abs(diff - d[at]) < 1e-6


def test_swiglu_gradient_against_autograd_and_differences():
    rng = np.random.default_rng(2)
    ab, dh = 2 * rng.standard_normal((4, 32)), rng.standard_normal((4, 16))
    d, terms = O.swiglu_backward(ab, dh)
    t = torch.tensor(ab, requires_grad=True)
    (torch.nn.functional.silu(t[:, :16]) * t[:, 16:] * torch.tensor(dh)).sum().backward()
    np.testing.assert_allclose(d, t.grad.numpy(), rtol=1e-12, atol=1e-14)
    assert (terms >= np.abs(d) * (1 - 1e-12)).all()
    h = 1e-5
    for at in ((0, 0), (3, 15), (1, 16), (2, 31)):
        up, down = ab.copy(), ab.copy()
        up[at] += h
        down[at] -= h
        diff = ((O.swiglu(up) - O.swiglu(down)) * dh).sum() / (2 * h)
        assert abs(diff - d[at]) < 1e-8


def test_mx8_codes_by_hand():
    v = np.zeros((1, 32))
    # amax 448: n = 0.  8..16 has steps of 1: ties at 8.5 (-> 8), 9.5 (-> 10); 256..448 steps of 32:
    # 272 (-> 256), 304 (-> 320); below 2^-6 steps of 2^-9: half of one (-> 0), three halves (-> 2)
    v[0, :9] = [448, 8.5, 9.5, 272, 304, 2.0**-10, 3 * 2.0**-10, -9.5, -0.0]
    c, s = O.quantize_mx8(v)
    assert s.tolist() == [[127]]
    assert O.values_mx8(c, s)[0, :9].tolist() == [448, 8, 10, 256, 320, 0, 2.0**-8, -10, 0]
    assert c[0, 8] == 128
    for amax, n in ((448.0, 0), (449.0, 1), (224.0, -1), (1.0, -8), (1.75, -8), (1.76, -7), (2.0**-140, -127),
                    (3.3e38, 120)):
        w = np.zeros((1, 32))
        w[0, 5] = -amax
        assert O.quantize_mx8(w)[1][0, 0] == n + 127, amax
    assert O.quantize_mx8(np.zeros((1, 32)))[1][0, 0] == 0
    for bad in (np.inf, -np.inf, np.nan):
        w = np.ones((1, 64))
        w[0, 40] = bad
        c, s = O.quantize_mx8(w)
        assert s.tolist() == [[119, 255]] and not c[0, 32:].any()
        vals = O.values_mx8(c, s)
        assert (vals[0, :32] == 1).all() and np.isnan(vals[0, 32:]).all()
    # every code of every sign comes back
    x = np.concatenate([O.E4M3, -O.E4M3, [448, 448]]).reshape(8, 32)
    x[:, 0] = 448
    c, s = O.quantize_mx8(x)
    assert (s == 127).all() and (O.values_mx8(c, s) == x).all()


# ----------------------------------------------------------------------------------------
# refusals of the C ABI
# ----------------------------------------------------------------------------------------
def _mm_calls(type=0, ld_a=64, ld_o=32, n_rows=8, off=FAKE, groups=2, b=FAKE, n=32, k=64, ty=0, a=FAKE,
              o=FAKE, ws=None, wsb=0):
    lib = L.load()
    return dict(out=lib.mok_grouped_mm(type, a, ld_a, n_rows, off, groups, b, n, k, ty, o, ld_o, ws, wsb, None),
                rows=lib.mok_grouped_mm_bwd_rows(type, o, ld_o, n_rows, off, groups, b, n, k, ty, a, ld_a,
                                                 ws, wsb, None),
                weights=lib.mok_grouped_mm_bwd_weights(type, o, ld_o, a, ld_a, None, 0, n_rows, off, groups,
                                                       n, k, ty, b, 0, ws, wsb, None))


@pytest.mark.parametrize("kw,code", [
    (dict(type=2, ty=2), L.MOK_E_UNSUPPORTED), (dict(type=-1), L.MOK_E_UNSUPPORTED),
    (dict(ty=1), L.MOK_E_UNSUPPORTED), (dict(type=1), L.MOK_E_UNSUPPORTED), (dict(ty=3), L.MOK_E_UNSUPPORTED),
    (dict(n_rows=-1), L.MOK_E_SHAPE), (dict(n_rows=(1 << 24) + 1), L.MOK_E_SHAPE),
    (dict(groups=0), L.MOK_E_SHAPE), (dict(groups=1025), L.MOK_E_SHAPE), (dict(k=0), L.MOK_E_SHAPE),
    (dict(k=60), L.MOK_E_SHAPE), (dict(k=65544, ld_a=65544), L.MOK_E_SHAPE), (dict(n=0), L.MOK_E_SHAPE),
    (dict(n=12), L.MOK_E_SHAPE), (dict(n=(1 << 20) + 8, ld_o=(1 << 20) + 8, k=8), L.MOK_E_SHAPE),
    (dict(n=1 << 20, ld_o=1 << 20, k=2048, ld_a=2048), L.MOK_E_SHAPE),
    (dict(ld_a=56), L.MOK_E_SHAPE), (dict(ld_a=68), L.MOK_E_SHAPE), (dict(ld_a=-64), L.MOK_E_SHAPE),
    (dict(ld_a=(1 << 21) + 8), L.MOK_E_SHAPE), (dict(ld_o=24), L.MOK_E_SHAPE), (dict(ld_o=36), L.MOK_E_SHAPE),
    (dict(ld_o=(1 << 21) + 8), L.MOK_E_SHAPE), (dict(a=None), L.MOK_E_NULL), (dict(o=None), L.MOK_E_NULL),
    (dict(b=None), L.MOK_E_NULL), (dict(off=None), L.MOK_E_NULL), (dict(a=FAKE + 8), L.MOK_E_SHAPE),
    (dict(o=FAKE + 2), L.MOK_E_SHAPE), (dict(b=FAKE + 8), L.MOK_E_SHAPE), (dict(off=FAKE + 2), L.MOK_E_SHAPE),
    (dict(ws=FAKE), L.MOK_E_WORKSPACE), (dict(ws=FAKE, wsb=L.MOK_MM_WORKSPACE_BYTES - 1), L.MOK_E_WORKSPACE),
    (dict(ws=FAKE + 8, wsb=L.MOK_MM_WORKSPACE_BYTES), L.MOK_E_SHAPE),
])
def test_grouped_mm_refuses(kw, code):
    assert set(_mm_calls(**kw).values()) == {code}


def test_grouped_mm_refuses_written_strides_and_8_bits():
    # a written matrix may not repeat one row
    assert _mm_calls(ld_o=0)["out"] == _mm_calls(ld_a=0)["rows"] == L.MOK_E_SHAPE
    fn = L.load().mok_grouped_mm_bwd_weights

    def call(type=0, a=FAKE, ld_a=64, s=FAKE, ld_s=2, k=64, ty=2, add=0):
        return fn(type, FAKE, 32, a, ld_a, s, ld_s, 8, FAKE, 2, 32, k, ty, FAKE, add, None, 0,
                  None)

    for kw in (dict(k=40), dict(ld_a=72), dict(ld_a=48), dict(ld_a=(1 << 22) + 16), dict(ld_s=1),
               dict(ld_s=(1 << 21) + 1), dict(a=FAKE + 4)):
        assert call(**kw) == L.MOK_E_SHAPE, kw
    assert call(ty=0, add=1) == L.MOK_E_UNSUPPORTED
    assert call(a=None) == L.MOK_E_NULL


def test_workspace_of_products():
    all_of = L.MOK_MM_WORKSPACE_BYTES
    w = L.mok_grouped_mm_workspace
    assert w(2, 16384, 1, 1024, 1024) == all_of  # 64 tiles of 256 steps
    assert w(2, 16384, 8, 4096, 7168) == w(2, 512, 1, 1024, 1024) == 0
    assert w(0, 2000, 1, 64, 8192) == w(1, 2000, 1, 8192, 64) == all_of
    assert w(0, 2000, 1, 8192, 64) == w(1, 2000, 1, 64, 8192) == w(0, 16384, 8, 7168, 2048) == 0
    assert w(0, 16384, 8, 4096, 7168) == w(1, 16384, 8, 4096, 7168) == L.MOK_MM_WORKSPACE_BYTES  # a last round of few tiles
    for bad, code in (((3, 8, 1, 64, 64), L.MOK_E_UNSUPPORTED), ((0, -1, 1, 64, 64), L.MOK_E_SHAPE),
                      ((0, 8, 0, 64, 64), L.MOK_E_SHAPE), ((2, 8, 1, 60, 64), L.MOK_E_SHAPE)):
        with pytest.raises(L.MokError) as e:
            w(*bad)
        assert e.value.code == code
    assert L.load().mok_grouped_mm_workspace(0, 8, 1, 64, 64, None) == L.MOK_E_NULL


def test_empty_calls_do_nothing():
    lib = L.load()
    got = _mm_calls(n_rows=0, a=None, o=None)
    assert got["out"] == got["rows"] == L.MOK_OK
    assert lib.mok_grouped_mm_bwd_weights(0, None, 32, None, 64, None, 0, 0, None, 2, 32, 64, 0, FAKE, 0,
                                          None, 0, None) == L.MOK_E_NULL  # (its result is 0, not nothing)
    assert lib.mok_quantize_mx8(0, None, 64, 0, 64, None, 64, None, 2, None) == L.MOK_OK
    assert lib.mok_dequantize_mx8(None, 64, None, 2, 0, 64, 0, None, 64, None) == L.MOK_OK
    assert lib.mok_swiglu_mx8(0, None, 64, 0, 32, None, 0, None, 32, None, 64, None, 2, None) == L.MOK_OK
    assert lib.mok_swiglu_mx8_bwd(0, None, 32, None, 64, None, 2, 0, 32, None, 0, None, 64, None, 0,
                                  None) == L.MOK_OK


@pytest.mark.parametrize("kw,code", [
    (dict(type=7), L.MOK_E_UNSUPPORTED), (dict(cols=48), L.MOK_E_SHAPE), (dict(cols=0), L.MOK_E_SHAPE),
    (dict(cols=65568), L.MOK_E_SHAPE), (dict(rows=-1), L.MOK_E_SHAPE), (dict(rows=1 << 31), L.MOK_E_SHAPE),
    (dict(ld=56), L.MOK_E_SHAPE), (dict(ld=0), L.MOK_E_SHAPE), (dict(ld=68), L.MOK_E_SHAPE),
    (dict(ld=2**30 + 8), L.MOK_E_SHAPE), (dict(ldc=48), L.MOK_E_SHAPE), (dict(ldc=72), L.MOK_E_SHAPE),
    (dict(ldc=2**30 + 16), L.MOK_E_SHAPE), (dict(lds=1), L.MOK_E_SHAPE), (dict(lds=2**30 + 1), L.MOK_E_SHAPE),
    (dict(v=None), L.MOK_E_NULL), (dict(c=None), L.MOK_E_NULL), (dict(s=None), L.MOK_E_NULL),
    (dict(v=FAKE + 4), L.MOK_E_SHAPE), (dict(c=FAKE + 8), L.MOK_E_SHAPE),
])
def test_mx8_quantisers_refuse(kw, code):
    a = dict(type=0, v=FAKE, ld=64, rows=4, cols=64, c=FAKE, ldc=64, s=FAKE, lds=2)
    a.update(kw)
    lib = L.load()
    assert lib.mok_quantize_mx8(a["type"], a["v"], a["ld"], a["rows"], a["cols"], a["c"], a["ldc"],
                                a["s"], a["lds"], None) == code
    assert lib.mok_dequantize_mx8(a["c"], a["ldc"], a["s"], a["lds"], a["rows"], a["cols"], a["type"],
                                  a["v"], a["ld"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(type=3), L.MOK_E_UNSUPPORTED), (dict(rows=-1), L.MOK_E_SHAPE), (dict(rows=1 << 31), L.MOK_E_SHAPE),
    (dict(inter=0), L.MOK_E_SHAPE), (dict(inter=48), L.MOK_E_SHAPE), (dict(inter=-32), L.MOK_E_SHAPE),
    (dict(inter=32800), L.MOK_E_SHAPE), (dict(groups=0), L.MOK_E_SHAPE), (dict(groups=1025), L.MOK_E_SHAPE),
    (dict(ld2=120), L.MOK_E_SHAPE), (dict(ld2=132), L.MOK_E_SHAPE), (dict(ld1=56), L.MOK_E_SHAPE),
    (dict(ld1=2**30 + 8), L.MOK_E_SHAPE), (dict(ldc=112), L.MOK_E_SHAPE), (dict(ldc=136), L.MOK_E_SHAPE),
    (dict(lds=3), L.MOK_E_SHAPE), (dict(two=None), L.MOK_E_NULL), (dict(one=None), L.MOK_E_NULL),
    (dict(c=None), L.MOK_E_NULL), (dict(s=None), L.MOK_E_NULL), (dict(two=FAKE + 8), L.MOK_E_SHAPE),
    (dict(one=FAKE + 2), L.MOK_E_SHAPE), (dict(c=FAKE + 8), L.MOK_E_SHAPE), (dict(off=FAKE + 1), L.MOK_E_SHAPE),
])
def test_swiglu_refuses(kw, code):
    a = dict(type=0, two=FAKE, ld2=128, one=FAKE, ld1=64, rows=4, inter=64, off=FAKE, groups=2, c=FAKE, ldc=128,
             s=FAKE, lds=4)
    a.update(kw)
    lib = L.load()
    assert lib.mok_swiglu_mx8(a["type"], a["two"], a["ld2"], a["rows"], a["inter"], a["off"], a["groups"],
                              a["one"], a["ld1"], a["c"], a["ldc"], a["s"], a["lds"], None) == code
    assert lib.mok_swiglu_mx8_bwd(a["type"], a["one"], a["ld1"], a["c"], a["ldc"], a["s"], a["lds"], a["rows"],
                                  a["inter"], a["off"], a["groups"], a["two"], a["ld2"], None, 0, None) == code
    if a["two"] and "one" in kw and a["one"]:  # the activation made again
        assert lib.mok_swiglu_mx8_bwd(a["type"], FAKE, 64, a["c"], a["ldc"], a["s"], a["lds"], a["rows"],
                                      a["inter"], a["off"], a["groups"], a["two"], a["ld2"], a["one"], a["ld1"],
                                      None) == code


def test_swiglu_refuses_written_rows_that_repeat():
    lib = L.load()
    assert lib.mok_swiglu_mx8(0, FAKE, 128, 4, 64, None, 0, FAKE, 0, FAKE, 128, FAKE, 4, None) == L.MOK_E_SHAPE
    assert lib.mok_swiglu_mx8_bwd(0, FAKE, 64, FAKE, 128, FAKE, 4, 4, 64, None, 0, FAKE, 0, None, 0,
                                  None) == L.MOK_E_SHAPE
    assert lib.mok_swiglu_mx8_bwd(0, FAKE, 64, FAKE, 128, FAKE, 4, 4, 64, None, 0, FAKE, 128, FAKE, 56,
                                  None) == L.MOK_E_SHAPE


# ----------------------------------------------------------------------------------------
# refusals of the torch-facing functions
# ----------------------------------------------------------------------------------------
def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


U8, I32, F32, F16 = torch.uint8, torch.int32, torch.float32, torch.float16


def _refuses(f, good, kw):
    with pytest.raises(ValueError) as e:
        f({**good, **kw})
    assert "on a GPU" not in str(e.value), kw


def test_grouped_mm_functions_refuse():
    good = dict(a=_t(6, 64), g=_t(6, 32), off=_t(3, dtype=I32), b=_t(2, 32, 64), out=None, dtype=None, add=False,
                s=None)
    calls = dict(
        out=lambda d: ops.grouped_mm(d["a"], d["off"], d["b"], out=d["out"], dtype=d["dtype"]),
        rows=lambda d: ops.grouped_mm_backward_rows(d["g"], d["off"], d["b"], out=d["out"], dtype=d["dtype"]),
        weights=lambda d: ops.grouped_mm_backward_weights(d["g"], d["a"], d["off"], a_scales=d["s"], out=d["out"],
                                                          dtype=d["dtype"] or F32, accumulate=d["add"]))
    for f in calls.values():
        with pytest.raises(ValueError, match="on a GPU"):
            f(good)
    for name in ("out", "rows"):
        for kw in (dict(off=_t(2, dtype=I32)), dict(off=_t(3, dtype=torch.int64)), dict(b=_t(2, 32, 64, dtype=F32)),
                   dict(b=_t(2, 64, 32).transpose(1, 2)), dict(b=_t(64, 64)), dict(dtype=F16),
                   dict(a=_t(6, 72), g=_t(6, 40)), dict(a=_t(6, 64, dtype=F16), g=_t(6, 32, dtype=F16)),
                   dict(a=_t(64, 6).t(), g=_t(32, 6).t()), dict(b=3)):
            _refuses(calls[name], good, kw)
    for kw in (dict(off=_t(3, dtype=torch.int64)), dict(off=_t(1, dtype=I32)), dict(off=_t(6, dtype=I32)[::2]),
               dict(g=_t(5, 32)), dict(g=_t(6, 32, dtype=F32)), dict(a=_t(6, 64, dtype=F16)), dict(dtype=F16),
               dict(a=_t(6, 64, dtype=U8)), dict(s=_t(6, 2, dtype=U8)), dict(add=True),
               dict(a=_t(6, 64, dtype=U8), s=_t(6, 3, dtype=U8)), dict(a=_t(6, 40, dtype=U8), s=_t(6, 1, dtype=U8))):
        _refuses(calls["weights"], good, kw)


def test_mx8_functions_refuse():
    for bad in (_t(4, 48), _t(4, 64, dtype=torch.float64), _t(4, 0)):
        with pytest.raises(ValueError):
            ops.quantize_mx8(bad)
    with pytest.raises(ValueError, match="on a GPU"):
        ops.quantize_mx8(_t(4, 64))
    with pytest.raises(ValueError, match="on a GPU"):
        ops.dequantize_mx8(_t(4, 64, dtype=U8), _t(4, 2, dtype=U8))
    for c, s, kw in ((_t(4, 64, dtype=U8), _t(4, 1, dtype=U8), {}), (_t(4, 48, dtype=U8), _t(4, 1, dtype=U8), {}),
                     (_t(4, 64, dtype=U8), _t(4, 2, dtype=U8), dict(dtype=torch.float64))):
        _refuses(lambda d: ops.dequantize_mx8(c, s, **kw), {}, {})
    good = dict(ab=_t(4, 128), dh=_t(4, 64), off=None, c=_t(4, 128, dtype=U8), s=_t(4, 4, dtype=U8))
    fwd = lambda d: ops.swiglu_mx8(d["ab"], d["off"])  # noqa: E731
    bwd = lambda d: ops.swiglu_mx8_backward(d["dh"], d["c"], d["s"], d["off"])  # noqa: E731
    for f in (fwd, bwd):
        with pytest.raises(ValueError, match="on a GPU"):
            f(good)
        for kw in (dict(ab=_t(4, 96), dh=_t(4, 48)), dict(ab=_t(4, 0), dh=_t(4, 0)),
                   dict(ab=_t(4, 128, dtype=torch.float64), dh=_t(4, 64, dtype=torch.float64)),
                   dict(ab=_t(128, 4).t(), dh=_t(64, 4).t()), dict(off=_t(3)), dict(off=_t(1, dtype=I32)),
                   dict(ab=_t(4, 2, 64), dh=_t(4, 2, 32))):
            _refuses(f, good, kw)
    for kw in (dict(c=_t(4, 64, dtype=U8)), dict(c=_t(4, 128)), dict(s=_t(4, 3, dtype=U8)), dict(s=_t(3, 4, dtype=U8))):
        _refuses(bwd, good, kw)


def test_sizes_past_32_bits_are_refused():
    big = 2**32 + 64
    off = torch.zeros(2, dtype=I32)
    with pytest.raises(ValueError, match="at most"):
        ops.grouped_mm(torch.empty(0, big, dtype=F16), off, torch.empty(0, 8, big, dtype=F16))
    with pytest.raises(ValueError, match="at most"):
        ops.grouped_mm_backward_weights(torch.empty(0, big, dtype=F16), torch.empty(0, 8, dtype=F16), off)
    with pytest.raises(ValueError, match="at most"):
        ops.quantize_mx8(torch.empty(0, big))
    with pytest.raises(ValueError, match="at most"):
        ops.swiglu_mx8(torch.empty(0, big))


def test_the_extension_module_passes_on_what_is_not_in_order():
    from mixture_experts_layer_mok_amd import _fast

    x, i = torch.zeros(4, 64), torch.zeros(4, 2, dtype=I32)
    counts = dict(grouped_mm=5, grouped_mm_backward_rows=5, grouped_mm_backward_weights=7, quantize_mx8=3,
                  dequantize_mx8=4, swiglu_mx8=5, swiglu_mx8_backward=7)
    for name, n in counts.items():
        f = getattr(_fast, name)
        assert f() is None and f(*[None] * n) is None and f(*[3] * n) is None
        assert f(*[x] * n) is None and f(*[i] * n) is None and f(*[x] * (n + 1)) is None
    with pytest.raises(TypeError):
        _fast.bind_more(1, 2)
    with pytest.raises(TypeError):
        _fast.bind_more(*["a"] * 8)
    with pytest.raises(ValueError):
        _fast.bind_more(*[0] * 8)
