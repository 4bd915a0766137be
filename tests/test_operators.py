"""CPU checks of the row operators and the MXFP4 operators: pins of their float64 forms
(autograd, differences, hand-worked codes), and the refusals of the C ABI and of the
torch-facing functions, which come before any GPU work."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_mok_amd import _lib as L
from mixture_experts_layer_mok_amd import ops
from oracle import operators as O

FAKE = 0x100000  # never dereferenced


def _routing(T, k, E, seed, masked=0.2):
    """pos of a random routing: rows in (expert, token, slot) order."""
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    ids = np.where(rng.random((T, k)) < masked, E, ids).reshape(-1)
    order = np.argsort(ids, kind="stable")
    R = int((ids < E).sum())
    pos = np.full(T * k, -1, np.int32)
    pos[order[:R]] = np.arange(R)
    return pos.reshape(T, k), R


def test_row_gradients_against_autograd_and_differences():
    pos, R = _routing(5, 3, 4, 1)
    rng = np.random.default_rng(2)
    x, w, dy = rng.standard_normal((5, 8)), rng.standard_normal((5, 3)), rng.standard_normal((5, 8))
    f = rng.standard_normal((R, 8))  # the experts: rows -> f * rows

    def loss(x, w):
        rows = O.permute(x, pos, np.zeros((R, 8)))
        return float((O.unpermute(f * rows, pos, w)[0] * dy).sum())

    rows = f * O.permute(x, pos, np.zeros((R, 8)))
    d_rows, dw, _ = O.unpermute_backward(dy, rows, pos, w, np.zeros((R, 8)))
    dx, _ = O.unpermute(f * d_rows, pos)
    xt, wt = (torch.tensor(v, requires_grad=True) for v in (x, w))
    y = torch.zeros(5, 8, dtype=torch.float64)
    for t in range(5):
        for j in range(3):
            if pos[t, j] >= 0:
                y = y + torch.nn.functional.one_hot(torch.tensor(t), 5).double()[:, None] * (
                    wt[t, j] * torch.tensor(f[pos[t, j]]) * xt[t])
    (y * torch.tensor(dy)).sum().backward()
    np.testing.assert_allclose(dx, xt.grad.numpy(), rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(dw, wt.grad.numpy(), rtol=1e-12, atol=1e-14)
    h = 1e-5
    for v, g in ((x, dx), (w, dw)):
        for i in np.ndindex(v.shape):
            keep = v[i]
            v[i] = keep + h
            up = loss(x, w)
            v[i] = keep - h
            down = loss(x, w)
            v[i] = keep
            assert abs((up - down) / (2 * h) - g[i]) < 1e-8


def test_mx4_codes_by_hand():
    v = np.zeros((1, 32))
    # amax 6: n = 0; ties at .25 (-> 0), .75 (-> 1), 1.25 (-> 1), 1.75 (-> 2), 2.5 (-> 2),
    # 3.5 (-> 4), 5 (-> 4)
    v[0, :12] = [6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.3, -1.6, -0.0, 2.51]
    c, s = O.quantize_mx4(v)
    assert s.tolist() == [[127]]
    assert c[0, :12].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 9, 11, 8, 5]
    # just above 6 * 2^n takes the next exponent; 6 * 2^n itself does not
    for amax, n in ((6.0, 0), (6.0625, 1), (3.0, -1), (3.03125, 0), (1.0, -2), (2.0**-126, -127),
                    (2.0**-140, -127), (3.3e38, 126)):
        w = np.zeros((1, 32))
        w[0, 5] = -amax
        assert O.quantize_mx4(w)[1][0, 0] == n + 127, amax
    assert O.quantize_mx4(np.zeros((1, 32)))[1][0, 0] == 0
    for bad in (np.inf, -np.inf, np.nan):
        w = np.ones((1, 64))
        w[0, 40] = bad
        c, s = O.quantize_mx4(w)
        assert s.tolist() == [[125, 255]] and not c[0, 32:].any()
        vals = O.values_mx4(O.pack4(c), s)
        assert (vals[0, :32] == 1).all() and np.isnan(vals[0, 32:]).all()


def test_mx4_packing_and_e4m3_values():
    c = np.arange(64, dtype=np.uint8).reshape(2, 32) % 16
    assert (O.unpack4(O.pack4(c)) == c).all()
    assert O.pack4(c)[0, 0] == 0x10  # element 0 in the low half
    codes = np.arange(256, dtype=np.uint8).reshape(8, 32)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(O.values_mx8(codes, np.full((8, 1), 127, np.uint8)), want)


# ----------------------------------------------------------------------------------------
# refusals of the C ABI
# ----------------------------------------------------------------------------------------
def _rows_calls(type=0, ld_x=64, pos=FAKE, T=4, k=2, cols=64, ld_r=64, n=8, x=FAKE, rows=FAKE,
                w=FAKE, dw=FAKE):
    lib = L.load()
    return dict(
        permute=lib.mok_permute(type, x, ld_x, pos, T, k, cols, rows, ld_r, n, None),
        permute_bwd=lib.mok_permute_bwd(type, rows, ld_r, n, pos, T, k, cols, x, ld_x, None),
        unpermute=lib.mok_unpermute(type, rows, ld_r, n, pos, w, T, k, cols, x, ld_x, None),
        unpermute_bwd=lib.mok_unpermute_bwd(type, x, ld_x, rows, ld_r, n, pos, w, T, k, cols, rows,
                                            ld_r, dw, None))


@pytest.mark.parametrize("kw,code", [
    (dict(type=3), L.MOK_E_UNSUPPORTED), (dict(type=-1), L.MOK_E_UNSUPPORTED),
    (dict(T=-1), L.MOK_E_SHAPE), (dict(T=(1 << 24) + 1, k=1), L.MOK_E_SHAPE),
    (dict(T=1 << 20, k=17), L.MOK_E_SHAPE), (dict(k=0), L.MOK_E_SHAPE), (dict(k=65), L.MOK_E_SHAPE),
    (dict(cols=0), L.MOK_E_SHAPE), (dict(cols=60), L.MOK_E_SHAPE),
    (dict(cols=65544, ld_x=65544, ld_r=65544), L.MOK_E_SHAPE), (dict(n=-1), L.MOK_E_SHAPE),
    (dict(n=1 << 31), L.MOK_E_SHAPE), (dict(ld_x=56), L.MOK_E_SHAPE), (dict(ld_r=68), L.MOK_E_SHAPE),
    (dict(ld_r=-64), L.MOK_E_SHAPE), (dict(ld_x=2**30 + 8), L.MOK_E_SHAPE),
    (dict(ld_r=2**30 + 8), L.MOK_E_SHAPE), (dict(pos=None), L.MOK_E_NULL), (dict(x=None), L.MOK_E_NULL),
    (dict(rows=None), L.MOK_E_NULL), (dict(x=FAKE + 8), L.MOK_E_SHAPE),
    (dict(rows=FAKE + 2), L.MOK_E_SHAPE), (dict(pos=FAKE + 1), L.MOK_E_SHAPE),
])
def test_row_operators_refuse(kw, code):
    assert set(_rows_calls(**kw).values()) == {code}


def test_row_operators_refuse_weights_and_written_strides():
    c = _rows_calls(w=None)
    assert c["unpermute"] == c["unpermute_bwd"] == L.MOK_E_NULL
    lib = L.load()
    assert lib.mok_unpermute_bwd(0, FAKE, 64, FAKE, 64, 8, FAKE, FAKE, 4, 2, 64, FAKE, 64, None,
                                 None) == L.MOK_E_NULL
    assert lib.mok_unpermute_bwd(0, FAKE, 64, FAKE, 64, 8, FAKE, FAKE, 4, 2, 64, FAKE, 64, FAKE + 2,
                                 None) == L.MOK_E_SHAPE
    # a written matrix may not repeat one row
    assert lib.mok_permute(0, FAKE, 64, FAKE, 4, 2, 64, FAKE, 0, 8, None) == L.MOK_E_SHAPE
    assert lib.mok_unpermute(0, FAKE, 64, 8, FAKE, FAKE, 4, 2, 64, FAKE, 0, None) == L.MOK_E_SHAPE


def test_empty_calls_do_nothing():
    assert set(_rows_calls(T=0, x=None, rows=None, pos=None, w=None, dw=None).values()) == {L.MOK_OK}
    lib = L.load()
    assert lib.mok_permute(0, None, 64, None, 4, 2, 64, None, 64, 0, None) == L.MOK_OK
    assert lib.mok_quantize_mx4(0, None, 64, 0, 64, None, 32, None, 2, None) == L.MOK_OK
    assert lib.mok_dequantize_mx4(None, 32, None, 2, 0, 64, 0, None, 64, None) == L.MOK_OK
    assert lib.mok_grouped_mx4(1, None, 32, None, 2, 0, None, 1, None, None, 64, 64, 0, None, 64,
                               None) == L.MOK_OK


@pytest.mark.parametrize("kw,code", [
    (dict(type=7), L.MOK_E_UNSUPPORTED), (dict(cols=48), L.MOK_E_SHAPE), (dict(cols=0), L.MOK_E_SHAPE),
    (dict(cols=65568), L.MOK_E_SHAPE), (dict(rows=-1), L.MOK_E_SHAPE), (dict(ld=56), L.MOK_E_SHAPE),
    (dict(ld=0), L.MOK_E_SHAPE), (dict(ld=68), L.MOK_E_SHAPE), (dict(ldc=24), L.MOK_E_SHAPE),
    (dict(ldc=40), L.MOK_E_SHAPE), (dict(ld=2**30 + 8), L.MOK_E_SHAPE),
    (dict(ldc=2**30 + 16), L.MOK_E_SHAPE), (dict(lds=2**30 + 1), L.MOK_E_SHAPE), (dict(lds=1), L.MOK_E_SHAPE), (dict(v=None), L.MOK_E_NULL),
    (dict(c=None), L.MOK_E_NULL), (dict(s=None), L.MOK_E_NULL), (dict(v=FAKE + 4), L.MOK_E_SHAPE),
    (dict(c=FAKE + 8), L.MOK_E_SHAPE),
])
def test_mx4_quantisers_refuse(kw, code):
    a = dict(type=0, v=FAKE, ld=64, rows=4, cols=64, c=FAKE, ldc=32, s=FAKE, lds=2)
    a.update(kw)
    lib = L.load()
    assert lib.mok_quantize_mx4(a["type"], a["v"], a["ld"], a["rows"], a["cols"], a["c"], a["ldc"],
                                a["s"], a["lds"], None) == code
    assert lib.mok_dequantize_mx4(a["c"], a["ldc"], a["s"], a["lds"], a["rows"], a["cols"], a["type"],
                                  a["v"], a["ld"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(fmt=2), L.MOK_E_UNSUPPORTED), (dict(ty=1), L.MOK_E_UNSUPPORTED),
    (dict(rows=-1), L.MOK_E_SHAPE), (dict(rows=(1 << 24) + 1), L.MOK_E_SHAPE),
    (dict(groups=0), L.MOK_E_SHAPE), (dict(groups=1025), L.MOK_E_SHAPE), (dict(k=48), L.MOK_E_SHAPE),
    (dict(k=0), L.MOK_E_SHAPE), (dict(n=12), L.MOK_E_SHAPE), (dict(n=0), L.MOK_E_SHAPE),
    (dict(n=1 << 20, k=2048, ld_out=1 << 20, ld_a=1024, ld_as=64), L.MOK_E_SHAPE),
    (dict(ld_a=16), L.MOK_E_SHAPE), (dict(ld_a=40), L.MOK_E_SHAPE), (dict(ld_as=1), L.MOK_E_SHAPE),
    (dict(fmt=0), L.MOK_E_SHAPE),  # e4m3 rows take k bytes
    (dict(ld_a=L.MOK_MX_MAX_LD + 16), L.MOK_E_SHAPE), (dict(ld_as=L.MOK_MX_MAX_LD + 1), L.MOK_E_SHAPE),
    (dict(ld_out=24), L.MOK_E_SHAPE), (dict(ld_out=(1 << 21) + 8), L.MOK_E_SHAPE), (dict(ld_out=68), L.MOK_E_SHAPE), (dict(a=None), L.MOK_E_NULL),
    (dict(as_=None), L.MOK_E_NULL), (dict(off=None), L.MOK_E_NULL), (dict(b=None), L.MOK_E_NULL),
    (dict(bs=None), L.MOK_E_NULL), (dict(out=None), L.MOK_E_NULL), (dict(a=FAKE + 8), L.MOK_E_SHAPE),
    (dict(b=FAKE + 4), L.MOK_E_SHAPE), (dict(out=FAKE + 8), L.MOK_E_SHAPE),
    (dict(off=FAKE + 2), L.MOK_E_SHAPE),
])
def test_grouped_mx4_refuses(kw, code):
    a = dict(fmt=1, a=FAKE, ld_a=32, as_=FAKE, ld_as=2, rows=8, off=FAKE, groups=2, b=FAKE, bs=FAKE,
             n=64, k=64, ty=0, out=FAKE, ld_out=64)
    a.update(kw)
    assert L.load().mok_grouped_mx4(*(a[n] for n in ("fmt", "a", "ld_a", "as_", "ld_as", "rows",
                                                     "off", "groups", "b", "bs", "n", "k", "ty",
                                                     "out", "ld_out")), None) == code


def test_schedule_layout():
    d = L.make_desc(128, 128, 64, 4, 2, M=32, S=2, comm_cus=8)
    off, pos = L.mok_schedule_layout(d)
    total = L.mok_workspace_size(d)
    assert off % 256 == 0 and pos % 256 == 0 and off != pos
    assert off + 5 * 4 <= total and pos + 128 * 2 * 4 <= total
    assert L.load().mok_schedule_layout(None, None, None) == L.MOK_E_NULL
    d.hidden = 100
    with pytest.raises(L.MokError) as e:
        L.mok_schedule_layout(d)
    assert e.value.code == L.MOK_E_SHAPE


# ----------------------------------------------------------------------------------------
# refusals of the torch-facing functions
# ----------------------------------------------------------------------------------------
def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def _row_tensors():
    return dict(x=_t(4, 64), rows=_t(8, 64), pos=_t(4, 2, dtype=torch.int32),
                w=_t(4, 2, dtype=torch.float32), dy=_t(4, 64), d_rows=_t(8, 64))


def _row_op(name, d):
    return {"permute": lambda: ops.permute(d["x"], d["pos"], d["rows"]),
            "permute_backward": lambda: ops.permute_backward(d["rows"], d["pos"], out=d["x"]),
            "unpermute": lambda: ops.unpermute(d["rows"], d["pos"], d["w"], out=d["x"]),
            "unpermute_backward": lambda: ops.unpermute_backward(d["dy"], d["rows"], d["pos"],
                                                                 d["w"], d["d_rows"])}[name]


ROW_OPS = ("permute", "permute_backward", "unpermute", "unpermute_backward")


@pytest.mark.parametrize("op", ROW_OPS)
def test_row_functions_want_gpu_tensors(op):
    with pytest.raises(ValueError, match="on a GPU"):
        _row_op(op, _row_tensors())()


@pytest.mark.parametrize("op", ROW_OPS)
@pytest.mark.parametrize("kw", [
    dict(pos=_t(4, 2, dtype=torch.int64)), dict(pos=_t(8, dtype=torch.int32)),
    dict(pos=_t(2, 4, dtype=torch.int32).t()), dict(rows=_t(8, 64, dtype=torch.float64)),
    dict(rows=_t(64, 8).t()), dict(rows=_t(8, 2, 32)),
])
def test_row_functions_refuse_tensors(op, kw):
    with pytest.raises(ValueError) as e:
        _row_op(op, {**_row_tensors(), **kw})()
    assert "on a GPU" not in str(e.value)


def test_row_functions_refuse_mismatches():
    d = _row_tensors()
    for op, kw in (("permute", dict(x=_t(5, 64))), ("permute", dict(x=_t(4, 72))),
                   ("permute", dict(x=_t(4, 64, dtype=torch.float16))),
                   ("permute", dict(rows=_t(1, 64).expand(8, 64))),
                   ("unpermute", dict(w=_t(4, 3, dtype=torch.float32))),
                   ("unpermute", dict(w=_t(4, 2))),
                   ("unpermute_backward", dict(dy=_t(3, 64))),
                   ("unpermute_backward", dict(d_rows=_t(7, 64)))):
        with pytest.raises(ValueError) as e:
            _row_op(op, {**d, **kw})()
        assert "on a GPU" not in str(e.value), (op, kw.keys())
    buf = _t(12, 64)
    with pytest.raises(ValueError, match="overlaps"):
        ops.permute(buf[:4], d["pos"], buf[2:10])


def test_mx4_functions_refuse():
    u8 = torch.uint8
    off = _t(3, dtype=torch.int32)
    good = dict(a=_t(4, 32, dtype=u8), s=_t(4, 2, dtype=u8), off=off, b=_t(2, 8, 32, dtype=u8),
                bs=_t(2, 8, 2, dtype=u8))

    def call(**kw):
        d = {**good, **kw}
        return ops.grouped_mx4(d["a"], d["s"], d["off"], d["b"], d["bs"],
                               dtype=d.get("dtype", torch.bfloat16))

    with pytest.raises(ValueError, match="on a GPU"):
        call()
    for kw in (dict(a=_t(4, 48, dtype=u8)), dict(a=_t(4, 32)), dict(s=_t(4, 3, dtype=u8)),
               dict(s=_t(5, 2, dtype=u8)), dict(off=_t(2, dtype=torch.int32)),
               dict(off=_t(3, dtype=torch.int64)), dict(b=_t(16, 32, dtype=u8)),
               dict(bs=_t(2, 8, 3, dtype=u8)), dict(b=_t(2, 8, 40, dtype=u8)),
               dict(b=_t(2, 32, 8, dtype=u8).transpose(1, 2)), dict(dtype=torch.float16)):
        with pytest.raises(ValueError) as e:
            call(**kw)
        assert "on a GPU" not in str(e.value), kw
    for bad in (_t(4, 48), _t(4, 64, dtype=torch.float64), _t(4, 0)):
        with pytest.raises(ValueError):
            ops.quantize_mx4(bad)
    with pytest.raises(ValueError, match="on a GPU"):
        ops.quantize_mx4(_t(4, 64))
    with pytest.raises(ValueError):
        ops.quantize_mx4(_t(4, 64).expand(4, 64)[:, ::1].unsqueeze(0).expand(2, 4, 64))
    with pytest.raises(ValueError, match="on a GPU"):
        ops.dequantize_mx4(_t(4, 32, dtype=u8), _t(4, 2, dtype=u8))
    with pytest.raises(ValueError):
        ops.dequantize_mx4(_t(4, 32, dtype=u8), _t(4, 1, dtype=u8))


def test_sizes_past_32_bits_are_refused():
    """Rows, slots and experts that the C ABI's 32-bit sizes would cut (tensors without memory)."""
    big = 2**32 + 64
    e = torch.empty(0, big)
    pos = torch.empty(0, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="at most"):
        ops.permute(e, pos, torch.empty(0, big))
    with pytest.raises(ValueError, match="at most"):
        ops.unpermute(e, pos, torch.empty(0, 2))
    with pytest.raises(ValueError, match="at most"):
        ops.permute(torch.empty(0, 64), torch.empty(0, big, dtype=torch.int32), torch.empty(0, 64))
    with pytest.raises(ValueError, match="at most"):
        ops.quantize_mx4(e)
    u8 = dict(dtype=torch.uint8)
    with pytest.raises(ValueError, match="at most"):
        ops.grouped_mx4(torch.empty(0, 32, **u8), torch.empty(0, 2, **u8), torch.empty(1, dtype=torch.int32),
                        torch.empty(0, big, 32, **u8), torch.empty(0, big, 2, **u8))


def test_the_layers_kernels_do_not_include_the_operators():
    """Counter summaries of the layer's kernels hold while only the operators' files change."""
    import os
    import re

    import bench

    names = os.listdir(bench.CSRC)
    assert set(bench.OPERATOR_SOURCES) <= set(names)
    for name in names:
        if name.endswith((".hip", ".h")) and name not in bench.OPERATOR_SOURCES:
            with open(os.path.join(bench.CSRC, name)) as f:
                included = re.findall(r'#include "([^"]+)"', f.read())
            assert not set(included) & set(bench.OPERATOR_SOURCES), name


def test_strides_of_no_rows_say_nothing():
    rows = torch.empty(0, 64).as_strided((0, 64), (1, 5))
    with pytest.raises(ValueError, match="on a GPU"):
        ops.permute_backward(rows, torch.full((3, 2), -1, dtype=torch.int32))
    with pytest.raises(ValueError, match="contiguous"):
        ops.permute_backward(torch.empty(5, 64).t(), torch.full((3, 2), -1, dtype=torch.int32))


def test_the_extension_module_passes_on_what_is_not_in_order():
    from mixture_experts_layer_mok_amd import _fast

    x, i = torch.zeros(4, 64), torch.zeros(4, 2, dtype=torch.int32)
    counts = dict(permute=3, permute_backward=3, unpermute=4, unpermute_backward=6, quantize_mx4=3,
                  dequantize_mx4=4, grouped_mx4=7)
    for name, n in counts.items():
        f = getattr(_fast, name)
        assert f() is None and f(*[None] * n) is None and f(*[3] * n) is None
        assert f(*[x] * n) is None and f(*[i] * n) is None and f(*[x] * (n + 1)) is None
    with pytest.raises(TypeError):
        _fast.bind(1, 2)
    with pytest.raises(TypeError):
        _fast.bind(len, len, *["a"] * 7)
    with pytest.raises(ValueError):
        _fast.bind(len, len, *[0] * 7)
