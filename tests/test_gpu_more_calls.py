"""The 16-bit grouped products and the functions of activations in 8 bits as calls, on a GPU: ordinary
calls take the extension module's way and give what the Python code gives, bit for bit; what is refused
is refused with nothing written; outputs count as changed; given streams, two streams at once, captured
graphs that overlap; a launch that fails is raised once; no extension module."""
import ctypes
import sys

import numpy as np
import pytest
import torch

import mixture_experts_layer_mok_amd as package
from mixture_experts_layer_mok_amd import _lib as L
from mixture_experts_layer_mok_amd import ops

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, FP, F32, U8 = torch.bfloat16, torch.float16, torch.float32, torch.uint8


def say(s):
    print(s, flush=True)


class Call:
    """A function's name, its arguments by name, outputs last, and which of them are outputs."""

    def __init__(self, fn, args, outs, fixed=None):
        self.fn, self.args, self.outs, self.fixed = fn, args, outs, fixed or {}

    def with_args(self, **kw):
        return Call(self.fn, {**self.args, **kw}, self.outs, self.fixed)

    def python(self, stream=None):
        return getattr(ops, self.fn)(**self.args, **self.fixed, stream=stream)

    def fast(self):
        a = {**self.args, **self.fixed}
        order = dict(grouped_mm=("a", "offsets", "b", "dtype", "out"),
                     grouped_mm_backward_rows=("d_out", "offsets", "b", "dtype", "out"),
                     grouped_mm_backward_weights=("d_out", "a", "offsets", "a_scales", "dtype", "out", "accumulate"),
                     quantize_mx8=("src", "codes", "scales"), dequantize_mx8=("codes", "scales", "dtype", "out"),
                     swiglu_mx8=("ab", "offsets", "h", "codes", "scales"),
                     swiglu_mx8_backward=("dh", "codes", "scales", "offsets", "d_ab", "h", "with_h"))[self.fn]
        default = dict(dtype=F32 if self.fn.endswith("weights") else BF if self.fn.startswith("de") else None,
                       accumulate=False, with_h=True)
        return getattr(ops._fast, self.fn)(*(a.get(k, default.get(k)) for k in order))

    def written(self):
        return [self.args[k] for k in self.outs]


def calls(seed=0, dtype=BF, rows=90, n=72, k=128, E=4):
    g = torch.Generator().manual_seed(seed)

    def rnd(*s, d=dtype):
        return torch.randn(*s, generator=g).to(DEV, d)

    def z(*s, d=dtype):
        return torch.zeros(*s, dtype=d, device=DEV)

    cut = np.sort(np.random.default_rng(seed).integers(0, rows - 9, E - 1))
    off = torch.tensor([0, *cut, rows - 9], dtype=torch.int32, device=DEV)
    a, dy, b = rnd(rows, k), rnd(rows, n), rnd(E, n, k)
    codes, scales = ops.quantize_mx8(a)
    ab, dh = rnd(rows, 2 * k), rnd(rows, k)
    c2, s2 = ops.quantize_mx8(ab)
    return dict(
        out=Call("grouped_mm", dict(a=a, offsets=off, b=b, out=z(rows, n)), ["out"]),
        rows=Call("grouped_mm_backward_rows", dict(d_out=dy, offsets=off, b=b, out=z(rows, k)), ["out"]),
        weights=Call("grouped_mm_backward_weights", dict(d_out=dy, a=a, offsets=off, out=z(E, n, k, d=F32)), ["out"]),
        held=Call("grouped_mm_backward_weights", dict(d_out=dy, a=codes, offsets=off, a_scales=scales,
                                                      out=z(E, n, k)), ["out"]),
        quantize=Call("quantize_mx8", dict(src=a, codes=z(rows, k, d=U8), scales=z(rows, k // 32, d=U8)),
                      ["codes", "scales"]),
        dequantize=Call("dequantize_mx8", dict(codes=codes, scales=scales, out=z(rows, k)), ["out"]),
        swiglu=Call("swiglu_mx8", dict(ab=ab, offsets=off, h=z(rows, k), codes=z(rows, 2 * k, d=U8),
                                       scales=z(rows, k // 16, d=U8)), ["h", "codes", "scales"]),
        swiglu_backward=Call("swiglu_mx8_backward", dict(dh=dh, codes=c2, scales=s2, offsets=off, d_ab=z(rows, 2 * k),
                                                         h=z(rows, k)), ["d_ab", "h"]))


NAMES = ["out", "rows", "weights", "held", "quantize", "dequantize", "swiglu",
         "swiglu_backward"]


def through_python(c):
    fresh = c.with_args(**{k: torch.zeros_like(c.args[k]) for k in c.outs})
    fresh.python(stream=torch.cuda.current_stream())  # a stream given: the Python code
    return fresh.written()


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
def test_both_ways_agree(dtype):
    for name, c in calls(dtype=dtype).items():
        say(f"[calls] {name} {dtype}")
        got = c.fast()
        assert got is not None
        got = list(got) if isinstance(got, tuple) else [got]
        assert all(g is o for g, o in zip(got, c.written()))
        for g, w in zip(got, through_python(c)):
            assert torch.equal(g, w)


@pytest.mark.parametrize("name", ["quantize", "dequantize", "swiglu", "swiglu_backward"])
def test_both_ways_agree_in_fp32(name):
    c = calls(dtype=BF)[name]
    c = c.with_args(**{k: v.float() for k, v in c.args.items() if v.dtype is BF})
    assert c.fast() is not None
    for g, w in zip(c.written(), through_python(c)):
        assert torch.equal(g, w)


@pytest.mark.parametrize("name", NAMES)
def test_outputs_made_by_the_call(name):
    c = calls()[name]
    c.args["offsets"] = torch.tensor([0, 20, 20, 50, 90], dtype=torch.int32, device=DEV)  # every row is covered
    if "offsets" not in calls()[name].args:
        del c.args["offsets"]
    bare = c.with_args(**{k: None for k in c.outs})
    if name == "held":
        bare.fixed = dict(dtype=BF)
    want = through_python(c)
    for got in (bare.fast(), bare.python(stream=torch.cuda.current_stream())):
        got = list(got) if isinstance(got, tuple) else [got]
        for g, w in zip(got, want):
            assert g.dtype == w.dtype and g.device == w.device and torch.equal(g, w) and not g.requires_grad


def test_fp32_results_and_accumulation():
    c = calls()
    for name in ("out", "rows"):
        for got in (c[name].with_args(out=None), c[name].with_args(out=None)):
            got.fixed = dict(dtype=F32)
            y, z = got.fast(), got.python(stream=torch.cuda.current_stream())
            n = int(c[name].args["offsets"][-1])
            assert y.dtype is F32 and torch.equal(y[:n], z[:n])
    for name in ("weights", "held"):
        d = c[name].with_args(out=torch.zeros(4, 72, 128, device=DEV))
        d.python()
        once = d.args["out"].clone()
        d.fixed = dict(accumulate=True)
        assert d.fast() is d.args["out"]
        assert torch.equal(d.args["out"], 2 * once)
        d.python(stream=torch.cuda.current_stream())
        assert torch.equal(d.args["out"], 2 * once + once)
        for bad in (d.with_args(out=None), d.with_args(out=torch.zeros(4, 72, 128, dtype=BF, device=DEV))):
            assert bad.fast() is None
            with pytest.raises(ValueError):
                bad.python()


def test_swiglu_without_offsets_and_without_h():
    c = calls()
    f, b = c["swiglu"], c["swiglu_backward"]
    h, codes, scales = ops.swiglu_mx8(f.args["ab"])
    c2, s2 = ops.quantize_mx8(f.args["ab"])
    assert torch.equal(codes, c2) and torch.equal(scales, s2)
    d, again = ops.swiglu_mx8_backward(b.args["dh"], codes, scales)
    for stream in (None, torch.cuda.current_stream()):
        d2, none = ops.swiglu_mx8_backward(b.args["dh"], codes, scales, with_h=False, stream=stream)
        assert none is None and torch.equal(d, d2)
        out = torch.empty_like(again)
        assert ops.swiglu_mx8_backward(b.args["dh"], codes, scales, h=out, with_h=False, stream=stream)[1] is out
        assert torch.equal(out, again)


def test_no_rows():
    e = torch.empty(0, 128, dtype=BF, device=DEV)
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    b = torch.ones(2, 72, 128, dtype=BF, device=DEV)
    for stream in (None, torch.cuda.current_stream()):
        assert ops.grouped_mm(e, off, b, stream=stream).shape == (0, 72)
        assert ops.grouped_mm_backward_rows(e[:, :72], off, b, stream=stream).shape == (0, 128)
        w = torch.full((2, 72, 128), 3.0, device=DEV)
        assert not ops.grouped_mm_backward_weights(e[:, :72], e, off, out=w, stream=stream).any()
        w = torch.full((2, 72, 128), 3.0, device=DEV)
        assert (ops.grouped_mm_backward_weights(e[:, :72], e, off, out=w, accumulate=True, stream=stream) == 3).all()
        c, s = ops.quantize_mx8(e, stream=stream)
        assert c.shape == (0, 128) and s.shape == (0, 4)
        assert ops.dequantize_mx8(c, s, stream=stream).shape == (0, 128)
        h, c, s = ops.swiglu_mx8(e, off, stream=stream)
        assert h.shape == (0, 64) and c.shape == (0, 128) and s.shape == (0, 4)
        d, h = ops.swiglu_mx8_backward(h, c, s, off, stream=stream)
        assert d.shape == (0, 128) and h.shape == (0, 64)
    x = torch.randn(3, 5, 64, device=DEV)
    c, s = ops.quantize_mx8(x)
    assert c.shape == (3, 5, 64) and s.shape == (3, 5, 2)
    c2, s2 = ops.quantize_mx8(x.view(15, 64), stream=torch.cuda.current_stream())
    assert torch.equal(c.view(15, 64), c2) and torch.equal(s.view(15, 2), s2)
    assert torch.equal(ops.dequantize_mx8(c, s, dtype=F32).view(15, 64), ops.dequantize_mx8(c2, s2, dtype=F32))


def wrong(t, how):
    """t with one thing about it wrong."""
    if how == "not a tensor":
        return 3
    if how == "cpu":
        return t.cpu()
    if how == "type":
        return t.to(torch.float64)
    if how == "axis":
        return t.reshape(-1)
    if how == "more":
        return torch.cat([t, t])
    if how == "less":
        return t[..., :-1]
    if how == "turned":
        return torch.empty(t.shape[::-1], dtype=t.dtype, device=t.device).permute(*range(t.dim() - 1, -1, -1))
    raise AssertionError(how)


@pytest.mark.parametrize("name", NAMES)
def test_refused_with_nothing_written(name):
    """Each argument in turn made wrong: the extension passes the call on, the function raises, and the
    other outputs hold what they held."""
    c = calls()[name]
    for arg in c.args:
        for how in ("not a tensor", "cpu", "type", "axis", "more", "less", "turned"):
            if how in ("axis", "turned") and c.args[arg].dim() < 2:
                continue
            if arg == "offsets" and how in ("more", "less") and name.startswith("swiglu"):
                continue  # any number of experts is in order there
            bad = c.with_args(**{o: torch.full_like(c.args[o], 5) for o in c.outs})
            bad.args[arg] = wrong(bad.args[arg], how)
            say(f"[calls] {name} {arg} {how}")
            assert bad.fast() is None
            with pytest.raises((ValueError, L.MokError)):
                bad.python()
            torch.cuda.synchronize()
            for o in c.outs:
                if o != arg:
                    assert (bad.args[o] == 5).all()


@pytest.mark.parametrize("name", NAMES)
def test_refused_where_an_output_is_an_input(name):
    c = calls()[name]
    for o in c.outs:
        for i in c.args:
            if i == o or c.args[i].numel() * c.args[i].element_size() < 32:
                continue
            need = max(v.numel() * v.element_size() for v in (c.args[o], c.args[i]))
            mem = torch.zeros(need + 64, dtype=U8, device=DEV)

            def put(t):
                return mem[:t.numel() * t.element_size()].view(t.dtype).view(t.shape)

            bad = c.with_args(**{i: put(c.args[i]), o: put(c.args[o])})
            say(f"[calls] {name} output {o} in {i}")
            assert bad.fast() is None
            with pytest.raises(ValueError, match="overlaps"):
                bad.python()


@pytest.fixture(params=[False, True], ids=["extension", "python"])
def stream(request):
    return torch.cuda.current_stream() if request.param else None


@pytest.mark.parametrize("name", NAMES)
def test_written_outputs_count_as_changed(name, stream):
    c = calls()[name]
    before = {k: v._version for k, v in c.args.items()}
    c.python(stream=stream)
    assert {k: v._version for k, v in c.args.items()} == {k: v + (k in c.outs) for k, v in before.items()}


@pytest.mark.parametrize("name", NAMES)
def test_results_have_no_graph_and_inference_mode(name, stream):
    c = calls()[name]
    for k, v in c.args.items():
        if v.is_floating_point() and k not in c.outs:
            v.requires_grad_(True)
    got = c.python(stream=stream)
    for t in got if isinstance(got, tuple) else [got]:
        assert not t.requires_grad and t.grad_fn is None
    want = [t.clone() for t in c.written()]
    with torch.inference_mode():
        d = c.with_args(**{o: torch.zeros_like(c.args[o]) for o in c.outs})
        d.python(stream=stream)
    assert all(torch.equal(o, w) for o, w in zip(d.written(), want))
    d.python(stream=stream)


def big(seed):
    """Sizes at which several forms run: whole and small tiles, few rows, split sums."""
    out = list(calls(seed=seed, rows=700, n=264, k=416, E=5).items())
    out += [(n + " deep", c) for n, c in calls(seed=seed + 9, rows=3000, n=40, k=1600, E=2).items()]
    out += [(n + " wide", c) for n, c in calls(seed=seed + 18, rows=1500, n=2048, k=2048, E=4).items() if n == "out"]
    return dict(out)


def test_two_streams_at_once():
    """The same functions on two streams with their own outputs, neither waiting for the other."""
    sets = [big(s) for s in (1, 2)]
    want = [{n: through_python(c) for n, c in d.items()} for d in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        for d, s in zip(sets, streams):
            with torch.cuda.stream(s):
                for c in d.values():
                    c.python()
    torch.cuda.synchronize()
    for d, w in zip(sets, want):
        for n, c in d.items():
            assert all(torch.equal(g, r) for g, r in zip(c.written(), w[n])), n


def test_two_graphs_replayed_on_two_streams():
    """Captured with workspaces of their own, replayed at once, with new routing written in between and
    eager work of the same functions beside them."""
    sets = [big(s) for s in (3, 4)]
    for d in sets:
        for c in d.values():
            assert c.fast() is not None
    torch.cuda.synchronize()
    graphs = []
    for d in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for c in d.values():
                assert c.fast() is not None
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in sets]
    for turn in range(4):
        for d in sets:
            for c in d.values():
                if "offsets" in c.args:
                    off = c.args["offsets"]
                    rows = next(v.shape[0] for k, v in c.args.items() if k in ("a", "d_out", "ab", "dh"))
                    last = max(2, rows // (turn + 1) - 7)
                    new = [0, *np.sort(np.random.default_rng(turn).integers(0, last, len(off) - 2)), last]
                    off.copy_(torch.tensor(new, dtype=torch.int32))
                for t in c.written():
                    t.zero_()
        want = [{n: through_python(c) for n, c in d.items()} for d in sets]
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        other = calls(seed=turn)["out"]
        other.python()
        torch.cuda.synchronize()
        for d, w in zip(sets, want):
            for n, c in d.items():
                assert all(torch.equal(g, r) for g, r in zip(c.written(), w[n])), (turn, n)


@pytest.mark.parametrize("forward", [True, False], ids=["out", "rows"])
def test_a_captured_product_with_any_routing(forward):
    """One capture at a share's buffer size, replayed with routings that ask for each form, for a last
    round of few tiles split along the sum, and for nothing: as the eager call each time."""
    rows, E, n, k = 16500, 8, *((1024, 4104) if forward else (4104, 1024))
    gen = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn(rows, k if forward else n, generator=gen, device=DEV).to(BF)
    b = (torch.randn(E, n, k, generator=gen, device=DEV) * 0.05).to(BF)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    fn = ops.grouped_mm if forward else ops.grouped_mm_backward_rows
    assert L.mok_grouped_mm_workspace(0 if forward else 1, rows, E, n, k) == L.MOK_MM_WORKSPACE_BYTES
    out = torch.full((rows, n if forward else k), 7.0, dtype=BF, device=DEV)
    fn(x, off, b, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fn(x, off, b, out=out)
    for counts in ([2053, 2030, 2048, 2061, 1999, 2001, 2077, 2040], [1, 0, 3, 0, 0, 2, 1, 0], [0] * 8,
                   [16500] + [0] * 7, [500, 530, 512, 498, 470, 513, 560, 500], [8300, 0, 0, 0, 0, 0, 0, 8200],
                   [70, 40, 60, 33, 64, 90, 20, 1]):
        say(f"[mm] captured {counts}")
        at = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        off.copy_(torch.from_numpy(at))
        want = torch.full_like(out, 7.0)
        fn(x, off, b, out=want)
        for _ in range(2):
            out.fill_(7.0)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
        assert bool((want[int(at[-1]):] == 7.0).all())
        # products of two bf16 values are exact in fp32; a sum of 4104 in any order is off by at most
        # 4104 * 2^-24 (and 1/1000 of that) of the sum of magnitudes, here and in the plain form, and the
        # result is then rounded by at most 2^-8 of itself
        for e in range(E):
            i, j = int(at[e]), int(at[e + 1])
            v, w = x[i:j].float(), b[e].float().t() if forward else b[e].float()
            plain, off_by = v @ w, 2 * 4104 * 1.001 * 2**-24 * (v.abs() @ w.abs())
            assert bool(((want[i:j].float() - plain).abs() <= 2**-8 * (plain.abs() + off_by) + off_by).all())


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_a_given_stream(raw):
    """Work goes to the stream that is given, a torch stream or its handle, behind what is on it."""
    for name, c in big(5).items():
        want = through_python(c)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        inputs = {k: v for k, v in c.args.items() if k not in c.outs}
        late = {k: torch.zeros_like(v) for k, v in inputs.items()}
        torch.cuda.synchronize()
        with torch.cuda.stream(side):  # the inputs are there only once the stream is at this point
            torch.cuda._sleep(2_000_000)
            for k, v in inputs.items():
                late[k].copy_(v)
        c.with_args(**late).python(stream=side.cuda_stream if raw else side)
        side.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(c.written(), want)), name


ENTRIES = dict(grouped_mm="mok_grouped_mm", grouped_mm_backward_rows="mok_grouped_mm_bwd_rows",
               grouped_mm_backward_weights="mok_grouped_mm_bwd_weights", quantize_mx8="mok_quantize_mx8",
               dequantize_mx8="mok_dequantize_mx8", swiglu_mx8="mok_swiglu_mx8",
               swiglu_mx8_backward="mok_swiglu_mx8_bwd")


@pytest.mark.parametrize("name", NAMES)
def test_a_failed_launch_is_raised_once(name):
    """Entry points that only report a failed launch, in place of the library's."""
    c = calls()[name]
    for t in c.written():
        t.fill_(5)
    ops.quantize_mx8(torch.zeros(1, 32, device=DEV))  # the extension module is bound
    lib, made = L.load(), []

    def stub(fn):
        def fail(*_):
            made.append(fn)
            return L.MOK_E_LAUNCH

        f = getattr(lib, fn)
        return ctypes.CFUNCTYPE(ctypes.c_int, *f.argtypes)(fail)

    stubs = [stub(fn) for fn in ENTRIES.values()]
    try:
        ops._fast.bind_more(*(ctypes.cast(s, ctypes.c_void_p).value for s in (*stubs, lib.mok_grouped_mm_workspace)))
        with pytest.raises(L.MokError) as e:
            c.python()
    finally:
        ops._bind(lib)
    assert e.value.code == L.MOK_E_LAUNCH and ENTRIES[c.fn] in str(e.value)
    assert made == [ENTRIES[c.fn]]
    torch.cuda.synchronize()
    assert all((t == 5).all() for t in c.written())


@pytest.mark.parametrize("name", NAMES)
def test_without_the_extension_module(name, monkeypatch):
    c = calls()[name]
    want = through_python(c)
    torch.cuda.synchronize()
    monkeypatch.delattr(package, "_fast", raising=False)
    monkeypatch.setitem(sys.modules, package.__name__ + "._fast", None)
    monkeypatch.setattr(ops, "_fast", None)
    monkeypatch.setattr(ops, "_bound", False)
    with pytest.warns(RuntimeWarning, match="_fast is not used"):
        c.python()
    assert ops._fast is None
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(c.written(), want))


def test_an_earlier_error_of_another_call():
    """The runtime remembers that a device number did not exist; the launch after it is in order."""
    lib = L.load()
    for name, c in calls().items():
        want = through_python(c)
        torch.cuda.synchronize()
        assert lib.hipSetDevice(4096) != 0
        c.python()
        lib.hipGetLastError()
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(c.written(), want)), name
