"""The row and MXFP4 functions as calls, on a GPU: ordinary calls take the extension module's
way and give what the Python code gives, bit for bit; what is refused is refused with nothing
written; work of two streams at once; captured graphs that overlap."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_mok_amd import _lib as L
from mixture_experts_layer_mok_amd import ops

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
NAMES = ["permute", "permute_backward", "unpermute", "unpermute_backward", "quantize_mx4",
         "dequantize_mx4", "grouped_mx4"]


def say(s):
    print(s, flush=True)


def data(seed=0, T=37, k=3, E=4, D=160, dtype=torch.bfloat16):
    """Arguments of every function, outputs last, by name."""
    g = torch.Generator().manual_seed(seed)
    pos = torch.randperm(T * k + 5, generator=g)[:T * k].to(torch.int32)
    pos[::7] = -1
    n = T * k + 5

    def rnd(*s):
        return torch.randn(*s, generator=g).to(DEV, dtype)

    pos = pos.view(T, k).to(DEV)
    x, rows, dy = rnd(T, D), rnd(n, D), rnd(T, D)
    w = torch.rand(T, k, generator=g).to(DEV)
    codes, scales = ops.quantize_mx4(rows)
    b, bs = ops.quantize_mx4(rnd(E, 72, D))
    cut = np.sort(np.random.default_rng(seed).integers(0, n, E - 1))
    off = torch.tensor([0, *cut, n], dtype=torch.int32, device=DEV)
    u8 = dict(dtype=torch.uint8, device=DEV)
    return dict(
        permute=[x, pos, torch.zeros_like(rows)], permute_backward=[rows, pos, torch.empty_like(x)],
        unpermute=[rows, pos, w, torch.empty_like(x)],
        unpermute_backward=[dy, rows, pos, w, torch.zeros_like(rows), torch.empty_like(w)],
        quantize_mx4=[rows, torch.empty(n, D // 2, **u8), torch.empty(n, D // 32, **u8)],
        dequantize_mx4=[codes, scales, torch.empty_like(rows)],
        grouped_mx4=[codes, scales, off, b, bs, torch.zeros(n, 72, dtype=torch.float32, device=DEV)])


OUTS = dict(permute=1, permute_backward=1, unpermute=1, unpermute_backward=2, quantize_mx4=2,
            dequantize_mx4=1, grouped_mx4=1)


def fast(name, *args):
    """The extension module's function; the output type that two of them take is bf16."""
    if name in ("dequantize_mx4", "grouped_mx4"):
        args = (*args[:-1], torch.bfloat16, args[-1])
    return getattr(ops._fast, name)(*args)


def through_python(name, args):
    n = OUTS[name]
    outs = [torch.zeros_like(t) for t in args[-n:]]
    a = args[:-n]
    stream = torch.cuda.current_stream()  # a stream given: the Python code
    if name == "unpermute_backward":
        ops.unpermute_backward(*a, outs[0], d_weights=outs[1], stream=stream)
    elif name == "quantize_mx4":
        ops.quantize_mx4(*a, codes=outs[0], scales=outs[1], stream=stream)
    elif name == "permute":
        ops.permute(*a, outs[0], stream=stream)
    else:
        getattr(ops, name)(*a, out=outs[0], stream=stream)
    return outs


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32],
                         ids=["bf16", "fp16", "fp32"])
def test_both_ways_agree(dtype):
    for name, args in data(dtype=dtype).items():
        say(f"[calls] {name} {dtype}")
        got = fast(name, *args)
        assert got is not None
        n = OUTS[name]
        got = list(got) if n > 1 else [got]
        assert all(g is a for g, a in zip(got, args[-n:]))
        for g, w in zip(got, through_python(name, args)):
            assert torch.equal(g, w)


@pytest.mark.parametrize("name,n", [("permute_backward", 1), ("unpermute", 1),
                                    ("unpermute_backward", 1), ("quantize_mx4", 2),
                                    ("dequantize_mx4", 1), ("grouped_mx4", 1)])
def test_outputs_made_by_the_call(name, n):
    args = data()[name]
    if name == "grouped_mx4":
        args[-1] = args[-1].to(torch.bfloat16)
        args[2][0], args[2][-1] = 0, len(args[0])  # every row of the output is written
    want = through_python(name, args)
    got = fast(name, *args[:-n], *[None] * n)
    got = list(got) if isinstance(got, tuple) else [got]
    for g, w in zip(got, want):
        assert g.dtype == w.dtype and g.device == w.device and torch.equal(g, w)


def test_three_axes_and_no_rows():
    x = torch.randn(3, 5, 64, device=DEV)
    c, s = ops.quantize_mx4(x)
    assert c.shape == (3, 5, 32) and s.shape == (3, 5, 2)
    c2, s2 = ops.quantize_mx4(x.view(15, 64), stream=torch.cuda.current_stream())
    assert torch.equal(c.view(15, 32), c2) and torch.equal(s.view(15, 2), s2)
    out = torch.empty_like(x)
    assert torch.equal(ops.dequantize_mx4(c, s, out=out).view(15, 64),
                       ops.dequantize_mx4(c2, s2, dtype=torch.float32))
    pos = torch.empty(0, 2, dtype=torch.int32, device=DEV)
    e = torch.empty(0, 64, device=DEV)
    assert ops.unpermute(x[0], pos, torch.empty(0, 2, device=DEV)).shape == (0, 64)
    assert ops.permute_backward(x[0], pos).shape == (0, 64)
    out = torch.full((4, 64), 3.0, device=DEV)
    assert (ops.permute(e, pos, out) == 3).all()
    rows = torch.empty(0, 64, device=DEV).as_strided((0, 64), (1, 5))
    pos = torch.full((3, 2), -1, dtype=torch.int32, device=DEV)
    for stream in (None, torch.cuda.current_stream()):
        y = ops.permute_backward(rows, pos, stream=stream)
        assert y.shape == (3, 64) and not y.any()


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
        return torch.empty(t.shape[::-1], dtype=t.dtype, device=t.device).permute(
            *range(t.dim() - 1, -1, -1))
    raise AssertionError(how)


@pytest.mark.parametrize("name", NAMES)
def test_refused_with_nothing_written(name):
    """Each argument in turn made wrong: the extension passes the call on, the function raises,
    and the other outputs hold what they held."""
    args = data()[name]
    n = OUTS[name]
    for i in range(len(args)):
        for how in ("not a tensor", "cpu", "type", "axis", "more", "less", "turned"):
            if how == "more" and ((name == "permute" and i == 2) or
                                  (name in ("permute_backward", "unpermute") and i == 0)):
                continue  # any number of rows is in order there
            if how in ("axis", "turned") and args[i].dim() < 2:
                continue
            bad = list(args)
            bad[-n:] = [torch.full_like(t, 5) for t in args[-n:]]
            bad[i] = wrong(bad[i], how)
            say(f"[calls] {name} argument {i} {how}")
            assert fast(name, *bad) is None
            kw = {}
            call = list(bad)
            if name in ("permute_backward", "unpermute", "dequantize_mx4", "grouped_mx4"):
                kw = dict(out=call.pop())
            with pytest.raises((ValueError, L.MokError)):
                getattr(ops, name)(*call, **kw)
            torch.cuda.synchronize()
            for j in range(len(args) - n, len(args)):
                if j != i:
                    assert (bad[j] == 5).all()


@pytest.mark.parametrize("name", NAMES)
def test_refused_where_an_output_is_an_input(name):
    """An output in the memory of an input (as bytes, where their types differ)."""
    args = data(T=64, k=2, D=128)[name]
    n = OUTS[name]
    for o in range(len(args) - n, len(args)):
        for i in range(len(args)):
            if i == o or args[i].numel() * args[i].element_size() < 32:
                continue
            bad = list(args)
            need = max(args[o].numel() * args[o].element_size(), args[i].numel() * args[i].element_size())
            mem = torch.zeros(need + 64, dtype=torch.uint8, device=DEV)

            def put(t):
                return mem[:t.numel() * t.element_size()].view(t.dtype).view(t.shape)

            bad[i], bad[o] = put(args[i]), put(args[o])
            say(f"[calls] {name} output {o} in input {i}")
            assert fast(name, *bad) is None
            kw = {}
            if name in ("permute_backward", "unpermute", "dequantize_mx4", "grouped_mx4"):
                kw = dict(out=bad.pop())
            with pytest.raises(ValueError, match="overlaps"):
                getattr(ops, name)(*bad, **kw)


def test_two_streams_at_once():
    """The same functions on two streams with their own outputs, neither waiting for the other."""
    sets = [data(seed=s, T=500, k=4, E=5, D=416) for s in (1, 2)]
    want = [{n: through_python(n, a) for n, a in d.items()} for d in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        for d, s in zip(sets, streams):
            with torch.cuda.stream(s):
                for name in NAMES:
                    getattr(ops, name)(*d[name]) if name in ("permute", "unpermute_backward", "quantize_mx4") \
                        else getattr(ops, name)(*d[name][:-1], out=d[name][-1])
    torch.cuda.synchronize()
    for d, w in zip(sets, want):
        for name in NAMES:
            for g, r in zip(d[name][-OUTS[name]:], w[name]):
                assert torch.equal(g, r)


def test_two_graphs_replayed_on_two_streams():
    sets = [data(seed=s, T=300, k=4, E=5, D=416) for s in (3, 4)]
    want = [{n: through_python(n, a) for n, a in d.items()} for d in sets]
    torch.cuda.synchronize()
    graphs = []
    for d in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for name in NAMES:
                assert fast(name, *d[name]) is not None
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        for d in sets:
            for name in NAMES:
                for t in d[name][-OUTS[name]:]:
                    t.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for d, w in zip(sets, want):
            for name in NAMES:
                for g, r in zip(d[name][-OUTS[name]:], w[name]):
                    assert torch.equal(g, r)


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_a_given_stream(raw):
    """Work goes to the stream that is given, a torch stream or its handle, behind what is on it."""
    for name, args in data(seed=5, T=200, k=2, D=256).items():
        want = through_python(name, args)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        n = OUTS[name]
        late = [t.clone() for t in args[:-n]]
        kept = [t.clone() for t in late]
        for t in late:
            t.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):  # the inputs are there only once the stream is at this point
            torch.cuda._sleep(2_000_000)
            for t, k in zip(late, kept):
                t.copy_(k)
        s = side.cuda_stream if raw else side
        if name in ("permute", "unpermute_backward", "quantize_mx4"):
            getattr(ops, name)(*late, *args[-n:], stream=s)
        else:
            getattr(ops, name)(*late, out=args[-1], stream=s)
        side.synchronize()
        for g, w in zip(args[-n:], want):
            assert torch.equal(g, w), name
