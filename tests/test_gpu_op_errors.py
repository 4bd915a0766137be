"""Errors around the row and MXFP4 functions' launches, on a GPU: a launch that fails is raised and
not repeated; an error that another call left behind is not taken for the launch's; without the
extension module every function runs."""
import ctypes
import sys

import pytest
import torch

import mixture_experts_layer_mok_amd as package
from mixture_experts_layer_mok_amd import _lib as L
from mixture_experts_layer_mok_amd import ops
from tests.test_gpu_op_calls import NAMES, OUTS, data, through_python

pytestmark = pytest.mark.gpu
ENTRIES = dict(permute="mok_permute", permute_backward="mok_permute_bwd", unpermute="mok_unpermute",
               unpermute_backward="mok_unpermute_bwd", quantize_mx4="mok_quantize_mx4",
               dequantize_mx4="mok_dequantize_mx4", grouped_mx4="mok_grouped_mx4")


def call(name, args):
    if name in ("permute", "unpermute_backward", "quantize_mx4"):
        return getattr(ops, name)(*args)
    return getattr(ops, name)(*args[:-1], out=args[-1])


@pytest.mark.parametrize("name", NAMES)
def test_a_failed_launch_is_raised_once(name):
    """Entry points that only report a failed launch, in place of the library's."""
    args = data()[name]
    outs = args[-OUTS[name]:]
    for t in outs:
        t.fill_(5)
    ops.quantize_mx4(torch.zeros(1, 32, device="cuda"))  # the extension module is bound
    calls = []

    def stub(fn):
        def fail(*_):
            calls.append(fn)
            return L.MOK_E_LAUNCH

        f = getattr(L.load(), fn)
        return ctypes.CFUNCTYPE(ctypes.c_int, *f.argtypes)(fail)

    stubs = [stub(fn) for fn in ENTRIES.values()]
    try:
        ops._fast.bind(torch.cuda.current_device, ops._raw_stream,
                       *(ctypes.cast(s, ctypes.c_void_p).value for s in stubs))
        with pytest.raises(L.MokError) as e:
            call(name, args)
    finally:
        ops._bind(L.load())
    assert e.value.code == L.MOK_E_LAUNCH and ENTRIES[name] in str(e.value)
    assert calls == [ENTRIES[name]]
    torch.cuda.synchronize()
    assert all((t == 5).all() for t in outs)


@pytest.mark.parametrize("name", NAMES)
def test_without_the_extension_module(name, monkeypatch):
    args = data()[name]
    n = OUTS[name]
    want = through_python(name, args)
    torch.cuda.synchronize()
    monkeypatch.delattr(package, "_fast", raising=False)
    monkeypatch.setitem(sys.modules, package.__name__ + "._fast", None)
    monkeypatch.setattr(ops, "_fast", None)
    monkeypatch.setattr(ops, "_bound", False)
    with pytest.warns(RuntimeWarning, match="_fast is not used"):
        call(name, args)
    call(name, args)
    assert ops._fast is None
    torch.cuda.synchronize()
    for g, w in zip(args[-n:], want):
        assert torch.equal(g, w)


@pytest.mark.parametrize("name", NAMES)
def test_an_earlier_error_of_another_call(name):
    """The runtime remembers that a device number did not exist; the launch after it is in order."""
    args = data()[name]
    n = OUTS[name]
    want = through_python(name, args)
    torch.cuda.synchronize()
    lib = L.load()
    ops._bind(lib)
    calls = []
    f = getattr(lib, ENTRIES[name])

    @ctypes.CFUNCTYPE(ctypes.c_int, *f.argtypes)
    def counted(*a):
        calls.append(f(*a))
        return calls[-1]

    try:
        ops._fast.bind(torch.cuda.current_device, ops._raw_stream,
                       *(ctypes.cast(counted if fn == ENTRIES[name] else getattr(lib, fn), ctypes.c_void_p).value
                         for fn in ENTRIES.values()))
        assert lib.hipSetDevice(4096) != 0
        call(name, args)
    finally:
        lib.hipGetLastError()
        ops._bind(lib)
    assert calls == [L.MOK_OK]
    torch.cuda.synchronize()
    for g, w in zip(args[-n:], want):
        assert torch.equal(g, w)
