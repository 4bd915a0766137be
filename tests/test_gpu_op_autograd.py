"""The row and MXFP4 functions beside autograd, on a GPU: they record nothing, and a backward pass
that saved a tensor which one of them has written to since raises."""
import pytest
import torch

from mixture_experts_layer_mok_amd import ops
from tests.test_gpu_op_calls import DEV, NAMES, OUTS, data

pytestmark = pytest.mark.gpu
VALUES = dict(permute=[0], permute_backward=[0], unpermute=[0, 2], unpermute_backward=[0, 1, 3],
              quantize_mx4=[0], dequantize_mx4=[], grouped_mx4=[])


def call(name, args, stream):
    if name in ("permute", "unpermute_backward", "quantize_mx4"):
        return getattr(ops, name)(*args, stream=stream)
    return getattr(ops, name)(*args[:-1], out=args[-1], stream=stream)


@pytest.fixture(params=[False, True], ids=["extension", "python"])
def stream(request):
    return torch.cuda.current_stream() if request.param else None


@pytest.mark.parametrize("name", NAMES)
def test_written_outputs_count_as_changed(name, stream):
    args = data()[name]
    outs = args[-OUTS[name]:]
    before = [t._version for t in outs]
    inputs = [t._version for t in args[:-len(outs)]]
    call(name, args, stream)
    assert [t._version for t in outs] == [v + 1 for v in before]
    assert [t._version for t in args[:-len(outs)]] == inputs


def test_a_graph_that_saved_an_output_raises(stream):
    args = data(dtype=torch.float32)["permute"]
    w = torch.ones_like(args[2], requires_grad=True)
    y = (w * args[2][:]).sum()  # saves a view of what is written next
    call("permute", args, stream)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


@pytest.mark.parametrize("name", NAMES)
def test_results_have_no_graph(name, stream):
    args = data(dtype=torch.float32)[name]
    for i in VALUES[name]:
        args[i].requires_grad_(True)
    got = call(name, args, stream)
    for t in got if isinstance(got, tuple) else [got]:
        assert not t.requires_grad and t.grad_fn is None


@pytest.mark.parametrize("name", NAMES)
def test_outputs_made_in_inference_mode(name, stream):
    """They have no version to count; inside the mode and outside."""
    args = data()[name]
    n = OUTS[name]
    call(name, args, stream)
    want = [t.clone() for t in args[-n:]]
    with torch.inference_mode():
        outs = [torch.zeros_like(t) for t in args[-n:]]
        call(name, args[:-n] + outs, stream)
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    call(name, args[:-n] + outs, stream)
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_outputs_made_by_the_call_have_no_graph(stream):
    x = torch.randn(4, 64, device=DEV, requires_grad=True)
    pos = torch.arange(4, dtype=torch.int32, device=DEV).view(4, 1)
    y = ops.permute_backward(x, pos, stream=stream)
    assert not y.requires_grad and torch.equal(y, x.detach())
    c, s = ops.quantize_mx4(x, stream=stream)
    assert not c.requires_grad and not s.requires_grad
