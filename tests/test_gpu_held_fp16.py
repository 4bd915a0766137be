"""The weights' gradient of fp16 rows from activations held in 8 bits, at the end of fp16's range, on a GPU.

Finite fp16 activations of 63,488 and more are held as 65,536 (code 256 at scale 2^8), which fp16 does not
have.  It enters the product as 65,504: off by 32, half of fp16's step there (eps / 2 of the value), and
nearer to the activation than 65,536 is.  Everything here is a whole number of 32s, and the sums are below
32 * 2^24, so that they are exact in fp32."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_mok_amd import ops
from oracle import operators as O
from tests.mm_forms import HELD_FP16

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


def entered(codes, scales):
    """The float64 values with which codes enter an fp16 product."""
    v = O.values_mx8(codes.cpu().numpy(), scales.cpu().numpy())
    with np.errstate(over="ignore"):
        half = v.astype(np.float16).astype(np.float64)
    return np.where(np.abs(v) == 65536, np.sign(v) * 65504, half)


@pytest.mark.parametrize("rows,n,k,form", HELD_FP16, ids=["small", "split", "whole"])
def test_the_largest_activations_stay_finite(rows, n, k, form):
    rng = np.random.default_rng(rows)
    some = np.array([0, 512, 40960, 57344, 63456, 63488, 64000, 65472, 65504])
    a = torch.from_numpy(rng.choice(np.concatenate([some, -some]), (rows, k))).to(FP)
    assert torch.isfinite(a).all()
    g = torch.from_numpy(rng.integers(-1, 2, (rows, n))).to(FP)
    off = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    codes, scales = ops.quantize_mx8(a.to(DEV))
    held = entered(codes, scales)
    assert (np.abs(held) == 65504).any() and np.isfinite(held).all()
    assert (np.abs(held - a.double().numpy()) <= np.abs(a.double().numpy()) * 2.0**-4).all()
    w = ops.grouped_mm_backward_weights(g.to(DEV), codes, off, a_scales=scales)
    assert np.array_equal(w[0].cpu().double().numpy(), g.double().numpy().T @ held)


def test_every_scale_and_code():
    """Row by row: 65,536 of any code and scale is 65,504, what is larger infinite, the rest as it was."""
    codes = torch.arange(256, device=DEV).to(torch.uint8)[None].repeat(256, 1)
    scales = torch.arange(256, device=DEV).to(torch.uint8)[:, None].repeat(1, 8)
    want = entered(codes, scales)
    g = torch.ones(256, 8, dtype=FP, device=DEV)
    for r in range(256):
        one = torch.tensor([r, r + 1], dtype=torch.int32, device=DEV)
        w = ops.grouped_mm_backward_weights(g, codes, one, a_scales=scales)[0].cpu().double().numpy()
        assert np.array_equal(w, np.broadcast_to(want[r], w.shape), equal_nan=True), r


def test_a_larger_value_is_infinite_alone():
    """An activation that fp16 does not have, among such that it has, in one block."""
    x = torch.full((1, 64), 65504.0)
    x[0, 5], x[0, 40] = 80000.0, -80000.0
    codes, scales = ops.quantize_mx8(x.to(DEV))
    off = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    w = ops.grouped_mm_backward_weights(torch.ones(1, 8, dtype=FP, device=DEV), codes, off, a_scales=scales)[0]
    want = torch.full((64,), 65504.0)
    want[5], want[40] = float("inf"), float("-inf")
    assert torch.equal(w.cpu(), want.expand(8, 64))
    # a product in bfloat16, whose range is float32's, has the held values themselves
    w = ops.grouped_mm_backward_weights(torch.ones(1, 8, dtype=BF, device=DEV), codes, off, a_scales=scales)[0]
    assert torch.equal(w.cpu().double(), torch.from_numpy(O.values_mx8(codes.cpu().numpy(), scales.cpu().numpy())).expand(8, 64))
