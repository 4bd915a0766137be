"""CPU checks of the exact-sum test of the grouped product: its conditions hold for its operands, and
it rejects sums in fewer bits, a dropped product and a dropped block."""
import numpy as np
import pytest
import torch

from oracle import operators as O
from tests import mx4_exact as X


def test_unit():
    v = np.array([[1.0, 0.0, 6.0], [0.375, 8.0, 2.0], [-2.0**-130, 1.0, 0.0]])
    assert X.unit(v).tolist() == [1.0, 0.125, 2.0**-130]
    assert X.unit(np.zeros((1, 4)))[0] == np.inf


def _accumulate(a, b, dtype, step):
    acc = torch.zeros(a.shape[0], b.shape[0], dtype=dtype)
    for k in range(0, a.shape[1], step):
        acc = (acc.double() + torch.from_numpy(a[:, k:k + step] @ b[:, k:k + step].T)).to(dtype)
    return acc.double().numpy()


@pytest.mark.parametrize("sign", [False, True])
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("K", [32, 96, 2080, 7168, 8448])
def test_every_result_is_exact_in_float32(K, fmt, sign):
    rng = np.random.default_rng(K)
    a, b = X.operand(rng, 40, K, fmt, sign)[2], X.operand(rng, 48, K, "e2m1", sign)[2]
    want, ok = X.exact(a, b, fmt)
    assert ok.all()
    at, bt = torch.from_numpy(a).float(), torch.from_numpy(b).float()
    assert X.off((at @ bt.T).double().numpy(), want, ok, torch.float32) == 0
    order = rng.permutation(K)
    assert X.off(_accumulate(a[:, order], b[:, order], torch.float32, 1 if K < 100 else 16), want, ok, torch.float32) == 0


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("K", [2080, 7168])
def test_what_is_rejected(K, fmt, out):
    rng = np.random.default_rng(K + 1)
    a, b = X.operand(rng, 40, K, fmt)[2], X.operand(rng, 48, K, "e2m1")[2]
    want, ok = X.exact(a, b, fmt)
    n = want.size

    def rejected(got):
        return X.off(X.nearest(got, out), want, ok, out)

    assert rejected(want) == 0
    for dtype in (torch.float16, torch.bfloat16):  # a rounded accumulator, every 64 elements
        assert rejected(np.nan_to_num(_accumulate(a, b, dtype, 64), posinf=0.0)) > n // 20
    dropped = a.copy()
    dropped[:, K - 32:] = 0
    assert rejected(dropped @ b.T) > n // 4
    if out is torch.float32:
        one = a.copy()
        one[:, 777] = 0
        assert rejected(one @ b.T) > n // 2


def test_the_quantised_normals_of_the_other_tests_are_exact_too():
    rng = np.random.default_rng(5)
    a = O.values_mx4(*_mx4(rng.standard_normal((6, 2080))))
    b = O.values_mx4(*_mx4(rng.standard_normal((5, 2080)) * 0.1))
    assert X.exact(a, b, "e2m1")[1].all()


def _mx4(x):
    c, s = O.quantize_mx4(x)
    return O.pack4(c), s
