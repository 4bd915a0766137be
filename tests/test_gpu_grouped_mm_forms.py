"""The grouped product of 16-bit rows in each of its forms, on a GPU, against float64.  The cases lie in
mm_forms.py with the form that each takes, which test_mm_forms.py holds against the code that chooses.
Whole numbers, so that the exact result is wanted (tolerances of the others: test_gpu_grouped_mm.py)."""
import pytest
import torch

from tests.mm_forms import FAR_OFFSETS, LEAST, MOST
from tests.test_gpu_grouped_mm import BF, DEV, F32, Case, check, say

pytestmark = pytest.mark.gpu


def short(v):
    return str(v)[:40].replace(" ", "").replace(str(MOST), "most").replace(str(LEAST), "least")


@pytest.mark.parametrize("kind,offsets,n,k,form", FAR_OFFSETS, ids=short)
def test_offsets_far_apart(kind, offsets, n, k, form):
    say("[mm] far offsets", kind, offsets, n, k, form)
    top = max(o for o in offsets if o < MOST)
    c = Case([top] + [0] * (len(offsets) - 2), n, k, BF, seed=41, whole=True, held=kind == "held")
    c.offsets = offsets
    c.off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    check(c, "weights" if kind == "held" else kind, F32, True)
