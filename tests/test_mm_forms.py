"""What the 16-bit grouped product answers to which form a call takes and how its sums are split.  The
kernels that need an answer are compiled apart, so the answers may not depend on what a compiler makes of
the arithmetic.  mm_forms_check.cpp computes them on the host."""
import os
import re
import subprocess

import pytest

from mixture_experts_layer_mok_amd import _lib as L
from mixture_experts_layer_mok_amd import build
from tests.mm_forms import (FAR_OFFSETS, FAR_ROWS, HELD_FP16, KINDS, LEAST, MOST, answers, compiler, form_cases,
                            forms_of, program)


def test_answers_do_not_depend_on_contraction(tmp_path):
    """The estimates, bit for bit, whether or not the compiler may fuse a multiplication and an addition
    where no pragma forbids it (for device code hipcc may by itself)."""
    said = []
    for how in ("off", "fast-honor-pragmas"):
        exe = program(tmp_path / how, "-mfma", f"-ffp-contract={how}")
        said.append(subprocess.run([exe, "sweep"], check=True, capture_output=True, text=True).stdout.splitlines())
    assert len(said[0]) > 100000
    bad = [(a, b) for a, b in zip(*said) if a != b]
    assert not bad and len(said[0]) == len(said[1]), bad[:4]


def test_device_code_fuses_nothing(tmp_path):
    """The kernels of one product as hipcc makes them: estimates are all that they compute on single
    floats, and no instruction of theirs multiplies and adds at once."""
    listing = str(tmp_path / "rows.s")
    subprocess.run([build.hipcc(), *build.HIPCC_FLAGS, "--cuda-device-only", "-S",
                    os.path.join(build.CSRC, "grouped_mm_rows.hip"), "-o", listing], check=True, capture_output=True)
    text = open(listing).read()
    assert len(re.findall(r"v_mul_f32", text)) > 20
    assert not re.findall(r"\b[vs]_(?:pk_)?(?:fma|mad)\w*_f32", text)


@pytest.mark.parametrize("kind,counts,n,k,want", [
    # at most 11 m-tiles of 128 times 32: one round of small ones at most.  112 steps of 0.72 us and 4,
    # less than 20.8 times the weights' 11.3
    ("out", [64] * 8, 4096, 7168, "only_small small 1 128"),
    ("out", [8] * 8, 4096, 7168, "only_small few 1 128"),
    # 71 x 16 whole tiles at most; 64 x 16 of them are four full rounds, 68 x 16 those and 64, in four items each
    ("out", [2048] * 8, 4096, 7168, "only_whole whole 1 256"),
    ("out", [2053, 2030, 2048, 2061, 1999, 2001, 2077, 2040], 4096, 7168, "only_whole whole 4 64"),
    # 2 x 56 small tiles, 64 steps: four items, 512 being the most
    ("rows", [256], 4096, 7168, "only_small small 4 128"),
    # 64 tiles of 256 steps: 512 items leave 7 units, of 37 steps
    ("weights", [16384], 1024, 1024, "only_small small 7 128"),
    ("weights", [2048] * 8, 4096, 7168, "only_whole whole 1 128"),
])
def test_known_answers(kind, counts, n, k, want):
    assert forms_of([(kind, counts, sum(counts), n, k)]) == [want]


def test_malformed_calls_are_refused():
    exe = program(os.path.join(build.BUILD, "mm_forms_check"))
    for line in ("", "0 1", "3 8 8 8 1 0 8", "0 8 8 8 1 0"):
        assert subprocess.run([exe, "calls"], input=line + "\n", text=True, capture_output=True).returncode == 1
    assert subprocess.run([exe], capture_output=True).returncode == 2
    assert compiler()


def test_rows_of_any_offsets():
    """An expert's rows lie in the matrix, and their number in 32 bits, whatever the offsets are."""
    ends = [LEAST, LEAST + 1, -1, 0, 1, 7, 2**24, 2**24 + 1, MOST - 1, MOST]
    lines = [(top, a, b) for top in (0, 1, 7, 2**24) for a in ends for b in ends]
    for (top, a, b), got in zip(lines, answers("rows", lines)):
        lo, hi = map(int, got.split())
        assert 0 <= lo <= MOST and 0 <= hi <= top
        assert list(range(lo, min(hi, lo + 9))) == list(range(max(a, 0), min(b, top, max(a, 0) + 9))), (top, a, b)
        assert max(hi - lo, 0) == max(min(b, top) - max(a, 0), 0)


def test_calls_with_far_offsets_reach_every_form():
    """(Run on a GPU by test_gpu_grouped_mm_forms.py; five rows belong to nobody.)"""
    lines = [(KINDS[kind], max(o for o in off if o < MOST) + 5, n, k, 1, *off) for kind, off, n, k, _ in FAR_OFFSETS]
    assert answers("calls", lines) == [c[-1] for c in FAR_OFFSETS]


@pytest.mark.parametrize("which,n,k", [(0, 2048, 4096), (1, 4096, 2048)])
def test_workspace_of_many_experts(which, n, k):
    """Whole tiles are split with at most 64 experts: with more, a call that launches nothing else has no
    use for a workspace; where the small tiles may run they may be split."""
    kind = ("out", "rows")[which]
    for groups, rows, launch, ws in ((64, 256 * 128, "only_whole", True), (65, 256 * 128, "only_whole", False),
                                     (1024, 256 * 128, "only_whole", False), (65, 4096, "both", True),
                                     (65, 30, "only_small", False)):
        assert forms_of([(kind, [1] * groups, rows, n, k)])[0].split()[0] == launch, (groups, rows)
        assert L.mok_grouped_mm_workspace(which, rows, groups, n, k) == ws * L.MOK_MM_WORKSPACE_BYTES, (groups, rows)


def test_held_fp16_cases_reach_every_form():
    """(Run on a GPU by test_gpu_held_fp16.py.)"""
    assert forms_of([("held", [rows], rows, n, k) for rows, n, k, _ in HELD_FP16]) == [c[-1] for c in HELD_FP16]


def test_cases_take_the_forms_they_are_named_for():
    """(Run on a GPU by test_gpu_grouped_mm_forms.py, with five rows more than are routed.)"""
    cases = form_cases()
    got = forms_of([(kind, counts, sum(counts) + 5, n, k) for kind, counts, n, k, _ in cases])
    assert not [(c, g) for c, g in zip(cases, got) if c[-1] != g]
    assert len({(c[0], c[-1]) for c in cases}) >= 20
    assert forms_of([(kind, counts, sum(counts) + 5, n, k) for kind, counts, n, k, _ in FAR_ROWS]) == \
        [c[-1] for c in FAR_ROWS]
