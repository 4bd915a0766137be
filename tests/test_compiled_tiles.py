"""The compiled loops of the 16-bit product's tiles.  Their MFMAs are inline assembly, so the compiler
places no wait states around them; the loops are right because between them nothing else touches the
sums.  Here the device code is compiled to assembly (no GPU needed) and every block that holds such a
loop, the ones with direct-to-LDS loads among MFMAs, is looked at."""
import os
import re
import subprocess

import pytest

from mixture_experts_layer_mok_amd import build

FILES = ["grouped_mm_out", "grouped_mm_rows", "grouped_mm_weights", "grouped_mm_held"]


def blocks(text):
    """(instructions, basic block by basic block) of an assembly listing."""
    cur = []
    for line in text.splitlines():
        if re.match(r"[A-Za-z_.][^\s]*:", line):
            yield cur
            cur = []
        elif line.startswith("\t") and not re.match(r"\t[.;]", line):
            cur.append(line.strip())
    yield cur


def is_loop(ops):
    return sum("v_mfma" in o for o in ops) >= 8 and any(o.startswith("buffer_load") and "lds" in o for o in ops)


def other_uses(ops):
    """Instructions of a block that touch accumulation registers and are no MFMA, or spill."""
    return [o for o in ops if ("v_mfma" not in o and re.search(r"\ba(\d+\b|\[\d+:\d+\])", o)) or
            o.startswith(("scratch_", "v_accvgpr"))]


@pytest.fixture(scope="module")
def listings(tmp_path_factory):
    out = tmp_path_factory.mktemp("asm")
    runs = {}
    for n in FILES:
        cmd = [build.hipcc(), *build.HIPCC_FLAGS, "--cuda-device-only", "-S",
               os.path.join(build.CSRC, n + ".hip"), "-o", str(out / (n + ".s"))]
        runs[n] = subprocess.Popen(cmd, stdout=subprocess.DEVNULL, stderr=subprocess.PIPE)
    for n, r in runs.items():
        err = r.communicate()[1]
        assert r.returncode == 0, err.decode()[-2000:]
    return {n: (out / (n + ".s")).read_text() for n in FILES}


@pytest.mark.parametrize("name", FILES)
def test_sums_are_touched_by_mfmas_alone(listings, name):
    loops = [b for b in blocks(listings[name]) if is_loop(b)]
    assert len(loops) >= (4 if "weights" in name or "held" in name else 8)  # two types of each tile
    for b in loops:
        assert not other_uses(b), other_uses(b)[:4]


@pytest.mark.parametrize("name", [f for f in FILES if f != "grouped_mm_out"])
def test_no_block_of_mfmas_touches_the_sums_otherwise(listings, name):
    """Also the blocks that a branch cuts a loop into, of which only one has loads to LDS.  (The forward's
    form of few rows has MFMAs that the compiler knows and sees to itself.)"""
    many = [b for b in blocks(listings[name]) if sum(bool(re.match(r"v_mfma\S+ a\[", o)) for o in b) >= 8]
    assert len(many) >= (8 if "rows" in name else 4)
    for b in many:
        assert not other_uses(b), other_uses(b)[:4]


@pytest.mark.parametrize("name", FILES)
def test_nothing_spills_to_memory(listings, name):
    assert set(re.findall(r"\.vgpr_spill_count:\s+(\d+)", listings[name])) == {"0"}
    assert set(re.findall(r"\.private_segment_fixed_size:\s+(\d+)", listings[name])) == {"0"}


def test_the_check_itself():
    good = ["v_mfma_f32_16x16x32_bf16 a[0:3], v[2:5], v[6:9], a[0:3]"] * 8 + ["buffer_load_dwordx4 v1, s[0:3], 0 offen lds"]
    assert is_loop(good) and not other_uses(good)
    for bad in ("v_accvgpr_read_b32 v1, a3", "v_mov_b32_e32 v1, a3", "scratch_load_dword v1, off, off", "ds_read_b128 a[4:7], v1"):
        assert other_uses(good + [bad]) == [bad]
    assert not is_loop(good[:8]) and not is_loop(good[-1:])
