"""Wait states of the loads written as inline assembly.  The compiler places none around or inside
it, so each such string has the ones gfx950 asks for:

- five between a vector instruction that writes a scalar register (v_readlane reloads a spilled
  one, and may stand right before the string) and a vector memory operation that reads it;
- one between a write of M0 and the direct-to-LDS load that reads M0.

An instruction is one state, s_nop n is n + 1."""
import os
import re

import pytest

from mixture_experts_layer_mok_amd import build

FILES = sorted(f for f in os.listdir(build.CSRC) if f.endswith((".h", ".hip")))
WITH_LOADS = {"gemm_bf16.h", "gemm_mx.h", "gemm_mx4.h"}


def strings(text):
    """The instruction lists of the asm statements of a source."""
    for m in re.finditer(r'\basm\s+volatile\s*\(\s*((?:"(?:[^"\\]|\\.)*"\s*)+)', text):
        code = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', m.group(1)))
        ops = [o.strip() for o in re.split(r"\\n(?:\\t)?|;", code) if o.strip()]
        if ops:
            yield ops


def states(ops):
    return sum(int(o.split()[1], 0) + 1 if o.split()[0] == "s_nop" else 1 for o in ops)


def missing(ops):
    """What a list of instructions leaves out; empty where nothing is."""
    found = []
    for i, op in enumerate(ops):
        if not re.match(r"(buffer|global|flat|scratch)_", op):
            continue
        if re.match(r"buffer_", op) and states(ops[:i]) < 5:
            found.append(f"{states(ops[:i])} of 5 states before {op}")
        if re.search(r"\blds\b|_lds_", op):
            at = [j for j in range(i) if re.match(r"s_mov_b32 m0\b", ops[j])]
            if not at or states(ops[at[-1] + 1:i]) < 1:
                found.append(f"no state between M0's write and {op}")
    return found


@pytest.mark.parametrize("name", FILES)
def test_loads_have_their_wait_states(name):
    with open(os.path.join(build.CSRC, name)) as f:
        loads = [ops for ops in strings(f.read()) if any(re.match(r"(buffer|global)_", o) for o in ops)]
    assert bool(loads) == (name in WITH_LOADS)
    assert [m for ops in loads for m in missing(ops)] == []


def test_the_check_itself():
    assert missing(["s_mov_b32 m0, %3", "s_nop 3", "buffer_load_dwordx4 %0, %1, %2 offen lds"]) == []
    assert len(missing(["s_mov_b32 m0, %3", "buffer_load_dwordx4 %0, %1, %2 offen lds"])) == 2
    assert len(missing(["s_mov_b32 m0, %3", "s_nop 2", "buffer_load_dwordx4 %0, %1, %2 offen lds"])) == 1
    assert len(missing(["s_nop 3", "s_mov_b32 m0, %1", "global_load_lds_dword %0, off"])) == 1
    assert missing(["s_mov_b32 m0, %1", "s_nop 0", "global_load_lds_dword %0, off"]) == []
    assert list(strings('asm volatile("s_nop 0\\n\\tv_mov_b32 %0, %1" "\\n\\ts_nop 4" : "=v"(x));')) == [
        ["s_nop 0", "v_mov_b32 %0, %1", "s_nop 4"]]
