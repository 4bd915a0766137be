"""Runs csrc/mm_forms_check.cpp: which form a call of the 16-bit grouped product takes (host only)."""
import os
import shutil
import subprocess

from mixture_experts_layer_mok_amd import build

KINDS = {"out": 0, "rows": 1, "weights": 2, "weights+": 2, "held": 2}


def compiler():
    """The compiler that hipcc drives."""
    return shutil.which("amdclang++") or "/opt/rocm/bin/amdclang++"


def program(exe, *flags):
    exe = str(exe)
    os.makedirs(os.path.dirname(exe), exist_ok=True)
    subprocess.run([compiler(), "-O2", "-std=c++17", "-Wall", "-Werror", *flags, "-o", exe,
                    os.path.join(build.CSRC, "mm_forms_check.cpp")], check=True)
    return exe


def forms_of(calls, ws=True):
    """calls: (kind, rows an expert, max_rows, n, k) each; "launched form parts tall" each."""
    lines = []
    for kind, counts, max_rows, n, k in calls:
        off = [0]
        for c in counts:
            off.append(off[-1] + c)
        lines.append(" ".join(map(str, [KINDS[kind], max_rows, n, k, int(ws), *off])))
    exe = program(os.path.join(build.BUILD, "mm_forms_check"))
    return subprocess.run([exe, "calls"], input="\n".join(lines) + "\n", check=True, capture_output=True,
                          text=True).stdout.splitlines()
