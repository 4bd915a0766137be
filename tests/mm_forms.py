"""Runs csrc/mm_forms_check.cpp: which form a call of the 16-bit grouped product takes (host only)."""
import functools
import os
import shutil
import subprocess

from mixture_experts_layer_mok_amd import build

KINDS = {"out": 0, "rows": 1, "weights": 2, "weights+": 2, "held": 2, "held+": 2}


def compiler():
    """The compiler that hipcc drives."""
    return shutil.which("amdclang++") or "/opt/rocm/bin/amdclang++"


@functools.lru_cache(None)
def program(exe, *flags):
    exe = str(exe)
    os.makedirs(os.path.dirname(exe), exist_ok=True)
    mine = f"{exe}.{os.getpid()}"  # (another process may be running, or making, the same)
    subprocess.run([compiler(), "-O2", "-std=c++17", "-Wall", "-Werror", *flags, "-o", mine,
                    os.path.join(build.CSRC, "mm_forms_check.cpp")], check=True)
    os.replace(mine, exe)
    return exe


def answers(what, lines):
    exe = program(os.path.join(build.BUILD, "mm_forms_check"))
    return subprocess.run([exe, what], input="\n".join(" ".join(map(str, v)) for v in lines) + "\n", check=True,
                          capture_output=True, text=True).stdout.splitlines()


def offsets_of(counts):
    off = [0]
    for c in counts:
        off.append(off[-1] + c)
    return off


def forms_of(calls, ws=True):
    """calls: (kind, rows an expert, max_rows, n, k) each; "launched form parts tall" each."""
    return answers("calls", [[KINDS[kind], max_rows, n, k, int(ws), *offsets_of(counts)]
                             for kind, counts, max_rows, n, k in calls])


# Offsets whose ranges end before they begin, as far apart as 32 bits allow: what the call has, the offsets
# in the place of its own, n, k, and what computes it.
LEAST, MOST = -2**31, 2**31 - 1
FAR_OFFSETS = [
    ("out", [MOST, LEAST, 0, 40, 60], 72, 136, "only_small few 1 128"),
    ("out", [0, 2000, LEAST], 1032, 520, "only_small small 1 128"),
    ("out", [0, 8400, LEAST], 2048, 4160, "both whole 8 256"),
    ("rows", [MOST, LEAST, 0, 40, 60], 72, 136, "only_small small 1 128"),
    ("rows", [0, 8400, LEAST], 4160, 2048, "both whole 8 256"),
    ("weights", [MOST, LEAST, 0, 40, 60], 72, 136, "only_small small 1 128"),
    ("weights", [0, 5000, LEAST], 136, 264, "only_small small 8 128"),
    ("weights", [0, 400, LEAST], 4104, 4064, "only_whole whole 1 128"),
    ("held", [MOST, LEAST, 0, 40, 60], 72, 160, "only_small small 1 128"),
    ("held", [0, 400, LEAST], 4104, 4064, "only_whole whole 1 128"),
]

# Rows of one expert, held in 8 bits, n, k, and what computes their weights' gradient.
HELD_FP16 = [
    (37, 72, 96, "only_small small 1 128"),
    (2500, 72, 64, "only_small small 5 128"),
    (300, 4104, 4064, "only_whole whole 1 128"),
]

# Cases of the three products by the form that computes them: kind, rows an expert, n, k, form.  An expert
# of many rows decides the form, the other has the count or the depth that is looked at.
ROWS = [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 192, 193, 255, 256, 257, 511, 513]
DEPTHS = [8, 16, 24, 56, 64, 72, 120, 128, 136, 184, 192, 200, 256, 264, 504, 520, 1032, 4104]
SHORT = [8, 56, 64, 72, 128, 136, 192, 200, 520]
SIXTY = [257 + i * 37 % 200 - 100 * (i % 5 == 0) for i in range(60)]
EIGHTY = [257 + i * 53 % 90 for i in range(78)] + [0, 3]


def form_cases():
    small, whole = "only_small small 1 128", "both whole 1 256"
    alone = "only_whole whole 1 256"
    c = []
    for r in ROWS:
        c.append(("out", [r, 2000], 1032, 520, small))
        c.append(("out", [r, 4200], 2040, 1032, whole))
        c.append(("rows", [4200, r], 1032, 2040, whole))
    for d in DEPTHS:
        c.append(("out", [90, 3000], 1032, d, small))
    for d in SHORT:
        c.append(("out", SIXTY, 2064, d, alone))
        c.append(("rows", SIXTY, d, 2064, alone))
        c.append(("out", EIGHTY, 2056, d, alone))
        c.append(("rows", EIGHTY, d, 2056, alone))
    # ends of the columns
    for cols in (2056, 2112, 2176, 2240, 2296):
        c.append(("out", SIXTY, cols, 72, alone))
        c.append(("rows", SIXTY, 72, cols, alone))
        c.append(("out", [100, 2900], cols // 2 - cols // 2 % 8, 200, small))
    # sums that are split, with more than 64 experts and with fewer; parts of 64, 128 and 256 rows
    c += [
        ("out", [100 + i % 9 for i in range(70)], 128, 4104, "only_small small 4 128"),
        ("rows", [100 + i % 9 for i in range(70)], 4104, 128, "only_small small 4 128"),
        ("rows", [3 * (i % 7) for i in range(70)], 8200, 136, "only_small small 4 128"),
        ("out", [600, 700], 264, 4104, "only_small small 4 128"),
        ("rows", [1, 200, 0, 77], 8200, 72, "only_small small 15 128"),
        ("out", [2053, 2030, 2048, 2061, 1999, 2001, 2077, 2040], 1024, 4104, "both whole 8 64"),
        ("rows", [2053, 2030, 2048, 2061, 1999, 2001, 2077, 2040], 4104, 1024, "both whole 8 64"),
        ("out", [8300], 2040, 4096, "both whole 8 128"),
        ("rows", [8300], 4096, 2040, "both whole 8 128"),
        ("out", [8400], 2048, 4160, "both whole 8 256"),
        ("rows", [0, 8400], 4160, 2048, "both whole 8 256"),
    ]
    # gradients of the weights, added to what is there, from 16 and from 8 bits
    for kind in ("weights+", "held+"):
        c += [
            (kind, [40, 0, 300], 136, 96, small),
            (kind, [5000, 1, 70], 136, 160, "only_small small 10 128"),
            (kind, [300, 1, 0], 2312, 2336, "only_small small 1 128"),
            (kind, [129, 0, 700], 2312, 2336, "only_whole whole 1 128"),
            (kind, [600, 20], 4104, 2080, "only_whole whole 1 128"),
            (kind, [130 + i % 3 for i in range(70)], 520, 544, "only_whole whole 1 128"),
        ]
    return c

# The same with rows 2^21 elements apart.
FAR_ROWS = [
    ("out", [300], 131080, 72, "only_whole whole 1 256"),
    ("rows", [300, 500], 72, 65536, "only_whole whole 1 256"),
    ("weights", [300], 4104, 4064, "only_whole whole 1 128"),
]


def short(v):
    return str(v)[:32].replace(" ", "").replace(str(MOST), "most").replace(str(LEAST), "least")
