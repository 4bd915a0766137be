"""Build the layer library (libmok.so) in-tree with hipcc for gfx950.

    python -m mixture_experts_layer_mok_amd.build [--jobs N]

Every .hip file under csrc/ is compiled to an object (in parallel), then linked into
mixture_experts_layer_mok_amd/libmok.so; csrc/fast_calls.cpp is compiled by the host
compiler to the extension module _fast.so, which the package also works without (where the
host compiler, Python's headers or torch are missing).  All device code is built with packed-FP32
instructions disabled (the compiler would otherwise form v_pk_* fp32 ops on its own).
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
OUT = os.path.join(HERE, "libmok.so")
FAST = os.path.join(HERE, "_fast.so")
BUILD = os.path.join(ROOT, "_build")

ARCH = "gfx950"
HIPCC_FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall", "-Wno-unused-result",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-Wno-inline-asm",
    "-I", os.path.join(ROOT, "include"),
]


def hipcc() -> str:
    for cand in (shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found; the layer library needs ROCm's hipcc")


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".hip"))


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-4] + ".o")
    cmd = [hipcc(), *HIPCC_FLAGS, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    noise = [ln for ln in r.stderr.splitlines() if "packed-fp32-ops" not in ln and ln.strip()]
    if noise:
        sys.stderr.write("\n".join(noise) + "\n")
    return obj


def _build_fast() -> None:
    """The extension module of ops.py's ordinary calls, against torch's headers and libraries
    (found at run time as the ones the importing process has loaded)."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    include = [d for p in [*cpp_extension.include_paths(), sysconfig.get_paths()["include"]]
               for d in ("-I", p)]
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DMOK_TORCH_VERSION="{torch.__version__}"', *include,
           os.path.join(CSRC, "fast_calls.cpp"), "-o", FAST + ".tmp", "-L", libs, "-ltorch_python",
           "-ltorch", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on fast_calls.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(FAST + ".tmp", FAST)


def _try_fast() -> bool:
    """_build_fast; where it fails, the reason on stderr and no module of an earlier build left."""
    try:
        _build_fast()
        return True
    except (ImportError, OSError, RuntimeError) as e:
        sys.stderr.write(f"_fast.so is not built (the operators' calls run without it): {e}\n")
        if os.path.exists(FAST):
            os.remove(FAST)
        return False


def build(jobs: int | None = None, verbose: bool = True) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    jobs = jobs or min(len(srcs) + 1, os.cpu_count() or 4, 8)
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        fast = ex.submit(_try_fast)
        objs = list(ex.map(_compile, srcs))
        with_fast = fast.result()
    tmp = OUT + ".tmp"
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, OUT)
    if verbose:
        print(f"built {OUT} from {len(srcs)} sources" + (f", and {FAST}" if with_fast else ""))
    return OUT


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--jobs", type=int, default=None)
    build(ap.parse_args().jobs)
