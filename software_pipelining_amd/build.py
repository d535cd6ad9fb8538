"""Build libtilepipe.so for gfx950 (hipcc) in-tree.

    python -m software_pipelining_amd.build [--jobs N]

Translation units compile in parallel into ``_build/`` at the repository root;
the shared library is written next to this file. The planners (tp_*plan.cpp) are
plain C++ and are compiled by g++ to keep them free of HIP. The direct binding of
the 8-bit layer's operators (tp_torch.cpp, against torch's own headers) becomes
_linear8.so beside the library; where it cannot be built, the operators are
called through ctypes.
"""
from __future__ import annotations

import argparse
import os
import subprocess
import sys
import time
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libtilepipe.so")
BINDING = os.path.join(PKG, "_linear8.so")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

# -packed-fp32-ops: no v_pk_{add,mul,fma}_f32 (results must stay bit-exact and
# some packed forms are not trusted); IEEE denormals; no FP contraction beyond
# the explicit fmaf calls.
HIP_FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-fvisibility=hidden",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-fno-gpu-flush-denormals-to-zero", "-ffp-contract=off",
    "-Wall", "-Wno-unused-command-line-argument",
]
CXX_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wall", "-Wextra", "-Werror"]

# The kernel families are instantiated per op and per half of the stage range
# (one compilation of tp_<family>_inst.hip each), heaviest first, so the
# pieces spread evenly over the compile jobs.
_OPS = (("scale2", "TP_OP_SCALE2"), ("horner32", "TP_OP_HORNER32"), ("copy", "TP_OP_COPY"))
_HALVES = ((1, 4), (5, 8))
INSTANCES = [
    (f"tp_{fam}_inst.hip", f"tp_{fam}_{op}_s{lo}_{hi}",
     [f"-DTP_INST_OP={macro}", f"-DTP_INST_SLO={lo}", f"-DTP_INST_SHI={hi}",
      f"-DTP_INST_FN=launch_{fam}_{op}_s{lo}_{hi}"])
    for fam in ("map2d", "map_split", "map") for lo, hi in reversed(_HALVES) for op, macro in _OPS
]
# The product's kernels, once per pair of 8-bit types (0: e4m3, 1: e5m2).
_EIGHT = ("e4m3", "e5m2")
INSTANCES = [
    ("tp_block_matmul_inst.hip", f"tp_block_matmul_{a}_{b}",
     [f"-DTP_INST_FA={i}", f"-DTP_INST_FB={j}", f"-DTP_INST_FN=launch_matmul_{a}_{b}"])
    for i, a in enumerate(_EIGHT) for j, b in enumerate(_EIGHT)
] + INSTANCES
HIP_SOURCES = ["tp_rms_norm.hip", "tp_rms_norm_grad.hip", "tp_block_quantize.hip", "tp_block_matmul.hip",
               "tp_chunk_copy.hip", "tp_row_shift.hip", "tp_wg_copy.hip", "tp_api.cpp"]
CXX_SOURCES = ["tp_plan.cpp", "tp_ops_plan.cpp"]


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    out = (r.stdout + r.stderr).strip()
    # hipcc's host pass does not know the packed-fp32 target feature: harmless
    lines = [ln for ln in out.splitlines() if "packed-fp32-ops" not in ln]
    if r.returncode != 0:
        raise RuntimeError("build failed: " + " ".join(cmd) + "\n" + "\n".join(lines))
    return "\n".join(lines)


def _compile(unit, save_temps: bool = False) -> str:
    """unit: a source file name, or (source, object stem, extra flags)."""
    src, stem, defs = (unit, os.path.splitext(unit)[0], []) if isinstance(unit, str) else unit
    obj = os.path.join(BUILD, stem + ".o")
    path = os.path.join(CSRC, src)
    if src in CXX_SOURCES:
        cmd = ["g++", *CXX_FLAGS, f"-I{INCLUDE}", f"-I{CSRC}", "-c", path, "-o", obj]
    else:
        cmd = [HIPCC, *HIP_FLAGS, *defs, "-x", "hip", f"-I{INCLUDE}", f"-I{CSRC}", "-c", path,
               "-o", obj]
        if save_temps:
            cmd += ["-save-temps=obj"]
    _run(cmd)
    return obj


def _compile_binding() -> str:
    """tp_torch.cpp to an object, against torch's headers."""
    import sysconfig

    from torch.utils import cpp_extension
    obj = os.path.join(BUILD, "tp_torch.o")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-D__HIP_PLATFORM_AMD__",
          f"-I{INCLUDE}", *("-isystem" + p for p in cpp_extension.include_paths()),
          f"-isystem{os.path.dirname(os.path.dirname(HIPCC))}/include",
          f"-isystem{sysconfig.get_paths()['include']}",
          "-c", os.path.join(CSRC, "tp_torch.cpp"), "-o", obj])
    return obj


def _link_binding(obj: str) -> None:
    """Linked after the library, which it finds beside itself."""
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + ".tmp%d" % os.getpid()
    _run(["g++", "-shared", "-o", tmp, obj, f"-L{PKG}", "-l:libtilepipe.so", f"-L{libs}", "-lc10",
          "-lc10_hip", "-ltorch_cpu", "-ltorch_hip", "-ltorch_python", "-Wl,-rpath,$ORIGIN"])
    os.replace(tmp, BINDING)


def _bind(compiled) -> bool:
    """Links the binding from its compilation's future. The library needs no torch
    and linear8.py no binding, so a failure is reported and does not end the
    build; a binding of an older build goes, since it may not fit the library."""
    try:
        _link_binding(compiled.result())
        return True
    except Exception as e:  # noqa: BLE001
        print(f"[build] without the direct binding ({os.path.basename(BINDING)}): {e}", file=sys.stderr)
        if os.path.exists(BINDING):
            os.remove(BINDING)
        return False


def build(jobs: int | None = None, verbose: bool = True, save_temps: bool = False) -> str:
    """Compile every translation unit, link libtilepipe.so and the direct binding;
    return the library's path."""
    os.makedirs(BUILD, exist_ok=True)
    t0 = time.time()
    units = HIP_SOURCES + INSTANCES + CXX_SOURCES
    jobs = jobs or min(len(units), max(1, os.cpu_count() or 1))
    with ThreadPoolExecutor(max_workers=jobs) as ex:
        binding = ex.submit(_compile_binding)
        objs = list(ex.map(lambda u: _compile(u, save_temps), units))
    tmp = LIB + ".tmp%d" % os.getpid()
    _run([HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs])
    os.replace(tmp, LIB)
    _bind(binding)
    if verbose:
        print(f"[build] {LIB} ({time.time() - t0:.1f}s)", file=sys.stderr)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--jobs", type=int, default=None)
    ap.add_argument("--save-temps", action="store_true",
                    help="keep the gfx950 assembly in _build/ for inspection")
    a = ap.parse_args()
    build(a.jobs, save_temps=a.save_temps)
