"""libtilepipe: software-pipelined global->LDS tile streaming for MI355X (gfx950).

The compute lives in hand-written HIP kernels inside ``libtilepipe.so`` behind a
C ABI (``include/tilepipe.h``). :mod:`software_pipelining_amd.tilepipe` is the
thin ctypes binding; it loads the library on first use and raises if it has not
been built; there is no CPU fallback. :mod:`software_pipelining_amd.linear8`
binds the 8-bit linear layer's operators; it needs torch and is imported when one
of its names is first used.
"""
from importlib.util import find_spec

from .tilepipe import (  # noqa: F401
    Align, TilepipeError, Path, Plan, Schedule, chunk_copy, device_check, lds_budget, library_path,
    map_2d, pipelined_map, plan_chunk_copy, plan_map, plan_map_2d, plan_row_shift,
    plan_workgroup_copy, row_shift, workgroup_copy, workgroup_copy_noalloc,
    workgroup_copy_workspace_bytes,
)

__all__ = [
    "Align", "BlockQuantized", "RmsNorm", "TilepipeError", "Path", "Plan", "Schedule",
    "block_matmul", "block_quantize", "chunk_copy", "device_check", "lds_budget",
    "library_path", "map_2d", "pipelined_map", "plan_chunk_copy", "plan_map", "plan_map_2d",
    "plan_row_shift", "plan_workgroup_copy", "rms_norm", "rms_norm_backward", "row_shift", "workgroup_copy",
    "workgroup_copy_noalloc", "workgroup_copy_workspace_bytes",
]

_LINEAR8 = ("BlockQuantized", "RmsNorm", "block_matmul", "block_quantize", "rms_norm", "rms_norm_backward")

if find_spec("torch") is None:      # a star import leaves out what cannot be had
    __all__ = [n for n in __all__ if n not in _LINEAR8]


def __getattr__(name):
    if name in _LINEAR8:
        from . import linear8
        globals().update({n: getattr(linear8, n) for n in _LINEAR8})
        return globals()[name]
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
