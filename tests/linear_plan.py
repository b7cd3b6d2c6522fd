"""What the library chooses to run for a product with FP4 weights, asked from
the probe library (host code, no GPU): for the tests that count which kernels
the cases of the GPU tests reach."""
import ctypes
import os
from collections import namedtuple

from microscaling_fp4_block_fp4q_amd import fp4q as F

PROBE_LIB = os.path.join(os.path.dirname(F.LIB_PATH), "libfp4q_probe.so")

KINDS = ("few", "tile32", "tile64", "tile128", "tile256")
FORMATS = {"mxfp4": F.E8M0, "nvfp4": F.E4M3}
DTYPES = {"f32": F.F32, "bf16": F.BF16, "f16": F.F16}
# the kernel's instantiation: kind, weight format and planes; few rows: weight-row tiles and whether per expert;
# tiles: gradient, 64-bit gather
Kernel = namedtuple("Kernel", "kind weights planes tiles grouped grad far")
Plan = namedtuple("Plan", "kernel copy gathered splits")

_lib = None


def plan(fmt, dt, grad, R, N, K, E=0, T=0, ld=0):
    """E: experts (0: dense); T, ld: x [T, ld] is gathered by rows (0: it is not)."""
    global _lib
    if _lib is None:
        _lib = ctypes.CDLL(PROBE_LIB)
        i, l = ctypes.c_int, ctypes.c_int64
        _lib.fp4q_probe_linear_plan.restype = None
        _lib.fp4q_probe_linear_plan.argtypes = [i, i, i, i, i, l, l, l, l, l, i, ctypes.POINTER(ctypes.c_int32)]
    out = (ctypes.c_int32 * 8)()
    _lib.fp4q_probe_linear_plan(grad, FORMATS[fmt], DTYPES[dt], E > 0, T > 0, T, ld, R, N, K, max(E, 1), out)
    kind, weights, planes, tiles, far, copy, gathered, splits = out
    few = kind == 0
    k = Kernel(KINDS[kind], weights, planes, tiles, E > 0 if few else None, None if few else bool(grad),
               None if few or grad or planes > 1 else bool(far))
    return Plan(k, bool(copy), bool(gathered), splits)


def every_kernel():
    """All instantiations that the library launches."""
    out = set()
    # weight format and planes: E8M0 with bf16, fp16, fp32; E4M3 with bf16, fp32; E4M3 as fp16 operands
    for weights, planes in ((0, 1), (0, 2), (0, 3), (1, 1), (1, 3), (2, 1)):
        out |= {Kernel("few", weights, planes, n, g, None, None) for n in (1, 2, 4) for g in (False, True)}
        out |= {Kernel(k, weights, planes, 0, None, True, None) for k in ("tile64", "tile128", "tile256")}
        out |= {Kernel(k, weights, planes, 0, None, False, far) for k in KINDS[1:]
                for far in ((False, True) if planes == 1 else (None,))}
    return out
