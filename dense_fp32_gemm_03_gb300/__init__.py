"""GB300-native FP32 GEMM (C = A * B, row-major, FFMA arithmetic) for sm_103a.

The product is the C-ABI library ``libsgemm.so`` (``include/sgemm.h``); this
package builds it (``_build``), binds it (``binding``) and provides the seeded
synthetic workloads (``workloads``).  The library's microscaled 4-bit
operators (``include/fp4.h``) are bound by ``fp4`` and its 8-bit integer operators
(``include/int8.h``) by ``int8``, which need torch to be imported; they are
loaded with the first of their names, so that the package itself needs none
(``sgemm_raw`` takes addresses).
"""
from .binding import (AUTO, GUARDED, SMALL, SPECIALIZED, STAGED, STREAMK, STREAMK_SMALL, TILED, TILED_SMALL, VARIANTS,
                      SgemmError, debug_expire_wait, debug_owner_publishes, load, query_device_status,
                      release_workspaces, select_variant, sgemm, sgemm_ex, sgemm_ex2, sgemm_host, sgemm_raw, sgemm_tf32, status_string,
                      ROW_MAJOR, COL_MAJOR, OP_N, OP_T,
                      variant_name, workspace_size)

_FP4 = ("Fp4Matrix", "Fp4Experts", "fp4_quantize", "fp4_matrix", "fp4_dequantize", "fp4_gemm", "fp4_linear",
        "fp4_experts", "fp4_moe")
_INT8 = ("Int8Matrix", "Int8Checkpoint", "int8_quantize", "int8_matrix", "int8_dequantize", "int8_gemm", "int8_linear",
         "int8_checkpoint", "int8_restore", "int8_weight_grad", "int8_swiglu", "int8_swiglu_backward")

__all__ = ["sgemm", "sgemm_ex", "sgemm_ex2", "sgemm_host", "ROW_MAJOR", "COL_MAJOR", "OP_N", "OP_T", "sgemm_tf32", "sgemm_raw", "select_variant", "workspace_size", "query_device_status",
           "debug_expire_wait", "debug_owner_publishes", "release_workspaces", "status_string", "variant_name", "load",
           "SgemmError", "VARIANTS", "AUTO", "GUARDED", "TILED", "STREAMK", "TILED_SMALL",
           "STREAMK_SMALL", "STAGED", "SPECIALIZED", "SMALL", *_FP4, *_INT8]


def __getattr__(name):
    if name in _FP4:
        from . import fp4 as module
        names = _FP4
    elif name in _INT8:
        from . import int8 as module
        names = _INT8
    else:
        raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
    globals().update({n: getattr(module, n) for n in names})
    return globals()[name]


def __dir__():
    return sorted({*globals(), *_FP4, *_INT8})
