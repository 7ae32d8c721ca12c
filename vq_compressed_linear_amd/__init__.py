"""MI355X-native HelixLinear (HXQ) forward pass.

The compute lives in libhxq (HIP kernels for gfx950 behind the C ABI declared
in include/hxq.h); this package is its Python binding plus a thin layer
object.  Importing it does not load the library; the first call does, and
raises if the library has not been built.

Compressed layers: HelixLinear (u8 and pk12 codebook indices).  The 8-bit path
beside it: Fp8Linear, Fp8Experts and RmsNorm.
"""

from ._binding import (  # noqa: F401
    HXQ_BF16,
    HXQ_E4M3,
    HXQ_F32,
    HXQ_FMT_PK12,
    HXQ_FMT_U8,
    HXQ_MAX_GROUP,
    HXQ_VARIANT_AUTO,
    HXQ_VARIANT_GEMM_BF16,
    HXQ_VARIANT_GEMM_BF16_T256,
    HXQ_VARIANT_GEMV_MFMA,
    HXQ_VARIANT_GEMV_VALU,
    HXQ_VARIANT_GENERIC,
    VARIANT_NAMES,
    HxqBwdLayer,
    HxqError,
    HxqLayer,
    hxq_dequant_bf16,
    hxq_linear_bwd_x,
    hxq_linear_bwd_x_grouped,
    hxq_linear_bwd_x_noalloc,
    hxq_linear_bwd_x_workspace,
    hxq_linear_fwd_grouped,
    hxq_linear_fwd_pk12,
    hxq_linear_fwd_u8,
    hxq_linear_fwd_ws,
    hxq_select_variant,
    hxq_sidecar_add,
    hxq_version,
    lib,
)
from .layer import HelixLinear  # noqa: F401

# The 8-bit path's names import torch; they are loaded on first use.
_FP8 = {
    "fp8_columns": "_binding_fp8",
    "fp8_scale_columns": "_binding_fp8",
    "hxq_linear_fwd_fp8": "_binding_fp8",
    "hxq_linear_fwd_fp8_experts": "_binding_fp8",
    "hxq_quant_fp8": "_binding_fp8",
    "hxq_quant_fp8_weight": "_binding_fp8",
    "hxq_rms_norm": "_binding_fp8",
    "hxq_rms_norm_bwd": "_binding_fp8",
    "Fp8Experts": "fp8",
    "Fp8Linear": "fp8",
    "RmsNorm": "fp8",
}


def __getattr__(name):
    if name not in _FP8:
        raise AttributeError("module %r has no attribute %r" % (__name__, name))
    import importlib

    value = getattr(importlib.import_module("." + _FP8[name], __name__), name)
    globals()[name] = value
    return value


def __dir__():
    return sorted(set(globals()) | set(_FP8))
