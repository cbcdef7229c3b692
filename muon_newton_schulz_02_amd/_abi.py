"""ctypes mirror of include/muon_adamw.h and include/ma_grads.h.

Argument marshalling only: every step of the optimizer runs in the HIP
library.  Loading fails loudly when the library has not been built; there is
no fallback path.
"""

from __future__ import annotations

import ctypes as C
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmuon_adamw.so")

MA_OK = 0
MA_ERR_INVALID_ARG = -1
MA_ERR_SHAPE = -2
MA_ERR_UNSUPPORTED = -3
MA_ERR_WORKSPACE = -4
MA_ERR_HIP = -5
MA_ERR_CAPTURE = -6

MA_GROUP_MUON, MA_GROUP_ADAMW, MA_GROUP_NONE = 0, 1, 2
MA_MODE_MUON_ADAMW, MA_MODE_ADAMW = 0, 1
MA_NS_BF16, MA_NS_FP32 = 0, 1
MA_LR_CONSTANT, MA_LR_COSINE_MIN = 0, 1
MA_PARAM_FP32, MA_PARAM_BF16 = 0, 1
MA_MAX_NDIM = 8
MA_ACT_GROUP = 32
MA_ACT_SILU, MA_ACT_GELU_TANH = 0, 1
MA_PROFILE_EVENTS = 5
MA_NOALLOC_SCRATCH_BYTES = 64 << 20


class ma_param_desc(C.Structure):
    _fields_ = [("name", C.c_char_p), ("ndim", C.c_int32),
                ("shape", C.POINTER(C.c_int64)), ("trainable", C.c_int32)]


class ma_plan_opts(C.Structure):
    _fields_ = [("mode", C.c_int32), ("moonlight_coefficient", C.c_double),
                ("overlap_groups", C.c_int32), ("param_dtype", C.c_int32)]


class ma_plan_entry(C.Structure):
    _fields_ = [("group", C.c_int32), ("bucket", C.c_int32),
                ("m", C.c_int64), ("n", C.c_int64), ("r", C.c_int64), ("c", C.c_int64),
                ("transposed", C.c_int32), ("lr_shape_scale", C.c_float),
                ("numel", C.c_int64), ("adam_offset", C.c_int64)]


class ma_state(C.Structure):
    _fields_ = [("muon_momentum", C.POINTER(C.c_void_p)),
                ("adam_m", C.POINTER(C.c_void_p)),
                ("adam_v", C.POINTER(C.c_void_p)),
                ("step", C.c_int64), ("device_step", C.c_void_p)]


class ma_hparams(C.Structure):
    _fields_ = [("lr", C.c_double), ("muon_lr_scale", C.c_double), ("muon_momentum", C.c_double),
                ("muon_nesterov", C.c_int32), ("muon_ns_steps", C.c_int32),
                ("ns_coeffs", C.c_double * 3), ("ns_precision", C.c_int32),
                ("ns_eps", C.c_double), ("beta1", C.c_double), ("beta2", C.c_double),
                ("eps", C.c_double), ("weight_decay", C.c_double),
                ("muon_weight_decay", C.c_double), ("max_grad_norm", C.c_double),
                ("lr_schedule", C.c_int32), ("warmup_steps", C.c_int64),
                ("total_steps", C.c_int64), ("min_lr_rate", C.c_double)]


# (name, restype, argtypes) of every exported symbol of muon_adamw.h
SIGNATURES = [
    ("muon_adamw_default_hparams", C.c_int, [C.POINTER(ma_hparams)]),
    ("muon_adamw_plan", C.c_int, [C.POINTER(ma_param_desc), C.c_int32,
                                  C.POINTER(ma_plan_opts), C.POINTER(C.c_void_p)]),
    ("muon_adamw_plan_size", C.c_int, [C.c_void_p, C.POINTER(C.c_int32)]),
    ("muon_adamw_plan_entry", C.c_int, [C.c_void_p, C.c_int32, C.POINTER(ma_plan_entry)]),
    ("muon_adamw_plan_dump", C.c_int, [C.c_void_p, C.c_char_p, C.c_size_t,
                                       C.POINTER(C.c_size_t)]),
    ("muon_adamw_workspace_size", C.c_int, [C.c_void_p, C.c_int32, C.POINTER(C.c_size_t)]),
    ("muon_adamw_step", C.c_int, [C.c_void_p, C.POINTER(C.c_void_p), C.POINTER(C.c_void_p),
                                  C.POINTER(ma_state), C.POINTER(ma_hparams),
                                  C.c_void_p, C.c_size_t, C.c_void_p, C.c_void_p,
                                  C.POINTER(C.c_void_p)]),
    ("muon_adamw_step_profiled", C.c_int, [C.c_void_p, C.POINTER(C.c_void_p),
                                           C.POINTER(C.c_void_p), C.POINTER(ma_state),
                                           C.POINTER(ma_hparams), C.c_void_p, C.c_size_t,
                                           C.c_void_p, C.c_void_p, C.POINTER(C.c_void_p),
                                           C.POINTER(C.c_void_p)]),
    ("muon_adamw_step_noalloc", C.c_int, [C.c_void_p, C.POINTER(C.c_void_p),
                                          C.POINTER(C.c_void_p), C.POINTER(ma_state),
                                          C.POINTER(ma_hparams), C.c_void_p, C.c_void_p,
                                          C.POINTER(C.c_void_p)]),
    ("muon_adamw_plan_free", None, [C.c_void_p]),
    ("muon_adamw_last_error", C.c_char_p, []),
    ("muon_adamw_version", C.c_char_p, []),
]

_I32, _I64, _P, _F64, _SZ = C.c_int32, C.c_int64, C.c_void_p, C.c_double, C.c_size_t

# and of ma_grads.h
GRAD_SIGNATURES = [
    ("ma_act_pitch", C.c_int, [_I64, C.POINTER(_I64), C.POINTER(_I64)]),
    ("ma_act_pack", C.c_int, [_P, _I32, _I64, _I64, _I64, _P, _P, _P]),
    ("ma_act_unpack", C.c_int, [_P, _P, _I64, _I64, _P, _I32, _I64, _P]),
    ("ma_embedding_lookup", C.c_int, [_P, _I32, _I64, _I64, _I64, _P, _I32, _I64, _F64, _P, _I32,
                                      _I64, _P]),
    ("ma_embedding_grad_workspace_size", C.c_int, [_I64, _I64, _I64, C.POINTER(_SZ)]),
    ("ma_embedding_grad", C.c_int, [_P, _I32, _I64, _P, _I32, _I64, _I64, _I64, _F64, _I64, _P,
                                    _I32, _I32, _P, _SZ, _P]),
    ("ma_linear_grad_workspace_size", C.c_int, [_I64, _I64, _I64, _I32, C.POINTER(_SZ)]),
    ("ma_linear_grad_workspace_size_at", C.c_int, [_P, _I32, _I64, _I64, _I64, _I64,
                                                   C.POINTER(_SZ)]),
    ("ma_linear_grad", C.c_int, [_P, _I32, _I64, _I64, _I64, _P, _P, _I64, _P, _I32, _I32, _P,
                                 _SZ, _P]),
    ("ma_glu_forward", C.c_int, [_P, _P, _I32, _I64, _I64, _I64, _I64, _I32, _P, _I64, _P, _P, _P,
                                 _P, _P]),
    ("ma_glu_backward", C.c_int, [_P, _I32, _I64, _I64, _I64, _P, _P, _P, _P, _I32, _P, _I64, _P,
                                  _I64, _P, _P, _P]),
]

_lib = None


def load(path: str = LIB_PATH):
    """Load the HIP library (once).  Raises if it is not built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            "libmuon_adamw.so is not built (%s); run "
            "`python -m muon_newton_schulz_02_amd.build` first" % path)
    lib = C.CDLL(path)
    for name, res, args in SIGNATURES + GRAD_SIGNATURES:
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib
