"""ctypes declarations of ``libflce.so`` (the C ABI in ``include/flce.h``).

Loading fails loudly when the library has not been built: there is no
fallback implementation.  Build it with ``__graft_entry__.build()`` or
``python -m linear_cross_entropy_tmem_gb300.build``.
"""
from __future__ import annotations

import ctypes
import os
from ctypes import POINTER, c_char_p, c_float, c_int, c_int32, c_int64, c_size_t, c_void_p

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_build", "libflce.so")


def torch_path() -> str:
    """The native marshalling's file.  It is compiled against one torch and one Python, which its name says: under
    another it is not found, rather than loaded."""
    import sysconfig

    import torch
    return os.path.join(os.path.dirname(LIB_PATH),
                        f"flce_torch-{torch.__version__}{sysconfig.get_config_var('EXT_SUFFIX')}")


FLCE_F32, FLCE_BF16, FLCE_F16 = 0, 1, 2
FLCE_RED_NONE, FLCE_RED_SUM, FLCE_RED_MEAN = 0, 1, 2
FLCE_FLAG_COMPACT_VALID = 1
FLCE_FLAG_BWD_RECOMPUTE = 2
FLCE_FLAG_BWD_KEEP_LOGITS = 4
FLCE_FLAG_FP32_FULL = 8
FLCE_FLAG_FROZEN_HEAD = 16
BWD_ALGOS = {"auto": 0, "recompute": FLCE_FLAG_BWD_RECOMPUTE, "keep_logits": FLCE_FLAG_BWD_KEEP_LOGITS}
REDUCTIONS = {"none": FLCE_RED_NONE, "sum": FLCE_RED_SUM, "mean": FLCE_RED_MEAN}

FLCE_OK = 0
FLCE_ERR_INVALID_ARG = 1
FLCE_ERR_UNSUPPORTED_DTYPE = 2
FLCE_ERR_DTYPE_MISMATCH = 3
FLCE_ERR_MISALIGNED = 4
FLCE_ERR_WORKSPACE_TOO_SMALL = 5
FLCE_ERR_CUDA = 6
FLCE_ERR_TARGET_OUT_OF_RANGE = 7
FLCE_ERR_TIMEOUT = 8
FLCE_ERR_UNSUPPORTED_DEVICE = 9


class FlceLaunchRecord(ctypes.Structure):
    """Mirror of ``flce_launch_record``."""
    _fields_ = [("begin_event", c_void_p), ("end_event", c_void_p), ("kind", c_int32), ("reserved", c_int32)]


LAUNCH_KINDS = {0: "fwd_logits", 1: "bwd_recompute", 2: "bwd_dweight", 3: "bwd_dhidden", 4: "other",
                5: "bwd_logit_grad"}


class FlceProblem(ctypes.Structure):
    """Mirror of ``flce_problem``."""
    _fields_ = [
        ("n_tokens", c_int64),
        ("hidden", c_int64),
        ("vocab", c_int64),
        ("hidden_dtype", c_int32),
        ("weight_dtype", c_int32),
        ("bias_dtype", c_int32),
        ("reduction", c_int32),
        ("logit_scale", c_float),
        ("final_logit_softcapping", c_float),
        ("ignore_index", c_int64),
        ("num_items_in_batch", ctypes.c_double),
        ("flags", ctypes.c_uint32),
        ("reserved", ctypes.c_uint32),
    ]


class FlceNormProblem(ctypes.Structure):
    """Mirror of ``flce_norm_problem``."""
    _fields_ = [
        ("rows", c_int64),
        ("cols", c_int64),
        ("x_stride", c_int64),
        ("residual_stride", c_int64),
        ("h_stride", c_int64),
        ("y_stride", c_int64),
        ("dresidual_stride", c_int64),
        ("dtype", c_int32),
        ("residual_dtype", c_int32),
        ("weight_dtype", c_int32),
        ("quant_group", c_int32),
        ("eps", c_float),
        ("weight_offset", c_float),
    ]


class FlceLogitsProblem(ctypes.Structure):
    """Mirror of ``flce_logits_problem``."""
    _fields_ = [
        ("rows", c_int64),
        ("vocab", c_int64),
        ("history", c_int64),
        ("n_bias", c_int64),
        ("logits_stride", c_int64),
        ("out_stride", c_int64),
        ("tokens_stride", c_int64),
        ("bias_ids_stride", c_int64),
        ("bias_stride", c_int64),
        ("mask_stride", c_int64),
        ("logits_dtype", c_int32),
        ("out_dtype", c_int32),
        ("tokens_i64", c_int32),
        ("bias_ids_i64", c_int32),
    ]


class FlceEmbeddingProblem(ctypes.Structure):
    """Mirror of ``flce_embedding_problem``."""
    _fields_ = [
        ("tokens", c_int64),
        ("vocab", c_int64),
        ("cols", c_int64),
        ("weight_stride", c_int64),
        ("out_stride", c_int64),
        ("padding", c_int64),
        ("weight_dtype", c_int32),
        ("out_dtype", c_int32),
        ("ids_i64", c_int32),
        ("accumulate", c_int32),
        ("scale", c_float),
        ("reserved", c_int32),
    ]


class FlceMxfp4Problem(ctypes.Structure):
    """Mirror of ``flce_mxfp4_problem``."""
    _fields_ = [("rows", c_int64), ("cols", c_int64), ("stride", c_int64), ("dtype", c_int32), ("reserved", c_int32)]


class FlceMxfp4LogitsProblem(ctypes.Structure):
    """Mirror of ``flce_mxfp4_logits_problem``."""
    _fields_ = [
        ("tokens", c_int64),
        ("vocab", c_int64),
        ("cols", c_int64),
        ("hidden_stride", c_int64),
        ("out_stride", c_int64),
        ("hidden_dtype", c_int32),
        ("out_dtype", c_int32),
        ("bias_dtype", c_int32),
        ("logit_scale", c_float),
        ("softcap", c_float),
        ("reserved", c_int32),
    ]


class FlceSampleProblem(ctypes.Structure):
    """Mirror of ``flce_sample_problem``."""
    _fields_ = [("rows", c_int64), ("vocab", c_int64), ("logits_stride", c_int64), ("logits_dtype", c_int32),
                ("reserved", c_int32)]


_LIB = None

# name -> (restype, argtypes); every function ``include/*.h`` declares.
class FlceTestingPlanInfo(ctypes.Structure):
    """Mirror of ``flce_testing_plan_info``."""
    _fields_ = [
        ("keep_logits", c_int32),
        ("dh_pair", c_int32),
        ("token_chunk_rows", c_int64),
        ("vocab_chunk_cols", c_int64),
        ("run_chunk_cols", c_int64),
        ("n_chunks", c_int64),
        ("dh_ksplit_max", c_int32),
        ("dh_ksplit", c_int32),
        ("fwd_pair", c_int32),
        ("fwd_splits", c_int32),
        ("fwd_tiles_per_split", c_int32),
        ("reserved", c_int32),
    ]


SIGNATURES = {
    "flce_workspace_size": (c_int, [POINTER(FlceProblem), c_int, POINTER(c_size_t)]),
    "flce_forward": (c_int, [POINTER(FlceProblem), c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                             c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "flce_backward": (c_int, [POINTER(FlceProblem), c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                              c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "flce_forward_backward": (c_int, [POINTER(FlceProblem), c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                      c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                      c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "flce_forward_noalloc": (c_int, [POINTER(FlceProblem), c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                     c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]),
    "flce_add_rms_norm": (c_int, [POINTER(FlceNormProblem)] + [c_void_p] * 7),
    "flce_add_rms_norm_fp8": (c_int, [POINTER(FlceNormProblem)] + [c_void_p] * 7),
    "flce_add_rms_norm_workspace_size": (c_int, [POINTER(FlceNormProblem), POINTER(c_size_t)]),
    "flce_add_rms_norm_backward": (c_int, [POINTER(FlceNormProblem)] + [c_void_p] * 9 + [c_size_t, c_void_p]),
    "flce_grad_norm_workspace_size": (c_int, [c_int64, POINTER(c_size_t)]),
    "flce_grad_norm": (c_int, [c_void_p, c_void_p, c_void_p, c_int64, c_void_p, c_void_p, c_size_t, c_void_p]),
    "flce_clip_grad_norm": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_int64, c_float, c_void_p, c_void_p,
                                    c_size_t, c_void_p]),
    "flce_process_logits_workspace_size": (c_int, [POINTER(FlceLogitsProblem), POINTER(c_size_t)]),
    "flce_process_logits": (c_int, [POINTER(FlceLogitsProblem)] + [c_void_p] * 14 + [c_size_t, c_void_p]),
    "flce_embedding": (c_int, [POINTER(FlceEmbeddingProblem)] + [c_void_p] * 4),
    "flce_embedding_workspace_size": (c_int, [POINTER(FlceEmbeddingProblem), POINTER(c_size_t)]),
    "flce_embedding_backward": (c_int, [POINTER(FlceEmbeddingProblem)] + [c_void_p] * 4 + [c_size_t, c_void_p]),
    "flce_mxfp4_size": (c_int, [POINTER(FlceMxfp4Problem), POINTER(c_size_t), POINTER(c_size_t)]),
    "flce_mxfp4_quantize": (c_int, [POINTER(FlceMxfp4Problem)] + [c_void_p] * 4),
    "flce_mxfp4_dequantize": (c_int, [POINTER(FlceMxfp4Problem)] + [c_void_p] * 4),
    "flce_mxfp4_logits_workspace_size": (c_int, [POINTER(FlceMxfp4LogitsProblem), POINTER(c_size_t)]),
    "flce_mxfp4_logits": (c_int, [POINTER(FlceMxfp4LogitsProblem)] + [c_void_p] * 6 + [c_size_t, c_void_p]),
    "flce_sample": (c_int, [POINTER(FlceSampleProblem)] + [c_void_p] * 10),
    "flce_read_device_status": (c_int, [c_void_p, c_void_p, POINTER(c_int)]),
    "flce_status_string": (c_char_p, [c_int]),
    "flce_abi_version": (c_int, []),
    "flce_testing_set_tuning": (c_int, [c_int64, c_int]),
    "flce_scale_gradient": (c_int, [c_void_p, c_void_p, c_int64, c_int32, c_void_p]),
    "flce_testing_set_gemm_mode": (c_int, [c_int]),
    "flce_testing_plan": (c_int, [POINTER(FlceProblem), c_int, c_int, POINTER(FlceTestingPlanInfo)]),
    "flce_testing_set_token_chunk": (c_int, [c_int64]),
    "flce_testing_set_launch_log": (c_int, [c_void_p, c_int32, POINTER(c_int32)]),
    "flce_testing_launch_count": (c_int64, []),
    "flce_testing_gemm": (c_int, [c_int, c_int, c_int64, c_int64, c_int64, c_void_p, c_int64, c_void_p, c_int64,
                                  c_void_p, c_int64, c_void_p]),
}


def load(path: str = LIB_PATH):
    """Load ``libflce.so`` once and declare every exported function."""
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(path):
        raise RuntimeError(
            f"libflce.so not found at {path}: build it with __graft_entry__.build() "
            "(the CUDA library is required; there is no CPU fallback)")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _LIB = lib
    return lib


# What flce_torch calls, in the order of its table.
_MARSHALLED = ("flce_add_rms_norm", "flce_add_rms_norm_fp8", "flce_add_rms_norm_workspace_size",
               "flce_add_rms_norm_backward", "flce_grad_norm_workspace_size", "flce_grad_norm", "flce_clip_grad_norm",
               "flce_process_logits_workspace_size", "flce_process_logits", "flce_embedding",
               "flce_embedding_workspace_size", "flce_embedding_backward", "flce_mxfp4_quantize",
               "flce_mxfp4_dequantize", "flce_mxfp4_logits_workspace_size", "flce_mxfp4_logits", "flce_sample")
_TORCH = None


def load_torch():
    """Load ``flce_torch``, the native marshalling of torch tensors, on the loaded library's functions."""
    global _TORCH
    if _TORCH is None:
        import importlib.machinery
        import importlib.util
        lib = load()
        path = torch_path()
        if not os.path.exists(path):
            raise RuntimeError(f"flce_torch not found at {path}: build it with __graft_entry__.build()")
        loader = importlib.machinery.ExtensionFileLoader("flce_torch", path)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("flce_torch", loader))
        loader.exec_module(module)
        module.bind(*(ctypes.cast(getattr(lib, name), c_void_p).value for name in _MARSHALLED))
        _TORCH = module
    return _TORCH


class FlceError(RuntimeError):
    def __init__(self, status: int, where: str = ""):
        lib = load()
        msg = lib.flce_status_string(status).decode()
        super().__init__(f"{where}: FLCE status {status} ({msg})" if where else f"FLCE status {status} ({msg})")
        self.status = status


def check(status: int, where: str = "") -> None:
    if status != FLCE_OK:
        raise FlceError(status, where)
