"""ctypes binding of libcattn's C ABI (declared in include/cattn.h).

Argument marshalling only: every step of the computation runs in the
library's CUDA kernels.  There is no fallback; if the shared library is
missing, importing this module raises.
"""

from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import struct
import sys
import warnings

import torch  # noqa: F401  (before the marshalling, which links against its libraries)

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libcattn.so")

OK = 0
ERR_INVALID_ARG = 1
ERR_UNSUPPORTED = 2
ERR_CUDA = 3
ERR_TIMEOUT = 4
ERR_TOO_LARGE = 5

STATUS_NAMES = {OK: "CATTN_OK", ERR_INVALID_ARG: "CATTN_ERR_INVALID_ARG",
                ERR_UNSUPPORTED: "CATTN_ERR_UNSUPPORTED", ERR_CUDA: "CATTN_ERR_CUDA",
                ERR_TIMEOUT: "CATTN_ERR_TIMEOUT", ERR_TOO_LARGE: "CATTN_ERR_TOO_LARGE"}



class Layout(ctypes.Structure):
    """cattn_layout: element strides (b, h, t) of a (B, H, T, D) tensor."""
    _fields_ = [("b", ctypes.c_longlong), ("h", ctypes.c_longlong), ("t", ctypes.c_longlong)]


class Dropout(ctypes.Structure):
    """cattn_dropout: drop probability p, generator seed, counter offset and
    the optional keep-bit cache (device pointer or None)."""
    _fields_ = [("p", ctypes.c_float), ("seed", ctypes.c_ulonglong), ("offset", ctypes.c_uint),
                ("mask", ctypes.c_void_p)]


# name -> (restype, argtypes), mirroring include/cattn.h
_vp, _i, _f, _sz, _u32 = (ctypes.c_void_p, ctypes.c_int, ctypes.c_float,
                          ctypes.c_size_t, ctypes.c_uint32)
_ll = ctypes.c_longlong
_L = Layout
_DP = ctypes.POINTER(Dropout)
SIGNATURES = {
    "attn_fwd": (_i, [_vp, _vp, _vp, _f, _i, _i, _i, _i, _vp, _vp, _vp]),
    "attn_fwd_ex": (_i, [_vp, _vp, _vp, _f, _i, _i, _i, _i, _vp, _vp, _vp, _vp]),
    "attn_bwd_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "attn_bwd_preprocess": (_i, [_vp, _vp, _i, _i, _i, _i, _vp, _vp]),
    "attn_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _f, _i, _i, _i, _i,
                      _vp, _vp, _vp, _vp, _sz, _vp]),
    "attn_bwd_ex": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _f, _i, _i, _i, _i,
                         _vp, _vp, _vp, _i, _vp, _sz, _vp]),
    "attn_bwd_noalloc": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _f, _i, _i, _i, _i,
                              _vp, _vp, _vp, _vp]),
    "attn_fwd_strided": (_i, [_vp, _L, _vp, _L, _vp, _L, _f, _i, _i, _i, _i, _vp, _L, _vp, _vp,
                              _vp]),
    "attn_bwd_strided": (_i, [_vp, _L, _vp, _L, _vp, _L, _vp, _L, _vp, _vp, _vp, _L, _f,
                              _i, _i, _i, _i, _vp, _L, _vp, _L, _vp, _L, _i, _vp, _sz, _vp]),
    "attn_fwd_dropout": (_i, [_vp, _L, _vp, _L, _vp, _L, _f, _i, _i, _i, _i, _DP, _vp, _L, _vp,
                              _vp, _vp]),
    "attn_bwd_dropout": (_i, [_vp, _L, _vp, _L, _vp, _L, _vp, _L, _vp, _vp, _vp, _L, _f,
                              _i, _i, _i, _i, _DP, _vp, _L, _vp, _L, _vp, _L, _i, _vp, _sz, _vp]),
    "attn_decode_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "attn_dropout_mask_bytes": (_sz, [_i, _i, _i]),
    "attn_decode": (_i, [_vp, _L, _vp, _L, _vp, _L, _f, _i, _i, _i, _i, _i, _vp, _L, _vp, _vp,
                         _sz, _vp]),
    "attn_paged_plan": (_i, [_vp, _vp, _vp, _ll, _vp, _vp, _i, _i, _i, _i, _ll, _vp, _vp, _vp, _vp,
                             _vp, _vp, _vp]),
    "attn_cache_append": (_i, [_vp, _L, _vp, _L, _ll, _i, _i, _i, _i, _vp, _vp, _L, _vp, _L, _vp,
                               _vp]),
    "attn_decode_paged_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "attn_decode_paged": (_i, [_vp, _L, _vp, _L, _vp, _L, _f, _i, _i, _i, _i, _i, _i, _i, _vp, _ll,
                               _i, _vp, _vp, _L, _vp, _vp, _sz, _vp]),
    "attn_page_select_workspace_bytes": (_sz, [_i, _i, _i]),
    "attn_page_select": (_i, [_vp, _L, _vp, _i, _i, _i, _i, _i, _i, _i, _vp, _ll, _i, _vp, _i, _i,
                              _i, _vp, _vp, _sz, _vp]),
    "attn_decode_sparse": (_i, [_vp, _L, _vp, _L, _vp, _L, _f, _i, _i, _i, _i, _i, _i, _i, _vp,
                                _ll, _i, _vp, _vp, _i, _vp, _L, _vp, _vp, _sz, _vp]),
    "attn_paged_call": (_i, [_i, ctypes.c_char_p, _i]),
    "cattn_get_device_status": (_i, [_i, _vp]),
    "cattn_set_wait_timeout_us": (None, [_u32]),
    "cattn_selftest_wait_timeout": (_i, [_u32, _vp]),
    "cattn_last_device_status": (_i, [_vp, _vp]),
    "cattn_selftest_wait_timeout_ws": (_i, [_u32, _vp, _vp]),
    "cattn_timing_enable": (None, [_i]),
    "cattn_timing_read": (_i, [ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_int), _i]),
    "cattn_status_string": (ctypes.c_char_p, [_i]),
    "cattn_version": (_i, []),
    "cattn_plan_passes": (_i, [_i, _i, _i, _i, ctypes.POINTER(ctypes.c_uint16), _i]),
    "cattn_last_cuda_error": (_i, []),
}


# attn_paged_call: the paged calls by number, and their words ("q" whole
# numbers and addresses, "d" the scale)
CALL_PAGED_PLAN, CALL_CACHE_APPEND, CALL_DECODE_PAGED, CALL_PAGE_SELECT, CALL_DECODE_SPARSE = range(5)
CALL_NAMES = ("attn_paged_plan", "attn_cache_append", "attn_decode_paged", "attn_page_select",
              "attn_decode_sparse")
CALL_WORDS = tuple(struct.Struct(f) for f in ("=18q", "=24q", "=12qd19q", "=23q", "=12qd21q"))


class CattnError(RuntimeError):
    def __init__(self, fn: str, status: int, cuda_error: int = 0):
        self.status = status
        self.cuda_error = cuda_error
        extra = f" (CUDA error {cuda_error})" if status == ERR_CUDA else ""
        super().__init__(f"{fn} failed: {STATUS_NAMES.get(status, status)}{extra}")


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError(
            f"libcattn.so not found at {path}; build it with "
            "`python causal_self_attention_flash_b200/build.py`")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


# CATTN_NOALLOC_SCRATCH_BYTES of include/cattn.h
NOALLOC_SCRATCH_BYTES = 64 << 20

LIB = load()


class LongWay:
    """Stands in for the marshalling of the paged calls: it recognises no
    arguments, so every call goes through the Python wrapper."""

    @staticmethod
    def _unknown(*args):
        return -1
    decode = append = plan = select = _unknown


def load_torch_calls():
    """The marshalling of the paged calls (csrc/torch_calls.cpp), set to make
    them through this process's libcattn; LongWay where there is none for this
    Python and torch (the library itself needs neither)."""
    path = os.path.join(HERE, f"_torch_calls-{sys.implementation.cache_tag}-"
                              f"torch{torch.__version__}.so")
    try:
        loader = importlib.machinery.ExtensionFileLoader(__package__ + "._torch_calls", path)
        module = importlib.util.module_from_spec(
            importlib.util.spec_from_file_location(loader.name, path, loader=loader))
        loader.exec_module(module)
    except ImportError as e:
        warnings.warn(f"{os.path.basename(path)} cannot be loaded ({e}): the paged calls take some "
                      "microseconds longer; build it with "
                      "`python causal_self_attention_flash_b200/build.py`", RuntimeWarning)
        return LongWay()
    module.use(ctypes.cast(LIB.attn_paged_call, ctypes.c_void_p).value)
    return module


TORCH_CALLS = load_torch_calls()
