"""ctypes declarations of the C interface in include/attn.h.

Loading fails loudly when the shared library has not been built: there is no
fallback implementation.
"""

import ctypes
import os

from .build import LIB_PATH

ATTN_OK = 0
ATTN_ERR_INVALID_ARG = 1
ATTN_ERR_UNSUPPORTED = 2
ATTN_ERR_CUDA = 3
ATTN_ERR_TIMEOUT = 4
ATTN_ERR_WORKSPACE = 5
ATTN_ERR_PAGE = 6
ATTN_ERR_FULL = 7

ATTN_BF16 = 0
ATTN_FP32 = 1
ATTN_FP8_E4M3 = 2

ATTN_STALL_NONE = 0
ATTN_STALL_FWD_SOFTMAX = 1
ATTN_STALL_BWD_COMPUTE = 2
ATTN_STALL_PAGED_TILE = 3
ATTN_STALL_PREFIX_SOFTMAX = 4
ATTN_STALL_LATENT_SOFTMAX = 5
ATTN_STALL_EVICT_READ = 8
ATTN_STALL_WEIGHTS_SUM = 9
ATTN_STALL_FP4_VALUES = 10

# every function the header declares, with its ctypes signature
EXPORTS = {
    "attn_workspace_size": (ctypes.c_size_t, [ctypes.c_void_p, ctypes.c_int]),
    "attn_fwd": (ctypes.c_int, [ctypes.c_void_p] * 7 + [ctypes.c_size_t, ctypes.c_void_p]),
    "attn_bwd": (ctypes.c_int, [ctypes.c_void_p] * 11 + [ctypes.c_size_t, ctypes.c_void_p]),
    "attn_bwd_preprocess": (ctypes.c_int, [ctypes.c_void_p] * 5 + [ctypes.c_size_t, ctypes.c_void_p]),
    "attn_bwd_main": (ctypes.c_int, [ctypes.c_void_p] * 8 + [ctypes.c_size_t, ctypes.c_void_p]),
    "attn_bwd_dq": (ctypes.c_int, [ctypes.c_void_p] * 3 + [ctypes.c_size_t, ctypes.c_void_p]),
    "attn_bwd_noalloc": (ctypes.c_int, [ctypes.c_void_p] * 11),
    "attn_decode_workspace_size": (ctypes.c_size_t, [ctypes.c_void_p, ctypes.c_int32]),
    "attn_decode": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32] + [ctypes.c_void_p] * 6
                    + [ctypes.c_size_t, ctypes.c_void_p]),
    "attn_decode_paged_workspace_size": (ctypes.c_size_t, [ctypes.c_void_p, ctypes.c_int32,
                                                           ctypes.c_void_p]),
    "attn_decode_paged": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32] + [ctypes.c_void_p] * 7
                          + [ctypes.c_size_t, ctypes.c_void_p]),
    "attn_decode_latent_workspace_size": (ctypes.c_size_t, [ctypes.c_void_p, ctypes.c_int32,
                                                            ctypes.c_void_p]),
    "attn_decode_latent": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32] + [ctypes.c_void_p] * 6
                           + [ctypes.c_size_t, ctypes.c_void_p]),
    "attn_pages_workspace_size": (ctypes.c_size_t, [ctypes.c_void_p, ctypes.c_int32]),
    "attn_pages_copy": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32,
                                       ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                       ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "attn_pages_extend": (ctypes.c_int, [ctypes.c_void_p] * 3 + [ctypes.c_int32, ctypes.c_void_p,
                                                                 ctypes.c_size_t,
                                                                 ctypes.c_void_p]),
    "attn_pages_fork": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                       ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                       ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                       ctypes.c_void_p]),
    "attn_pages_free": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                       ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "attn_pages_compact": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                          ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                          ctypes.c_void_p]),
    "attn_pages_store_fp4": (ctypes.c_int, [ctypes.c_void_p] * 8 + [ctypes.c_size_t,
                                                                    ctypes.c_void_p]),
    "attn_pages_load_fp4": (ctypes.c_int, [ctypes.c_void_p] * 8 + [ctypes.c_size_t,
                                                                   ctypes.c_void_p]),
    "attn_decode_fp4_workspace_size": (ctypes.c_size_t, [ctypes.c_void_p, ctypes.c_int32,
                                                         ctypes.c_void_p]),
    "attn_decode_fp4": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32] + [ctypes.c_void_p] * 7
                        + [ctypes.c_size_t, ctypes.c_void_p]),
    "attn_key_weights": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32] + [ctypes.c_void_p] * 6
                         + [ctypes.c_int64, ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p,
                            ctypes.c_size_t, ctypes.c_void_p]),
    "attn_pages_evict_workspace_size": (ctypes.c_size_t, [ctypes.c_void_p, ctypes.c_int32,
                                                          ctypes.c_int32, ctypes.c_void_p,
                                                          ctypes.c_int32]),
    "attn_pages_evict": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                        ctypes.c_int32, ctypes.c_void_p, ctypes.c_int64,
                                        ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                        ctypes.c_void_p]),
    "attn_selftest_timeout": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_uint64, ctypes.c_void_p]),
    "attn_debug_stall": (ctypes.c_int, [ctypes.c_int32, ctypes.c_uint64]),
    "attn_check": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),
    "attn_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "attn_last_error": (ctypes.c_char_p, []),
}


class AttnParams(ctypes.Structure):
    """Mirror of `attn_params`."""

    _fields_ = [
        ("B", ctypes.c_int32), ("H", ctypes.c_int32), ("N", ctypes.c_int32),
        ("d", ctypes.c_int32), ("dtype", ctypes.c_int32), ("scale", ctypes.c_float),
        ("causal", ctypes.c_int32), ("dropout_p", ctypes.c_float),
        ("philox_seed", ctypes.c_uint64), ("philox_offset", ctypes.c_uint64),
        ("key_lens", ctypes.c_void_p), ("block_mask", ctypes.c_void_p),
        ("block_mask_head_stride", ctypes.c_int64),
        ("stride_b", ctypes.c_int64), ("stride_h", ctypes.c_int64),
        ("stride_n", ctypes.c_int64),
        ("H_kv", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("kv_stride_b", ctypes.c_int64), ("kv_stride_h", ctypes.c_int64),
        ("kv_stride_n", ctypes.c_int64),
        ("q_descale", ctypes.c_float), ("k_descale", ctypes.c_float),
        ("v_descale", ctypes.c_float), ("reserved2", ctypes.c_int32),
    ]


class AttnPages(ctypes.Structure):
    """Mirror of `attn_pages`."""

    _fields_ = [
        ("table", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
        ("max_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32), ("shared_len", ctypes.c_int32),
    ]


class AttnPageTable(ctypes.Structure):
    """Mirror of `attn_page_table`."""

    _fields_ = [
        ("table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("lens", ctypes.c_void_p),
        ("refs", ctypes.c_void_p), ("rows", ctypes.c_int32), ("max_pages", ctypes.c_int32),
        ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32),
    ]


class AttnPool(ctypes.Structure):
    """Mirror of `attn_pool`."""

    _fields_ = [("base", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("page_bytes", ctypes.c_int64)]


class AttnFp4(ctypes.Structure):
    """Mirror of `attn_fp4`."""

    _fields_ = [
        ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
        ("code_page", ctypes.c_int64), ("code_head", ctypes.c_int64),
        ("scale_page", ctypes.c_int64), ("scale_head", ctypes.c_int64),
        ("descale", ctypes.c_float), ("reserved", ctypes.c_int32),
    ]


class AttnRows(ctypes.Structure):
    """Mirror of `attn_rows`."""

    _fields_ = [
        ("base", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
        ("head_stride", ctypes.c_int64), ("row_stride", ctypes.c_int64),
        ("row_bytes", ctypes.c_int32), ("reserved", ctypes.c_int32),
    ]


class AttnError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"{message} (status {status})")
        self.status = status


_lib = None


def lib():
    """The loaded shared library; raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"CUDA library {LIB_PATH} is not built; run "
                "`python -m exact_attention_12_gb300.build` (needs nvcc)")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in EXPORTS.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def check_status(status, what):
    if status != ATTN_OK:
        detail = lib().attn_last_error().decode(errors="replace")
        raise AttnError(status, f"{what}: {detail}")
