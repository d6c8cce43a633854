"""ctypes loader for libccv.so, the CUDA library behind include/ccv.h and
include/ccv_layer.h.

There is no fallback: if the library has not been built, loading raises.
"""
from __future__ import annotations

import ctypes
import os
import re

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_build", "libccv.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "ccv.h")
LAYER_HEADER = os.path.join(os.path.dirname(HERE), "include", "ccv_layer.h")

P = ctypes.c_void_p
I64 = ctypes.c_int64
I32 = ctypes.c_int
F32 = ctypes.c_float


class PagedStream(ctypes.Structure):
    """struct ccv_paged_stream of include/ccv.h."""
    _fields_ = [("x", P), ("x_stride_t", I64), ("weight", P), ("w_stride_c", I64),
                ("w_stride_w", I64), ("out", P), ("out_stride_t", I64), ("off_s", I32),
                ("ws", I32)]


# Argument lists, in the order of the declarations in include/ccv.h.
SIGNATURES = {
    "ccv_status_string": ([I32], ctypes.c_char_p),
    "ccv_version": ([], I32),
    "ccv_fwd": ([P, I64, I64, P, I64, I64, P, I64, I64, P,
                 P, I64, I64, I64, I32, I32, P, I32, P, P,
                 I32, I32, I32, I32, I32, P, P], I32),
    "ccv_update": ([P, I64, I64, I64, P, I64, I64, I64, P, I64, I64, P,
                    P, I64, I64, I64, I32, I32, P, I32, I32, I32,
                    I32, I32, I32, P, P], I32),
    "ccv_update_spec": ([P, I64, I64, I64, P, I64, I64, I64, P, I64, I64, P,
                         P, I64, I64, I64, I32, I32, P, P,
                         P, I64, I64, I64, I64, I32, P, I64, I64, I32,
                         I32, I32, I32, I32, I32, I32, P, P], I32),
    "paged_sconv_seq_metadata": ([P, I32, I32, I32, P, P, I32, P], I32),
    "paged_sconv_fwd": ([P, I64, P, I64, I64, I64, I32, I32, I32, I32,
                         P, I64, I64, P, I64, P, P, P, P, I64, I32, I32,
                         P, I32, I32, I32, I32, I32, I32, P, P], I32),
    "paged_sconv_fwd_with_metadata": ([P, I64, P, I64, I64, I64, I32, I32, I32, I32,
                                       P, I64, I64, P, I64, P, P, I32, I32, P, P,
                                       P, P, I64, I32, I32, I32, I32, I32, I32, I32, I32,
                                       P, P], I32),
    "paged_sconv_fwd_streams": ([P, I32, P, I64, I64, I64, I32, I32, I32, I32,
                                 P, P, P, P, I64, I32, I32, P, I32, I32, I32, I32, P, P], I32),
}


class HeadsView(ctypes.Structure):
    """struct ccv_heads_view of include/ccv_layer.h."""
    _fields_ = [("data", P), ("stride_row", I64), ("stride_tok", I64), ("stride_head", I64),
                ("stride_dim", I64)]


class GdrArgs(ctypes.Structure):
    """struct ccv_gdr_args of include/ccv_layer.h."""
    _fields_ = [("q", HeadsView), ("k", HeadsView), ("v", HeadsView), ("out", HeadsView),
                ("g", P), ("beta", P), ("gate_stride_row", I64), ("gate_stride_tok", I64),
                ("gate_stride_head", I64), ("a_log", P), ("dt_bias", P), ("state", P),
                ("s_stride_line", I64), ("s_stride_head", I64), ("s_stride_v", I64),
                ("s_stride_k", I64), ("num_lines", I32), ("num_k_heads", I32),
                ("num_v_heads", I32), ("dim_k", I32), ("dim_v", I32), ("scale", F32),
                ("qk_l2norm", I32), ("pad_slot_id", I32)]


# Argument lists of include/ccv_layer.h, in the order of its declarations.
LAYER_SIGNATURES = {
    "gdr_fwd": ([P, P, I32, P, P, I32, P, I64, P, P], I32),
    "gdr_fwd_workspace": ([I32, I32, I32, I32, I32, I32], I64),
    "gdr_update": ([P, P, P, P, I64, I64, I32, I32, I32, P, P], I32),
    "gated_rms_norm": ([P, P, P, P, I32, I32, I32, F32, I32, I32, P], I32),
    "residual_rms_norm": ([P, I64, I64, P, I64, I64, I32, P, P, P, I64, I64, P, I64, I64,
                           P, I64, I64, I32, I32, F32, F32, F32, P], I32),
    "spec_verify": ([P, I32, I64, I64, P, I64, I64, P, I64, I64, P, P, P, I64, I64, P, I64,
                     P, P, I32, I32, I32, P, I64, P, P], I32),
    "spec_verify_workspace": ([I32, I32, I32], I64),
}

_LIB = None


class CcvError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


def load():
    """Load libccv.so once.  Raises if it has not been built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"libccv.so is not built ({LIB_PATH} missing); build it with "
                "`python -c 'import __graft_entry__ as g; g.build()'`")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in (*SIGNATURES.items(), *LAYER_SIGNATURES.items()):
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _LIB = lib
    return _LIB


def status_string(status: int) -> str:
    return load().ccv_status_string(int(status)).decode()


def declared_functions(header: str = HEADER):
    """Names of the functions declared in include/ccv.h (or the given header)."""
    text = open(header).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(\w+)\s*\(", text, flags=re.M)
