"""ctypes declarations of libcpattn.so (the C ABI in include/cp_attn.h).

Loading fails loudly when the library has not been built: there is no other
implementation of these calls.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import threading

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "lib", "libcpattn.so")

# status codes (cp_status)
CP_OK = 0
CP_ERR_INVALID_ARG = -1
CP_ERR_NOT_DIVISIBLE = -2
CP_ERR_UNSUPPORTED_COMBO = -3
CP_ERR_ALIGNMENT = -4
CP_ERR_CUDA = -5
CP_ERR_TIMEOUT = -6
CP_ERR_WORKSPACE = -7
CP_ERR_UNSUPPORTED_DEVICE = -8

CP_BF16 = 0
CP_F32 = 1
CP_LAP_FUSED = 0
CP_LAP_STEPWISE = 1

class ScoreRule(ctypes.Structure):
    """cp_score_rule."""
    _fields_ = [("softcap", ctypes.c_float), ("slopes", ctypes.c_void_p), ("causal", ctypes.c_int),
                ("prefix_lens", ctypes.c_void_p), ("q_docs", ctypes.c_void_p), ("kv_docs", ctypes.c_void_p),
                ("q_pos0", ctypes.c_int64), ("kv_pos0", ctypes.c_int64)]


class QkRule(ctypes.Structure):
    """cp_qk_rule."""
    _fields_ = [("norm", ctypes.c_int), ("eps", ctypes.c_float), ("q_weight", ctypes.c_void_p),
                ("k_weight", ctypes.c_void_p), ("weight_dt", ctypes.c_int), ("pairs", ctypes.c_int),
                ("interleaved", ctypes.c_int), ("freqs", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("positions_shared", ctypes.c_int), ("axes", ctypes.c_int), ("pair_axis", ctypes.c_char_p)]


class Q4Cache(ctypes.Structure):
    """cp_q4_cache."""
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("block_table", ctypes.c_void_p), ("num_pages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("max_pages", ctypes.c_int)]


# every symbol include/cp_attn.h declares, with (restype, argtypes)
_vp, _i, _i64, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
_ip = ctypes.POINTER(ctypes.c_int)
_rule = ctypes.POINTER(ScoreRule)
_qk = ctypes.POINTER(QkRule)
_q4 = ctypes.POINTER(Q4Cache)
_i64p = ctypes.POINTER(ctypes.c_int64)
SIGNATURES = {
    "cp_status_string": (ctypes.c_char_p, [_i]),
    "cp_version": (_i, []),
    "cp_block_attn_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i64, _i64, _i64, _i, _vp]),
    "cp_lse_merge": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp]),
    "cp_ulysses_seq2head": (_i, [_vp, _vp, _i, _i, _i, _i, _i, _i, _vp]),
    "cp_ulysses_head2seq": (_i, [_vp, _vp, _i, _i, _i, _i, _i, _i, _vp]),
    "cp_ulysses_anything_seq2head": (_i, [_vp, _vp, _i, _i, _i, _i, _i, _i, _vp]),
    "cp_ulysses_anything_head2seq": (_i, [_vp, _vp, _i, _i, _i, _i, _i, _i, _vp]),
    "cp_attention_validate": (_i, [_i, _i, _i, _i, _i, _i, _i, _i]),
    "cp_ring_shard_table": (_i, [_i, _i, _i, _ip, _ip]),
    "cp_attention_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i, _i, _i]),
    "cp_attention_launch_count": (_i, [_i, _i, _i, _i, _i, _i, _i, _i]),
    "cp_attention_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _i, _i, _vp, _sz, _i, _i, _vp]),
    "cp_check_device_status": (_i, [_vp]),
    "cp_debug_bounded_wait_probe": (_i, [_i, _vp]),
    "cp_attention_fwd_no_alloc": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _i, _i, _i, _i, _vp]),
    "cp_attention_host_buffer_size": (_sz, [_i, _i, _i, _i, _i, _i, _i, _i]),
    "cp_attention_fwd_masked": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _i, _i, _vp, _sz, _i, _i,
                                     _vp]),
    "cp_attention_fwd_host": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _i, _i, _vp, _sz, _i, _i, _i,
                                   _vp]),
    "cp_attention_bwd_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i, _i]),
    "cp_attention_bwd_launch_count": (_i, [_i, _i, _i, _i, _i, _i, _i]),
    "cp_attention_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _i, _i, _vp, _sz,
                              _i, _vp]),
    "cp_scored_attn_validate": (_i, [_i, _i, _i, _i, _i, _i, _f, _rule, _i]),
    "cp_scored_attn_workspace_size": (_sz, [_i, _i, _i, _i, _i]),
    "cp_scored_attn_bwd_workspace_size": (_sz, [_i, _i, _i, _i, _i]),
    "cp_scored_attn_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _rule, _vp, _sz, _i, _i, _vp]),
    "cp_scored_attn_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _rule, _vp,
                                _sz, _i, _i, _i, _vp]),
    "cp_paged_kv_append": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i, _vp]),
    "cp_paged_attn_workspace_size": (_sz, [_i, _i, _i, _i, _i]),
    "cp_paged_attn_workspace_size_for": (_sz, [_i, _i, _i, _i, _i, _i, _i]),
    "cp_paged_attn_decode": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _f, _vp, _vp, _sz,
                                  _i, _i, _vp]),
    "cp_qk_norm_rope_fwd": (_i, [_vp, _vp, _vp, _vp, _i64p, _i, _i, _i, _i, _i, _qk, _i, _vp]),
    "cp_qk_norm_rope_bwd_workspace_size": (_sz, [_i]),
    "cp_qk_norm_rope_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64p, _i, _i, _i, _i, _i, _qk, _vp, _sz, _i, _i,
                                 _vp]),
    "cp_paged_kv_append_q4": (_i, [_vp, _vp, _q4, _vp, _vp, _i, _i, _i, _i, _i, _vp]),
    "cp_paged_kv_read_q4": (_i, [_q4, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp]),
    "cp_paged_attn_q4_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i, _i]),
    "cp_paged_attn_decode_q4": (_i, [_vp, _q4, _vp, _vp, _vp, _i, _i, _i, _i, _f, _f, _vp, _vp, _sz, _i, _i, _vp]),
}
CP_NO_ALLOC_WORKSPACE_BYTES = 64 * 1024 * 1024

_lock = threading.RLock()
_lib = None
_bind = None


class CpError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                if not os.path.exists(LIB_PATH):
                    raise RuntimeError(
                        f"libcpattn.so is not built ({LIB_PATH}); run "
                        "`python -m context_attention_dits_gb300.build`")
                L = ctypes.CDLL(LIB_PATH)
                for name, (res, args) in SIGNATURES.items():
                    fn = getattr(L, name)
                    fn.restype = res
                    fn.argtypes = args
                _lib = L
    return _lib


def bind():
    """The compiled marshalling of the calls whose host time counts, over the library that lib() loads."""
    global _bind
    if _bind is None:
        with _lock:
            if _bind is None:
                from .build import bind_path
                path = bind_path()  # (torch is loaded now, and with it the libraries that the module needs)
                if path is None:
                    raise RuntimeError("these calls need a torch for CUDA")
                if not os.path.exists(path):
                    raise RuntimeError(f"the compiled marshalling is not built for this torch ({path}); run "
                                       "`python -m context_attention_dits_gb300.build`")
                spec = importlib.util.spec_from_file_location("_cpbind", path)
                module = importlib.util.module_from_spec(spec)
                spec.loader.exec_module(module)
                module.init(lib()._handle)
                _bind = module
    return _bind


def status_string(status: int) -> str:
    return lib().cp_status_string(int(status)).decode()


def check(status: int, where: str) -> None:
    if status != CP_OK:
        raise CpError(status, where)
