"""ctypes binding of libmxscale's C ABI (include/mxscale.h).

Argument marshalling only: every step of the rearrange runs in the library's
CUDA kernels.  The library is loaded from this package directory; if it is
missing the first call raises, there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import re
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmxscale.so")
HEADER = os.path.join(os.path.dirname(PKG), "include", "mxscale.h")

MX_OK, MX_ERR_INVALID_ARG, MX_ERR_MISALIGNED, MX_ERR_UNSUPPORTED, MX_ERR_CUDA = range(5)
MX_GROUPS_M, MX_GROUPS_K = 0, 1
MX_PATH_AUTO, MX_PATH_TMA, MX_PATH_WORD, MX_PATH_BYTE, MX_PATH_FLAT = range(5)
MX_MAX_GROUPS = 64
PATHS = {"auto": MX_PATH_AUTO, "tma": MX_PATH_TMA, "word": MX_PATH_WORD, "byte": MX_PATH_BYTE,
         "flat": MX_PATH_FLAT}
PATH_NAMES = {v: k for k, v in PATHS.items()}

MX_F32, MX_BF16, MX_F16, MX_E4M3, MX_E5M2 = range(5)
MX_TILES_NONE, MX_TILES_NARROW, MX_TILES_SPLIT_2, MX_TILES_SPLIT_4, MX_TILES_SPLIT_8 = 0, 1, 2, 4, 8
MX_TILES_WIDE, MX_TILES_PAIRS, MX_TILES_PAIRS_ACROSS = 16, 32, 33
MX_B_NK, MX_B_KN = 0, 1
B_LAYOUTS = {"nk": MX_B_NK, "kn": MX_B_KN}

_lock = threading.Lock()
_lib = None

_I64, _I32, _P, _U32P = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.POINTER(ctypes.c_uint32)

_SIGNATURES = {
    "mx_rearranged_size": (ctypes.c_size_t, [ctypes.c_int, _I64, _I64, _I32]),
    "mx_rearrange_m_groups": (ctypes.c_int, [_P, _I64, _I64, _I64, _P, _I32, _P, _P]),
    "mx_rearrange_k_groups": (ctypes.c_int, [_P, _I64, _I64, _I64, _P, _I32, _P, _P]),
    "mx_rearrange_ex": (ctypes.c_int, [ctypes.c_int, _P, _I64, _I64, _I64, _P, _I32, _P, ctypes.c_int, _P]),
    "mx_select_path": (ctypes.c_int, [ctypes.c_int, _P, _I64, _I64, _I64]),
    "mx_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "mx_device_flags": (ctypes.c_int, [_U32P, ctypes.c_int]),
    "mx_selftest_bounded_wait": (ctypes.c_int, [_I64, _P]),
    "mx_unrearrange_m_groups": (ctypes.c_int, [_P, _I64, _I64, _P, _I32, _P, _I64, _P]),
    "mx_unrearrange_k_groups": (ctypes.c_int, [_P, _I64, _I64, _P, _I32, _P, _I64, _P]),
    "mx_padded_group_starts": (ctypes.c_int, [ctypes.c_int, _I64, _I64, _P, _I32, _P, _P]),
    "mx_expert_sort_workspace": (ctypes.c_size_t, [_I64, _I32]),
    "mx_expert_sort": (ctypes.c_int, [_P, _I32, _I64, _I32, _I32, _P, _P, _P, _P, _P]),
    "mx_dispatch_rows": (ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _I64, _P, _I32, _P, _I32, _P, _I64, _P]),
    "mx_combine_rows": (ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _I64, _P, _I32, _P, _P, _I64, _P]),
    "mx_combine_rows_backward": (ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _I64, _P, _I64, _P, _I32, _P, _I32, _P,
                                                _P, _I64, _P, _P]),
    "mx_quantize_rows": (ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _I64, _I32, ctypes.c_int, _P, _I32, _P, _I32, _P,
                                        _I64, _P, _I64, _I64, _P]),
    "mx_padded_rows": (_I64, [_I64, _I32]),
    "mx_quantize_cols": (ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _I64, _P, _I32, ctypes.c_int, _P, _I64, _P, _I64,
                                        _P]),
    "mx_quantize_blocks": (ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _I64, _I64, _I64, ctypes.c_int, _P, _I64, _I64,
                                          _P, _P]),
    "mx_grouped_matmul_m": (ctypes.c_int, [_P, ctypes.c_int, _I64, _P, _I64, _I64, _P, ctypes.c_int, ctypes.c_int, _I64,
                                           _I64, _P, _I64, _I64, _I64, _I32, _I64, _I64, _I64, _P, _I32, _P,
                                           ctypes.c_int, _I64, _P]),
    "mx_grouped_matmul_k": (ctypes.c_int, [_P, ctypes.c_int, _I64, _P, _I64, _P, ctypes.c_int, _I64, _P, _I64, _I64,
                                           _I64, _I64, _P, _I32, _P, ctypes.c_int, _I64, _I64, _P]),
    "mx_select_tiles": (ctypes.c_int, [ctypes.c_int, _I64, _I64, _I64, _I32, _I32]),
    "mx_last_cuda_error": (ctypes.c_int, []),
    "mx_version": (ctypes.c_int, []),
}


class MxError(RuntimeError):
    def __init__(self, where: str, status: int):
        extra = f", CUDA error {mx_last_cuda_error()}" if status == MX_ERR_CUDA else ""
        super().__init__(f"{where}: {status_string(status)} (status {status}{extra})")
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                if not os.path.exists(LIB_PATH):
                    raise RuntimeError(
                        f"libmxscale.so is missing at {LIB_PATH}; build it with "
                        "`python -m scale_factor_layout_b200._build` (nvcc, sm_100a)")
                handle = ctypes.CDLL(LIB_PATH)
                for name, (res, args) in _SIGNATURES.items():
                    f = getattr(handle, name)
                    f.restype, f.argtypes = res, args
                _lib = handle
    return _lib


def declared_symbols(header: str = HEADER):
    """Function names declared in include/mxscale.h."""
    text = open(header).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(mx_[a-z_0-9]+)\s*\(", text)))


def status_string(status: int) -> str:
    return lib().mx_status_string(status).decode()


def mx_rearranged_size(dim: int, rows: int, cols: int, num_groups: int) -> int:
    return int(lib().mx_rearranged_size(dim, rows, cols, num_groups))


def mx_rearrange_m_groups(scales: int, rows: int, cols: int, row_stride: int, group_end_offsets: int,
                          num_groups: int, out: int, stream: int) -> int:
    return lib().mx_rearrange_m_groups(scales, rows, cols, row_stride, group_end_offsets, num_groups, out, stream)


def mx_rearrange_k_groups(scales: int, rows: int, cols: int, row_stride: int, group_end_offsets: int,
                          num_groups: int, out: int, stream: int) -> int:
    return lib().mx_rearrange_k_groups(scales, rows, cols, row_stride, group_end_offsets, num_groups, out, stream)


def mx_rearrange_ex(dim: int, scales: int, rows: int, cols: int, row_stride: int, group_end_offsets: int,
                    num_groups: int, out: int, path: int, stream: int) -> int:
    return lib().mx_rearrange_ex(dim, scales, rows, cols, row_stride, group_end_offsets, num_groups, out,
                                 path, stream)


def mx_unrearrange_m_groups(blocked: int, rows: int, cols: int, group_end_offsets: int, num_groups: int,
                            scales: int, row_stride: int, stream: int) -> int:
    return lib().mx_unrearrange_m_groups(blocked, rows, cols, group_end_offsets, num_groups, scales, row_stride,
                                         stream)


def mx_unrearrange_k_groups(blocked: int, rows: int, cols: int, group_end_offsets: int, num_groups: int,
                            scales: int, row_stride: int, stream: int) -> int:
    return lib().mx_unrearrange_k_groups(blocked, rows, cols, group_end_offsets, num_groups, scales, row_stride,
                                         stream)


def mx_padded_group_starts(dim: int, rows: int, cols: int, group_end_offsets: int, num_groups: int, starts: int,
                           stream: int) -> int:
    return lib().mx_padded_group_starts(dim, rows, cols, group_end_offsets, num_groups, starts, stream)


def mx_select_path(dim: int, scales: int, rows: int, cols: int, row_stride: int) -> int:
    return int(lib().mx_select_path(dim, scales, rows, cols, row_stride))


def mx_device_flags(clear: bool = False) -> int:
    v = ctypes.c_uint32(0)
    st = lib().mx_device_flags(ctypes.byref(v), 1 if clear else 0)
    if st != MX_OK:
        raise MxError("mx_device_flags", st)
    return int(v.value)


def mx_selftest_bounded_wait(limit_cycles: int, stream: int = 0) -> int:
    return lib().mx_selftest_bounded_wait(limit_cycles, stream)


def mx_last_cuda_error() -> int:
    return int(lib().mx_last_cuda_error())


def mx_version() -> int:
    return int(lib().mx_version())


def mx_expert_sort_workspace(tokens: int, choices: int) -> int:
    return int(lib().mx_expert_sort_workspace(tokens, choices))


def mx_expert_sort(expert_ids: int, id_bytes: int, tokens: int, choices: int, num_experts: int, group_ends: int,
                   row_of_slot: int, slot_of_row: int, workspace: int, stream: int) -> int:
    return lib().mx_expert_sort(expert_ids, id_bytes, tokens, choices, num_experts, group_ends, row_of_slot,
                                slot_of_row, workspace, stream)


def mx_dispatch_rows(x: int, dtype: int, tokens: int, cols: int, x_stride: int, row_of_slot: int, choices: int,
                     group_ends: int, num_experts: int, out: int, out_stride: int, stream: int) -> int:
    return lib().mx_dispatch_rows(x, dtype, tokens, cols, x_stride, row_of_slot, choices, group_ends, num_experts, out,
                                  out_stride, stream)


def mx_combine_rows(rows: int, dtype: int, tokens: int, cols: int, rows_stride: int, row_of_slot: int, choices: int,
                    weights: int, y: int, y_stride: int, stream: int) -> int:
    return lib().mx_combine_rows(rows, dtype, tokens, cols, rows_stride, row_of_slot, choices, weights, y, y_stride,
                                 stream)


def mx_combine_rows_backward(grad: int, dtype: int, tokens: int, cols: int, grad_stride: int, rows: int,
                             rows_stride: int, row_of_slot: int, choices: int, group_ends: int, num_experts: int,
                             weights: int, d_rows: int, d_rows_stride: int, d_weights: int, stream: int) -> int:
    return lib().mx_combine_rows_backward(grad, dtype, tokens, cols, grad_stride, rows, rows_stride, row_of_slot,
                                          choices, group_ends, num_experts, weights, d_rows, d_rows_stride, d_weights,
                                          stream)


def mx_quantize_rows(x: int, dtype: int, rows: int, cols: int, x_stride: int, block: int, out_dtype: int,
                     row_of_slot: int, choices: int, group_ends: int, num_experts: int, q: int, q_stride: int,
                     scales: int, scale_row_stride: int, scale_block_stride: int, stream: int) -> int:
    return lib().mx_quantize_rows(x, dtype, rows, cols, x_stride, block, out_dtype, row_of_slot, choices, group_ends,
                                  num_experts, q, q_stride, scales, scale_row_stride, scale_block_stride, stream)


def mx_padded_rows(rows: int, num_groups: int) -> int:
    return int(lib().mx_padded_rows(rows, num_groups))


def mx_quantize_cols(x: int, dtype: int, rows: int, cols: int, x_stride: int, group_ends: int, num_groups: int,
                     out_dtype: int, q: int, q_stride: int, scales: int, scale_stride: int, stream: int) -> int:
    return lib().mx_quantize_cols(x, dtype, rows, cols, x_stride, group_ends, num_groups, out_dtype, q, q_stride,
                                  scales, scale_stride, stream)


def mx_quantize_blocks(x: int, dtype: int, groups: int, rows: int, cols: int, x_group_stride: int, x_stride: int,
                       out_dtype: int, q: int, q_group_stride: int, q_stride: int, scales: int, stream: int) -> int:
    return lib().mx_quantize_blocks(x, dtype, groups, rows, cols, x_group_stride, x_stride, out_dtype, q,
                                    q_group_stride, q_stride, scales, stream)


def mx_grouped_matmul_m(a: int, a_dtype: int, a_stride: int, a_scales: int, a_scale_row_stride: int,
                        a_scale_block_stride: int, b: int, b_dtype: int, b_layout: int, b_group_stride: int,
                        b_stride: int, b_scales: int, b_scale_group_stride: int, b_scale_n_stride: int,
                        b_scale_k_stride: int, block: int, rows: int, n: int, k: int, group_ends: int,
                        num_groups: int, out: int, out_dtype: int, out_stride: int, stream: int) -> int:
    return lib().mx_grouped_matmul_m(a, a_dtype, a_stride, a_scales, a_scale_row_stride, a_scale_block_stride, b,
                                     b_dtype, b_layout, b_group_stride, b_stride, b_scales, b_scale_group_stride,
                                     b_scale_n_stride, b_scale_k_stride, block, rows, n, k, group_ends, num_groups,
                                     out, out_dtype, out_stride, stream)


def mx_grouped_matmul_k(a: int, a_dtype: int, a_stride: int, a_scales: int, a_scale_stride: int, b: int, b_dtype: int,
                        b_stride: int, b_scales: int, b_scale_stride: int, padded_rows: int, m: int, n: int,
                        group_ends: int, num_groups: int, out: int, out_dtype: int, out_group_stride: int,
                        out_stride: int, stream: int) -> int:
    return lib().mx_grouped_matmul_k(a, a_dtype, a_stride, a_scales, a_scale_stride, b, b_dtype, b_stride, b_scales,
                                     b_scale_stride, padded_rows, m, n, group_ends, num_groups, out, out_dtype,
                                     out_group_stride, out_stride, stream)


def mx_select_tiles(dim: int, m: int, n: int, k: int, num_groups: int, sms: int) -> int:
    return int(lib().mx_select_tiles(dim, m, n, k, num_groups, sms))
