"""Mixture-of-experts operators on torch tensors.

Slots (token, choice) sorted by expert, token rows copied into expert order and
summed back with their weights, 8-bit quantization with a power-of-two scale
for each block, and the grouped 8-bit product that reads those scales.  A
forward pass of an expert layer and its weight:

    order  = expert_sort(expert_ids, num_experts)
    q, s   = quantize_rows(x, order=order)              # tokens to experts, in 8 bits
    wq, ws = quantize_blocks(weight)                    # [G, n, k], once
    rows   = grouped_matmul(q, s, wq, ws, order.group_ends)
    y      = combine_rows(rows, order, weights)

and its backward pass:

    d_rows, d_weights = combine_rows_backward(grad, rows, order, weights)
    dq, ds = quantize_rows(d_rows, dtype=torch.float8_e5m2)
    d_x_rows = grouped_matmul(dq, ds, wq, ws, order.group_ends, b_layout="kn")
    d_x    = combine_rows(d_x_rows, order)
    d_weight = grouped_matmul_k(*quantize_cols(d_rows, order.group_ends, dtype=torch.float8_e5m2),
                                *quantize_cols(dispatch_rows(x, order), order.group_ends), order.group_ends)

``dispatch_rows`` and ``combine_rows`` are differentiable, backward and once;
forward-mode derivatives raise.  The other calls take no part in
differentiation: their results carry no gradient, whatever their inputs do.
All calls run on torch's current stream of the tensors' device, allocate their
outputs with torch and may be captured in a CUDA graph (after one call on the
device).  An ``out`` that is given must not overlap an input.
"""
from __future__ import annotations

import functools
import math
from typing import NamedTuple

import torch
from torch.autograd import forward_ad

from . import _binding as B

FLOATS = {torch.float32: B.MX_F32, torch.bfloat16: B.MX_BF16, torch.float16: B.MX_F16}
EIGHT_BIT = {torch.float8_e4m3fn: B.MX_E4M3, torch.float8_e5m2: B.MX_E5M2}
MAX_SLOTS = 2**31 - 2**14   # the library's largest extent; choices go into it as 32-bit numbers


class ExpertOrder(NamedTuple):
    """Where the slots of [tokens, choices] went: ``group_ends`` int32[experts]
    (cumulative rows), ``row_of_slot`` int32[tokens, choices] (-1: no row) and
    ``slot_of_row`` int32[tokens * choices] (-1 behind the last group)."""

    group_ends: torch.Tensor
    row_of_slot: torch.Tensor
    slot_of_row: torch.Tensor


def _up(n: int, m: int) -> int:
    return -(-n // m) * m


_entries: dict = {}


def _call(name: str, device: torch.device, *args) -> None:
    """An entry point on torch's current stream of ``device``.  These calls take
    less time on the GPU than in Python when they are small, so they go to the
    library's functions directly."""
    fn = _entries.get(name)
    if fn is None:
        fn = _entries[name] = getattr(B.lib(), name)
    index = device.index
    stream = torch._C._cuda_getCurrentRawStream(index)
    if index == torch._C._cuda_getDevice():
        st = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            st = fn(*args, stream)
    if st != B.MX_OK:
        raise B.MxError(name, st)


def _check_cuda(**tensors) -> None:
    device = None
    for name, t in tensors.items():
        if t is None:
            continue
        at = t.get_device()
        if at < 0:
            raise ValueError(f"{name} must be a CUDA tensor")
        if device is None:
            device = at
        elif at != device:
            raise ValueError(f"{name} is on {t.device}, the other tensors on cuda:{device}")


def _check_matrix(name: str, t: torch.Tensor, dtypes) -> None:
    if t.dim() != 2 or t.dtype not in dtypes:
        raise ValueError(f"{name} must be a 2-D tensor of {', '.join(str(d) for d in dtypes)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must be dense along columns (stride(1) == 1)")


def _row_stride(t: torch.Tensor, multiple: int = 1) -> int:
    """Elements between rows; of a single row, any that suits."""
    return t.stride(-2) if t.shape[-2] > 1 else _up(max(t.shape[-1], 1), multiple)


def _check_ends(name: str, t: torch.Tensor) -> None:
    if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 1-D int32 tensor")
    if not 1 <= t.numel() <= B.MX_MAX_GROUPS:
        raise ValueError(f"{name} must hold 1 to {B.MX_MAX_GROUPS} groups")


def _check_order(order: ExpertOrder) -> None:
    _check_ends("order.group_ends", order.group_ends)
    r = order.row_of_slot
    if r.dtype != torch.int32 or r.dim() != 2 or not r.is_contiguous() or r.shape[1] < 1:
        raise ValueError("order.row_of_slot must be a contiguous int32 tensor [tokens, choices]")
    if r.numel() > MAX_SLOTS:
        raise ValueError(f"order.row_of_slot must hold at most {MAX_SLOTS} slots")


def _wants_derivative(t: torch.Tensor, u: torch.Tensor | None = None) -> bool:
    """Whether a result has to go through an autograd function.  A tangent of forward
    mode has to as well: the functions have no rule for it, so that it raises there."""
    if torch.is_grad_enabled() and (t.requires_grad or (u is not None and u.requires_grad)):
        return True
    return forward_ad._current_level >= 0 and (forward_ad.unpack_dual(t).tangent is not None or (
        u is not None and forward_ad.unpack_dual(u).tangent is not None))


def _check_out(out: torch.Tensor, shape, dtypes) -> None:
    if tuple(out.shape) != tuple(shape) or out.dtype not in dtypes or (shape[-1] > 1 and out.stride(-1) != 1):
        raise ValueError(f"out must be a {', '.join(str(d) for d in dtypes)} tensor of shape {tuple(shape)}, "
                         "dense along columns")
    if _wants_derivative(out):
        raise ValueError("out cannot be a tensor that needs a gradient")


def _overlap(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Whether two tensors may share a byte: their spans do, and they are not columns
    of one matrix beside each other."""
    if not a.numel() or not b.numel():
        return False
    es, fs = a.element_size(), b.element_size()
    span_a = (sum((n - 1) * s for n, s in zip(a.shape, a.stride())) + 1) * es
    span_b = (sum((n - 1) * s for n, s in zip(b.shape, b.stride())) + 1) * fs
    p, q = a.data_ptr(), b.data_ptr()
    if p + span_a <= q or q + span_b <= p:
        return False
    # rows start at multiples of `pitch` from the first one's start
    pitch = math.gcd(*(s * es for n, s in zip(a.shape[:-1], a.stride()) if n > 1),
                     *(s * fs for n, s in zip(b.shape[:-1], b.stride()) if n > 1))
    if pitch == 0:
        return True
    at = (q - p) % pitch
    return at < ((a.shape[-1] - 1) * a.stride(-1) + 1) * es or at + ((b.shape[-1] - 1) * b.stride(-1) + 1) * fs > pitch


def _check_apart(out: torch.Tensor, **inputs) -> None:
    for name, t in inputs.items():
        if t is not None and _overlap(out, t):
            raise ValueError(f"out overlaps {name}")


def _written(out: torch.Tensor) -> torch.Tensor:
    """A caller's tensor after a kernel has been launched that writes it: autograd is told."""
    if not out.is_inference():
        torch.autograd.graph.increment_version(out)
    return out


@functools.lru_cache(maxsize=1024)
def _sort_workspace(tokens: int, choices: int) -> int:
    return B.mx_expert_sort_workspace(tokens, choices)


def expert_sort(expert_ids: torch.Tensor, num_experts: int) -> ExpertOrder:
    """Sort the slots of ``expert_ids`` (int32 or int64 [tokens, choices]) by
    expert, stable; ids outside [0, num_experts) get no row."""
    if expert_ids.dim() != 2 or expert_ids.dtype not in (torch.int32, torch.int64) or not expert_ids.is_contiguous():
        raise ValueError("expert_ids must be a contiguous int32 or int64 tensor [tokens, choices]")
    if not 1 <= num_experts <= B.MX_MAX_GROUPS:
        raise ValueError(f"num_experts must be 1 to {B.MX_MAX_GROUPS}")
    _check_cuda(expert_ids=expert_ids)
    T, k = expert_ids.shape
    if k < 1:
        raise ValueError("expert_ids must have at least one choice a token")
    dev, i32, S = expert_ids.device, torch.int32, T * k
    if S > MAX_SLOTS:
        raise ValueError(f"expert_ids must hold at most {MAX_SLOTS} slots")
    ends = torch.empty_strided((num_experts,), (1,), dtype=i32, device=dev)
    row_of_slot = torch.empty_strided((T, k), (k, 1), dtype=i32, device=dev)
    slot_of_row = torch.empty_strided((S,), (1,), dtype=i32, device=dev)
    need = _sort_workspace(T, k)
    # held until both kernels are on the stream: from then on whoever gets this memory on the same stream comes after
    # them, but a thread that shares the stream could be given it between them
    workspace = torch.empty_strided((need,), (1,), dtype=torch.uint8, device=dev) if need else None
    _call("mx_expert_sort", dev, expert_ids.data_ptr(), 4 if expert_ids.dtype == i32 else 8, T, k, num_experts,
          ends.data_ptr(), row_of_slot.data_ptr(), slot_of_row.data_ptr(), workspace.data_ptr() if need else 0)
    return ExpertOrder(ends, row_of_slot, slot_of_row)


# ------------------------------------------------------------------ rows to experts and back
def _dispatch(x, order, out=None):
    T, k = order.row_of_slot.shape
    y = x.new_empty(T * k, x.shape[1]) if out is None else out
    _call("mx_dispatch_rows", x.device, x.data_ptr(), FLOATS[x.dtype], T, x.shape[1], _row_stride(x),
          order.row_of_slot.data_ptr(), k, order.group_ends.data_ptr(), order.group_ends.numel(), y.data_ptr(),
          _row_stride(y))
    return y if out is None else _written(out)


def _combine(rows, order, weights, out=None):
    T, k = order.row_of_slot.shape
    y = rows.new_empty(T, rows.shape[1]) if out is None else out
    _call("mx_combine_rows", rows.device, rows.data_ptr(), FLOATS[rows.dtype], T, rows.shape[1], _row_stride(rows),
          order.row_of_slot.data_ptr(), k, 0 if weights is None else weights.data_ptr(), y.data_ptr(), _row_stride(y))
    return y if out is None else _written(out)


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, group_ends, row_of_slot, slot_of_row):
        ctx.save_for_backward(group_ends, row_of_slot, slot_of_row)
        return _dispatch(x, ExpertOrder(group_ends, row_of_slot, slot_of_row))

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        return _combine(grad.contiguous(), ExpertOrder(*ctx.saved_tensors), None), None, None, None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, weights, group_ends, row_of_slot, slot_of_row):
        ctx.weighted = weights is not None
        ctx.save_for_backward(group_ends, row_of_slot, slot_of_row, *((rows, weights) if ctx.weighted else ()))
        return _combine(rows, ExpertOrder(group_ends, row_of_slot, slot_of_row), weights)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        order = ExpertOrder(*ctx.saved_tensors[:3])
        grad = grad.contiguous()
        if not ctx.weighted:
            return _dispatch(grad, order), None, None, None, None
        d_rows, d_weights = combine_rows_backward(grad, ctx.saved_tensors[3], order, ctx.saved_tensors[4])
        return d_rows, d_weights, None, None, None


def dispatch_rows(x: torch.Tensor, order: ExpertOrder, out: torch.Tensor | None = None) -> torch.Tensor:
    """Token rows ``x`` [tokens, cols] in expert order: [tokens * choices, cols],
    zeros behind the last group.  Differentiable in x (without ``out``)."""
    _check_matrix("x", x, FLOATS)
    _check_order(order)
    _check_cuda(x=x, group_ends=order.group_ends, row_of_slot=order.row_of_slot, out=out)
    T, k = order.row_of_slot.shape
    if x.shape[0] != T:
        raise ValueError(f"x has {x.shape[0]} rows, the order {T} tokens")
    wants_grad = _wants_derivative(x)
    if out is not None:
        if wants_grad:
            raise ValueError("out cannot be given where a gradient is wanted")
        _check_out(out, (T * k, x.shape[1]), (x.dtype,))
        _check_apart(out, x=x, group_ends=order.group_ends, row_of_slot=order.row_of_slot)
    return _Dispatch.apply(x, *order) if wants_grad else _dispatch(x, order, out)


def _check_rows_of(order: ExpertOrder, rows: torch.Tensor) -> None:
    if rows.shape[0] != order.row_of_slot.numel():
        raise ValueError(f"rows has {rows.shape[0]} rows, the order {order.row_of_slot.numel()} slots")


def _check_weights(order: ExpertOrder, weights: torch.Tensor) -> None:
    if weights.dtype != torch.float32 or weights.shape != order.row_of_slot.shape or not weights.is_contiguous():
        raise ValueError("weights must be a contiguous float32 tensor [tokens, choices]")


def combine_rows(rows: torch.Tensor, order: ExpertOrder, weights: torch.Tensor | None = None,
                 out: torch.Tensor | None = None) -> torch.Tensor:
    """The sum of each token's rows, times ``weights`` (float32 [tokens, choices])
    if given: [tokens, cols].  Slots without a row add nothing.  Differentiable
    in rows and weights (without ``out``); without weights it is the gradient of
    ``dispatch_rows``."""
    _check_matrix("rows", rows, FLOATS)
    _check_order(order)
    _check_cuda(rows=rows, group_ends=order.group_ends, row_of_slot=order.row_of_slot, weights=weights, out=out)
    _check_rows_of(order, rows)
    if weights is not None:
        _check_weights(order, weights)
    wants_grad = _wants_derivative(rows, weights)
    if out is not None:
        if wants_grad:
            raise ValueError("out cannot be given where a gradient is wanted")
        _check_out(out, (order.row_of_slot.shape[0], rows.shape[1]), (rows.dtype,))
        _check_apart(out, rows=rows, row_of_slot=order.row_of_slot, weights=weights)
    return _Combine.apply(rows, weights, *order) if wants_grad else _combine(rows, order, weights, out)


def combine_rows_backward(grad: torch.Tensor, rows: torch.Tensor, order: ExpertOrder, weights: torch.Tensor):
    """Gradients of ``combine_rows``: (d_rows like rows, d_weights float32 [tokens, choices])."""
    _check_matrix("grad", grad, FLOATS)
    _check_matrix("rows", rows, FLOATS)
    _check_order(order)
    _check_weights(order, weights)
    _check_cuda(grad=grad, rows=rows, group_ends=order.group_ends, row_of_slot=order.row_of_slot, weights=weights)
    _check_rows_of(order, rows)
    T, k = order.row_of_slot.shape
    if grad.dtype != rows.dtype or tuple(grad.shape) != (T, rows.shape[1]):
        raise ValueError(f"grad must be a {rows.dtype} tensor of shape ({T}, {rows.shape[1]})")
    d_rows = rows.new_empty(T * k, rows.shape[1])
    if rows.shape[1] == 0:
        return d_rows, torch.zeros_like(weights)
    d_weights = torch.empty_like(weights)
    _call("mx_combine_rows_backward", rows.device, grad.data_ptr(), FLOATS[rows.dtype], T, rows.shape[1],
          _row_stride(grad), rows.data_ptr(), _row_stride(rows), order.row_of_slot.data_ptr(), k,
          order.group_ends.data_ptr(), order.group_ends.numel(), weights.data_ptr(), d_rows.data_ptr(),
          _row_stride(d_rows), d_weights.data_ptr())
    return d_rows, d_weights


# ------------------------------------------------------------------ quantization
def _eight_bit_rows(shape, dtype, device) -> torch.Tensor:
    """8-bit rows that start on 16-byte boundaries, as the product reads them."""
    stride = _up(shape[-1], 16)
    strides = (stride, 1) if len(shape) == 2 else (shape[1] * stride, stride, 1)
    return torch.empty_strided(shape, strides, dtype=dtype, device=device)


def _check_eight_bit(dtype) -> None:
    if dtype not in EIGHT_BIT:
        raise ValueError("dtype must be torch.float8_e4m3fn or torch.float8_e5m2")


def quantize_rows(x: torch.Tensor, block: int = 128, dtype: torch.dtype = torch.float8_e4m3fn,
                  order: ExpertOrder | None = None):
    """``x`` [rows, cols] in 8 bits with one scale for each ``block`` (128 or 32)
    columns of a row: (values [rows, cols], E8M0 bytes uint8 [rows, blocks]).
    With ``order`` the rows are tokens and the result is that of
    ``quantize_rows(dispatch_rows(x, order))``, in one pass.  Scales of 128 lie
    block by block in memory (strides (1, rows)), those of 32 row by row, as
    ``rearrange_m_groups`` reads them."""
    _check_matrix("x", x, FLOATS)
    _check_eight_bit(dtype)
    if block not in (32, 128):
        raise ValueError("block must be 128 or 32")
    rows, cols = x.shape
    slots, k, ends, G = 0, 0, 0, 0
    _check_cuda(x=x, **({} if order is None else {"group_ends": order.group_ends, "row_of_slot": order.row_of_slot}))
    out_rows = rows
    if order is not None:
        _check_order(order)
        if order.row_of_slot.shape[0] != rows:
            raise ValueError(f"x has {rows} rows, the order {order.row_of_slot.shape[0]} tokens")
        k = order.row_of_slot.shape[1]
        slots, ends, G = order.row_of_slot.data_ptr(), order.group_ends.data_ptr(), order.group_ends.numel()
        out_rows = rows * k
    q = _eight_bit_rows((out_rows, cols), dtype, x.device)
    blocks = _up(cols, block) // block
    if block == 128:
        row_stride, block_stride = 1, out_rows
    else:
        row_stride, block_stride = blocks, 1
    scales = torch.empty_strided((out_rows, blocks), (row_stride, block_stride), dtype=torch.uint8, device=x.device)
    if out_rows and cols:
        _call("mx_quantize_rows", x.device, x.data_ptr(), FLOATS[x.dtype], rows, cols, _row_stride(x), block,
              EIGHT_BIT[dtype], slots, k, ends, G, q.data_ptr(), _row_stride(q, 16), scales.data_ptr(), row_stride,
              block_stride)
    return q, scales


def quantize_cols(x: torch.Tensor, group_ends: torch.Tensor, dtype: torch.dtype = torch.float8_e4m3fn):
    """``x`` [rows, cols] in 8 bits with one scale for each 128 rows of a group in
    a column, groups padded to 128 rows with zeros: (values [padded rows, cols],
    E8M0 bytes uint8 [padded rows / 128, cols]), the operands of ``grouped_matmul_k``."""
    _check_matrix("x", x, FLOATS)
    _check_eight_bit(dtype)
    _check_ends("group_ends", group_ends)
    _check_cuda(x=x, group_ends=group_ends)
    rows, cols = x.shape
    padded = _up(rows, 128) + 128 * group_ends.numel()   # mx_padded_rows
    q = _eight_bit_rows((padded, cols), dtype, x.device)
    scales = torch.empty((padded // 128, cols), dtype=torch.uint8, device=x.device)
    if cols:
        _call("mx_quantize_cols", x.device, x.data_ptr(), FLOATS[x.dtype], rows, cols, _row_stride(x),
              group_ends.data_ptr(), group_ends.numel(), EIGHT_BIT[dtype], q.data_ptr(), _row_stride(q),
              scales.data_ptr(), cols)
    return q, scales


def quantize_blocks(x: torch.Tensor, dtype: torch.dtype = torch.float8_e4m3fn):
    """Matrices ``x`` [groups, rows, cols] (weights) in 8 bits with one scale for
    each 128 x 128 block: (values, E8M0 bytes uint8 [groups, row blocks, column blocks])."""
    if x.dim() != 3 or x.dtype not in FLOATS:
        raise ValueError("x must be a 3-D float32, bfloat16 or float16 tensor")
    if x.shape[2] > 1 and x.stride(2) != 1:
        raise ValueError("x must be dense along columns (stride(2) == 1)")
    _check_eight_bit(dtype)
    _check_cuda(x=x)
    G, rows, cols = x.shape
    q = _eight_bit_rows((G, rows, cols), dtype, x.device)
    scales = torch.empty((G, _up(rows, 128) // 128, _up(cols, 128) // 128), dtype=torch.uint8, device=x.device)
    if x.numel():
        q_stride = _row_stride(q, 16)
        _call("mx_quantize_blocks", x.device, x.data_ptr(), FLOATS[x.dtype], G, rows, cols, x.stride(0),
              _row_stride(x), EIGHT_BIT[dtype], q.data_ptr(), rows * q_stride, q_stride, scales.data_ptr())
    return q, scales


# ------------------------------------------------------------------ product
def _scale_bytes(name: str, s: torch.Tensor) -> torch.Tensor:
    if s.dtype not in (torch.uint8, torch.float8_e8m0fnu):
        raise ValueError(f"{name} must be E8M0 bytes (uint8 or float8_e8m0fnu)")
    return s


def _check_shape(name: str, t: torch.Tensor, shape) -> None:
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def grouped_matmul(a: torch.Tensor, a_scales: torch.Tensor, b: torch.Tensor, b_scales: torch.Tensor,
                   group_ends: torch.Tensor, block: int = 128, b_layout: str = "nk",
                   out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """Rows of ``a`` [rows, k] times their group's matrix of ``b`` ([groups, n, k],
    or [groups, k, n] with b_layout "kn"): [rows, n], zeros behind the last group.

    block 128: a_scales [rows, k blocks], b_scales [groups, rows of b / 128,
    columns of b / 128], any strides (``quantize_rows``, ``quantize_blocks``).
    block 32: both in the blocked layout, a_scales from ``rearrange_m_groups`` of
    [rows, k / 32], b_scales from that of [groups * n, k / 32] with n rows a group."""
    _check_matrix("a", a, EIGHT_BIT)
    if b.dim() != 3 or b.dtype not in EIGHT_BIT or (b.shape[2] > 1 and b.stride(2) != 1):
        raise ValueError("b must be a 3-D float8_e4m3fn or float8_e5m2 tensor, dense along columns")
    if b_layout not in B.B_LAYOUTS:
        raise ValueError('b_layout must be "nk" or "kn"')
    if block not in (32, 128) or (block == 32 and b_layout != "nk"):
        raise ValueError('block must be 128, or 32 with b_layout "nk"')
    if out_dtype not in FLOATS:
        raise ValueError("out_dtype must be float32, bfloat16 or float16")
    _check_ends("group_ends", group_ends)
    _scale_bytes("a_scales", a_scales)
    _scale_bytes("b_scales", b_scales)
    _check_cuda(a=a, a_scales=a_scales, b=b, b_scales=b_scales, group_ends=group_ends, out=out)
    rows, k = a.shape
    G = group_ends.numel()
    n = b.shape[1] if b_layout == "nk" else b.shape[2]
    _check_shape("b", b, (G, n, k) if b_layout == "nk" else (G, k, n))
    if k < 1:
        raise ValueError("the contraction must have at least one value")
    a_row, a_block, b_group, b_n, b_k = 0, 0, 0, 0, 0
    if block == 128:
        kb, nb = _up(k, 128) // 128, _up(n, 128) // 128
        _check_shape("a_scales", a_scales, (rows, kb))
        _check_shape("b_scales", b_scales, (G, nb, kb) if b_layout == "nk" else (G, kb, nb))
        a_row, a_block = a_scales.stride()
        b_group, b_n, b_k = b_scales.stride()
        if b_layout == "kn":
            b_n, b_k = b_k, b_n
    else:
        cols = _up(k, 32) // 32
        for name, s, need in (("a_scales", a_scales, B.mx_rearranged_size(B.MX_GROUPS_M, rows, cols, G)),
                              ("b_scales", b_scales, G * _up(n, 128) * _up(cols, 4))):
            if not s.is_contiguous() or s.numel() < need:
                raise ValueError(f"{name} must be a contiguous blocked buffer of at least {need} bytes")
    if out is None:
        y = torch.empty_strided((rows, n), (n, 1), dtype=out_dtype, device=a.device)
    else:
        _check_out(out, (rows, n), (out_dtype,))
        _check_apart(out, a=a, a_scales=a_scales, b=b, b_scales=b_scales, group_ends=group_ends)
        y = out
    _call("mx_grouped_matmul_m", a.device, a.data_ptr(), EIGHT_BIT[a.dtype], _row_stride(a, 16), a_scales.data_ptr(),
          a_row, a_block, b.data_ptr(), EIGHT_BIT[b.dtype], B.B_LAYOUTS[b_layout], b.stride(0), _row_stride(b, 16),
          b_scales.data_ptr(), b_group, b_n, b_k, block, rows, n, k, group_ends.data_ptr(), G, y.data_ptr(),
          FLOATS[out_dtype], _row_stride(y))
    return y if out is None else _written(out)


def grouped_matmul_k(a: torch.Tensor, a_scales: torch.Tensor, b: torch.Tensor, b_scales: torch.Tensor,
                     group_ends: torch.Tensor, out_dtype: torch.dtype = torch.bfloat16,
                     out: torch.Tensor | None = None) -> torch.Tensor:
    """For each group the product over its rows, a^T b: [groups, m, n], from
    operands [padded rows, m] and [padded rows, n] as ``quantize_cols`` gives
    them; ``group_ends`` are those of the rows without padding."""
    _check_matrix("a", a, EIGHT_BIT)
    _check_matrix("b", b, EIGHT_BIT)
    if out_dtype not in FLOATS:
        raise ValueError("out_dtype must be float32, bfloat16 or float16")
    _check_ends("group_ends", group_ends)
    _scale_bytes("a_scales", a_scales)
    _scale_bytes("b_scales", b_scales)
    _check_cuda(a=a, a_scales=a_scales, b=b, b_scales=b_scales, group_ends=group_ends, out=out)
    padded, m = a.shape
    n, G = b.shape[1], group_ends.numel()
    if padded < 128 or padded % 128 or b.shape[0] != padded:
        raise ValueError("a and b must have the same number of rows, a multiple of 128, as quantize_cols gives them")
    for name, s, cols in (("a_scales", a_scales, m), ("b_scales", b_scales, n)):
        _check_shape(name, s, (padded // 128, cols))
        if cols > 1 and s.stride(1) != 1:
            raise ValueError(f"{name} must be dense along columns (stride(1) == 1)")
    if out is None:
        y = torch.empty_strided((G, m, n), (m * n, n, 1), dtype=out_dtype, device=a.device)
    else:
        _check_out(out, (G, m, n), (out_dtype,))
        _check_apart(out, a=a, a_scales=a_scales, b=b, b_scales=b_scales, group_ends=group_ends)
        y = out
    _call("mx_grouped_matmul_k", a.device, a.data_ptr(), EIGHT_BIT[a.dtype], _row_stride(a, 16), a_scales.data_ptr(),
          _row_stride(a_scales), b.data_ptr(), EIGHT_BIT[b.dtype], _row_stride(b, 16), b_scales.data_ptr(),
          _row_stride(b_scales), padded, m, n, group_ends.data_ptr(), G, y.data_ptr(), FLOATS[out_dtype],
          y.stride(0), _row_stride(y))
    return y if out is None else _written(out)
