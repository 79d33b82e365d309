"""Strides that no memory has are refused before anything is computed from
them: neither a product of theirs nor their bytes may wrap round 64 bits."""
import pytest

pytest.importorskip("torch")

from scale_factor_layout_b200 import _binding as B  # noqa: E402
from test_moe_abi import BACKWARD, BLOCKS, COLS, COMBINE, DISPATCH, PRODUCT, PRODUCT_K, ROWS, call  # noqa: E402

OK, INVALID, UNSUPPORTED = B.MX_OK, B.MX_ERR_INVALID_ARG, B.MX_ERR_UNSUPPORTED
F32 = B.MX_F32


@pytest.mark.parametrize("name,defaults,kwargs,status", [
    # 2^25 rows of 2^39 are 2^64 elements, which is 0 in 64 bits: the matrices overlap
    ("mx_grouped_matmul_m", PRODUCT, dict(n=2**25 + 1, b_stride=2**39, b_group_stride=64, out_stride=2**26), INVALID),
    ("mx_grouped_matmul_m", PRODUCT, dict(b_layout=B.MX_B_KN, k=2**25, b_stride=2**39, a_stride=2**25, b_group_stride=64), INVALID),
    ("mx_grouped_matmul_k", PRODUCT_K, dict(m=2**27 + 1, a_stride=2**28, a_scale_stride=2**28, out_stride=2**37, out_group_stride=2**37), INVALID),
    ("mx_grouped_matmul_k", PRODUCT_K, dict(m=2**28 + 1, a_stride=2**29, a_scale_stride=2**29, out_dtype=B.MX_BF16, out_stride=2**36, out_group_stride=32), INVALID),
    ("mx_quantize_blocks", BLOCKS, dict(rows=2**25 + 1, q_stride=2**39, q_group_stride=64, x_group_stride=2**32), INVALID),
    # bytes, not elements, are what a stride has to fit
    ("mx_grouped_matmul_m", PRODUCT, dict(out_dtype=F32, out_stride=2**38), UNSUPPORTED),
    ("mx_grouped_matmul_m", PRODUCT, dict(out_stride=2**39), UNSUPPORTED),
    ("mx_grouped_matmul_m", PRODUCT, dict(a_stride=2**40), UNSUPPORTED),
    ("mx_grouped_matmul_k", PRODUCT_K, dict(out_stride=2**38, out_group_stride=2**50), UNSUPPORTED),
    ("mx_grouped_matmul_k", PRODUCT_K, dict(out_group_stride=2**38), UNSUPPORTED),
    ("mx_dispatch_rows", DISPATCH, dict(x_stride=2**62), UNSUPPORTED),
    ("mx_dispatch_rows", DISPATCH, dict(dtype=F32, out_stride=2**38), UNSUPPORTED),
    ("mx_combine_rows", COMBINE, dict(rows_stride=2**62), UNSUPPORTED),
    ("mx_combine_rows", COMBINE, dict(y_stride=2**39), UNSUPPORTED),
    ("mx_combine_rows_backward", BACKWARD, dict(grad_stride=2**62), UNSUPPORTED),
    ("mx_combine_rows_backward", BACKWARD, dict(rows_stride=2**62), UNSUPPORTED),
    ("mx_combine_rows_backward", BACKWARD, dict(d_rows_stride=2**39), UNSUPPORTED),
    ("mx_quantize_rows", ROWS, dict(x_stride=2**62), UNSUPPORTED),
    ("mx_quantize_rows", ROWS, dict(q_stride=2**40), UNSUPPORTED),
    ("mx_quantize_rows", ROWS, dict(scale_row_stride=2**62), UNSUPPORTED),
    ("mx_quantize_rows", ROWS, dict(scale_block_stride=2**40), UNSUPPORTED),
    ("mx_quantize_cols", COLS, dict(x_stride=2**62), UNSUPPORTED),
    ("mx_quantize_cols", COLS, dict(q_stride=2**62), UNSUPPORTED),
    ("mx_quantize_cols", COLS, dict(scale_stride=2**40), UNSUPPORTED),
    ("mx_quantize_blocks", BLOCKS, dict(x_stride=2**62), UNSUPPORTED),
    ("mx_quantize_blocks", BLOCKS, dict(x_group_stride=2**62), UNSUPPORTED),
    ("mx_quantize_blocks", BLOCKS, dict(q_group_stride=2**40), UNSUPPORTED),
    # the largest that fit get past these checks (to a misaligned pointer, or nothing to do)
    ("mx_grouped_matmul_m", PRODUCT, dict(out_dtype=F32, out_stride=2**38 - 1, out=0x8002), B.MX_ERR_MISALIGNED),
    ("mx_grouped_matmul_m", PRODUCT, dict(num_groups=1, b_group_stride=2**62, out=0x8001), B.MX_ERR_MISALIGNED),
    ("mx_grouped_matmul_m", PRODUCT, dict(a_stride=2**40 - 16, b_stride=2**30, b_group_stride=31 * 2**30 + 64, out=0x8001), B.MX_ERR_MISALIGNED),
    ("mx_grouped_matmul_m", PRODUCT, dict(b_stride=2**30, b_group_stride=31 * 2**30 + 63), INVALID),
    ("mx_grouped_matmul_k", PRODUCT_K, dict(num_groups=1, out_group_stride=2**62, out=0x8001), B.MX_ERR_MISALIGNED),
    ("mx_dispatch_rows", DISPATCH, dict(x_stride=2**39 - 1, out=0x9001), B.MX_ERR_MISALIGNED),
    ("mx_quantize_blocks", BLOCKS, dict(groups=1, x_group_stride=2**62, q_group_stride=2**62, x=0x1001), B.MX_ERR_MISALIGNED),
    ("mx_quantize_rows", ROWS, dict(x_stride=2**39 - 1, rows=0), OK),
])
def test_strides(mxlib, name, defaults, kwargs, status):
    assert call(name, defaults, **kwargs) == status
