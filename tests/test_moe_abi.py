"""The mixture-of-experts entry points refuse bad arguments before they touch
the device: C statuses, and the torch wrappers' checks on CPU tensors."""
import pytest

torch = pytest.importorskip("torch")

from scale_factor_layout_b200 import _binding as B  # noqa: E402
import scale_factor_layout_b200 as mxs  # noqa: E402

OK, INVALID, MISALIGNED, UNSUPPORTED = B.MX_OK, B.MX_ERR_INVALID_ARG, B.MX_ERR_MISALIGNED, B.MX_ERR_UNSUPPORTED
BIG = 2**31


def call(name, defaults, **kwargs):
    assert set(kwargs) <= set(defaults), kwargs
    return getattr(B, name)(**{**defaults, **kwargs})


SORT = dict(expert_ids=0x1000, id_bytes=8, tokens=16, choices=2, num_experts=8, group_ends=0x2000, row_of_slot=0x3000,
            slot_of_row=0x4000, workspace=0, stream=0)
DISPATCH = dict(x=0x1000, dtype=B.MX_BF16, tokens=16, cols=64, x_stride=64, row_of_slot=0x3000, choices=2,
                group_ends=0x2000, num_experts=8, out=0x9000, out_stride=64, stream=0)
COMBINE = dict(rows=0x1000, dtype=B.MX_BF16, tokens=16, cols=64, rows_stride=64, row_of_slot=0x3000, choices=2,
               weights=0x2000, y=0x9000, y_stride=64, stream=0)
BACKWARD = dict(grad=0x1000, dtype=B.MX_BF16, tokens=16, cols=64, grad_stride=64, rows=0x5000, rows_stride=64,
                row_of_slot=0x3000, choices=2, group_ends=0x2000, num_experts=8, weights=0x6000, d_rows=0x9000,
                d_rows_stride=64, d_weights=0xa000, stream=0)
ROWS = dict(x=0x1000, dtype=B.MX_BF16, rows=16, cols=64, x_stride=64, block=128, out_dtype=B.MX_E4M3, row_of_slot=0,
            choices=0, group_ends=0, num_experts=0, q=0x9000, q_stride=64, scales=0xa000, scale_row_stride=1,
            scale_block_stride=16, stream=0)
COLS = dict(x=0x1000, dtype=B.MX_BF16, rows=16, cols=64, x_stride=64, group_ends=0x2000, num_groups=2,
            out_dtype=B.MX_E4M3, q=0x9000, q_stride=64, scales=0xa000, scale_stride=64, stream=0)
BLOCKS = dict(x=0x1000, dtype=B.MX_BF16, groups=2, rows=16, cols=64, x_group_stride=1024, x_stride=64,
              out_dtype=B.MX_E4M3, q=0x9000, q_group_stride=1024, q_stride=64, scales=0xa000, stream=0)
PRODUCT = dict(a=0x1000, a_dtype=B.MX_E4M3, a_stride=64, a_scales=0x2000, a_scale_row_stride=1, a_scale_block_stride=16,
               b=0x4000, b_dtype=B.MX_E4M3, b_layout=B.MX_B_NK, b_group_stride=2048, b_stride=64, b_scales=0x6000,
               b_scale_group_stride=1, b_scale_n_stride=1, b_scale_k_stride=1, block=128, rows=16, n=32, k=64,
               group_ends=0x7000, num_groups=2, out=0x8000, out_dtype=B.MX_BF16, out_stride=32, stream=0)
PRODUCT_K = dict(a=0x1000, a_dtype=B.MX_E4M3, a_stride=64, a_scales=0x2000, a_scale_stride=64, b=0x4000,
                 b_dtype=B.MX_E4M3, b_stride=32, b_scales=0x6000, b_scale_stride=32, padded_rows=256, m=64, n=32,
                 group_ends=0x7000, num_groups=2, out=0x8000, out_dtype=B.MX_F32, out_group_stride=2048, out_stride=32,
                 stream=0)


@pytest.mark.parametrize("name,defaults,kwargs,status", [
    ("mx_expert_sort", SORT, dict(num_experts=0), INVALID),
    ("mx_expert_sort", SORT, dict(num_experts=65), INVALID),
    ("mx_expert_sort", SORT, dict(id_bytes=2), INVALID),
    ("mx_expert_sort", SORT, dict(choices=0), INVALID),
    ("mx_expert_sort", SORT, dict(tokens=-1), INVALID),
    ("mx_expert_sort", SORT, dict(tokens=2**30, choices=2), INVALID),
    ("mx_expert_sort", SORT, dict(expert_ids=0), INVALID),
    ("mx_expert_sort", SORT, dict(group_ends=0), INVALID),
    ("mx_expert_sort", SORT, dict(tokens=100000), INVALID),          # workspace missing
    ("mx_expert_sort", SORT, dict(expert_ids=0x1004), MISALIGNED),
    ("mx_dispatch_rows", DISPATCH, dict(dtype=B.MX_E4M3), INVALID),
    ("mx_dispatch_rows", DISPATCH, dict(x_stride=63), INVALID),
    ("mx_dispatch_rows", DISPATCH, dict(out=0), INVALID),
    ("mx_dispatch_rows", DISPATCH, dict(tokens=BIG), INVALID),
    ("mx_dispatch_rows", DISPATCH, dict(x=0x1001), MISALIGNED),
    ("mx_dispatch_rows", DISPATCH, dict(tokens=0), OK),
    ("mx_dispatch_rows", DISPATCH, dict(cols=0), OK),
    ("mx_combine_rows", COMBINE, dict(dtype=9), INVALID),
    ("mx_combine_rows", COMBINE, dict(y_stride=10), INVALID),
    ("mx_combine_rows", COMBINE, dict(row_of_slot=0), INVALID),
    ("mx_combine_rows", COMBINE, dict(weights=0x2002), MISALIGNED),
    ("mx_combine_rows", COMBINE, dict(tokens=0), OK),
    ("mx_combine_rows_backward", BACKWARD, dict(weights=0), INVALID),
    ("mx_combine_rows_backward", BACKWARD, dict(cols=0), INVALID),
    ("mx_combine_rows_backward", BACKWARD, dict(d_rows_stride=1), INVALID),
    ("mx_combine_rows_backward", BACKWARD, dict(d_weights=0xa001), MISALIGNED),
    ("mx_quantize_rows", ROWS, dict(block=64), INVALID),
    ("mx_quantize_rows", ROWS, dict(out_dtype=B.MX_BF16), INVALID),
    ("mx_quantize_rows", ROWS, dict(dtype=B.MX_E4M3), INVALID),
    ("mx_quantize_rows", ROWS, dict(q_stride=63), INVALID),
    ("mx_quantize_rows", ROWS, dict(scale_row_stride=0), INVALID),
    ("mx_quantize_rows", ROWS, dict(row_of_slot=0x3000), INVALID),   # no choices, no ends
    ("mx_quantize_rows", ROWS, dict(scales=0), INVALID),
    ("mx_quantize_rows", ROWS, dict(rows=0), OK),
    ("mx_quantize_cols", COLS, dict(num_groups=65), INVALID),
    ("mx_quantize_cols", COLS, dict(scale_stride=63), INVALID),
    ("mx_quantize_cols", COLS, dict(group_ends=0), INVALID),
    ("mx_quantize_cols", COLS, dict(group_ends=0x2002), MISALIGNED),
    ("mx_quantize_cols", COLS, dict(cols=0, x_stride=0, q_stride=0, scale_stride=0), OK),
    ("mx_quantize_blocks", BLOCKS, dict(q_group_stride=100), INVALID),
    ("mx_quantize_blocks", BLOCKS, dict(x=0), INVALID),
    ("mx_quantize_blocks", BLOCKS, dict(groups=0), OK),
    ("mx_grouped_matmul_m", PRODUCT, dict(k=0), INVALID),
    ("mx_grouped_matmul_m", PRODUCT, dict(block=16), INVALID),
    ("mx_grouped_matmul_m", PRODUCT, dict(a_dtype=B.MX_BF16), INVALID),
    ("mx_grouped_matmul_m", PRODUCT, dict(out_dtype=B.MX_E4M3), INVALID),
    ("mx_grouped_matmul_m", PRODUCT, dict(b_layout=2), INVALID),
    ("mx_grouped_matmul_m", PRODUCT, dict(b_group_stride=1024), INVALID),
    ("mx_grouped_matmul_m", PRODUCT, dict(num_groups=65), INVALID),
    ("mx_grouped_matmul_m", PRODUCT, dict(out_stride=31), INVALID),
    ("mx_grouped_matmul_m", PRODUCT, dict(group_ends=0), INVALID),
    ("mx_grouped_matmul_m", PRODUCT, dict(a=0x1008), MISALIGNED),
    ("mx_grouped_matmul_m", PRODUCT, dict(a_stride=72), MISALIGNED),
    ("mx_grouped_matmul_m", PRODUCT, dict(b_group_stride=2056), MISALIGNED),
    ("mx_grouped_matmul_m", PRODUCT, dict(out=0x8001), MISALIGNED),
    ("mx_grouped_matmul_m", PRODUCT, dict(block=32, a_scales=0x2004), MISALIGNED),
    ("mx_grouped_matmul_m", PRODUCT, dict(block=32, b_layout=B.MX_B_KN, b_group_stride=4096), UNSUPPORTED),
    ("mx_grouped_matmul_m", PRODUCT, dict(k=2**25 + 16, a_stride=2**26, b_stride=2**26, b_group_stride=2**31), UNSUPPORTED),
    ("mx_grouped_matmul_m", PRODUCT, dict(n=2**30, out_stride=2**30, b_group_stride=2**36), UNSUPPORTED),
    ("mx_grouped_matmul_m", PRODUCT, dict(b_stride=2**40, b_group_stride=2**62), UNSUPPORTED),
    ("mx_grouped_matmul_m", PRODUCT, dict(rows=0), OK),
    ("mx_grouped_matmul_k", PRODUCT_K, dict(padded_rows=200), INVALID),
    ("mx_grouped_matmul_k", PRODUCT_K, dict(padded_rows=0), INVALID),
    ("mx_grouped_matmul_k", PRODUCT_K, dict(out_group_stride=100), INVALID),
    ("mx_grouped_matmul_k", PRODUCT_K, dict(a_scale_stride=63), INVALID),
    ("mx_grouped_matmul_k", PRODUCT_K, dict(b_stride=40), MISALIGNED),
    ("mx_grouped_matmul_k", PRODUCT_K, dict(padded_rows=2**25 + 128), UNSUPPORTED),
    ("mx_grouped_matmul_k", PRODUCT_K, dict(m=0), OK),
])
def test_statuses(mxlib, name, defaults, kwargs, status):
    assert call(name, defaults, **kwargs) == status


def test_sizes(mxlib):
    assert B.mx_padded_rows(0, 1) == 128 and B.mx_padded_rows(129, 3) == 256 + 384
    assert B.mx_padded_rows(-1, 1) == 0 and B.mx_padded_rows(5, 0) == 0 and B.mx_padded_rows(5, 65) == 0
    assert B.mx_expert_sort_workspace(10, 2) == 0 and B.mx_expert_sort_workspace(-1, 2) == 0
    assert B.mx_expert_sort_workspace(100000, 2) > 0


def refuse(fn, *args, match=None, **kwargs):
    with pytest.raises(ValueError, match=match):
        fn(*args, **kwargs)


def test_wrappers_refuse():
    """Every check that needs no device, on CPU tensors (which are refused last)."""
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)   # noqa: E731
    f8 = lambda *s: torch.zeros(s, dtype=torch.float8_e4m3fn)   # noqa: E731
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)   # noqa: E731
    ids = torch.zeros(4, 2, dtype=torch.int64)
    order = mxs.ExpertOrder(i32(3), i32(4, 2), i32(8))
    x = torch.zeros(4, 16)
    refuse(mxs.expert_sort, ids, 3, match="CUDA")
    refuse(mxs.expert_sort, ids, 65, match="num_experts")
    refuse(mxs.expert_sort, ids.float(), 3, match="int32 or int64")
    refuse(mxs.expert_sort, ids.t(), 3, match="contiguous")
    refuse(mxs.expert_sort, ids.view(-1), 3, match="tokens, choices")
    refuse(mxs.dispatch_rows, x, order, match="CUDA")
    refuse(mxs.dispatch_rows, x.double(), order, match="float32")
    refuse(mxs.dispatch_rows, x.t(), order, match="dense")
    refuse(mxs.dispatch_rows, x, order._replace(row_of_slot=ids), match="row_of_slot")
    refuse(mxs.dispatch_rows, x, order._replace(group_ends=i32(65)), match="groups")
    refuse(mxs.combine_rows, x, order, match="CUDA")
    refuse(mxs.combine_rows, x[0], order, match="2-D")
    refuse(mxs.combine_rows_backward, x, x, order, torch.zeros(4, 2).double(), match="weights")
    refuse(mxs.quantize_rows, x, match="CUDA")
    refuse(mxs.quantize_rows, x, block=64, match="block")
    refuse(mxs.quantize_rows, x, dtype=torch.int8, match="float8")
    refuse(mxs.quantize_cols, x, i32(3).long(), match="int32")
    refuse(mxs.quantize_cols, x, i32(3), match="CUDA")
    refuse(mxs.quantize_blocks, x, match="3-D")
    refuse(mxs.quantize_blocks, x[None], match="CUDA")
    a, b, s, ends = f8(4, 32), f8(2, 8, 32), u8(4, 1), i32(2)
    refuse(mxs.grouped_matmul, a, s, b, u8(2, 1, 1), ends, match="CUDA")
    refuse(mxs.grouped_matmul, a.float(), s, b, s, ends, match="float8")
    refuse(mxs.grouped_matmul, a, s, b, s, ends, block=64, match="block")
    refuse(mxs.grouped_matmul, a, s, b, s, ends, block=32, b_layout="kn", match="block")
    refuse(mxs.grouped_matmul, a, s, b, s, ends, b_layout="mn", match="b_layout")
    refuse(mxs.grouped_matmul, a, s.float(), b, s, ends, match="E8M0")
    refuse(mxs.grouped_matmul, a, s, b, s, ends, out_dtype=torch.float64, match="out_dtype")
    refuse(mxs.grouped_matmul_k, f8(128, 8), u8(1, 8), f8(128, 8), u8(1, 8), ends, match="CUDA")
    refuse(mxs.grouped_matmul_k, f8(128, 8), u8(1, 8), f8(128, 8), u8(1, 8), ends, out_dtype=torch.int8, match="out_dtype")


def test_rows_too_long_off_8_byte_boundaries():
    """Such rows are indexed by halves of 16 bits, in 31 bits."""
    n = 2**30 + 1
    assert call("mx_dispatch_rows", DISPATCH, dtype=B.MX_F32, tokens=1, cols=n, x_stride=n, out_stride=n) == UNSUPPORTED
