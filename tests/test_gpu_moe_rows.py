"""Slots sorted by expert, rows to experts and back, and quantization, against
plain forms in 64 bits: every type, odd widths, strides, choices and group
counts, dropped slots, empty groups, values at the types' borders."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import moe_reference as ref  # noqa: E402
import scale_factor_layout_b200 as mxs  # noqa: E402

pytestmark = pytest.mark.gpu

BF, HF, FL = torch.bfloat16, torch.float16, torch.float32
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2


def order_for(rng, T, k, E, lo=-2, hi=2, id_type=torch.int64):
    """(ids, the framework's order, the plain one); some ids outside [0, E)."""
    ids = rng.integers(lo, E + hi, size=(T, k))
    plain = ref.sort(ids, E)
    return mxs.expert_sort(torch.from_numpy(ids).to(id_type).cuda(), E), plain


def matrix(rng, rows, cols, dtype, pad=0):
    """A matrix on the GPU whose rows are `pad` elements apart, NaN between, and its CPU copy."""
    v = torch.from_numpy(rng.standard_normal((rows, cols))).to(dtype)
    buf = torch.full((rows, cols + pad), float("nan"), dtype=dtype, device="cuda")
    buf[:, :cols] = v.cuda()
    return buf[:, :cols], v


@pytest.mark.parametrize("T,k,E,id_type", [
    (0, 1, 1, torch.int64), (1, 1, 1, torch.int32), (1, 8, 64, torch.int64), (7, 3, 5, torch.int32), (33, 1, 64, torch.int64),
    (1000, 8, 64, torch.int64), (1024, 8, 33, torch.int64), (1025, 8, 32, torch.int32), (3001, 7, 64, torch.int64),
    (40000, 9, 17, torch.int64), (300001, 1, 3, torch.int32),
])
def test_sort(mxlib, T, k, E, id_type):
    rng = np.random.default_rng(T + k)
    order, (ends, row, slot) = order_for(rng, T, k, E, id_type=id_type)
    assert np.array_equal(order.group_ends.cpu().numpy(), ends)
    assert np.array_equal(order.row_of_slot.cpu().numpy(), row)
    assert np.array_equal(order.slot_of_row.cpu().numpy(), slot)


@pytest.mark.parametrize("only", [0, 5, 63, -1, 64, 2**31 - 1, -2**31])
def test_sort_one_expert_or_none(mxlib, only):
    """Every slot at one expert (the sort's counters all in one place), or at none."""
    for n in (50, 20000):
        ids = np.full((n, 2), only, np.int64)
        ends, row, slot = ref.sort(ids, 64)
        order = mxs.expert_sort(torch.from_numpy(ids).cuda(), 64)
        assert np.array_equal(order.group_ends.cpu().numpy(), ends)
        assert np.array_equal(order.row_of_slot.cpu().numpy(), row)
        assert np.array_equal(order.slot_of_row.cpu().numpy(), slot)


def test_sort_ids_past_32_bits(mxlib):
    """Ids that are valid only in their low 32 bits have no row."""
    ids = torch.tensor([[1, 2**32 + 1, -2**63, 0, 2**40]], device="cuda")
    order = mxs.expert_sort(ids, 4)
    assert order.row_of_slot.tolist() == [[1, -1, -1, 0, -1]]
    assert order.group_ends.tolist() == [1, 2, 2, 2]


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (5, 8, 64), (130, 3, 7), (257, 9, 4)])
@pytest.mark.parametrize("C,pad", [(1, 0), (7, 0), (8, 8), (64, 3), (1408, 0), (2056, 8)])
@pytest.mark.parametrize("dtype", [BF, HF, FL])
def test_dispatch_and_combine(mxlib, T, k, E, C, pad, dtype):
    rng = np.random.default_rng(C + T)
    order, (ends, row, slot) = order_for(rng, T, k, E)
    x, x_cpu = matrix(rng, T, C, dtype, pad)
    rows, rows_cpu = matrix(rng, T * k, C, dtype, pad)
    got = mxs.dispatch_rows(x, order)
    assert torch.equal(got.cpu(), ref.dispatch(x_cpu, slot, k))

    # 32-bit sums of k products: each step is off by at most 2^-24 of the magnitudes so far;
    # then one rounding to the type
    half = torch.finfo(dtype).eps / 2
    for w in (None, torch.from_numpy(rng.standard_normal((T, k))).float()):
        y = mxs.combine_rows(rows, order, None if w is None else w.cuda()).cpu().double()
        want, mag = ref.combine(rows_cpu, row, w)
        assert ((y - want).abs() <= (k + 1) * 2.0 ** -24 * mag + half * want.abs() + 1e-7 * (dtype == HF)).all()

    g, g_cpu = matrix(rng, T, C, dtype, pad)
    w = torch.from_numpy(rng.standard_normal((T, k))).float()
    d_rows, d_w = mxs.combine_rows_backward(g, rows, order, w.cuda())
    want = torch.zeros(T * k, C, dtype=torch.float64)
    dots = torch.zeros(T, k, dtype=torch.float64)
    mags = torch.zeros(T, k, dtype=torch.float64)
    for r, s in enumerate(slot):
        if s >= 0:
            t, j = divmod(int(s), k)
            want[r] = g_cpu[t].double() * float(w[t, j])
            prod = g_cpu[t].double() * rows_cpu[r].double()
            dots[t, j], mags[t, j] = prod.sum(), prod.abs().sum()
    # one product in 32 bits, one rounding to the type (subnormal halves are off by 2^-25)
    assert ((d_rows.cpu().double() - want).abs() <= (half + 2.0 ** -24) * 1.01 * want.abs() + 2.0 ** -25 * (dtype == HF)).all()
    assert (d_rows.cpu()[torch.from_numpy(slot < 0)] == 0).all()
    assert ((d_w.cpu().double() - dots).abs() <= (C + 1) * 2.0 ** -24 * mags).all()


def test_combine_ignores_rows_that_no_slot_has(mxlib):
    """NaN in rows behind the last group and in weights of dropped slots reaches nothing."""
    ids = torch.tensor([[0, 9], [9, 9], [1, 0]], device="cuda")
    order = mxs.expert_sort(ids, 2)
    rows = torch.ones(6, 40, device="cuda", dtype=BF)
    rows[3:] = float("nan")
    w = torch.tensor([[2.0, float("nan")], [float("nan"), float("nan")], [3.0, 4.0]], device="cuda")
    y = mxs.combine_rows(rows, order, w)
    assert y[0].eq(2).all() and y[1].eq(0).all() and y[2].eq(7).all()
    d_rows, d_w = mxs.combine_rows_backward(torch.ones(3, 40, device="cuda", dtype=BF), rows, order, w)
    assert d_rows[3:].eq(0).all() and d_w.tolist() == [[40.0, 0.0], [0.0, 0.0], [40.0, 40.0]]


def test_bad_indexes_are_skipped(mxlib):
    """Rows that do not exist are neither read nor written."""
    row = torch.tensor([[0, 7], [-5, 2**31 - 1], [3, -2**31]], dtype=torch.int32, device="cuda")
    order = mxs.ExpertOrder(torch.tensor([4], dtype=torch.int32, device="cuda"), row, torch.zeros(6, dtype=torch.int32, device="cuda"))
    buf = torch.full((10, 16), 5.0, device="cuda")
    mxs.dispatch_rows(torch.arange(3.0, device="cuda")[:, None].expand(3, 16).contiguous() + 1, order, out=buf[2:8])
    assert buf[:2].eq(5).all() and buf[8:].eq(5).all()
    assert buf[2].eq(1).all() and buf[5].eq(3).all() and buf[6:8].eq(0).all()
    y = mxs.combine_rows(torch.ones(6, 16, device="cuda"), order)
    assert y[0].eq(1).all() and y[1].eq(0).all() and y[2].eq(1).all()
    q, _ = mxs.quantize_rows(torch.ones(3, 16, device="cuda"), order=order)
    assert q.shape == (6, 16)


def test_autograd(mxlib):
    """Gradients of dispatch and combine against the formula's and against
    differences; a gradient that is broadcast over rows (a sum's) too."""
    rng = np.random.default_rng(3)
    order, (ends, row, slot) = order_for(rng, 9, 3, 4)
    x = torch.from_numpy(rng.standard_normal((9, 24))).float().cuda().requires_grad_()
    w = torch.from_numpy(rng.standard_normal((9, 3))).float().cuda().requires_grad_()
    mixed = torch.from_numpy(rng.standard_normal((9, 24))).float().cuda()

    def loss(x, w):
        return (mxs.combine_rows(mxs.dispatch_rows(x, order).square(), order, w) * mixed).sum()

    dx, dw = torch.autograd.grad(loss(x, w), (x, w))
    live = torch.from_numpy(row >= 0).cuda()
    wl = torch.where(live, w.detach(), 0).sum(1, keepdim=True).double()
    want_x = 2 * x.detach().double() * mixed.double() * wl
    want_w = torch.where(live, (x.detach().double().square() * mixed).sum(1, keepdim=True), 0)
    assert (dx.double() - want_x).abs().max() <= 20 * 2.0 ** -24 * (want_x.abs().max() * 3 + 1)
    assert (dw.double() - want_w).abs().max() <= 50 * 2.0 ** -24 * (x.detach().double().square() * mixed.double().abs()).sum(1).max()
    # differences: the loss is quadratic in x and linear in w, so central differences are exact but for rounding
    step = 0.25
    for t, c in ((0, 0), (4, 13), (8, 23)):
        e = torch.zeros_like(x)
        e[t, c] = step
        num = (loss(x.detach() + e, w.detach()) - loss(x.detach() - e, w.detach())) / (2 * step)
        assert abs(float(num) - float(dx[t, c])) <= 1e-3 * (1 + abs(float(num)))
    for t, j in ((0, 0), (5, 2)):
        e = torch.zeros_like(w)
        e[t, j] = step
        num = (loss(x.detach(), w.detach() + e) - loss(x.detach(), w.detach() - e)) / (2 * step)
        assert abs(float(num) - float(dw[t, j])) <= 1e-3 * (1 + abs(float(num)))
    (db,) = torch.autograd.grad(mxs.dispatch_rows(x, order).sum(), x)
    assert torch.equal(db, live.sum(1, keepdim=True).float().expand(9, 24))
    rows = torch.ones(27, 24, device="cuda", requires_grad=True)
    (dr,) = torch.autograd.grad(mxs.combine_rows(rows, order).sum(), rows)
    assert torch.equal(dr[:, 0], torch.from_numpy((slot >= 0).astype(np.float32)).cuda())


# ------------------------------------------------------------------ quantization
def hard_values(rng, rows, cols, dtype):
    """Blocks of every size of magnitude, with zeros, borders between scales and ties between 8-bit values."""
    v = rng.standard_normal((rows, cols)) * 2.0 ** rng.integers(-30, 12, size=(rows, 1))
    v[rng.random((rows, cols)) < 0.3] *= 2.0 ** -9
    ties = rng.integers(-64, 65, size=(rows, cols)) / 32.0
    v = np.where(rng.random((rows, 1)) < 0.4, ties, v)
    v[rng.random(rows) < 0.1] = 0.0
    border = rng.random(rows) < 0.2
    v[border, 0] = 448.0 * 2.0 ** rng.integers(-12, 5, size=border.sum())
    return torch.from_numpy(v).to(dtype)


def check_quantized(q, s, want):
    values, scale = want
    assert np.array_equal(s.cpu().numpy(), scale)
    assert np.array_equal(q.float().cpu().double().numpy(), values, equal_nan=True)


@pytest.mark.parametrize("R,C,pad", [(1, 1, 0), (3, 128, 0), (33, 129, 0), (32, 256, 8), (70, 1000, 0), (5, 2056, 3), (257, 40, 0)])
@pytest.mark.parametrize("block", [128, 32])
@pytest.mark.parametrize("dtype,to", [(BF, E4), (HF, E5), (FL, E4), (BF, E5)])
def test_quantize_rows(mxlib, R, C, pad, block, dtype, to):
    rng = np.random.default_rng(R + C)
    v = hard_values(rng, R, C, dtype)
    buf = torch.full((R, C + pad), float("nan"), dtype=dtype, device="cuda")
    buf[:, :C] = v.cuda()
    q, s = mxs.quantize_rows(buf[:, :C], block=block, dtype=to)
    assert q.dtype == to and q.shape == (R, C) and (R == 1 or q.stride(0) % 16 == 0)
    check_quantized(q, s, ref.quantize(v, to, 1, block))


@pytest.mark.parametrize("T,k,E,C,block", [(1, 1, 1, 128, 128), (40, 3, 5, 300, 128), (65, 8, 64, 264, 32), (130, 2, 9, 1001, 128)])
def test_quantize_rows_in_expert_order(mxlib, T, k, E, C, block):
    """One pass gives what dispatch and quantization give, zeros behind the last group."""
    rng = np.random.default_rng(C)
    order, _ = order_for(rng, T, k, E)
    x = hard_values(rng, T, C, BF).cuda()
    q, s = mxs.quantize_rows(x, block=block, order=order)
    q2, s2 = mxs.quantize_rows(mxs.dispatch_rows(x, order), block=block)
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)


@pytest.mark.parametrize("sizes,C,pad", [([1], 1, 0), ([0, 5, 128, 0, 129], 40, 0), ([300], 136, 8), ([127, 1, 0, 400], 257, 0), ([0, 0], 16, 0)])
@pytest.mark.parametrize("dtype,to", [(BF, E4), (FL, E5), (HF, E4)])
def test_quantize_cols(mxlib, sizes, C, pad, dtype, to):
    rng = np.random.default_rng(C)
    R = sum(sizes) + 3   # three rows behind the last group
    v = hard_values(rng, C, R, dtype).t().contiguous()
    buf = torch.full((R, C + pad), float("nan"), dtype=dtype, device="cuda")
    buf[:, :C] = v.cuda()
    ends = np.cumsum(sizes)
    q, s = mxs.quantize_cols(buf[:, :C], torch.tensor(ends, dtype=torch.int32, device="cuda"), dtype=to)
    check_quantized(q, s, ref.quantize(ref.pad_groups(v, ends), to, 128, 1))


@pytest.mark.parametrize("G,R,C", [(1, 1, 1), (3, 128, 128), (2, 130, 257), (5, 40, 1000)])
@pytest.mark.parametrize("dtype,to", [(BF, E4), (FL, E5)])
def test_quantize_blocks(mxlib, G, R, C, dtype, to):
    rng = np.random.default_rng(C)
    v = torch.stack([hard_values(rng, R, C, dtype) for _ in range(G)])
    q, s = mxs.quantize_blocks(v.cuda(), dtype=to)
    for g in range(G):
        check_quantized(q[g], s[g], ref.quantize(v[g], to, 128, 128))


def test_quantize_not_finite(mxlib):
    """A block with a NaN or an infinity is NaN, in scale and values; its neighbours are not."""
    x = torch.ones(4, 384, device="cuda", dtype=BF)
    x[0, 5], x[1, 130], x[2, 383], x[3, 0] = float("nan"), float("inf"), float("-inf"), 3.38e38
    q, s = mxs.quantize_rows(x)
    check_quantized(q, s, ref.quantize(x.cpu(), E4, 1, 128))
    q, s = mxs.quantize_blocks(x[None])
    check_quantized(q[0], s[0], ref.quantize(x.cpu(), E4, 128, 128))
    ends = torch.tensor([2, 4], dtype=torch.int32, device="cuda")
    q, s = mxs.quantize_cols(x, ends)
    # padding of a block that is not finite stays zero
    want, byte = ref.quantize(ref.pad_groups(x.cpu(), [2, 4]), E4, 128, 1)
    want[2:128], want[130:] = 0, 0
    check_quantized(q, s, (want, byte))


def test_quantize_tiny(mxlib):
    """Subnormal inputs and magnitudes below the smallest scale."""
    x = torch.tensor([[1e-40, -3e-39, 2.0 ** -149, 0.0], [2.0 ** -126, 2.0 ** -118, -2.0 ** -127, 2.0 ** -119]])
    q, s = mxs.quantize_rows(x.cuda())
    check_quantized(q, s, ref.quantize(x, E4, 1, 128))


@pytest.mark.parametrize("dtype", [BF, HF, FL])
@pytest.mark.parametrize("offset", [1, 2, 3, 4, 8])
@pytest.mark.parametrize("C,stride", [(37, 45), (64, 80), (129, 130), (530, 544)])
def test_rows_that_start_anywhere(mxlib, dtype, offset, C, stride):
    """Inputs and outputs at every alignment give what aligned ones give, and nothing beside them is written."""
    rng = np.random.default_rng(C + offset)
    T, k, E = 45, 2, 3
    order, (ends, row, slot) = order_for(rng, T, k, E)

    def view(rows, fill=None):
        buf = torch.full((rows * stride + 64,), 77.0, dtype=dtype, device="cuda")
        v = buf[offset: offset + rows * stride].view(rows, stride)[:, :C]
        if fill is not None:
            v.copy_(fill)
        return buf, v

    x = hard_values(rng, T, C, dtype).cuda()
    rows = torch.from_numpy(rng.standard_normal((T * k, C))).to(dtype).cuda()
    w = torch.from_numpy(rng.standard_normal((T, k))).float().cuda()
    (_, xv), (_, rv) = view(T, x), view(T * k, rows)
    buf, out = view(T * k)
    assert torch.equal(mxs.dispatch_rows(xv, order, out=out), mxs.dispatch_rows(x, order))
    gaps = torch.ones_like(buf, dtype=torch.bool)
    gaps[offset: offset + T * k * stride].view(T * k, stride)[:, :C] = False
    assert buf[gaps].eq(77).all()
    buf, out = view(T)
    # sums of the same terms in the same order, whatever is loaded at once
    assert torch.equal(mxs.combine_rows(rv, order, w, out=out), mxs.combine_rows(rows, order, w))
    gaps = torch.ones_like(buf, dtype=torch.bool)
    gaps[offset: offset + T * stride].view(T, stride)[:, :C] = False
    assert buf[gaps].eq(77).all()
    (a, b), (c, d) = mxs.combine_rows_backward(xv, rv, order, w), mxs.combine_rows_backward(x, rows, order, w)
    assert torch.equal(a, c)
    mag = torch.from_numpy(np.stack([[float((x[t].double() * rows[row[t, j]].double()).abs().sum()) if row[t, j] >= 0 else 0.0
                                      for j in range(k)] for t in range(T)])).cuda()
    assert ((b - d).double().abs() <= 2 * (C + 1) * 2.0 ** -24 * mag).all()   # sums in another order
    e = torch.tensor(ends, dtype=torch.int32, device="cuda")
    for got, want in ((mxs.quantize_rows(xv), mxs.quantize_rows(x)), (mxs.quantize_rows(xv, block=32, order=order), mxs.quantize_rows(x, block=32, order=order)),
                      (mxs.quantize_cols(rv, e), mxs.quantize_cols(rows, e)), (mxs.quantize_blocks(xv[None]), mxs.quantize_blocks(x[None]))):
        assert torch.equal(got[0].view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("offset,stride", [(0, 300), (1, 301), (8, 304), (4, 308)])
def test_quantized_rows_that_start_anywhere(mxlib, offset, stride):
    """8-bit outputs at any alignment through the C entry points; the bytes between rows are left alone."""
    from scale_factor_layout_b200 import _binding as B

    rng = np.random.default_rng(offset)
    R, C = 70, 299
    x = hard_values(rng, R, C, BF).cuda()
    stream = torch.cuda.current_stream().cuda_stream
    ends = torch.tensor([40, 70], dtype=torch.int32, device="cuda")
    P = B.mx_padded_rows(R, 2)

    def check(rows, call, want_q, want_s):
        buf = torch.full((rows * stride + 16,), 0xA5, dtype=torch.uint8, device="cuda")
        s = torch.zeros(want_s.numel(), dtype=torch.uint8, device="cuda")
        assert call(buf.data_ptr() + offset, s.data_ptr()) == B.MX_OK
        torch.cuda.synchronize()
        body = buf[offset: offset + rows * stride].view(rows, stride)
        assert torch.equal(body[:, :C], want_q.view(torch.uint8).reshape(rows, C)) and torch.equal(s, want_s.reshape(-1))
        assert body[:, C:].eq(0xA5).all() and buf[:offset].eq(0xA5).all() and buf[offset + rows * stride:].eq(0xA5).all()

    q, s = mxs.quantize_rows(x)
    check(R, lambda p, t: B.mx_quantize_rows(x.data_ptr(), B.MX_BF16, R, C, C, 128, B.MX_E4M3, 0, 0, 0, 0, p, stride, t, 1, R, stream), q, s.t().contiguous())
    q, s = mxs.quantize_cols(x, ends)
    check(P, lambda p, t: B.mx_quantize_cols(x.data_ptr(), B.MX_BF16, R, C, C, ends.data_ptr(), 2, B.MX_E4M3, p, stride, t, C, stream), q, s)
    q, s = mxs.quantize_blocks(x[None])
    check(R, lambda p, t: B.mx_quantize_blocks(x.data_ptr(), B.MX_BF16, 1, R, C, R * C, C, B.MX_E4M3, p, R * stride, stride, t, stream), q, s)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("C", [1, 2, 3, 6, 7, 8, 9, 15, 16, 17, 23, 31, 257, 4095, 4097, 8231])
@pytest.mark.parametrize("k", [1, 3])
def test_dispatch_of_odd_strides(mxlib, dtype, C, k):
    """Each row starts at another alignment, in the tokens and in expert order: the same bits arrive, and no gap is written."""
    rng = np.random.default_rng(C + k)
    T, E = 19, 4
    order, (ends, row, slot) = order_for(rng, T, k, E)
    bits = torch.from_numpy(rng.integers(-32768, 32768, size=(T, C + C % 2 + 3)).astype(np.int16))
    x = bits.cuda().view(dtype)[:, 1:C + 1]
    stride = C + 5 + C % 2
    buf = torch.full((T * k * stride + 8,), 77, dtype=torch.int16, device="cuda")
    out = buf[3: 3 + T * k * stride].view(T * k, stride)[:, :C]
    mxs.dispatch_rows(x, order, out=out.view(dtype))
    want = torch.full((T * k * stride + 8,), 77, dtype=torch.int16)
    inner = want[3: 3 + T * k * stride].view(T * k, stride)
    inner[:, :C] = 0
    for t in range(T):
        for j in range(k):
            if row[t, j] >= 0:
                inner[row[t, j], :C] = bits[t, 1:C + 1]
    assert torch.equal(buf.cpu(), want)
