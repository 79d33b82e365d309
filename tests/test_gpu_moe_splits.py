"""Products whose tiles' contraction is shared by a cluster of CTAs, and weight
gradients on the other tiles that few shapes take: against 64-bit products of
the dequantized operands.  Each case names the tiles that it is there for."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import moe_reference as ref  # noqa: E402
import scale_factor_layout_b200 as mxs  # noqa: E402
from scale_factor_layout_b200 import _binding as B  # noqa: E402

BF, HF, FL = torch.bfloat16, torch.float16, torch.float32
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
SMS = 148

# sizes of groups, rows behind them, N, K, tiles
ROWS = [
    ([260], 0, 2100, 1100, 2),                # 9 steps: 8 and 1
    ([300, 7], 5, 520, 1000, 2),
    ([1], 0, 130, 2050, 4),                   # 17 steps: 8, 8, 1 and none
    ([77, 0, 100], 5, 257, 2176, 4),
    ([130, 1], 0, 900, 2064, 4),
    ([150], 0, 1100, 4224, 4),                # 33 steps: 12, 12, 9 and none
    ([0, 0], 3, 40, 2048, 4),                 # nothing but rows behind the last group
    ([1], 0, 1, 4224, 8),                     # 33 steps: four of 8, one of 1, three of none
    ([200, 0], 7, 257, 4224, 8),
    ([5, 120], 0, 130, 8304, 8),              # 65 steps: five of 12, one of 5, two of none
    ([128], 0, 128, 4096, 8),
]
# sizes of groups, columns of a, columns of b, tiles
OUTER = [
    ([2100], 130, 257, 4), ([4100, 0], 130, 40, 4), ([700, 2000], 257, 288, 2), ([0, 4300], 1, 257, 4),
    ([4200], 129, 72, 8), ([12000, 0, 300], 40, 130, 8), ([4224], 128, 1, 8),
    ([700, 0, 129, 1, 300, 128, 0, 40], 100, 2600, B.MX_TILES_WIDE), ([100, 300] * 4, 77, 2441, B.MX_TILES_WIDE),
    ([1000, 0, 333], 1000, 1300, B.MX_TILES_PAIRS), ([600], 2000, 1301, B.MX_TILES_PAIRS),
    ([300], 1285, 2049, B.MX_TILES_PAIRS_ACROSS), ([200, 0, 77], 1029, 2573, B.MX_TILES_PAIRS_ACROSS),
    ([900, 0, 1300], 1400, 2560, B.MX_TILES_PAIRS_ACROSS),
]


def padded(sizes):
    return ref.up(sum(sizes), 128) + 128 * len(sizes)


def test_tiles_of_the_cases(mxlib):
    """What each case is there for, also where there is no GPU."""
    for sizes, behind, N, K, tiles in ROWS:
        assert B.mx_select_tiles(B.MX_GROUPS_M, sum(sizes) + behind, N, K, len(sizes), SMS) == tiles, (sizes, N, K)
    for sizes, M, N, tiles in OUTER:
        assert B.mx_select_tiles(B.MX_GROUPS_K, M, N, padded(sizes), len(sizes), SMS) == tiles, (sizes, M, N)
    assert B.mx_select_tiles(B.MX_GROUPS_M, 131072, 1408, 7168, 8, SMS) == B.MX_TILES_PAIRS
    assert B.mx_select_tiles(B.MX_GROUPS_M, 128, 1408, 7168, 64, SMS) == B.MX_TILES_WIDE
    assert B.mx_select_tiles(B.MX_GROUPS_M, 128, 1408, 512, 4, SMS) == B.MX_TILES_NARROW
    for bad in ((2, 1, 1, 1, 1, SMS), (0, 0, 1, 1, 1, SMS), (0, 1, 0, 1, 1, SMS), (0, 1, 1, 0, 1, SMS), (0, 1, 1, 1, 65, SMS),
                (0, 1, 1, 1, 0, SMS), (0, 1, 1, 1, 1, 0), (0, 2**31, 1, 1, 1, SMS)):
        assert B.mx_select_tiles(*bad) == B.MX_TILES_NONE


def operand(gen, shape, dtype):
    """8-bit values whose rows start on 16-byte boundaries, NaN between them."""
    v = (torch.randn(shape, device="cuda", generator=gen) * (60 if dtype is E4 else 8000)).to(dtype)
    buf = torch.full((*shape[:-1], ref.up(shape[-1], 16) + 16), 0x7F, dtype=torch.uint8, device="cuda")
    buf[..., :shape[-1]] = v.view(torch.uint8)
    return buf.view(dtype)[..., :shape[-1]]


def scales(gen, shape, dtype):
    low = 112 if dtype is E4 else 105
    return torch.randint(low, low + 12, shape, dtype=torch.uint8, device="cuda", generator=gen)


def wide(q, s, rows, cols):
    """Quantized values as 64-bit numbers, scales of blocks of rows x cols."""
    p = ref.powers(s).cuda()
    return q.double() * p.repeat_interleave(rows, -2)[..., :q.shape[-2], :].repeat_interleave(cols, -1)[..., :q.shape[-1]]


def near(got, want, mag, steps, parts):
    """A matrix instruction adds 32 products to the sum; with every term cut to 23 bits below the largest
    each is off by at most 33 * 2^-23 of the magnitudes (4 instructions a step of 128).  Parts are added up
    in 32 bits, each addition off by at most 2^-24 of them.  Then one rounding to the output's type, which
    is off by half a step of the value or of the type's smallest number."""
    info = torch.finfo(got.dtype)
    err = (4 * steps * 33 * 2.0 ** -23 + (parts - 1) * 2.0 ** -24) * mag
    tol = err + info.eps / 2 * (want.abs() + err) + info.smallest_normal * info.eps / 2
    off = (got.double() - want).abs()
    assert bool((off <= tol).all()), f"{int((off > tol).sum())} of {off.numel()} values off, worst by {float((off - tol).max())}"


def outputs(shape, dtype):
    """None (dense rows), rows on 16-byte boundaries with gaps, rows off them; NaN around the last two."""
    yield None, None
    for stride, first in ((ref.up(shape[-1], 8) + 8, 8), (shape[-1] + 3 + shape[-1] % 2, 1)):
        rows = int(np.prod(shape[:-1]))
        buf = torch.full((first + rows * stride,), float("nan"), dtype=dtype, device="cuda")
        yield buf, buf[first:].view(*shape[:-1], stride)[..., :shape[-1]]


def same_in_every_output(call, shape, dtype):
    first = None
    for buf, out in outputs(shape, dtype):
        got = call(out)
        if out is None:
            first = got
            continue
        assert torch.equal(got, first)
        got.zero_()
        assert int((~buf.isnan()).sum()) == out.numel(), "something beside the output was written"
    return first


@pytest.mark.gpu
@pytest.mark.parametrize("sizes,behind,N,K,tiles", ROWS)
@pytest.mark.parametrize("ta,tb,out", [(E4, E4, BF), (E5, E4, FL), (E4, E5, HF)])
@pytest.mark.parametrize("form", ["nk", "kn", "blocked"])
def test_split_rows_in_groups(mxlib, sizes, behind, N, K, tiles, ta, tb, out, form):
    assert torch.cuda.get_device_properties(0).multi_processor_count == SMS
    gen = torch.Generator(device="cuda").manual_seed(N + K)
    R, G, ends = sum(sizes) + behind, len(sizes), np.cumsum(sizes)
    e = torch.tensor(ends, dtype=torch.int32, device="cuda")
    a, b = operand(gen, (R, K), ta), operand(gen, (G, K, N) if form == "kn" else (G, N, K), tb)
    KB, NB, cols = ref.up(K, 128) // 128, ref.up(N, 128) // 128, ref.up(K, 32) // 32
    if form == "blocked":
        sa, sb = scales(gen, (R, cols), ta), scales(gen, (G * N, cols), tb)
        even = torch.arange(1, G + 1, dtype=torch.int32, device="cuda") * N
        ra, rb = mxs.rearrange_m_groups(sa, e), mxs.rearrange_m_groups(sb, even)
        got = same_in_every_output(lambda o: mxs.grouped_matmul(a, ra, b, rb, e, block=32, out_dtype=out, out=o), (R, N), out)
        av, bv = wide(a, sa, 1, 32), wide(b.reshape(G * N, K), sb, 1, 32).view(G, N, K)
    else:
        sa, sb = scales(gen, (KB, R), ta).t(), scales(gen, (G, KB, NB) if form == "kn" else (G, NB, KB), tb)
        got = same_in_every_output(lambda o: mxs.grouped_matmul(a, sa, b, sb, e, b_layout=form, out_dtype=out, out=o), (R, N), out)
        av, bv = wide(a, sa, 1, 128), wide(b, sb, 128, 128)
    begin = 0
    for g, end in enumerate(ends):
        m = bv[g] if form == "kn" else bv[g].t()
        near(got[begin:end], av[begin:end] @ m, av[begin:end].abs() @ m.abs(), KB, tiles)
        begin = end
    assert got[begin:].eq(0).all() and mxs.mx_device_flags() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("sizes,M,N,tiles", OUTER)
@pytest.mark.parametrize("ta,tb,out", [(E5, E4, BF), (E4, E4, FL), (E4, E5, HF)])
def test_weight_gradients_on_every_kind_of_tile(mxlib, sizes, M, N, tiles, ta, tb, out):
    assert torch.cuda.get_device_properties(0).multi_processor_count == SMS
    gen = torch.Generator(device="cuda").manual_seed(M + N)
    G, ends, P = len(sizes), np.cumsum(sizes), padded(sizes)
    real = ref.pad_groups(torch.ones(sum(sizes), 1), ends).bool()[:, 0].cuda()
    a, b = operand(gen, (P, M), ta), operand(gen, (P, N), tb)
    a.view(torch.uint8)[~real] = 0
    b.view(torch.uint8)[~real] = 0
    sa, sb = scales(gen, (P // 128, M), ta), scales(gen, (P // 128, N), tb)
    e = torch.tensor(ends, dtype=torch.int32, device="cuda")
    got = same_in_every_output(lambda o: mxs.grouped_matmul_k(a, sa, b, sb, e, out_dtype=out, out=o), (G, M, N), out)
    av, bv, at = wide(a, sa, 128, 1), wide(b, sb, 128, 1), 0
    for g, n in enumerate(sizes):
        x, y, steps = av[at:at + n], bv[at:at + n], ref.up(n, 128) // 128
        near(got[g], x.t() @ y, x.t().abs() @ y.abs(), steps, tiles if tiles <= 8 else 1)
        at += ref.up(n, 128)
    assert mxs.mx_device_flags() == 0


@pytest.mark.gpu
def test_accuracy_of_one_long_sum(mxlib):
    """The longest sum that one accumulator takes in the measured work: a weight gradient over 131072
    rows of one group, of positive values.  Each instruction, of 32 products, cuts the running sum to 23 bits
    behind its first: 2^-23 of it, 4096 times."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    R, M = 131072, 2560
    assert B.mx_select_tiles(B.MX_GROUPS_K, M, M, R + 128, 1, SMS) == B.MX_TILES_PAIRS
    a, b = (torch.zeros(R + 128, M, dtype=torch.uint8, device="cuda") for _ in range(2))
    for t in (a, b):
        for at in range(0, R, 16384):
            t[at:at + 16384] = (torch.randn(16384, M, device="cuda", generator=gen) * 60).to(E4).view(torch.uint8) & 0x7F
    s = torch.full((R // 128 + 1, M), 120, dtype=torch.uint8, device="cuda")
    ends = torch.tensor([R], dtype=torch.int32, device="cuda")
    a, b = a.view(E4), b.view(E4)
    got = mxs.grouped_matmul_k(a, s, b, s, ends, out_dtype=FL)[0, :128, -128:].double()
    want = a[:, :128].double().t() @ b[:, -128:].double() * 2.0 ** -14
    err = float(((got - want) / want).abs().max())
    print(f"largest relative error of sums of {R} positive products: {err:.3g}")
    assert err <= R / 32 * 2.0 ** -23
    assert mxs.mx_device_flags() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("R,G,N,K", [(128, 64, 1408, 2048), (5000, 8, 1408, 4096), (120, 2, 257, 4224)])
def test_larger_products_repeat_bit_for_bit(mxlib, R, G, N, K):
    gen = torch.Generator(device="cuda").manual_seed(R)
    a, b = operand(gen, (R, K), E4), operand(gen, (G, N, K), E4)
    sa, sb = scales(gen, (R, ref.up(K, 128) // 128), E4), scales(gen, (G, ref.up(N, 128) // 128, ref.up(K, 128) // 128), E4)
    ends = torch.sort(torch.randint(0, R, (G,), device="cuda", generator=gen, dtype=torch.int32)).values
    first = mxs.grouped_matmul(a, sa, b, sb, ends)
    for _ in range(20):
        assert torch.equal(mxs.grouped_matmul(a, sa, b, sb, ends), first)
    assert mxs.mx_device_flags() == 0
