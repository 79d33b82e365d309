"""The grouped 8-bit product against 64-bit products of the dequantized
operands: both layouts of the weights, groups along the contraction, scales of
128 and of 32 in the blocked layout, all types, odd sizes, empty groups, rows
behind the last group, strides."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import moe_reference as ref  # noqa: E402
import scale_factor_layout_b200 as mxs  # noqa: E402

pytestmark = pytest.mark.gpu

BF, HF, FL = torch.bfloat16, torch.float16, torch.float32
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2


def operand(rng, shape, dtype):
    """8-bit values on the GPU with rows on 16-byte boundaries, and as 64-bit numbers."""
    v = torch.from_numpy(rng.standard_normal(shape) * (60 if dtype is E4 else 8000)).float().to(dtype)
    buf = torch.full((*shape[:-1], ref.up(shape[-1], 16) + 16), float("nan"), dtype=torch.float32).to(dtype).cuda()
    buf.view(torch.uint8)[..., :shape[-1]] = v.view(torch.uint8).cuda()
    return buf[..., :shape[-1]], v.double()


def scales(rng, shape, dtype):
    low = 112 if dtype is E4 else 105
    return torch.from_numpy(rng.integers(low, low + 12, size=shape, dtype=np.uint8))


def check(got, want, mag, K):
    """A matrix instruction adds 32 products to the sum; with every term cut to 23
    bits below the largest, each of the K / 32 of them is off by at most 33 * 2^-23
    of the magnitudes so far.  Then one rounding to the output's type."""
    half = torch.finfo(got.dtype).eps / 2
    steps = ref.up(K, 128) // 32
    got = got.cpu().double()
    tol = steps * 33 * 2.0 ** -23 * mag + half * want.abs() + (2.0 ** -25 if half == 2.0 ** -11 else 0)
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}: " \
                          f"{got[bad][:4].tolist()} for {want[bad][:4].tolist()}"


def by_group(a, b_of, ends, N):
    out = torch.zeros(a.shape[0], N, dtype=torch.float64)
    mag = torch.zeros_like(out)
    begin = 0
    for g, e in enumerate(ends):
        out[begin:e] = a[begin:e] @ b_of(g)
        mag[begin:e] = a[begin:e].abs() @ b_of(g).abs()
        begin = e
    return out, mag


ROW_CASES = [
    # sizes of groups, rows behind them, N, K
    ([1], 0, 1, 1), ([1], 0, 16, 32), ([128], 0, 128, 128), ([128], 0, 256, 256), ([5], 2, 300, 100),
    ([0, 130, 1, 0], 0, 257, 128), ([300, 7], 5, 520, 1000), ([64, 0, 200, 3, 129], 1, 384, 640),
    ([1] * 64, 0, 96, 272), ([0, 0], 9, 40, 64),
]


@pytest.mark.parametrize("sizes,behind,N,K", ROW_CASES)
@pytest.mark.parametrize("ta,tb,out", [(E4, E4, BF), (E5, E4, FL), (E4, E5, HF)])
@pytest.mark.parametrize("layout", ["nk", "kn"])
def test_rows_in_groups(mxlib, sizes, behind, N, K, ta, tb, out, layout):
    rng = np.random.default_rng(N + K)
    R, G = sum(sizes) + behind, len(sizes)
    ends = np.cumsum(sizes)
    a, av = operand(rng, (R, K), ta)
    b, bv = operand(rng, (G, N, K) if layout == "nk" else (G, K, N), tb)
    KB, NB = ref.up(K, 128) // 128, ref.up(N, 128) // 128
    sa = scales(rng, (R, KB), ta)
    sb = scales(rng, (G, NB, KB) if layout == "nk" else (G, KB, NB), tb)
    av = av * ref.spread(ref.powers(sa), 128, 1, K)
    bv = bv * ref.spread(ref.spread(ref.powers(sb), 128, 1, bv.shape[1]), 128, 2, bv.shape[2])
    want, mag = by_group(av, lambda g: bv[g].t() if layout == "nk" else bv[g], ends, N)
    e = torch.tensor(ends, dtype=torch.int32, device="cuda")
    for row_major in (True, False):   # scales row by row, and block by block
        s = sa.cuda() if row_major else sa.t().contiguous().cuda().t()
        got = mxs.grouped_matmul(a, s, b, sb.cuda(), e, b_layout=layout, out_dtype=out)
        check(got, want, mag, K)
    assert mxs.mx_device_flags() == 0


@pytest.mark.parametrize("sizes,behind,N,K", ROW_CASES)
@pytest.mark.parametrize("ta,tb,out", [(E4, E4, BF), (E5, E5, FL)])
def test_blocked_scales(mxlib, sizes, behind, N, K, ta, tb, out):
    rng = np.random.default_rng(N + K)
    R, G = sum(sizes) + behind, len(sizes)
    ends = np.cumsum(sizes)
    a, av = operand(rng, (R, K), ta)
    b, bv = operand(rng, (G, N, K), tb)
    cols = ref.up(K, 32) // 32
    sa, sb = scales(rng, (R, cols), ta), scales(rng, (G * N, cols), tb)
    av = av * ref.spread(ref.powers(sa), 32, 1, K)
    bv = bv * ref.spread(ref.powers(sb), 32, 1, K).view(G, N, K)
    want, mag = by_group(av, lambda g: bv[g].t(), ends, N)
    e = torch.tensor(ends, dtype=torch.int32, device="cuda")
    even = torch.arange(1, G + 1, dtype=torch.int32, device="cuda") * N
    got = mxs.grouped_matmul(a, mxs.rearrange_m_groups(sa.cuda(), e), b, mxs.rearrange_m_groups(sb.cuda(), even), e,
                             block=32, out_dtype=out)
    check(got, want, mag, K)
    assert mxs.mx_device_flags() == 0


@pytest.mark.parametrize("sizes,M,N", [
    ([1], 1, 1), ([128], 128, 256), ([256], 128, 128), ([5, 0, 300], 40, 72), ([130, 1, 127, 128], 129, 300),
    ([0, 0], 16, 16), ([1] * 64, 64, 48), ([700], 257, 520),
])
@pytest.mark.parametrize("ta,tb,out", [(E5, E4, BF), (E4, E4, FL), (E4, E5, HF)])
def test_contraction_in_groups(mxlib, sizes, M, N, ta, tb, out):
    rng = np.random.default_rng(M + N)
    R, G = sum(sizes), len(sizes)
    ends = np.cumsum(sizes)
    P = ref.up(R, 128) + 128 * G
    real = ref.pad_groups(torch.ones(R, 1), ends).bool()[:, 0]
    a, av = operand(rng, (P, M), ta)
    b, bv = operand(rng, (P, N), tb)
    for q, v in ((a, av), (b, bv)):
        q.view(torch.uint8)[~real.cuda()] = 0
        v[~real] = 0
    sa, sb = scales(rng, (P // 128, M), ta), scales(rng, (P // 128, N), tb)
    av, bv = av * ref.spread(ref.powers(sa), 128, 0, P), bv * ref.spread(ref.powers(sb), 128, 0, P)
    want, mag = torch.zeros(G, M, N, dtype=torch.float64), torch.zeros(G, M, N, dtype=torch.float64)
    at = 0
    for g, n in enumerate(sizes):
        want[g] = av[at:at + n].t() @ bv[at:at + n]
        mag[g] = av[at:at + n].abs().t() @ bv[at:at + n].abs()
        at += ref.up(n, 128)
    got = mxs.grouped_matmul_k(a, sa.cuda(), b, sb.cuda(), torch.tensor(ends, dtype=torch.int32, device="cuda"), out_dtype=out)
    check(got, want, mag, max(sizes))
    assert mxs.mx_device_flags() == 0


def test_accuracy_of_long_sums(mxlib):
    """Long contractions of positive values, where a short accumulator would lose bits."""
    rng = np.random.default_rng(0)
    K = 8192
    a, av = operand(rng, (128, K), E4)
    b, bv = operand(rng, (1, 128, K), E4)
    a.view(torch.uint8).bitwise_and_(0x7f)
    b.view(torch.uint8).bitwise_and_(0x7f)
    s = torch.full((128, K // 128), 120, dtype=torch.uint8, device="cuda")
    got = mxs.grouped_matmul(a, s, b, s[None, :1], torch.tensor([128], dtype=torch.int32, device="cuda"), out_dtype=FL)
    want = (av.abs() @ bv[0].abs().t()) * 2.0 ** -14
    err = ((got.cpu().double() - want).norm() / want.norm()).item()
    print(f"relative error of sums of {K} positive products: {err:.3g}")
    assert err <= K / 32 * 2.0 ** -23
