"""The mixture-of-experts operators as they are used: one layer forward and
backward against 64 bits, captured and replayed graphs, several streams and
threads, large products on both kernels, and offsets past 32 bits."""
import threading

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import moe_reference as ref  # noqa: E402
import scale_factor_layout_b200 as mxs  # noqa: E402

pytestmark = pytest.mark.gpu

BF, E4, E5 = torch.bfloat16, torch.float8_e4m3fn, torch.float8_e5m2


def wide(q, s, rows, cols):
    """Quantized values as 64-bit numbers on the GPU, blocks of rows x cols."""
    p = ref.powers(s).cuda()
    return q.double() * p.repeat_interleave(rows, -2)[..., :q.shape[-2], :].repeat_interleave(cols, -1)[..., :q.shape[-1]]


def near(got, want, mag, K, out_eps):
    """32-bit sums of K products by matrix instructions of 32 with every term cut to
    23 bits below the largest, then one rounding to the output's type."""
    tol = (ref.up(K, 128) // 32) * 33 * 2.0 ** -23 * mag + out_eps / 2 * want.abs()
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), f"{int((err > tol).sum())} values off, worst by {float((err - tol).max())}"


def layer(x, weight, ids, w, grad):
    """One expert layer, forward and backward, with every intermediate result."""
    order = mxs.expert_sort(ids, weight.shape[0])
    q, s = mxs.quantize_rows(x, order=order)
    wq, ws = mxs.quantize_blocks(weight)
    rows = mxs.grouped_matmul(q, s, wq, ws, order.group_ends)
    y = mxs.combine_rows(rows, order, w)
    d_rows, d_w = mxs.combine_rows_backward(grad, rows, order, w)
    dq, ds = mxs.quantize_rows(d_rows, dtype=E5)
    d_in = mxs.grouped_matmul(dq, ds, wq, ws, order.group_ends, b_layout="kn")
    d_x = mxs.combine_rows(d_in, order)
    gq, gs = mxs.quantize_cols(d_rows, order.group_ends, dtype=E5)
    xq, xs = mxs.quantize_cols(mxs.dispatch_rows(x, order), order.group_ends)
    d_weight = mxs.grouped_matmul_k(gq, gs, xq, xs, order.group_ends, out_dtype=torch.float32)
    return dict(order=order, q=q, s=s, wq=wq, ws=ws, rows=rows, y=y, d_rows=d_rows, d_w=d_w, dq=dq, ds=ds, d_in=d_in,
                d_x=d_x, gq=gq, gs=gs, xq=xq, xs=xs, d_weight=d_weight)


def inputs(seed, T=300, k=3, E=5, C=264, N=400):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, C, device="cuda", generator=g).to(BF)
    weight = (torch.randn(E, N, C, device="cuda", generator=g) / C ** 0.5).to(BF)
    ids = torch.randint(-1, E, (T, k), device="cuda", generator=g)
    ids[ids == 2] = 3   # an expert with no tokens
    w = torch.rand(T, k, device="cuda", generator=g)
    grad = torch.randn(T, N, device="cuda", generator=g).to(BF)
    return x, weight, ids, w, grad


def test_layer_forward_and_backward(mxlib):
    x, weight, ids, w, grad = inputs(0)
    r = layer(x, weight, ids, w, grad)
    E, N, C = weight.shape
    ends = [0, *r["order"].group_ends.tolist()]
    a, b = wide(r["q"], r["s"], 1, 128), wide(r["wq"], r["ws"], 128, 128)
    da, ga, xa = wide(r["dq"], r["ds"], 1, 128), wide(r["gq"], r["gs"], 128, 1), wide(r["xq"], r["xs"], 128, 1)
    # each product from its own quantized operands
    at = 0
    for e in range(E):
        lo, hi = ends[e], ends[e + 1]
        near(r["rows"][lo:hi], a[lo:hi] @ b[e].t(), a[lo:hi].abs() @ b[e].t().abs(), C, torch.finfo(BF).eps)
        near(r["d_in"][lo:hi], da[lo:hi] @ b[e], da[lo:hi].abs() @ b[e].abs(), N, torch.finfo(BF).eps)
        g, i = ga[at:at + hi - lo], xa[at:at + hi - lo]
        near(r["d_weight"][e], g.t() @ i, g.t().abs() @ i.abs(), max(1, hi - lo), torch.finfo(torch.float32).eps)
        at += ref.up(hi - lo, 128)
    assert r["rows"][ends[-1]:].eq(0).all() and r["d_in"][ends[-1]:].eq(0).all()
    # quantization: e4m3 is off by at most 2^-4 of a value (or, below its normal numbers, 2^-10 of the block's scale)
    full = mxs.dispatch_rows(x, r["order"]).double()
    step = a.new_tensor(2.0) ** (r["s"].double() - 127 - 10)
    assert ((a - full).abs() <= 2.0 ** -4 * full.abs() + step.repeat_interleave(128, 1)[:, :C]).all()
    # the whole layer against unquantized 64-bit values: two operands with relative errors up to
    # 2^-4 each, spread as rounding errors are, leave a few percent of the norm
    live = (ids >= 0)
    want = torch.zeros(x.shape[0], N, dtype=torch.float64, device="cuda")
    for e in range(E):
        for j in range(ids.shape[1]):
            t = (ids[:, j] == e).nonzero()[:, 0]
            want[t] += w[t, j, None].double() * (x[t].double() @ weight[e].double().t())
    assert float((r["y"].double() - want).norm() / want.norm()) < 2 * 2.0 ** -4
    assert live.any() and mxs.mx_device_flags() == 0


def results(r):
    return [t for v in r.values() for t in (v if isinstance(v, tuple) else (v,))]


def same(a, b):
    return all(torch.equal(p.view(torch.uint8) if p.element_size() == 1 else p, q.view(torch.uint8) if q.element_size() == 1 else q)
               for p, q in zip(results(a), results(b)))


def test_calls_repeat_bit_for_bit(mxlib):
    args = inputs(1)
    first = layer(*args)
    for _ in range(3):
        assert same(first, layer(*args))


def test_graphs(mxlib):
    """The layer captured twice; the two graphs replay at once on two streams, with new inputs."""
    want = [layer(*inputs(s)) for s in (2, 3)]
    graphs = []
    for s in (4, 5):
        static = [t.clone() for t in inputs(s)]
        layer(*static)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = layer(*static)
        graphs.append((g, static, out, torch.cuda.Stream()))
    for (g, static, out, stream), seed in zip(graphs, (2, 3)):
        for dst, src in zip(static, inputs(seed)):
            dst.copy_(src)
    torch.cuda.synchronize()
    for _ in range(5):
        for g, static, out, stream in graphs:
            with torch.cuda.stream(stream):
                g.replay()
    torch.cuda.synchronize()
    for (g, static, out, stream), w in zip(graphs, want):
        assert same(out, w)
    assert mxs.mx_device_flags() == 0


def test_threads_and_streams(mxlib):
    seeds = range(10, 16)
    args = [inputs(s, T=500 + 40 * s, C=128 + 8 * s) for s in seeds]
    want = [layer(*a) for a in args]
    torch.cuda.synchronize()
    errors = []

    def work(a, w):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(4):
                    got = layer(*a)
                stream.synchronize()
                if not same(got, w):
                    errors.append("differs")
        except Exception as exc:  # noqa: BLE001
            errors.append(repr(exc))

    threads = [threading.Thread(target=work, args=p) for p in zip(args, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not errors, errors
    assert mxs.mx_device_flags() == 0


def test_nothing_to_do(mxlib):
    """No tokens, rows, columns or groups' rows: empty results, or zeros where a result has a size."""
    dev = "cuda"
    order = mxs.expert_sort(torch.zeros(0, 2, dtype=torch.int64, device=dev), 3)
    assert order.group_ends.tolist() == [0, 0, 0] and order.row_of_slot.shape == (0, 2)
    none = torch.empty(0, 40, device=dev, dtype=BF)
    assert mxs.dispatch_rows(none, order).shape == (0, 40)
    assert mxs.combine_rows(none, order).shape == (0, 40)
    d_rows, d_w = mxs.combine_rows_backward(none, none, order, torch.empty(0, 2, device=dev))
    assert d_rows.shape == (0, 40) and d_w.shape == (0, 2)
    q, s = mxs.quantize_rows(none, order=order)
    assert q.shape == (0, 40) and s.shape == (0, 1)
    q, s = mxs.quantize_rows(torch.empty(5, 0, device=dev))
    assert q.shape == (5, 0) and s.shape == (5, 0)
    ends = torch.zeros(2, dtype=torch.int32, device=dev)
    q, s = mxs.quantize_cols(none, ends)
    assert q.shape == (256, 40) and q.float().eq(0).all() and s.eq(0).all()
    got = mxs.grouped_matmul_k(q, s, q, s, ends)
    assert got.shape == (2, 40, 40) and got.eq(0).all()
    wq, ws = mxs.quantize_blocks(torch.randn(2, 24, 40, device=dev))
    assert mxs.quantize_blocks(torch.empty(0, 24, 40, device=dev))[0].shape == (0, 24, 40)
    assert mxs.grouped_matmul(*mxs.quantize_rows(none), wq, ws, ends).shape == (0, 24)
    x = torch.randn(7, 40, device=dev, dtype=BF)
    assert mxs.grouped_matmul(*mxs.quantize_rows(x), wq, ws, ends).eq(0).all()       # all rows behind the last group
    empty = mxs.quantize_blocks(torch.empty(2, 0, 40, device=dev))
    assert mxs.grouped_matmul(*mxs.quantize_rows(x), *empty, ends).shape == (7, 0)
    assert mxs.mx_device_flags() == 0


def operand(gen, shape, dtype):
    v = (torch.randn(shape, device="cuda", generator=gen) * (60 if dtype is E4 else 8000)).to(dtype)
    buf = torch.zeros((*shape[:-1], ref.up(shape[-1], 16)), dtype=torch.uint8, device="cuda").view(dtype)
    buf.view(torch.uint8)[..., :shape[-1]] = v.view(torch.uint8)
    return buf[..., :shape[-1]]


def scales(gen, shape, dtype):
    low = 112 if dtype is E4 else 105
    return torch.randint(low, low + 12, shape, dtype=torch.uint8, device="cuda", generator=gen)


@pytest.mark.parametrize("sizes,behind,N,K", [
    ([1000, 0, 333], 700, 1000, 1300),     # 256-row tiles, a half-empty one, rows behind, narrow last columns
    ([129, 255, 256, 257, 511], 0, 288, 512), ([4000], 1, 2320, 144), ([5, 3000, 7, 1500], 0, 130, 2048),
    ([90] * 64, 33, 520, 400), ([300] * 64, 0, 96, 128),
    ([20000, 5], 100, 1, 48), ([9000] * 3, 0, 40, 200),   # pairs on narrow tiles
    # many short tiles, ragged ends stored element by element, and a run of empty tiles at the end: a
    # warp still busy with its stores must not lose its next tile to the ones announced after it
    ([1187, 0, 1700, 1102, 742, 1326, 2740, 2043, 656, 426, 668, 1061, 208, 916, 453, 583], 490, 4080, 1408),
])
@pytest.mark.parametrize("ta,tb,out", [(E4, E4, BF), (E5, E4, torch.float32)])
@pytest.mark.parametrize("form", ["nk", "kn", "blocked"])
def test_larger_products(mxlib, sizes, behind, N, K, ta, tb, out, form):
    gen = torch.Generator(device="cuda").manual_seed(N + K)
    R, G, ends = sum(sizes) + behind, len(sizes), np.cumsum(sizes)
    e = torch.tensor(ends, dtype=torch.int32, device="cuda")
    a, b = operand(gen, (R, K), ta), operand(gen, (G, K, N) if form == "kn" else (G, N, K), tb)
    KB, NB, cols = ref.up(K, 128) // 128, ref.up(N, 128) // 128, ref.up(K, 32) // 32
    if form == "blocked":
        sa, sb = scales(gen, (R, cols), ta), scales(gen, (G * N, cols), tb)
        even = torch.arange(1, G + 1, dtype=torch.int32, device="cuda") * N
        got = mxs.grouped_matmul(a, mxs.rearrange_m_groups(sa, e), b, mxs.rearrange_m_groups(sb, even), e, block=32, out_dtype=out)
        av, bv = wide(a, sa, 1, 32), wide(b.reshape(G * N, K), sb, 1, 32).view(G, N, K)
    else:
        sa, sb = scales(gen, (KB, R), ta).t(), scales(gen, (G, KB, NB) if form == "kn" else (G, NB, KB), tb)
        got = mxs.grouped_matmul(a, sa, b, sb, e, b_layout=form, out_dtype=out)
        av, bv = wide(a, sa, 1, 128), wide(b, sb, 128, 128)
    begin = 0
    for g, end in enumerate(ends):
        m = bv[g] if form == "kn" else bv[g].t()
        near(got[begin:end], av[begin:end] @ m, av[begin:end].abs() @ m.abs(), K, torch.finfo(out).eps)
        begin = end
    assert got[begin:].eq(0).all() and mxs.mx_device_flags() == 0


@pytest.mark.parametrize("sizes,M,N", [([1000, 0, 333, 5], 1000, 1300), ([700, 2000], 257, 288), ([3000], 1408, 520), ([60] * 64, 300, 272),
                                       ([900, 0, 1300], 1400, 2560), ([2000, 500], 2560, 1400)])   # one of them is computed across
@pytest.mark.parametrize("ta,tb,out", [(E5, E4, BF), (E4, E4, torch.float32)])
def test_larger_weight_gradients(mxlib, sizes, M, N, ta, tb, out):
    gen = torch.Generator(device="cuda").manual_seed(M + N)
    R, G, ends = sum(sizes), len(sizes), np.cumsum(sizes)
    P = ref.up(R, 128) + 128 * G
    real = ref.pad_groups(torch.ones(R, 1), ends).bool()[:, 0].cuda()
    a, b = operand(gen, (P, M), ta), operand(gen, (P, N), tb)
    a.view(torch.uint8)[~real] = 0
    b.view(torch.uint8)[~real] = 0
    sa, sb = scales(gen, (P // 128, M), ta), scales(gen, (P // 128, N), tb)
    got = mxs.grouped_matmul_k(a, sa, b, sb, torch.tensor(ends, dtype=torch.int32, device="cuda"), out_dtype=out)
    av, bv, at = wide(a, sa, 128, 1), wide(b, sb, 128, 1), 0
    for g, n in enumerate(sizes):
        x, y = av[at:at + n], bv[at:at + n]
        near(got[g], x.t() @ y, x.t().abs() @ y.abs(), max(n, 1), torch.finfo(out).eps)
        at += ref.up(n, 128)
    assert mxs.mx_device_flags() == 0


@pytest.mark.parametrize("ends", [[40, 30, 60], [-5, 10, 10], [100, 500, 20], [2**31 - 1, 0, 3]])
def test_bad_ends_are_clamped(mxlib, ends):
    """Ends that go back, below zero or past the rows give what the clamped ends give."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    R, N, K = 60, 64, 128
    good = ref.clamp_ends(ends, R)
    e, c = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in (ends, good))
    a, b, sa, sb = operand(gen, (R, K), E4), operand(gen, (3, N, K), E4), scales(gen, (R, 1), E4), scales(gen, (3, 1, 1), E4)
    assert torch.equal(mxs.grouped_matmul(a, sa, b, sb, e), mxs.grouped_matmul(a, sa, b, sb, c))
    x = torch.randn(R, 40, device="cuda", generator=gen)
    (q, s), (q2, s2) = mxs.quantize_cols(x, e), mxs.quantize_cols(x, c)
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)
    # padded operands end with the buffer: rows past it are zeros, their scales are not read
    P = q.shape[0]
    got = mxs.grouped_matmul_k(q, s, q, s, e)
    assert got.shape == (3, 40, 40) and bool(torch.isfinite(got).all()) and P == ref.up(R, 128) + 3 * 128
    assert mxs.mx_device_flags() == 0


def test_offsets_past_32_bits(mxlib):
    """Matrices of more than 2^31 elements (and, in 16 bits, 2^32 bytes)."""
    T, k, C = 150001, 2, 7184   # 300002 rows: 2.155e9 elements
    ids = torch.tensor([[0, 1]], device="cuda").repeat(T, 1)
    order = mxs.expert_sort(ids, 2)
    x = torch.randn(T, C, device="cuda", dtype=BF)
    rows = mxs.dispatch_rows(x, order)
    assert torch.equal(rows[:T], x) and torch.equal(rows[T:], x)
    y = mxs.combine_rows(rows, order)
    assert torch.equal(y, (x.float() * 2).to(BF))
    del y
    q, s = mxs.quantize_rows(x, order=order)
    del rows
    sample = torch.tensor([0, T - 1, T, 2 * T - 1, 250000], device="cuda")
    q1, s1 = mxs.quantize_rows(x[sample % T])
    assert torch.equal(q[sample].view(torch.uint8), q1.view(torch.uint8)) and torch.equal(s[sample], s1)
    # a product whose operand and output both pass 2^31 elements
    gen = torch.Generator(device="cuda").manual_seed(0)
    N = 7200
    b = operand(gen, (2, N, C), E4)
    sb = scales(gen, (2, ref.up(N, 128) // 128, ref.up(C, 128) // 128), E4)
    got = mxs.grouped_matmul(q, s, b, sb, order.group_ends)
    for r in sample.tolist():
        g = int(r >= T)
        x1, b1 = wide(q[r:r + 1], s[r:r + 1], 1, 128), wide(b[g], sb[g], 128, 128)
        near(got[r:r + 1], x1 @ b1.t(), x1.abs() @ b1.t().abs(), C, torch.finfo(BF).eps)
    assert mxs.mx_device_flags() == 0
