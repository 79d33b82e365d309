"""The torch calls of the mixture-of-experts operators as programs mix them:
threads on one stream, outputs given by the caller, hand-made orders."""
import threading

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import moe_reference as ref  # noqa: E402
import scale_factor_layout_b200 as mxs  # noqa: E402

pytestmark = pytest.mark.gpu


def test_sorts_of_threads_on_one_stream(mxlib):
    """Sorts with a workspace, made by several threads on the default stream with other work of theirs between."""
    rng = np.random.default_rng(0)
    ids = [rng.integers(-1, 9 + i, size=(3000 + 700 * i, 3)) for i in range(6)]
    want = [ref.sort(v, 8 + i) for i, v in enumerate(ids)]
    args = [torch.from_numpy(v).cuda() for v in ids]
    torch.cuda.synchronize()
    errors = []

    def work(i):
        try:
            got = []
            for _ in range(40):
                got.append(mxs.expert_sort(args[i], 8 + i))
                torch.full((37888,), 255, dtype=torch.uint8, device="cuda")   # as large as a workspace
            for order in got:
                for t, w in zip(order, want[i]):
                    if not np.array_equal(t.cpu().numpy(), w):
                        errors.append(f"thread {i} got another order")
                        return
        except Exception as exc:  # noqa: BLE001
            errors.append(repr(exc))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(ids))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not errors, errors
    assert mxs.mx_device_flags() == 0


@pytest.mark.parametrize("ends", [[100, 500, 20], [-5, 30, 10], [2**31 - 1, 0, 3], [45, 20, -2**31], [-1, -7, -2**31]])
@pytest.mark.parametrize("C", [24, 33])
def test_bad_ends_of_an_order_are_clamped(mxlib, ends, C):
    """Ends that go back, below zero or past the rows are read as everywhere: rows of a group that they
    cover are not zeroed as rows behind the last group."""
    T, k = 30, 2
    good = ref.clamp_ends(ends, T * k)
    row = torch.arange(T * k, dtype=torch.int32).view(T, k)
    row[row >= good[-1]] = -1
    row = row.cuda()
    bad, order = (mxs.ExpertOrder(torch.tensor(e, dtype=torch.int32, device="cuda"), row, row.reshape(-1)) for e in (ends, good))
    gen = torch.Generator(device="cuda").manual_seed(C)
    x, rows = (torch.randn(n, C, device="cuda", generator=gen).bfloat16() for n in (T, T * k))
    w = torch.rand(T, k, device="cuda", generator=gen)
    assert torch.equal(mxs.dispatch_rows(x, bad), mxs.dispatch_rows(x, order))
    for got, want in zip(mxs.combine_rows_backward(x, rows, bad, w), mxs.combine_rows_backward(x, rows, order, w)):
        assert torch.equal(got, want)
    for block in (32, 128):
        (q, s), (q2, s2) = mxs.quantize_rows(x, block=block, order=bad), mxs.quantize_rows(x, block=block, order=order)
        assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)
    assert (mxs.dispatch_rows(x, bad).abs().sum(1) > 0).sum() == good[-1]


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("sizes,behind,N,K", [
    ([200], 40, 131, 256),            # 128 x 128 tiles
    ([100] * 12, 0, 2441, 128),       # 128 x 256 tiles
    ([600, 0, 1000], 70, 2437, 256),  # pairs of CTAs
    ([40], 0, 129, 2304),             # a contraction that CTAs share
])
def test_products_write_nothing_beside_their_rows(mxlib, sizes, behind, N, K, out):
    """Rows that start on 16-byte boundaries and end off them, in the middle of a larger matrix."""
    gen = torch.Generator(device="cuda").manual_seed(N)
    R, G = sum(sizes) + behind, len(sizes)
    ends = torch.tensor(np.cumsum(sizes), dtype=torch.int32, device="cuda")
    (a, sa), (b, sb) = mxs.quantize_rows(torch.randn(R, K, device="cuda", generator=gen)), mxs.quantize_blocks(torch.randn(G, N, K, device="cuda", generator=gen))
    P = ref.up(R, 128) + 128 * G
    at, sat = mxs.quantize_cols(torch.randn(R, 300, device="cuda", generator=gen), ends)
    bt, sbt = mxs.quantize_cols(torch.randn(R, N, device="cuda", generator=gen), ends)
    assert at.shape[0] == P

    def check(call, shape):
        want = call(None)
        stride = ref.up(N, 8) + 8
        buf = torch.full((int(np.prod(shape[:-1])) + 2, stride), 77.0, dtype=out, device="cuda")
        inner = buf[1:-1].view(*shape[:-1], stride)[..., :N]
        assert inner.data_ptr() % 16 == 0 and torch.equal(call(inner), want)
        assert buf[:, N:].eq(77).all() and buf[0].eq(77).all() and buf[-1].eq(77).all()

    check(lambda o: mxs.grouped_matmul(a, sa, b, sb, ends, out_dtype=out, out=o), (R, N))
    check(lambda o: mxs.grouped_matmul_k(at, sat, bt, sbt, ends, out_dtype=out, out=o), (G, 300, N))
    check(lambda o: mxs.grouped_matmul_k(bt, sbt, bt, sbt, ends, out_dtype=out, out=o), (G, N, N))
    assert mxs.mx_device_flags() == 0


def test_a_captured_training_step(mxlib):
    """Dispatch and combine with their autograd backward in one graph, replayed on new inputs; a sort of
    more slots than one CTA takes, so that its workspace is the graph's."""
    T, k, E, C = 1100, 3, 5, 72
    gen = torch.Generator(device="cuda").manual_seed(0)

    def fresh():
        return (torch.randn(T, C, device="cuda", generator=gen), torch.rand(T, k, device="cuda", generator=gen),
                torch.randint(-1, E, (T, k), device="cuda", generator=gen))

    def step(x, w, ids):
        order = mxs.expert_sort(ids, E)
        y = mxs.combine_rows(mxs.dispatch_rows(x, order).square(), order, w)
        return (y, *torch.autograd.grad(y.sin().sum(), (x, w)))

    x, w, ids = fresh()
    x.requires_grad_()
    w.requires_grad_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x, w, ids)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(x, w, ids)
    for _ in range(3):
        new = fresh()
        with torch.no_grad():
            for dst, src in zip((x, w, ids), new):
                dst.copy_(src)
        graph.replay()
        want = step(new[0].requires_grad_(), new[1].requires_grad_(), new[2])
        for a, b in zip(got, want):
            assert torch.equal(a, b)
