"""What the torch calls of the mixture-of-experts operators do around their
launches, on the CPU: the library is left out or called for sizes only."""
import weakref

import pytest

torch = pytest.importorskip("torch")

import scale_factor_layout_b200 as mxs  # noqa: E402
from scale_factor_layout_b200 import moe  # noqa: E402


@pytest.fixture
def launches(monkeypatch):
    """CPU tensors pass for CUDA ones, and launches are recorded instead of made: (name, arguments)."""
    calls = []
    monkeypatch.setattr(moe, "_check_cuda", lambda **tensors: None)
    monkeypatch.setattr(moe, "_call", lambda name, device, *args: calls.append((name, args)))
    return calls


@pytest.mark.parametrize("tokens", [3, 5000])
def test_a_sort_holds_its_memory_until_its_launches(mxlib, launches, monkeypatch, tokens):
    """The memory of every pointer that the library is given belongs to a live tensor while it launches."""
    made, empty = [], torch.empty_strided

    def recorded(*args, **kwargs):
        t = empty(*args, **kwargs)
        made.append((t.data_ptr(), t.numel(), weakref.ref(t)))
        return t

    def call(name, device, *args):
        dead = [(at, n) for at, n, ref in made if n and ref() is None]
        assert not dead, f"{name} is given memory that has been freed"
        launches.append((name, args))

    monkeypatch.setattr(torch, "empty_strided", recorded)
    monkeypatch.setattr(moe, "_call", call)
    mxs.expert_sort(torch.zeros(tokens, 2, dtype=torch.int64), 8)
    assert [name for name, _ in launches] == ["mx_expert_sort"]
    needed = moe.B.mx_expert_sort_workspace(tokens, 2)
    assert (needed > 0) == (tokens == 5000) and sum(n == needed for _, n, _ in made) == (needed > 0)


def small_order(tokens=4, choices=2, experts=3):
    i32 = torch.int32
    return mxs.ExpertOrder(torch.zeros(experts, dtype=i32), torch.zeros(tokens, choices, dtype=i32),
                           torch.zeros(tokens * choices, dtype=i32))


@pytest.mark.parametrize("no_grad", [False, True])
def test_forward_mode_derivatives_are_refused(launches, no_grad):
    """There are none: a tangent raises, and does not vanish from the result."""
    from torch.autograd import forward_ad

    order, x, rows, w = small_order(), torch.ones(4, 16), torch.ones(8, 16), torch.ones(4, 2)
    with forward_ad.dual_level(), torch.set_grad_enabled(not no_grad):
        dual = lambda t: forward_ad.make_dual(t, torch.ones_like(t))   # noqa: E731
        for call in (lambda: mxs.dispatch_rows(dual(x), order), lambda: mxs.combine_rows(dual(rows), order),
                     lambda: mxs.combine_rows(dual(rows), order, w), lambda: mxs.combine_rows(rows, order, dual(w)),
                     lambda: mxs.combine_rows(dual(rows), order, dual(w))):
            with pytest.raises(NotImplementedError, match="forward mode"):
                call()
        with pytest.raises(ValueError, match="gradient"):
            mxs.dispatch_rows(dual(x), order, out=torch.empty(8, 16))
        with pytest.raises(ValueError, match="gradient"):
            mxs.combine_rows(rows, order, dual(w), out=torch.empty(4, 16))
        # without a tangent the calls are what they are elsewhere
        assert mxs.dispatch_rows(x, order).shape == (8, 16) and mxs.combine_rows(rows, order, w).shape == (4, 16)


def out_calls():
    """(name, call(out), shape, dtype) of every call that takes an output."""
    f8, u8 = torch.float8_e4m3fn, torch.uint8
    order, ends = small_order(), torch.zeros(2, dtype=torch.int32)
    a, b, at, bt = (torch.zeros(s, dtype=f8) for s in ((4, 32), (2, 16, 32), (256, 16), (256, 32)))
    s = lambda *shape: torch.zeros(shape, dtype=u8)   # noqa: E731
    return [
        ("dispatch_rows", lambda out: mxs.dispatch_rows(torch.ones(4, 16), order, out=out), (8, 16)),
        ("combine_rows", lambda out: mxs.combine_rows(torch.ones(8, 16), order, torch.ones(4, 2), out=out), (4, 16)),
        ("grouped_matmul", lambda out: mxs.grouped_matmul(a, s(4, 1), b, s(2, 1, 1), ends, out_dtype=torch.float32, out=out), (4, 16)),
        ("grouped_matmul_k", lambda out: mxs.grouped_matmul_k(at, s(2, 16), bt, s(2, 32), ends, out_dtype=torch.float32, out=out), (2, 16, 32)),
    ]


OUT_CALLS = ["dispatch_rows", "combine_rows", "grouped_matmul", "grouped_matmul_k"]


@pytest.mark.parametrize("name", OUT_CALLS)
def test_a_written_output_is_known_to_autograd(launches, name):
    """Writing into `out` counts as the change in place that it is: what was saved for a backward
    pass and is overwritten raises there, instead of giving gradients from the new values."""
    call, shape = next(c[1:] for c in out_calls() if c[0] == name)
    out = torch.ones(shape)
    leaf = torch.ones(shape, requires_grad=True)
    loss = (leaf * out).sum()
    assert call(out) is out
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():   # tensors without such a count
        assert call(torch.ones(shape)).shape == shape


@pytest.mark.parametrize("name", OUT_CALLS)
def test_an_output_that_needs_a_gradient_is_refused(launches, name):
    """Its gradient would be that of the values before the call."""
    call, shape = next(c[1:] for c in out_calls() if c[0] == name)
    leaf = torch.ones(shape, requires_grad=True)
    for out in (leaf, leaf * 2):
        with pytest.raises(ValueError, match="gradient"):
            call(out)
    with torch.no_grad():   # a parameter filled outside of any graph
        assert call(leaf) is leaf


def test_an_output_that_overlaps_an_input_is_refused(launches):
    """Kernels read rows while others are written: the same memory cannot be both."""
    order, f32 = small_order(), torch.float32
    buf = torch.ones(16, 16)
    with pytest.raises(ValueError, match="out overlaps x"):
        mxs.dispatch_rows(buf[:4], order, out=buf[:8])
    with pytest.raises(ValueError, match="out overlaps x"):
        mxs.dispatch_rows(buf[7:11], order, out=buf[:8])
    with pytest.raises(ValueError, match="out overlaps rows"):
        mxs.combine_rows(buf[:8], order, out=buf[:4])
    with pytest.raises(ValueError, match="out overlaps rows"):
        mxs.combine_rows(buf[:8, :8], order, out=buf[4:8, 7:15])
    w = torch.ones(8, 2)
    with pytest.raises(ValueError, match="out overlaps weights"):
        mxs.combine_rows(torch.ones(8, 2), order, w[:4], out=w[2:6])
    memory = torch.zeros(1 << 14, dtype=torch.uint8)
    f8, ends = torch.float8_e4m3fn, torch.zeros(2, dtype=torch.int32)
    a, b, sa, sb = (torch.zeros(s, dtype=t) for s, t in (((4, 32), f8), ((2, 16, 32), f8), ((4, 1), torch.uint8), ((2, 1, 1), torch.uint8)))
    place = lambda like, at: memory[at: at + like.numel()].view(like.dtype).view(like.shape)   # noqa: E731
    out = memory[:4 * 16 * 4].view(f32).view(4, 16)
    for i, name in enumerate(("a", "a_scales", "b", "b_scales")):
        given = [a, sa, b, sb]
        given[i] = place(given[i], 255)   # the last byte of out
        with pytest.raises(ValueError, match=f"out overlaps {name}"):
            mxs.grouped_matmul(*given, ends, out_dtype=f32, out=out)
        given[i] = place(given[i], 256)
        assert mxs.grouped_matmul(*given, ends, out_dtype=f32, out=out) is out
    at, bt, s, t = (torch.zeros(s, dtype=d) for s, d in (((256, 16), f8), ((256, 32), f8), ((2, 16), torch.uint8), ((2, 32), torch.uint8)))
    out = memory[:2 * 16 * 32 * 4].view(f32).view(2, 16, 32)
    with pytest.raises(ValueError, match="out overlaps b"):
        mxs.grouped_matmul_k(at, s, place(bt, 4000), t, ends, out_dtype=f32, out=out)


def test_an_output_beside_its_input_is_taken(launches):
    """Neighbours in one buffer do not overlap: rows behind rows, columns beside columns, every other row."""
    order, buf = small_order(), torch.ones(16, 32)
    assert mxs.dispatch_rows(buf[8:12], order, out=buf[:8]).shape == (8, 32)
    assert mxs.dispatch_rows(buf[:4, :16], order, out=buf[:8, 16:]).shape == (8, 16)
    assert mxs.combine_rows(buf[0::2], order, out=buf[1::2][:4]).shape == (4, 32)
    assert mxs.combine_rows(buf[:8, 20:30], order, out=buf[2:6, 10:20]).shape == (4, 10)
    assert mxs.combine_rows(buf[:8, :0], order, out=buf[:4, :0]).shape == (4, 0)
    one = small_order(tokens=1, choices=1)
    assert mxs.combine_rows(buf[:1, :8], one, out=buf[:1, 8:16]).shape == (1, 8)
    with pytest.raises(ValueError, match="overlaps"):
        mxs.combine_rows(buf[:1, :8], one, out=buf[:1, 7:15])


@pytest.mark.parametrize("choices", [2**31 - 2**14 + 1, 2**32 + 2])
def test_more_slots_than_31_bits_are_refused(mxlib, launches, choices):
    """Their number would lose its upper bits on the way into the library."""
    ids = torch.empty(1, choices, dtype=torch.int32, device="meta")
    with pytest.raises(ValueError, match="slots"):
        mxs.expert_sort(ids, 4)
    order = small_order()._replace(row_of_slot=ids)
    x = torch.empty(1, 16, device="meta")
    for call in (lambda: mxs.dispatch_rows(x, order), lambda: mxs.quantize_rows(x, order=order),
                 lambda: mxs.combine_rows(torch.empty(choices, 16, device="meta"), order),
                 lambda: mxs.combine_rows_backward(x, torch.empty(choices, 16, device="meta"), order, torch.empty(1, choices, device="meta"))):
        with pytest.raises(ValueError, match="slots"):
            call()
    assert not launches
    most = torch.empty(1, 2**31 - 2**14, dtype=torch.int32, device="meta")
    assert mxs.expert_sort(most, 4).row_of_slot.shape == most.shape


@pytest.mark.parametrize("name", OUT_CALLS)
def test_an_output_that_carries_a_tangent_is_refused(launches, name):
    """Its tangent would be that of the values before the call."""
    from torch.autograd import forward_ad

    call, shape = next(c[1:] for c in out_calls() if c[0] == name)
    with forward_ad.dual_level():
        with pytest.raises(ValueError, match="gradient"):
            call(forward_ad.make_dual(torch.ones(shape), torch.ones(shape)))
        plain = torch.ones(shape)
        assert call(plain) is plain
    outside = torch.ones(shape)
    with torch.inference_mode():   # a tensor that was made outside of it
        before = outside._version
        assert call(outside) is outside and outside._version > before
