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
