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
