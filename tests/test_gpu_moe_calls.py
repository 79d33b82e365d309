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
