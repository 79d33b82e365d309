"""Plain forms of the mixture-of-experts operators in 64 bits on the CPU, from
their definitions, for the tests of the CUDA path."""
from __future__ import annotations

import numpy as np
import torch

FEXP = {torch.float8_e4m3fn: 8, torch.float8_e5m2: 15}
FRACTION = {torch.float8_e4m3fn: (3, -6), torch.float8_e5m2: (2, -14)}


def up(n, m):
    return -(-n // m) * m


def sort(ids: np.ndarray, E: int):
    """(group_ends, row_of_slot, slot_of_row) of integer ids [tokens, choices]."""
    flat = ids.reshape(-1)
    slots = [s for e in range(E) for s in np.flatnonzero(flat == e)]
    ends = np.cumsum([int((flat == e).sum()) for e in range(E)])
    row = np.full(flat.size, -1)
    slot = np.full(flat.size, -1)
    row[slots] = np.arange(len(slots))
    slot[:len(slots)] = slots
    return ends, row.reshape(ids.shape), slot


def dispatch(x: torch.Tensor, slot: np.ndarray, k: int) -> torch.Tensor:
    out = torch.zeros(len(slot), x.shape[1], dtype=x.dtype)
    live = slot >= 0
    out[torch.from_numpy(live)] = x[torch.from_numpy(slot[live] // k)]
    return out


def combine(rows: torch.Tensor, row: np.ndarray, w):
    """(sum, sum of magnitudes) in 64 bits."""
    T, k = row.shape
    y = torch.zeros(T, rows.shape[1], dtype=torch.float64)
    mag = torch.zeros_like(y)
    for t in range(T):
        for j in range(k):
            if row[t, j] >= 0:
                v = rows[row[t, j]].double() * (1.0 if w is None else float(w[t, j]))
                y[t] += v
                mag[t] += v.abs()
    return y, mag


def quantize_block(v: np.ndarray, dtype):
    """(values, scale byte) of one block given as float64."""
    if not np.isfinite(v).all():
        return np.full(v.shape, np.nan), 255
    amax, top = float(np.abs(v).max(initial=0.0)), 1.75 * 2.0 ** FEXP[dtype]
    e = -127
    while e < 127 and amax > top * 2.0 ** e:
        e += 1
    bits, low = FRACTION[dtype]
    x = v / 2.0 ** e
    _, exp = np.frexp(x)
    step = 2.0 ** (np.maximum(exp - 1, low) - bits)
    return np.rint(x / step) * step, e + 127   # rint: ties to even


def quantize(x: torch.Tensor, dtype, rows: int, cols: int):
    """(values, bytes) of a matrix in blocks of rows x cols."""
    v = x.double().numpy()
    R, C = v.shape
    out = np.zeros((R, C))
    scale = np.zeros((up(R, rows) // rows, up(C, cols) // cols), np.uint8)
    for i in range(scale.shape[0]):
        for j in range(scale.shape[1]):
            at = np.s_[i * rows:(i + 1) * rows, j * cols:(j + 1) * cols]
            out[at], scale[i, j] = quantize_block(v[at], dtype)
    return out, scale


def clamp_ends(ends, rows):
    """Group ends as the kernels read them: monotone and within the rows."""
    out, last = [], 0
    for e in ends:
        last = min(max(int(e), last), rows)
        out.append(last)
    return out


def pad_groups(x: torch.Tensor, ends) -> torch.Tensor:
    P = up(x.shape[0], 128) + 128 * len(ends)
    out = torch.zeros(P, x.shape[1], dtype=x.dtype)
    at = begin = 0
    for e in ends:
        out[at:at + e - begin] = x[begin:e]
        at, begin = at + up(e - begin, 128), e
    return out


def powers(s: torch.Tensor) -> torch.Tensor:
    """E8M0 bytes as 64-bit numbers."""
    return torch.from_numpy(np.ldexp(1.0, s.cpu().numpy().astype(np.int64) - 127))


def spread(s: torch.Tensor, block: int, dim: int, size: int) -> torch.Tensor:
    return s.repeat_interleave(block, dim).narrow(dim, 0, size)
