"""The operators of an 8-bit mixture-of-experts layer, as measured work.

Four operators and the calls that a training or serving step makes of them:

* dispatch: slots (token, choice) sorted by expert, and the tokens' rows copied into that order;
* combine: the weighted sum of a token's rows, and its gradient;
* quantize: rows, columns of a group, or square blocks to 8-bit floating point, with one power-of-two
  scale (E8M0) for each block of 128 (or 32) values;
* product: the grouped matrix product of such operands, with groups along the rows (forward, and the
  gradient of the input) or along the contraction (the gradient of the weights).

Each has a plain form in elementary torch operations and the framework's call beside it.
"""
import math

import numpy as np
import torch

own = False

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3": E4M3, "e5m2": E5M2}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1, "e5m2": 1}
FMAX_EXP = {"e4m3": 8, "e5m2": 15}   # the largest finite value is 1.75 * 2^this in both types
BLOCK = 128


def up(n, m):
    return -(-n // m) * m


def listed():
    return [
        # One decoding step of 16 sequences, 8 of 64 experts each, rows of the 7168-wide model of the
        # repository's scale tensors (224 scales of 32): the latency of a sort and a small copy.
        dict(name="dispatch_decode", op="dispatch", T=16, k=8, E=64, C=7168, dtype="bf16", local=64, train=False),
        # A training step: 131072 rows (the repository's row count) from 16384 tokens, with the gradient.
        dict(name="dispatch_train", op="dispatch", T=16384, k=8, E=8, C=7168, dtype="bf16", local=8, train=True),
        # Serving on one of four expert-parallel ranks: 16 of 64 experts are here, the other slots are
        # dropped; an odd number of tokens and choices, rows in 32 bits.
        dict(name="combine_local_odd", op="combine", T=1003, k=7, E=64, C=1408, dtype="fp32", local=16, train=False),
        # A training step's way back: the weighted sum, then the gradients of rows and weights.
        dict(name="combine_train", op="combine", T=16384, k=8, E=8, C=4096, dtype="bf16", local=8, train=True),
        # A decoding step's activations: 128 rows.
        dict(name="quantize_rows_decode", op="quantize", kind="rows", R=128, C=7168, G=1, dtype="bf16", to="e4m3"),
        # A training step's expert inputs: tokens copied to their experts and quantized in one pass.
        dict(name="quantize_dispatch_train", op="quantize", kind="dispatch", R=16384, k=8, C=7168, G=8, dtype="bf16", to="e4m3"),
        # Output gradients for the weight gradient: blocks of 128 rows of a group, ragged groups.
        dict(name="quantize_cols_train", op="quantize", kind="cols", R=131072, C=1408, G=8, dtype="bf16", to="e5m2"),
        # Expert weights of one decoding step: 128 rows over 64 experts; the weights' bytes bound it.
        dict(name="product_decode", op="product", kind="nk", R=128, G=64, N=1408, K=7168, a="e4m3", b="e4m3", out="bf16", used=1.0),
        # A training step's expert product: 131072 rows, ragged groups.
        dict(name="product_forward", op="product", kind="nk", R=131072, G=8, N=1408, K=7168, a="e4m3", b="e4m3", out="bf16", used=1.0),
        # The gradient of the input with the forward weights as they are stored; odd sizes, some rows unused.
        dict(name="product_dgrad_odd", op="product", kind="kn", R=16301, G=16, N=4080, K=1408, a="e5m2", b="e4m3", out="bf16", used=0.97),
        # The gradient of the weights: the contraction runs over each group's rows.
        dict(name="product_wgrad", op="product", kind="wgrad", R=131072, G=8, N=7168, K=1408, a="e5m2", b="e4m3", out="bf16", used=1.0),
        # Scales for blocks of 32 in the blocked layout: the activations' scales are rearranged, then read.
        dict(name="product_blocked32", op="product", kind="blocked32", R=16384, G=8, N=4096, K=4096, a="e4m3", b="e4m3", out="bf16", used=1.0),
    ]


def spread(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dispatch", "combine", "quantize", "product"])
    if op in ("dispatch", "combine"):
        k = rng.randint(1, 8)
        E = rng.randint(k, 64)
        C = spread(rng, 64, 7168)
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        most = int(min(131072, 1.8e9 / (C * SIZE[dtype]))) // k
        return dict(op=op, T=spread(rng, 1, most), k=k, E=E, C=C, dtype=dtype,
                    local=rng.choice([E, E, rng.randint(1, E)]), train=rng.random() < 0.5)
    if op == "quantize":
        kind = rng.choice(["rows", "dispatch", "cols", "blocks", "rows32"])
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        G, C, k = rng.randint(1, 64), spread(rng, 32, 7168), rng.randint(1, min(8, 8))
        if kind == "dispatch":
            G = max(G, k)
        most = int(9e8 / C) // (k if kind == "dispatch" else 1)
        R = spread(rng, 1, min(131072 // (k if kind == "dispatch" else 1), most))
        if kind == "blocks":
            R = spread(rng, 1, max(1, min(8192, int(9e8 / C / G))))
        return dict(op=op, kind=kind, R=R, C=C, G=G, dtype=dtype, to=rng.choice(["e4m3", "e5m2"]), k=k)
    kind = rng.choice(["nk", "kn", "wgrad", "blocked32"])
    G = rng.choice([1, rng.randint(2, 16), rng.randint(17, 64)])
    N, K = spread(rng, 64, 7168), spread(rng, 64, 7168)
    R = spread(rng, 1, max(1, min(131072, int(1.3e12 / (N * K)))))
    while G * N * K > 1.2e9:
        G //= 2
    if kind == "blocked32":
        K = up(K, 32)
    return dict(op="product", kind=kind, R=R, G=max(G, 1), N=N, K=K, a=rng.choice(["e4m3", "e5m2"]), b="e4m3",
                out=rng.choice(["bf16", "fp16"]), used=rng.choice([1.0, 1.0, 0.9]))


# ------------------------------------------------------------------ inputs
def group_sizes(seed, rows, G):
    """Ragged sizes with the skew of a trained router; with many groups some are empty."""
    r = np.random.default_rng(seed)
    p = np.exp(0.7 * r.standard_normal(G))
    if G >= 4:
        p[r.integers(0, G)] = 0.0
    return r.multinomial(rows, p / p.sum())


def route(gen, T, k, E, local):
    """Expert ids and weights of a softmax router with uneven experts; ids past `local` are another rank's."""
    logits = torch.randn(T, E, device="cuda", generator=gen) + 0.7 * torch.randn(E, device="cuda", generator=gen)
    top, ids = logits.topk(k, dim=1)
    return ids.contiguous(), top.softmax(1).contiguous()


def ends_of(sizes):
    return torch.tensor(np.cumsum(sizes), dtype=torch.int32, device="cuda")


def padded_rows(shape, dtype):
    """An 8-bit matrix whose rows start on 16-byte boundaries, as tensor copies need."""
    return torch.zeros(*shape[:-1], up(shape[-1], 16), dtype=dtype, device="cuda")[..., :shape[-1]]


def eight_bit(gen, shape, dtype):
    """Values as a quantized block holds them: the block's largest in the type's last two binades."""
    q = padded_rows(shape, dtype)
    scale = 100.0 if dtype is E4M3 else 12800.0
    flat = q.view(torch.uint8) if q.dim() == 2 else q.view(torch.uint8).view(shape[0], shape[1], -1)
    step = max(1, (1 << 28) // max(1, shape[-1] * (shape[1] if len(shape) == 3 else 1)))
    for at in range(0, shape[0], step):
        v = torch.randn(min(step, shape[0] - at), *shape[1:], device="cuda", generator=gen)
        flat[at:at + step] = (v * scale).clamp_(-4 * scale, 4 * scale).to(dtype).view(torch.uint8)
    return q


def scale_bytes(gen, shape, dtype):
    """E8M0 bytes around those of unit-variance data."""
    low = 115 if dtype is E4M3 else 108
    return torch.randint(low, low + 8, shape, dtype=torch.uint8, device="cuda", generator=gen)


def to_blocked(s, G, N):
    """Equal groups' row-major scales (G * N, cols) in the blocked 128x4 layout, as weights are laid out once."""
    cols = s.shape[1]
    p = torch.zeros(G, up(N, 128), up(cols, 4), dtype=torch.uint8, device="cuda")
    p[:, :N, :cols] = s.view(G, N, cols)
    return p.view(G, up(N, 128) // 128, 4, 32, up(cols, 4) // 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(-1).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    op = case["op"]
    if op in ("dispatch", "combine"):
        T, k, C, dt = case["T"], case["k"], case["C"], TYPES[case["dtype"]]
        s["ids"], s["w"] = route(gen, T, k, case["E"], case["local"])
        if op == "dispatch":
            s["x"] = torch.randn(T, C, device="cuda", generator=gen).to(dt)
            if case["train"]:
                s["grad"] = torch.randn(T * k, C, device="cuda", generator=gen, dtype=dt)
        else:
            s["rows"] = torch.randn(T * k, C, device="cuda", generator=gen, dtype=dt)
            if case["train"]:
                s["grad"] = torch.randn(T, C, device="cuda", generator=gen, dtype=dt)
            # the order that the dispatch of the same step made
            s["order"] = plain_order(s["ids"], case["local"])
    elif op == "quantize":
        R, C, dt = case["R"], case["C"], TYPES[case["dtype"]]
        shape = (case["G"], R, C) if case["kind"] == "blocks" else (R, C)
        # activations and gradients: rows of uneven size
        rows = torch.randn(*shape[:-1], 1, device="cuda", generator=gen).exp()
        s["x"] = torch.randn(*shape, device="cuda", generator=gen, dtype=dt) * rows.to(dt)
        if case["kind"] == "dispatch":
            ids, _ = route(gen, R, case["k"], case["G"], case["G"])
            s["order"] = plain_order(ids, case["G"])
        s["sizes"] = [int(v) for v in group_sizes(seed, R, case["G"])]
        s["ends"] = ends_of(s["sizes"])
    else:
        R, G, N, K, kind = case["R"], case["G"], case["N"], case["K"], case["kind"]
        s["sizes"] = [int(v) for v in group_sizes(seed, int(R * case["used"]), G)]
        s["ends"] = ends_of(s["sizes"])
        KB, NB = up(K, BLOCK) // BLOCK, up(N, BLOCK) // BLOCK
        ta, tb = TYPES[case["a"]], TYPES[case["b"]]
        if kind == "wgrad":
            # operands in padded groups, as quantization of columns lays them out: zeros behind each group
            P = up(R, BLOCK) + BLOCK * G
            real = torch.zeros(P, dtype=torch.bool, device="cuda")
            at = 0
            for n in s["sizes"]:
                real[at:at + n] = True
                at += up(n, BLOCK)
            s["a"], s["b"] = eight_bit(gen, (P, K), ta), eight_bit(gen, (P, N), tb)
            s["a"].view(torch.uint8)[~real] = 0
            s["b"].view(torch.uint8)[~real] = 0
            s["sa"], s["sb"] = scale_bytes(gen, (P // BLOCK, K), ta), scale_bytes(gen, (P // BLOCK, N), tb)
        elif kind == "blocked32":
            s["a"], s["b"] = eight_bit(gen, (R, K), ta), eight_bit(gen, (G, N, K), tb)
            s["sa"], s["sb_rows"] = scale_bytes(gen, (R, K // 32), ta), scale_bytes(gen, (G * N, K // 32), tb)
            s["sb"] = to_blocked(s["sb_rows"], G, N)
        else:
            s["a"] = eight_bit(gen, (R, K), ta)
            s["b"] = eight_bit(gen, (G, N, K) if kind == "nk" else (G, K, N), tb)
            s["sa"] = scale_bytes(gen, (KB, R), ta).t()   # block-major, as quantization of rows writes them
            s["sb"] = scale_bytes(gen, (G, NB, KB) if kind == "nk" else (G, KB, NB), tb)
    return s


# ------------------------------------------------------------------ plain forms
def plain_order(ids, E):
    """(group_ends, row_of_slot, slot_of_row): slots with an id in [0, E), sorted by id and then by slot."""
    T, k = ids.shape
    flat = ids.reshape(-1).long()
    valid = (flat >= 0) & (flat < E)
    key = torch.where(valid, flat, E)
    slot = torch.argsort(key, stable=True)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=ids.device).scatter_add_(0, key, torch.ones_like(key))
    ends = counts[:E].cumsum(0).int()
    row = torch.empty_like(slot)
    row[slot] = torch.arange(T * k, device=ids.device)
    inside = torch.arange(T * k, device=ids.device) < ends[-1]
    slot_of_row = torch.where(inside, slot, -1).int()
    row_of_slot = torch.where(valid, row, -1).int().view(T, k)
    return ends, row_of_slot, slot_of_row


def plain_dispatch(x, slot_of_row, k):
    rows = x[slot_of_row.clamp(min=0).long() // k]
    return rows.masked_fill_((slot_of_row < 0)[:, None], 0)


def plain_combine(rows, row_of_slot, w, dtype):
    T, k = row_of_slot.shape
    total = torch.zeros(T, rows.shape[1], device=rows.device, dtype=torch.float32)
    for j in range(k):
        r = row_of_slot[:, j].long()
        part = rows[r.clamp(min=0)].float()
        if w is not None:
            part = part * w[:, j, None]
        total += part.masked_fill_((r < 0)[:, None], 0)
    return total.to(dtype)


def plain_combine_backward(grad, rows, row_of_slot, slot_of_row, w):
    T, k = row_of_slot.shape
    token, live = slot_of_row.clamp(min=0).long() // k, (slot_of_row >= 0)[:, None]
    g = grad[token].float()
    weight = w.reshape(-1)[slot_of_row.clamp(min=0).long()]
    d_rows = (g * weight[:, None]).masked_fill_(~live, 0).to(rows.dtype)
    dots = (g * rows.float()).sum(1)
    r = row_of_slot.reshape(-1).long()
    d_w = torch.where(r >= 0, dots[r.clamp(min=0)], 0).view(T, k)
    return d_rows, d_w


def power(n, dtype):
    """2^n, put together from its bits: torch's pow and ldexp may be off in the last place."""
    return ((n.long() + 1023) << 52).view(torch.float64).to(dtype)


def plain_quantize(x, dims, to):
    """x viewed in blocks, `dims` the axes of one block: 8-bit values and scale bytes."""
    x = x.float()
    amax = x.abs().amax(dims, keepdim=True)
    m, e = torch.frexp(amax)                        # amax = m * 2^e with m in [0.5, 1)
    e = e - 1 - FMAX_EXP[to] + (m > 0.875).int()    # amax <= 1.75 * 2^(e + FMAX_EXP)
    e = torch.where(amax == 0, -127, e).clamp(-127, 127)
    return (x * power(-e, torch.float32)).to(TYPES[to]), (e + 127).to(torch.uint8)


def in_blocks(x, rows, cols):
    """(..., R, C) padded with zeros and viewed as (..., R / rows, rows, C / cols, cols)."""
    R, C = x.shape[-2:]
    p = torch.zeros(*x.shape[:-2], up(R, rows), up(C, cols), dtype=x.dtype, device=x.device)
    p[..., :R, :C] = x
    return p.view(*x.shape[:-2], up(R, rows) // rows, rows, up(C, cols) // cols, cols)


def padded_groups(x, sizes):
    """Rows of each group from a multiple of 128 on, zeros between, as columns are quantized."""
    P = up(x.shape[0], BLOCK) + BLOCK * len(sizes)
    out = torch.zeros(P, x.shape[1], dtype=x.dtype, device=x.device)
    at = begin = 0
    for n in sizes:
        out[at:at + n] = x[begin:begin + n]
        at, begin = at + up(n, BLOCK), begin + n
    return out


def plain_quantize_case(s, x):
    kind, C = s["kind"], s["C"]
    if kind == "cols":
        p = padded_groups(x, s["sizes"])
        q, e = plain_quantize(in_blocks(p, BLOCK, 1), (-3, -1), s["to"])
        return q.view(p.shape), e.view(-1, C)
    if kind == "blocks":
        G, R, C = x.shape
        v = in_blocks(x, BLOCK, BLOCK)
        q, e = plain_quantize(v, (-3, -1), s["to"])
        return q.view(G, up(R, BLOCK), up(C, BLOCK))[:, :R, :C], e.view(G, v.shape[1], v.shape[3])
    block = 32 if kind == "rows32" else BLOCK
    if kind == "dispatch":
        x = plain_dispatch(x, s["order"][2], s["k"])
    q, e = plain_quantize(in_blocks(x, 1, block), (-1,), s["to"])
    return q.view(x.shape[0], -1)[:, :C], e.view(x.shape[0], -1)


def decode(e, dtype):
    """E8M0 bytes as the powers of two they stand for."""
    return power(e.int() - 127, dtype)


def dequantized(s, dtype):
    """Operands a (rows, contraction) and b of a case as full numbers."""
    kind = s["kind"]
    if kind == "wgrad":
        return (s["a"].to(dtype) * decode(s["sa"], dtype).repeat_interleave(BLOCK, 0),
                s["b"].to(dtype) * decode(s["sb"], dtype).repeat_interleave(BLOCK, 0))
    if kind == "blocked32":
        G, N, K = s["b"].shape
        return (s["a"].to(dtype) * decode(s["sa"], dtype).repeat_interleave(32, 1),
                s["b"].to(dtype) * decode(s["sb_rows"], dtype).repeat_interleave(32, 1).view(G, N, K))
    b = s["b"]
    sb = decode(s["sb"], dtype).repeat_interleave(BLOCK, 1)[:, :b.shape[1]].repeat_interleave(BLOCK, 2)[:, :, :b.shape[2]]
    sa = decode(s["sa"], dtype).repeat_interleave(BLOCK, 1)[:, :s["a"].shape[1]]
    return s["a"].to(dtype) * sa, b.to(dtype) * sb


def plain_product(s, dtype, out_dtype):
    a, b = dequantized(s, dtype)
    kind, begin = s["kind"], 0
    if kind == "wgrad":
        out = torch.zeros(len(s["sizes"]), s["K"], s["N"], dtype=out_dtype, device="cuda")
        for g, n in enumerate(s["sizes"]):
            out[g] = a[begin:begin + n].t() @ b[begin:begin + n]
            begin += up(n, BLOCK)
        return out
    out = torch.zeros(s["R"], s["N"], dtype=out_dtype, device="cuda")
    for g, n in enumerate(s["sizes"]):
        out[begin:begin + n] = a[begin:begin + n] @ (b[g] if kind == "kn" else b[g].t())
        begin += n
    return out


# ------------------------------------------------------------------ one pass
def scales_out(s):
    """Scale bytes as the powers of two they stand for."""
    return s.view(torch.float8_e8m0fnu)


def run(state):
    return run_own(state) if own else run_plain(state)


def run_plain(s):
    op = s["op"]
    if op == "dispatch":
        order = plain_order(s["ids"], s["local"])
        out = [*order, plain_dispatch(s["x"], order[2], s["k"])]
        if s["train"]:
            out.append(plain_combine(s["grad"], order[1], None, s["grad"].dtype))
        return out
    if op == "combine":
        ends, row, slot = s["order"]
        out = [plain_combine(s["rows"], row, s["w"], s["rows"].dtype)]
        if s["train"]:
            out += plain_combine_backward(s["grad"], s["rows"], row, slot, s["w"])
        return out
    if op == "quantize":
        q, e = plain_quantize_case(s, s["x"])
        return [q, scales_out(e)]
    return plain_product(s, torch.float32, TYPES[s["out"]])


def run_own(s):
    import scale_factor_layout_b200 as mxs
    op = s["op"]
    if op == "dispatch":
        order = mxs.expert_sort(s["ids"], s["local"])
        out = [*order, mxs.dispatch_rows(s["x"], order)]
        if s["train"]:
            out.append(mxs.combine_rows(s["grad"], order))
        return out
    if op == "combine":
        order = mxs.ExpertOrder(*s["order"])
        out = [mxs.combine_rows(s["rows"], order, s["w"])]
        if s["train"]:
            out += mxs.combine_rows_backward(s["grad"], s["rows"], order, s["w"])
        return out
    if op == "quantize":
        kind, to = s["kind"], TYPES[s["to"]]
        if kind == "cols":
            q, e = mxs.quantize_cols(s["x"], s["ends"], dtype=to)
        elif kind == "blocks":
            q, e = mxs.quantize_blocks(s["x"], dtype=to)
        else:
            order = mxs.ExpertOrder(*s["order"]) if kind == "dispatch" else None
            q, e = mxs.quantize_rows(s["x"], block=32 if kind == "rows32" else BLOCK, dtype=to, order=order)
        return [q, scales_out(e)]
    kind, out = s["kind"], TYPES[s["out"]]
    if kind == "wgrad":
        return mxs.grouped_matmul_k(s["a"], s["sa"], s["b"], s["sb"], s["ends"], out_dtype=out)
    if kind == "blocked32":
        sa = mxs.rearrange_m_groups(s["sa"], s["ends"])
        return mxs.grouped_matmul(s["a"], sa, s["b"], s["sb"], s["ends"], block=32, out_dtype=out)
    return mxs.grouped_matmul(s["a"], s["sa"], s["b"], s["sb"], s["ends"], b_layout=kind, out_dtype=out)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op in ("dispatch", "combine"):
        T, k, C, es = case["T"], case["k"], case["C"], SIZE[case["dtype"]]
        S = T * k
        if op == "dispatch":
            data = 8 * S + 8 * S + (T + S) * C * es
            return {"bytes": data * 1.0 + ((S + T) * C * es if case["train"] else 0), "flops": S * C if case["train"] else 0}
        live = S * case["local"] / case["E"]
        data = live * C * es + 8 * S + T * C * es
        if case["train"]:   # the rows are read once for both directions
            data += T * C * es + S * C * es + 4 * S
        return {"bytes": data, "flops": 2 * S * C * (3 if case["train"] else 1)}
    if op == "quantize":
        R, C, kind = case["R"], case["C"], case["kind"]
        rows_in = R * (case["G"] if kind == "blocks" else 1)
        rows_out = R * case["k"] if kind == "dispatch" else rows_in
        per = {"rows32": 32, "blocks": BLOCK * BLOCK}.get(kind, BLOCK)
        return {"bytes": rows_in * C * SIZE[case["dtype"]] + rows_out * C * (1 + 1 / per), "flops": 3 * rows_out * C}
    R, G, N, K = int(case["R"] * case["used"]), case["G"], case["N"], case["K"]
    scale = 33 / 32 if case["kind"] == "blocked32" else 129 / 128
    busy = min(G, R)
    if case["kind"] == "wgrad":
        data = R * (N + K) * scale + G * N * K * SIZE[case["out"]]
    else:
        data = R * K * scale + busy * N * K + case["R"] * N * SIZE[case["out"]]
    return {"bytes": data, "flops": 2 * R * N * K}


# ------------------------------------------------------------------ from the definitions, in 64 bits
def two(n):
    """2^n from a table of exact values, n in [-200, 200]."""
    return torch.tensor([2.0 ** i for i in range(-200, 201)], dtype=torch.float64, device="cuda")[n.long() + 200]


def exact_blocks(x, block_of_row, block_of_col, n_rows, n_cols, to):
    """Values and scales of a matrix from its definition; block_of_*: the block that each row and column is in."""
    top = torch.zeros(n_rows, x.shape[1], dtype=torch.float64, device=x.device)
    top.index_reduce_(0, block_of_row, x.abs(), "amax")
    amax = torch.zeros(n_rows, n_cols, dtype=torch.float64, device=x.device)
    amax.index_reduce_(1, block_of_col, top, "amax")
    m, e = torch.frexp(amax / (1.75 * 2.0 ** FMAX_EXP[to]))   # the quotient is a power of two where m is a half
    e = torch.where(amax == 0, -127, e - (m == 0.5).int()).clamp(-127, 127)
    scale = two(e)
    del top
    v = x / scale[:, block_of_col][block_of_row]
    bits, low = (3, -6) if to == "e4m3" else (2, -14)
    step = two((torch.frexp(v)[1] - 1).clamp(min=low) - bits)
    return torch.round(v / step) * step, scale   # torch.round takes halves to the even neighbour


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "dispatch":
        k, ids = case["k"], s["ids"].reshape(-1).cpu().numpy()
        order = np.argsort(ids, kind="stable")
        order = order[ids[order] < case["local"]]
        ends = np.searchsorted(ids[order], np.arange(case["local"]), side="right").astype(np.int32)
        slot = np.full(ids.size, -1, np.int32)
        slot[:order.size] = order
        row = np.full(ids.size, -1, np.int32)
        row[order] = np.arange(order.size, dtype=np.int32)
        rows = torch.zeros(ids.size, case["C"], dtype=s["x"].dtype, device="cuda")
        rows[:order.size] = s["x"][torch.from_numpy(order // k).cuda()]
        out = [torch.from_numpy(ends), torch.from_numpy(row).view(-1, k), torch.from_numpy(slot), rows]
        if case["train"]:
            token = torch.from_numpy(order // k).cuda()
            dx = torch.zeros(case["T"], case["C"], dtype=torch.float64, device="cuda")
            for at in range(0, order.size, 16384):
                n = min(16384, order.size - at)
                dx.index_add_(0, token[at:at + n], s["grad"][at:at + n].double())
            out.append(dx)
        return out
    if op == "combine":
        slot = s["order"][2].long()
        live = int((slot >= 0).sum())
        slot, k, T, C = slot[:live], case["k"], case["T"], case["C"]
        w = s["w"].double().reshape(-1)
        y = torch.zeros(T, C, dtype=torch.float64, device="cuda")
        d_rows = torch.zeros(T * k, C, dtype=torch.float32, device="cuda") if case["train"] else None
        d_w = torch.zeros(T * k, dtype=torch.float64, device="cuda")
        for at in range(0, live, 16384):
            part = slot[at:at + 16384]
            rows = s["rows"][at:at + part.numel()].double()
            y.index_add_(0, part // k, rows * w[part, None])
            if case["train"]:
                g = s["grad"][part // k].double()
                d_rows[at:at + part.numel()] = (g * w[part, None]).float()
                d_w[part] = (g * rows).sum(1)
        return [y, d_rows, d_w.view(T, k)] if case["train"] else [y]
    if op == "quantize":
        kind, to, C = case["kind"], case["to"], case["C"]
        x = s["x"]
        if kind == "blocks":
            G, R, _ = x.shape
            at_row, at_col = torch.arange(R, device="cuda") // BLOCK, torch.arange(C, device="cuda") // BLOCK
            got = [exact_blocks(x[g].double(), at_row, at_col, up(R, BLOCK) // BLOCK, up(C, BLOCK) // BLOCK, to) for g in range(G)]
            return [torch.stack([v for v, _ in got]).float(), torch.stack([e for _, e in got])]
        if kind == "cols":
            x = padded_groups(x, s["sizes"])
            at_row, at_col = torch.arange(x.shape[0], device="cuda") // BLOCK, torch.arange(C, device="cuda")
            v, e = exact_blocks(x.double(), at_row, at_col, x.shape[0] // BLOCK, C, to)
            return [v, e]
        if kind == "dispatch":
            slot = s["order"][2].long()
            token = torch.where(slot >= 0, slot // case["k"], 0)
            x = x[token] * (slot >= 0)[:, None]
        block = 32 if kind == "rows32" else BLOCK
        at_col = torch.arange(C, device="cuda") // block
        vs, es = [], []
        for at in range(0, x.shape[0], 16384):
            part = x[at:at + 16384].double()
            v, e = exact_blocks(part, torch.arange(part.shape[0], device="cuda"), at_col, part.shape[0], up(C, block) // block, to)
            vs.append(v.float())   # 8-bit values: nothing is lost
            es.append(e)
        return [torch.cat(vs), torch.cat(es)]
    G, K, N, kind = case["G"], case["K"], case["N"], case["kind"]
    wide = lambda t, n, dim, size: two(t.int() - 127).repeat_interleave(n, dim).narrow(dim, 0, size)   # noqa: E731
    begin = 0
    if kind == "wgrad":
        out = torch.zeros(G, K, N, dtype=torch.float64, device="cuda")
        for g, n in enumerate(s["sizes"]):
            rows = slice(begin, begin + up(n, BLOCK))
            blocks = slice(begin // BLOCK, (begin + up(n, BLOCK)) // BLOCK)
            a = s["a"][rows].double() * wide(s["sa"][blocks], BLOCK, 0, up(n, BLOCK))
            b = s["b"][rows].double() * wide(s["sb"][blocks], BLOCK, 0, up(n, BLOCK))
            out[g] = torch.einsum("rm,rn->mn", a, b)
            begin += up(n, BLOCK)
        return out
    out = torch.zeros(case["R"], N, dtype=torch.float64, device="cuda")
    for g, n in enumerate(s["sizes"]):
        rows = slice(begin, begin + n)
        if kind == "blocked32":
            a = s["a"][rows].double() * wide(s["sa"][rows], 32, 1, K)
            b = s["b"][g].double() * wide(s["sb_rows"].view(G, N, -1)[g], 32, 1, K)
        else:
            a = s["a"][rows].double() * wide(s["sa"][rows], BLOCK, 1, K)
            b = s["b"][g].double()
            b = b * two(s["sb"][g].int() - 127).repeat_interleave(BLOCK, 0)[:b.shape[0]].repeat_interleave(BLOCK, 1)[:, :b.shape[1]]
        out[rows] = torch.einsum("rk,kn->rn" if kind == "kn" else "rk,nk->rn", a, b)
        begin += n
    return out
