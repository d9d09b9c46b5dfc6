"""The operators that train an expert layer, as cases to be measured.

The experts' product on 16-bit weights (`moe_grouped_gemm`), forward and with the weights read the other way for the
rows' gradient, the weights' gradient (`moe_grouped_gemm_wgrad`), and activation checkpoints in 8 bits: rows to 8-bit
floating point with one power-of-two scale per 32 values and back (`mxfp8_quantize`, `mxfp8_dequantize`), and
SiLU-and-mul that keeps its input so, with the backward pass that reads it (`mxfp8_silu_mul`, `mxfp8_silu_mul_backward`).

`run` computes a case in plain torch where `own` is false and by the library's calls where it is true.
"""
import math

import torch

own = False

if torch.cuda.is_available():
    DEVICE = "cuda"
else:
    DEVICE = "cpu"

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}
MOST = 448.0  # the largest 8-bit magnitude (four exponent bits, three mantissa bits)


def listed():
    return [
        # one token through a 1/8 slice of the intermediate dimension: the latency of the smallest product
        {"name": "forward_token", "kind": "forward", "T": 1, "topk": 8, "E": 64, "G": 64, "N": 512, "K": 7168, "bm": 16,
         "dtype": "bf16", "out": "bf16", "gather": True},
        # gate_up of a decode batch on one GPU's 48 of 384 experts: the weights are read once
        {"name": "forward_decode", "kind": "forward", "T": 128, "topk": 8, "E": 48, "G": 384, "N": 4096, "K": 7168,
         "bm": 16, "dtype": "bf16", "out": "bf16", "gather": True},
        # gate_up of a training step's 4096 tokens on 16 experts, ragged rows per expert
        {"name": "forward_train", "kind": "forward", "T": 4096, "topk": 8, "E": 16, "G": 16, "N": 4096, "K": 7168,
         "bm": 128, "dtype": "bf16", "out": "bf16", "gather": True},
        # down of a prompt on 48 of 384 experts, fp16, some 85 rows an expert
        {"name": "forward_down", "kind": "forward", "T": 4096, "topk": 8, "E": 48, "G": 384, "N": 7168, "K": 2048,
         "bm": 128, "dtype": "fp16", "out": "fp32", "gather": False},
        # the rows' gradient of the training step's gate_up
        {"name": "rows_grad_train", "kind": "rows_grad", "T": 4096, "topk": 8, "E": 16, "G": 16, "N": 7168, "K": 4096,
         "bm": 128, "dtype": "bf16", "out": "bf16", "gather": False},
        # odd sizes, a slice of the experts, few rows each
        {"name": "rows_grad_odd", "kind": "rows_grad", "T": 333, "topk": 3, "E": 10, "G": 13, "N": 1384, "K": 1000,
         "bm": 32, "dtype": "fp16", "out": "fp16", "gather": False},
        # the weights' gradient of the training step's gate_up, kept in 32 bits
        {"name": "weights_grad_train", "kind": "weights_grad", "T": 4096, "topk": 8, "E": 16, "G": 16, "N": 4096,
         "K": 7168, "bm": 128, "dtype": "bf16", "out": "fp32", "gather": True},
        # a small layer's, odd sizes, long runs of rows for few weights
        {"name": "weights_grad_odd", "kind": "weights_grad", "T": 2777, "topk": 2, "E": 4, "G": 4, "N": 264, "K": 712,
         "bm": 128, "dtype": "fp16", "out": "fp16", "gather": False},
        # token rows of a small batch kept in 8 bits for the backward pass, and taken back
        {"name": "checkpoint_small", "kind": "checkpoint", "rows": 64, "K": 7168, "dtype": "bf16"},
        # the same of a long batch
        {"name": "checkpoint_train", "kind": "checkpoint", "rows": 16384, "K": 7168, "dtype": "bf16"},
        # the activation between the products with its gradient: a small batch's rows
        {"name": "silu_small", "kind": "silu", "rows": 200, "spare": 56, "I": 416, "dtype": "fp32"},
        # and those of the training step, half a block of padding an expert behind them
        {"name": "silu_train", "kind": "silu", "rows": 32768, "spare": 1024, "I": 2048, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _block(T, topk, G, rng):
    """Rows per block by the tokens an expert is expected to get; 64 now and then."""
    per = T * topk / G
    bm = 16 if per <= 6 else 32 if per <= 40 else 128
    return 64 if per > 6 and rng.random() < 0.15 else bm


def draw(rng):
    kind = rng.choice(["forward", "forward", "rows_grad", "rows_grad", "weights_grad", "weights_grad", "checkpoint",
                       "silu"])
    if kind == "checkpoint":
        rows = _log(rng, 1, 16384)
        return {"kind": kind, "rows": rows, "K": 32 * _log(rng, 1, max(1, min(512, 16384 * 112 // rows))),
                "dtype": rng.choice(["bf16", "fp16", "fp32"])}
    if kind == "silu":
        rows = _log(rng, 1, 32768)
        return {"kind": kind, "rows": rows, "spare": rng.choice([0, rng.randint(1, 512)]),
                "I": 32 * _log(rng, 1, max(1, min(224, 32768 * 32 // rows))), "dtype": rng.choice(["bf16", "fp16", "fp32"])}
    while True:
        G = _log(rng, 1, 384)
        E = G if rng.random() < 0.5 else max(1, G // rng.choice([2, 3, 4, 8]))
        topk = rng.randint(1, min(8, G))
        T = _log(rng, 1, 4096)
        if E < G and T * topk * E < 16 * G:  # a slice that hardly any token chose says nothing
            continue
        dtype = rng.choice(["bf16", "fp16"])
        N, K = 8 * _log(rng, 1, 1024), 8 * _log(rng, 1, 1024)
        slots = T * topk * E / G
        if E * N * K <= 1.2e9 and slots * N * K <= 0.9e12 and (slots + E * 128) * max(N, K) <= 4e8:
            return {"kind": kind, "T": T, "topk": topk, "E": E, "G": G, "N": N, "K": K, "bm": _block(T, topk, G, rng),
                    "dtype": dtype, "out": rng.choice([dtype, dtype, "fp32"]),
                    "gather": kind != "rows_grad" and rng.random() < 0.5}


# ------------------------------------------------------------------ inputs


def _plan(ids, E, bm):
    """The aligned order of routed ids [T, topk]: sorted slots, expert of each block, padded rows; and, as a program
    without such a product keeps it, each expert's first row and number of rows."""
    flat = ids.reshape(-1).long()
    n = flat.numel()
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    order = torch.argsort(key, stable=True)
    counts = torch.bincount(key, minlength=E + 1)[:E]
    padded = (counts + bm - 1) // bm * bm
    live = int(counts.sum())
    ordered = key[order[:live]]
    starts = padded.cumsum(0) - padded
    at = starts[ordered] + torch.arange(live, device=ids.device) - (counts.cumsum(0) - counts)[ordered]
    capacity = n + E * (bm - 1)
    slots = torch.full((capacity,), n, dtype=torch.int32, device=ids.device)
    slots[at] = order[:live].int()
    rows = int(padded.sum())
    blocks = torch.full(((capacity + bm - 1) // bm,), -1, dtype=torch.int32, device=ids.device)
    blocks[: rows // bm] = torch.repeat_interleave(torch.arange(E, device=ids.device), padded // bm).int()
    return {"sorted": slots, "expert_ids": blocks, "ntpp": torch.tensor([rows], dtype=torch.int32, device=ids.device),
            "rows": rows, "capacity": capacity, "runs": list(zip(starts.tolist(), counts.tolist()))}


def prepare(case, seed):
    rng = torch.Generator(device=DEVICE).manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=rng, device=DEVICE)  # noqa: E731
    empty = lambda *shape, dtype: torch.zeros(*shape, dtype=dtype, device=DEVICE)  # noqa: E731
    kind, dtype = case["kind"], DTYPES[case["dtype"]]
    if kind in ("checkpoint", "silu"):
        rows = case["rows"] + case.get("spare", 0)
        K = case["K"] if kind == "checkpoint" else 2 * case["I"]
        # activations: channels of different sizes, a few of them far larger
        size = torch.exp2(0.5 * normal(K)) * torch.where(torch.rand(K, generator=rng, device=DEVICE) < 0.01, 12.0, 1.0)
        state = {"case": case, "x": (normal(rows, K) * size).to(dtype),
                 "q": empty(rows, K, dtype=torch.uint8), "s": empty(rows, K // 32, dtype=torch.uint8)}
        if kind == "checkpoint":
            state["values"] = empty(rows, K, dtype=dtype if case["dtype"] != "fp16" else torch.float32)
        else:
            state["rows"] = torch.tensor([case["rows"]], dtype=torch.int32, device=DEVICE)
            state["dh"] = (0.1 * normal(rows, K // 2)).to(dtype)
            state["h"], state["again"] = empty(rows, K // 2, dtype=dtype), empty(rows, K // 2, dtype=dtype)
            state["dgu"] = empty(rows, K, dtype=dtype)
        return state
    T, topk, E, G, bm, N, K = (case[k] for k in ("T", "topk", "E", "G", "bm", "N", "K"))
    # how many rows the experts get is the case's, so that outputs have one size; which tokens and which of the
    # resident experts they are is the seed's
    ids = torch.rand(T, G, generator=torch.Generator(device=DEVICE).manual_seed(1), device=DEVICE).topk(topk, dim=1)[1]
    label = torch.cat((torch.randperm(E, generator=rng, device=DEVICE), torch.arange(E, G, device=DEVICE)))
    ids = label[ids][torch.randperm(T, generator=rng, device=DEVICE)]
    plan = _plan(ids.int(), E, bm)
    state = {"case": case, "plan": plan}
    state["a"] = normal(T if case["gather"] else plan["capacity"], K).to(dtype)
    if kind == "weights_grad":
        state["dout"] = (0.1 * normal(plan["capacity"], N)).to(dtype)
        state["dw"] = empty(E, N, K, dtype=DTYPES[case["out"]])
        if own:
            import w4a16_grouped_gemm_amd as w
            nbytes = w.moe_grouped_gemm_wgrad_workspace_bytes(E, N, K, plan["capacity"])
            state["workspace"] = empty(nbytes, dtype=torch.uint8) if nbytes else None
        return state
    shape = (E, N, K) if kind == "forward" else (E, K, N)
    state["w"] = torch.empty(*shape, dtype=dtype, device=DEVICE)
    for e in range(E):  # an expert at a time: the 32-bit numbers of all would be twice the weights
        state["w"][e] = normal(*shape[1:]) * K**-0.5
    state["out"] = empty(plan["capacity"], N, dtype=DTYPES[case["out"]])
    return state


# ------------------------------------------------------------------ one pass


def run(state):
    return _own(state) if own else _plain(state)


def _own(state):
    import w4a16_grouped_gemm_amd as w

    case, plan = state["case"], state.get("plan")
    kind = case["kind"]
    if kind == "checkpoint":
        w.mxfp8_quantize(state["x"], state["q"], state["s"])
        w.mxfp8_dequantize(state["q"], state["s"], state["values"])
        return state["values"]
    if kind == "silu":
        w.mxfp8_silu_mul(state["x"], state["h"], state["q"], state["s"], num_rows=state["rows"])
        w.mxfp8_silu_mul_backward(state["q"], state["s"], state["dh"], state["dgu"], h=state["again"],
                                  num_rows=state["rows"])
        n = case["rows"]
        return state["h"][:n], state["dgu"][:n], state["again"][:n]
    if kind == "weights_grad":
        w.moe_grouped_gemm_wgrad(state["dout"], state["a"], case["T"], case["topk"], plan["sorted"],
                                 plan["expert_ids"], plan["ntpp"], case["bm"], state["dw"], gather=case["gather"],
                                 workspace=state["workspace"])
        return state["dw"]
    w.moe_grouped_gemm(state["a"], case["T"], case["topk"], plan["sorted"], plan["expert_ids"], plan["ntpp"],
                       case["bm"], state["w"], state["out"], gather=case["gather"], transposed=kind == "rows_grad")
    return state["out"][: plan["rows"]]


def _checkpoint(x):
    """Rows [.., K] of 32 bits -> the values that their 8-bit codes and scales stand for. Division by a power of two is
    exact; a block of 32 that holds an infinity or a NaN becomes NaN."""
    blocks = x.unflatten(-1, (-1, 32))
    most = blocks.abs().amax(-1, keepdim=True)
    finite = torch.isfinite(most)
    mantissa, exponent = torch.frexp(torch.where(finite, most, 0.0))
    # most = mantissa 2^exponent, mantissa in [0.5, 1): at most 448 = 0.875 * 2^9 after the division
    exponent = torch.where(mantissa > 0.875, exponent - 8, exponent - 9).clamp(min=-127)
    scale = torch.exp2(exponent.double())
    v = torch.where(finite, (blocks / scale).float(), 0.0)
    step = torch.exp2((torch.frexp(v)[1] - 1).clamp(min=-6).float() - 3)  # three mantissa bits, down to 2^-6
    return torch.where(finite, torch.round(v / step) * step * scale, math.nan).float().flatten(-2)


def _plain(state):
    case, plan = state["case"], state.get("plan")
    kind = case["kind"]
    if kind == "checkpoint":
        return _checkpoint(state["x"].float()).to(state["values"].dtype)
    if kind == "silu":
        x = state["x"][: case["rows"]].float()
        gate, up = x.chunk(2, dim=-1)
        h = gate / (1 + torch.exp(-gate)) * up
        gate, up = _checkpoint(x).chunk(2, dim=-1)
        dh = state["dh"][: case["rows"]].float()
        sig = 1 / (1 + torch.exp(-gate))
        dgu = torch.cat((dh * up * sig * (1 + gate * (1 - sig)), dh * gate * sig), dim=-1)
        return tuple(t.to(state["x"].dtype) for t in (h, dgu, gate * sig * up))
    slots = plan["sorted"].long()
    if kind == "weights_grad":
        dw = torch.empty_like(state["dw"])
        for e, (first, count) in enumerate(plan["runs"]):
            rows = slice(first, first + count)
            a = state["a"][slots[rows] // case["topk"]] if case["gather"] else state["a"][rows]
            dw[e] = state["dout"][rows].float().T @ a.float()
        return dw
    out = torch.zeros(plan["rows"], case["N"], dtype=state["out"].dtype, device=slots.device)
    for e, (first, count) in enumerate(plan["runs"]):
        if count:
            rows = slice(first, first + count)
            a = state["a"][slots[rows] // case["topk"]] if case["gather"] else state["a"][rows]
            w = state["w"][e].float()
            out[rows] = (a.float() @ (w.T if kind == "forward" else w)).to(out.dtype)
    return out


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    kind, size = case["kind"], SIZES[case["dtype"]]
    if kind == "checkpoint":  # values in, codes and scales out and in again, values out
        n = case["rows"] * case["K"]
        return {"bytes": n * (size + 2 * (1 + 1 / 32) + (2 if case["dtype"] == "bf16" else 4)), "flops": 0}
    if kind == "silu":  # gate and up in, h and the checkpoint out; the checkpoint and dh in, dgu and h out
        n = case["rows"] * case["I"]
        return {"bytes": n * (3 * size + 2 * (1 + 1 / 32) + 2 * (1 + 1 / 32) + 4 * size), "flops": 20 * n}
    T, topk, E, G, N, K = (case[k] for k in ("T", "topk", "E", "G", "N", "K"))
    slots = T * topk * E / G  # rows that carry a slot, as expected of the routing
    tokens = T * (1 - math.prod(max(0, G - E - j) / (G - j) for j in range(topk)))  # tokens with such a row
    a = (tokens if case["gather"] else slots) * K * size
    if kind == "weights_grad":  # experts without a row get zeros
        return {"bytes": a + slots * N * size + E * N * K * SIZES[case["out"]], "flops": 2 * slots * N * K}
    active = E * (1 - (1 - topk / G) ** T)  # experts that any token chose
    return {"bytes": a + active * N * K * size + slots * N * SIZES[case["out"]], "flops": 2 * slots * N * K}


# ------------------------------------------------------------------ the definition in 64 bits


def _nearest(x):
    """The value of the nearest 8-bit code times the block's scale, found among all codes, a tie to the even one."""
    code = torch.arange(127, device=x.device, dtype=torch.float64)
    e, m = torch.floor(code / 8), code % 8
    levels = torch.where(e == 0, m * 2.0**-9, torch.exp2(e - 7) * (1 + m / 8))
    middles = (levels[1:] + levels[:-1]) / 2
    blocks = x.reshape(x.shape[0], -1, 32)
    out = torch.empty_like(blocks)
    for r in range(0, x.shape[0], 1024):
        b = blocks[r : r + 1024]
        most = b.abs().amax(-1, keepdim=True)
        e = torch.ceil(torch.log2((most / MOST).clamp(min=2.0**-1000)))
        e = torch.where(MOST * torch.exp2(e - 1) >= most, e - 1, torch.where(MOST * torch.exp2(e) < most, e + 1, e))
        unit = torch.exp2(e.clamp(min=-127.0))
        v = (b / unit).abs()
        below = torch.searchsorted(middles, v, right=False)  # the number of middles under v
        tie = (below < 126) & (v == middles[below.clamp(max=125)])
        below = torch.where(tie & (below % 2 == 1), below + 1, below)
        out[r : r + 1024] = torch.sign(b) * levels[below] * unit
    return out.view(x.shape)


def exact(case, seed):
    state = prepare(case, seed)
    kind = case["kind"]
    if kind == "checkpoint":
        return _nearest(state["x"].double())
    if kind == "silu":
        I, n = case["I"], case["rows"]
        x = state["x"][:n].double()
        h = x[:, :I] * torch.sigmoid(x[:, :I]) * x[:, I:]
        x = _nearest(x)
        g, u, dh = x[:, :I], x[:, I:], state["dh"][:n].double()
        silu = g * torch.sigmoid(g)
        slope = torch.sigmoid(g) + silu * torch.sigmoid(-g)
        return h, torch.cat((dh * u * slope, dh * silu), dim=-1), silu * u
    plan, topk, bm = state["plan"], case["topk"], case["bm"]
    M = plan["rows"]
    live = torch.nonzero(plan["sorted"][:M] < case["T"] * topk).flatten()
    source = plan["sorted"][live].long() // topk if case["gather"] else live
    expert = plan["expert_ids"][live // bm]
    if kind == "weights_grad":
        total = torch.zeros(case["E"], case["N"], case["K"], dtype=torch.float64, device=DEVICE)
    else:
        total = torch.zeros(M, case["N"], dtype=torch.float64, device=DEVICE)
    for e in range(case["E"]):
        mine = torch.nonzero(expert == e).flatten()
        if mine.numel():
            a = state["a"][source[mine]].double()
            if kind == "weights_grad":
                total[e] = torch.matmul(state["dout"][live[mine]].double().T.contiguous(), a)
            else:
                w = state["w"][e].double()
                total[live[mine]] = a @ (w.T.contiguous() if kind == "forward" else w)
    return total
