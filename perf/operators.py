"""The grouped-layout and microscaled (MXFP4) operators of the expert layer, as cases to be measured.

Rows sorted by expert and back (`moe_permute`, `moe_unpermute` and their gradients), bf16/fp16/fp32 rows
to 4-bit floating point with one power-of-two scale per 32 values and back (`mxfp4_quantize`,
`mxfp4_silu_mul_quantize`, `mxfp4_dequantize`), and the experts' product on such operands (`mxfp4_moe_gemm`).

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

# the eight magnitudes of a 4-bit float with two exponent bits and one mantissa bit; code 8 + i is -LEVELS[i]
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # a handful of requests decoding on one GPU's 48 of 384 experts: latency of the smallest call
        {"name": "permute_decode", "kind": "permute", "T": 4, "topk": 8, "E": 48, "G": 384, "H": 7168, "bm": 16,
         "dtype": "bf16"},
        # a prompt of 4096 tokens whose 64 experts are all resident, rows grouped for 128-row tiles
        {"name": "permute_prefill", "kind": "permute", "T": 4096, "topk": 8, "E": 64, "G": 64, "H": 7168, "bm": 128,
         "dtype": "bf16"},
        # a training step's gradient of the grouped rows, summed back per token
        {"name": "permute_bwd", "kind": "permute_bwd", "T": 2048, "topk": 8, "E": 64, "G": 64, "H": 7168, "bm": 128,
         "dtype": "bf16"},
        # decode: fp32 expert rows of one GPU's slice, weighted and summed into bf16
        {"name": "unpermute_decode", "kind": "unpermute", "T": 128, "topk": 8, "E": 48, "G": 384, "H": 7168, "bm": 16,
         "dtype": "fp32", "out": "bf16"},
        # the same of a long prompt, all experts resident
        {"name": "unpermute_prefill", "kind": "unpermute", "T": 4096, "topk": 8, "E": 64, "G": 64, "H": 7168,
         "bm": 128, "dtype": "bf16", "out": "bf16"},
        # the gradient of the weighted sum in a training step: rows and routing weights
        {"name": "unpermute_bwd", "kind": "unpermute_bwd", "T": 4096, "topk": 8, "E": 64, "G": 64, "H": 4096,
         "bm": 128, "dtype": "bf16", "out": "bf16"},
        # odd sizes, a slice of the experts, fp32 training
        {"name": "unpermute_bwd_odd", "kind": "unpermute_bwd", "T": 333, "topk": 3, "E": 10, "G": 13, "H": 1001,
         "bm": 32, "dtype": "fp32", "out": "fp32"},
        # activations of a decode batch to 4 bits and back
        {"name": "quantize_decode", "kind": "quantize", "rows": 128, "K": 7168, "dtype": "bf16"},
        # activations of a long prompt
        {"name": "quantize_prefill", "kind": "quantize", "rows": 16384, "K": 7168, "dtype": "bf16"},
        # gate_up of a decode batch on 48 of 384 experts: the weights are read once
        {"name": "gate_up_decode", "kind": "gate_up", "T": 128, "topk": 8, "E": 48, "G": 384, "N": 4096, "K": 7168,
         "bm": 16, "even": False, "out": "bf16"},
        # gate_up of a prompt with exactly 128 rows for each of 48 experts
        {"name": "gate_up_prefill", "kind": "gate_up", "T": 768, "topk": 8, "E": 48, "G": 48, "N": 4096, "K": 7168,
         "bm": 128, "even": True, "out": "bf16"},
        # SiLU-and-mul to 4 bits and the down product of a long prompt, ragged rows per expert
        {"name": "down_prefill", "kind": "down", "T": 4096, "topk": 8, "E": 16, "G": 16, "N": 7168, "K": 2048,
         "bm": 128, "even": False, "out": "bf16"},
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
    kind = rng.choice(["permute", "permute_bwd", "unpermute", "unpermute_bwd", "quantize", "gate_up", "gate_up", "down"])
    if kind == "quantize":
        rows = _log(rng, 1, 16384)
        return {"kind": kind, "rows": rows, "K": 32 * _log(rng, 1, max(1, min(512, 16384 * 224 // rows))),
                "dtype": rng.choice(["bf16", "fp16", "fp32"])}
    while True:
        G = _log(rng, 1, 384)
        E = G if rng.random() < 0.5 else max(1, G // rng.choice([2, 3, 4, 8]))
        topk = rng.randint(1, min(8, G))
        T = _log(rng, 1, 4096)
        if E < G and T * topk * E < 16 * G:  # a slice that hardly any token chose says nothing
            continue
        case = {"kind": kind, "T": T, "topk": topk, "E": E, "G": G}
        if kind in ("gate_up", "down"):
            N, K = 16 * _log(rng, 4, 512), 32 * _log(rng, 1, 224)
            case.update(N=N, K=K, bm=_block(T, topk, G, rng), even=False, out=rng.choice(["bf16", "fp16", "fp32"]))
            blocks = (T * topk * E / G + E * case["bm"]) / case["bm"]
            if E * N * K <= 1.5e9 and blocks * N * K <= 4e9 and T * topk * E / G * N * K <= 4.8e11:
                return case
        else:
            H = _log(rng, 64, 7168)
            H += rng.choice([0, 0, (-H) % 8, (-H) % 64])
            dtype = rng.choice(["bf16", "fp16", "fp32"])
            case.update(H=H, bm=_block(T, topk, G, rng), dtype=dtype)
            if kind.startswith("unpermute"):
                case["out"] = rng.choice(["bf16", "fp16", "fp32"]) if dtype == "fp32" else dtype
            if T * topk * H * (2 if dtype == "fp32" else 1) <= 4096 * 8 * 4096:
                return case


# ------------------------------------------------------------------ inputs


def _plan(ids, E, bm):
    """The aligned order of routed ids [T, topk]: sorted slots, expert of each block, padded rows."""
    flat = ids.reshape(-1).long()
    n = flat.numel()
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    order = torch.argsort(key, stable=True)
    counts = torch.bincount(key, minlength=E + 1)[:E]
    padded = (counts + bm - 1) // bm * bm
    live = int(counts.sum())
    ordered = key[order[:live]]
    at = (padded.cumsum(0) - padded)[ordered] + torch.arange(live, device=ids.device) - (counts.cumsum(0) - counts)[ordered]
    capacity = n + E * (bm - 1)
    slots = torch.full((capacity,), n, dtype=torch.int32, device=ids.device)
    slots[at] = order[:live].int()
    rows = int(padded.sum())
    blocks = torch.full(((capacity + bm - 1) // bm,), -1, dtype=torch.int32, device=ids.device)
    blocks[: rows // bm] = torch.repeat_interleave(torch.arange(E, device=ids.device), padded // bm).int()
    slot_rows = torch.full((n,), -1, dtype=torch.int32, device=ids.device)
    slot_rows[order[:live]] = at.int()
    return {"sorted": slots, "expert_ids": blocks, "ntpp": torch.tensor([rows], dtype=torch.int32, device=ids.device),
            "rows": rows, "slot_rows": slot_rows.view(ids.shape), "capacity": capacity}


def _codes(x):
    """Rows [.., K] of 32 or 64 bits -> the code (0..15) of each value and the scale byte of each 32 (255: not finite).
    Division by a power of two is exact in either."""
    blocks = x.unflatten(-1, (-1, 32))
    most = blocks.abs().amax(-1)
    finite = torch.isfinite(most)
    exponent = torch.frexp(torch.where(finite, most, 0.0))[1] - 1  # floor(log2) of what is not zero
    scale = torch.where(most == 0, torch.zeros_like(exponent), (exponent - 2 + 127).clamp(min=0))
    inverse = torch.exp2(127 - scale.double()).to(x.dtype)
    v = torch.where(finite[..., None], blocks * inverse[..., None], 0.0)
    m = v.abs()
    code = (m > 0.25).to(torch.uint8)  # ties to the level whose mantissa bit is 0
    code += m >= 0.75
    code += m > 1.25
    code += m >= 1.75
    code += m > 2.5
    code += m >= 3.5
    code += m > 5.0
    code += 8 * (v < 0).to(torch.uint8)
    return code.flatten(-2), torch.where(finite, scale, 255).to(torch.uint8)


def _pack(code):
    """Two codes a byte, the even one in the low half."""
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _values(q, s, dtype=torch.float32):
    """Packed codes [.., K/2] and scale bytes [.., K/32] -> the values they stand for."""
    table = torch.tensor(LEVELS + tuple(-v for v in LEVELS), dtype=dtype, device=q.device)
    code = torch.stack((q & 15, q >> 4), -1).flatten(-2)
    scale = torch.where(s == 255, math.nan, torch.exp2(s.double() - 127)).to(dtype)
    return (table[code.int()].unflatten(-1, (-1, 32)) * scale[..., None]).flatten(-2)


def prepare(case, seed):
    rng = torch.Generator(device=DEVICE).manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=rng, device=DEVICE)  # noqa: E731
    empty = lambda *shape, dtype: torch.zeros(*shape, dtype=dtype, device=DEVICE)  # noqa: E731
    kind = case["kind"]
    if kind == "quantize":
        rows, K = case["rows"], case["K"]
        # activations: channels of different sizes, a few of them far larger
        size = torch.exp2(normal(K)) * torch.where(torch.rand(K, generator=rng, device=DEVICE) < 0.01, 30.0, 1.0)
        return {"case": case, "x": (normal(rows, K) * size).to(DTYPES[case["dtype"]]),
                "q": empty(rows, K // 2, dtype=torch.uint8), "s": empty(rows, K // 32, dtype=torch.uint8),
                "values": empty(rows, K, dtype=DTYPES[case["dtype"]] if case["dtype"] != "fp16" else torch.float32)}
    T, topk, E, G, bm = (case[k] for k in ("T", "topk", "E", "G", "bm"))
    # how many rows the experts get is the case's, so that outputs have one size; which tokens and which of the
    # resident experts they are is the seed's
    if case.get("even"):
        ids = (torch.arange(T * topk, device=DEVICE) % G).view(T, topk)
    else:
        ids = torch.rand(T, G, generator=torch.Generator(device=DEVICE).manual_seed(1), device=DEVICE).topk(topk, dim=1)[1]
    label = torch.cat((torch.randperm(E, generator=rng, device=DEVICE), torch.arange(E, G, device=DEVICE)))
    ids = label[ids][torch.randperm(T, generator=rng, device=DEVICE)]
    state = {"case": case, "plan": _plan(ids.int(), E, bm), "weights": normal(T, topk).softmax(-1)}
    capacity = state["plan"]["capacity"]
    if kind in ("gate_up", "down"):
        N, K = case["N"], case["K"]
        w_q = torch.randint(0, 256, (E, N, K // 2), generator=rng, dtype=torch.uint8, device=DEVICE)
        w_s = torch.randint(118, 122, (E, N, K // 32), generator=rng, dtype=torch.uint8, device=DEVICE)
        if kind == "gate_up":
            code, state["a_s"] = _codes(normal(T, K))
            state["a_q"] = _pack(code)
        else:  # gate and up halves of the aligned rows; padding rows are zero, as the product leaves them
            real = state["plan"]["sorted"] < T * topk
            state["gu"] = (normal(capacity, 2 * K) * real[:, None]).bfloat16()
            state["a_q"] = empty(capacity, K // 2, dtype=torch.uint8)
            state["a_s"] = empty(capacity, K // 32, dtype=torch.uint8)
        state["w_q"], state["w_s"] = w_q, w_s
        state["out"] = empty(capacity, N, dtype=DTYPES[case["out"]])
        if own:  # weights are laid out once, at load
            import w4a16_grouped_gemm_amd as w
            state["packed"] = empty(w.mxfp4_packed_bytes(E, N, K), dtype=torch.uint8)
            w.mxfp4_repack(w_q, w_s, state["packed"])
        return state
    H, dtype = case["H"], DTYPES[case["dtype"]]
    if kind == "permute":
        state["x"] = normal(T, H).to(dtype)
        state["xp"] = empty(capacity, H, dtype=dtype)
        state["slot_rows"] = empty(T, topk, dtype=torch.int32)
    elif kind == "permute_bwd":
        state["dxp"] = normal(capacity, H).to(dtype)
        state["dx"] = empty(T, H, dtype=dtype)
    else:
        state["y"] = normal(capacity, H).to(dtype)
        state["out"] = empty(T, H, dtype=DTYPES[case["out"]])
        if kind == "unpermute_bwd":
            state["dout"] = normal(T, H).to(DTYPES[case["out"]])
            state["dy"] = empty(capacity, H, dtype=dtype)
            state["dweights"] = empty(T, topk, dtype=torch.float32)
    return state


# ------------------------------------------------------------------ one pass


def run(state):
    return _own(state) if own else _plain(state)


def _own(state):
    import w4a16_grouped_gemm_amd as w

    case, plan = state["case"], state.get("plan")
    kind = case["kind"]
    if kind == "quantize":
        w.mxfp4_quantize(state["x"], state["q"], state["s"])
        w.mxfp4_dequantize(state["q"], state["s"], state["values"])
        return state["values"]
    if kind == "permute":
        w.moe_permute(state["x"], plan["sorted"], plan["ntpp"], case["topk"], state["xp"], state["slot_rows"])
        return state["xp"][: plan["rows"]], state["slot_rows"]
    if kind == "permute_bwd":
        w.moe_permute_backward(state["dxp"], plan["slot_rows"], state["dx"])
        return state["dx"]
    if kind == "unpermute":
        w.moe_unpermute(state["y"], plan["slot_rows"], state["out"], topk_weights=state["weights"])
        return state["out"]
    if kind == "unpermute_bwd":
        w.moe_unpermute_backward(state["dout"], state["y"], plan["slot_rows"], state["weights"], plan["sorted"],
                                 plan["ntpp"], state["dy"], state["dweights"])
        return state["dy"][: plan["rows"]], state["dweights"]
    topk = case["topk"]  # gate_up gathers token rows, down reads the aligned rows in place
    if kind == "down":
        w.mxfp4_silu_mul_quantize(state["gu"], state["a_q"], state["a_s"], num_rows=plan["ntpp"])
    w.mxfp4_moe_gemm(state["a_q"], state["a_s"], case["T"], topk, plan["sorted"], plan["expert_ids"], plan["ntpp"],
                     case["bm"], case["E"], state["packed"], state["out"], gather=kind == "gate_up")
    return state["out"][: plan["rows"]]


def _plain(state):
    case, plan = state["case"], state.get("plan")
    kind = case["kind"]
    if kind == "quantize":
        code, s = _codes(state["x"].float())
        return _values(_pack(code), s).to(state["values"].dtype)
    n = case["T"] * case["topk"]
    slots = plan["sorted"][: plan["rows"]].long()
    real = slots < n
    token = (slots // case["topk"]).clamp(max=case["T"] - 1)
    if kind == "permute":
        back = torch.full((n + 1,), -1, dtype=torch.int32, device=slots.device)
        back[slots] = torch.arange(plan["rows"], dtype=torch.int32, device=slots.device)
        return state["x"][token] * real[:, None], back[:n].view(case["T"], case["topk"])
    rows = plan["slot_rows"].long()
    has = rows >= 0
    if kind == "permute_bwd":
        return (state["dxp"][rows.clamp(min=0)].float() * has[..., None]).sum(1).to(state["dx"].dtype)
    if kind == "unpermute":
        picked = state["y"][rows.clamp(min=0)].float()
        return (picked * (state["weights"] * has)[..., None]).sum(1).to(state["out"].dtype)
    if kind == "unpermute_bwd":
        dout = state["dout"].float()
        weight = torch.where(real, state["weights"].reshape(-1)[slots.clamp(max=n - 1)], 0.0)
        dy = (dout[token] * weight[:, None]).to(state["y"].dtype)
        dweights = (state["y"][rows.clamp(min=0)].float() * dout[:, None]).sum(-1) * has
        return dy, dweights
    if kind == "gate_up":
        a = _values(state["a_q"], state["a_s"])[token]
    else:
        gate, up = state["gu"][: plan["rows"]].double().chunk(2, dim=-1)
        code, s = _codes(gate / (1 + torch.exp(-gate)) * up)
        a = _values(_pack(code), s)
    used = plan["rows"] // case["bm"]
    blocks = (a * real[:, None]).view(used, case["bm"], case["K"])
    weights = _values(state["w_q"], state["w_s"]).transpose(1, 2)[plan["expert_ids"][:used].long()].contiguous()
    return torch.bmm(blocks, weights).flatten(0, 1).to(state["out"].dtype)


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    kind = case["kind"]
    if kind == "quantize":  # values in, codes and scales out, values out
        n = case["rows"] * case["K"]
        return {"bytes": n * (size[case["dtype"]] + 0.5 + 1 / 32 + (2 if case["dtype"] == "bf16" else 4)), "flops": 0}
    T, topk, E, G = case["T"], case["topk"], case["E"], case["G"]
    slots = T * topk * E / G  # rows that carry a slot, as expected of the routing
    tokens = T * (1 - math.prod(max(0, G - E - j) / (G - j) for j in range(topk)))  # tokens with such a row
    if kind in ("gate_up", "down"):
        N, K = case["N"], case["K"]
        active = E * (1 - (1 - topk / G) ** T)  # experts that any token chose
        a = tokens * K * (0.5 + 1 / 32) if kind == "gate_up" else slots * K * 4
        return {"bytes": active * N * K * (0.5 + 1 / 32) + a + slots * N * size[case["out"]], "flops": 2 * slots * N * K}
    row = case["H"] * size[case["dtype"]]
    if kind == "permute":
        return {"bytes": tokens * row + slots * row + 8 * T * topk, "flops": 0}
    if kind == "permute_bwd":
        return {"bytes": slots * row + T * row + 4 * T * topk, "flops": slots * case["H"]}
    out = case["H"] * size[case["out"]]
    if kind == "unpermute":
        return {"bytes": slots * row + T * out + 8 * T * topk, "flops": 2 * slots * case["H"]}
    return {"bytes": tokens * out + 2 * slots * row + 16 * T * topk, "flops": 3 * slots * case["H"]}


# ------------------------------------------------------------------ the definition in 64 bits


def _level(x):
    """The nearest 4-bit level of |x| / 2^e with its sign, e from the largest of each 32: by distance to each level."""
    blocks = x.reshape(x.shape[0], -1, 32)
    out = torch.empty_like(blocks)
    for r in range(0, x.shape[0], 2048):
        b = blocks[r : r + 2048]
        most = b.abs().amax(-1, keepdim=True)
        e = torch.floor(torch.log2(most.clamp(min=2.0**-1000)))
        e = torch.where(torch.exp2(e + 1) <= most, e + 1, torch.where(torch.exp2(e) > most, e - 1, e))
        unit = torch.exp2((e - 2).clamp(min=-127.0))
        m = (b / unit).abs()
        best, far = torch.zeros_like(m), m.clone()
        for i, level in enumerate(LEVELS[1:], 1):
            d = (m - level).abs()
            nearer = (d < far) | ((d == far) & (i % 2 == 0))  # a tie goes to the even code
            best, far = torch.where(nearer, torch.full_like(m, level), best), torch.minimum(d, far)
        out[r : r + 2048] = torch.sign(b) * best * unit
    return out.view(x.shape)


def _wide(q, s):
    """Packed codes and scale bytes in 64 bits, by the bits of a code: sign, two of exponent, one of mantissa."""
    code = torch.empty(q.shape[:-1] + (2 * q.shape[-1],), dtype=torch.float64, device=q.device)
    for half in (0, 1):
        c = ((q >> (4 * half)) & 15).double()
        sign = 1 - 2 * (c >= 8).double()
        c = c % 8
        e, m = torch.floor(c / 2), c % 2
        code[..., half::2] = sign * torch.where(e == 0, 0.5 * m, torch.exp2(e - 1) * (1 + 0.5 * m))
    return code * torch.exp2(s.double() - 127).repeat_interleave(32, dim=-1)


def exact(case, seed):
    state = prepare(case, seed)
    kind = case["kind"]
    if kind == "quantize":
        return _level(state["x"].double())
    T, topk, E, bm = case["T"], case["topk"], case["E"], case["bm"]
    plan = state["plan"]
    M = plan["rows"]
    live = torch.nonzero(plan["sorted"][:M] < T * topk).flatten()
    slot = plan["sorted"][live].long()
    if kind == "permute":
        xp = torch.zeros(M, case["H"], dtype=torch.float64, device=DEVICE)
        xp[live] = state["x"].double()[slot // topk]
        return xp, None
    if kind in ("permute_bwd", "unpermute"):
        given = state["dxp"] if kind == "permute_bwd" else state["y"]
        total = torch.zeros(T, case["H"], dtype=torch.float64, device=DEVICE)
        weight = torch.ones(T * topk, device=DEVICE) if kind == "permute_bwd" else state["weights"].reshape(-1)
        for j in range(topk):  # one slot of every token at a time
            mine = slot % topk == j
            total[slot[mine] // topk] += given[live[mine]].double() * weight[slot[mine]].double()[:, None]
        return total
    if kind == "unpermute_bwd":
        dy = torch.zeros(M, case["H"], dtype=torch.float64, device=DEVICE)
        above = state["dout"].double()[slot // topk]
        dy[live] = above * state["weights"].reshape(-1)[slot].double()[:, None]
        dweights = torch.zeros(T * topk, dtype=torch.float64, device=DEVICE)
        dweights[slot] = (above * state["y"][live].double()).sum(-1)
        return dy, dweights.view(T, topk)
    out = torch.zeros(M, case["N"], dtype=torch.float64, device=DEVICE)
    expert = plan["expert_ids"][live // bm]
    if kind == "gate_up":
        a = _wide(state["a_q"], state["a_s"])
        source = slot // topk
    else:
        g = state["gu"][:M].double()
        a = _level(g[:, : case["K"]] * torch.sigmoid(g[:, : case["K"]]) * g[:, case["K"] :])
        source = live
    for e in range(E):
        mine = expert == e
        if bool(mine.any()):
            out[live[mine]] = a[source[mine]] @ _wide(state["w_q"][e], state["w_s"][e]).T.contiguous()
    return out
