"""Routings and plain 64-bit references of the experts' product, its gradients and 8-bit checkpoints."""
from __future__ import annotations

import torch

import w4a16_grouped_gemm_amd as w

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SUM_STEP = 2.0**-23  # an fp32 addition, rounded to nearest or towards zero, is off by less than this of its result


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


class Routing:
    """Routed ids of T tokens over G experts, the first E of them resident, aligned on the GPU."""

    def __init__(self, T, topk, E, G, bm, seed=0, only=None):
        g = torch.Generator().manual_seed(seed)
        if only is None:
            ids = torch.rand(T, G, generator=g).topk(topk, dim=1)[1] if T else torch.zeros(0, topk)
        else:  # every slot to one of these experts
            ids = torch.tensor(only)[torch.randint(0, len(only), (T, topk), generator=g)]
        self.T, self.topk, self.E, self.bm, self.n = T, topk, E, bm, T * topk
        self.ids = ids.int().cuda()
        buf = w.align_buffers(T, topk, E, bm)
        w.moe_align(self.ids, E, bm, buf["sorted_token_ids"], buf["expert_ids"], buf["num_tokens_post_padded"],
                    buf["expert_counts"], buf["workspace"])
        self.sorted, self.expert_ids, self.ntpp = (buf[k] for k in ("sorted_token_ids", "expert_ids",
                                                                    "num_tokens_post_padded"))
        self.capacity = self.sorted.numel()
        self.rows = int(self.ntpp.item())
        slots = self.sorted[: self.rows].cpu().long()
        self.live = torch.nonzero(slots < self.n).flatten()
        self.token = slots[self.live] // topk
        self.expert = self.expert_ids.cpu()[self.live // bm].long()

    def args(self):
        return self.T, self.topk, self.sorted, self.expert_ids, self.ntpp, self.bm

    def source(self, gather):
        return self.token if gather else self.live


def product(r: Routing, a, weights, gather, transposed):
    """(out, sum of the products' magnitudes) in 64 bits, [rows, N]; a and weights on the CPU."""
    N = weights.shape[2] if transposed else weights.shape[1]
    out, size = torch.zeros(r.rows, N, dtype=torch.float64), torch.zeros(r.rows, N, dtype=torch.float64)
    source = r.source(gather)
    for e in r.expert.unique().tolist():
        if not 0 <= e < weights.shape[0]:
            continue
        mine = r.expert == e
        x, m = a[source[mine]].double(), weights[e].double()
        m = m if transposed else m.T
        out[r.live[mine]], size[r.live[mine]] = x @ m, x.abs() @ m.abs()
    return out, size


def weight_gradient(r: Routing, dout, a, E, gather):
    N, K = dout.shape[1], a.shape[1]
    dw, size = torch.zeros(E, N, K, dtype=torch.float64), torch.zeros(E, N, K, dtype=torch.float64)
    source = r.source(gather)
    for e in r.expert.unique().tolist():
        if not 0 <= e < E:
            continue
        mine = r.expert == e
        d, x = dout[r.live[mine]].double(), a[source[mine]].double()
        dw[e], size[e] = d.T @ x, d.abs().T @ x.abs()
    return dw, size


def sum_error(size, terms, dtype):
    """Bound of |out - ref|: `terms` additions in fp32, each off by less than SUM_STEP of a partial sum that is at most
    `size`, and one rounding to dtype (of a value of at most `size`, hence the reference's own magnitude apart)."""
    return terms * SUM_STEP * size


def check(got, ref, size, terms, what):
    """|got - ref| within the sums' error and one rounding to got's type."""
    dtype = got.dtype
    got = got.cpu().double()
    sums = sum_error(size, terms, dtype)
    rounding = half_step(dtype) * (ref.abs() + sums) if dtype != torch.float32 else 0.0
    tiny = 2.0**-25 if dtype == torch.float16 else 2.0**-133  # half a step below the type's normal numbers
    err, tol = (got - ref).abs(), sums + rounding + tiny
    bad = ~(err <= tol)
    print(f"  {what}: max err/tol {float((err / tol).max()) if err.numel() else 0:.4f}", flush=True)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, e.g. {torch.nonzero(bad)[:5].tolist()}"


MOST = 448.0


def levels():
    code = torch.arange(127, dtype=torch.float64)
    e, m = torch.floor(code / 8), code % 8
    return torch.where(e == 0, m * 2.0**-9, torch.exp2(e - 7) * (1 + m / 8))


def quantize8(x):
    """x [rows, K] on the CPU -> code bytes [rows, K] and scale bytes [rows, K / 32], from the definition."""
    lv = levels()
    middle = (lv[1:] + lv[:-1]) / 2
    b = x.double().reshape(x.shape[0], -1, 32)
    finite = torch.isfinite(b).all(-1)
    clean = torch.where(torch.isfinite(b), b, 0.0)
    most = clean.abs().amax(-1)
    byte = torch.zeros_like(most, dtype=torch.int64)
    for s in range(254):  # the smallest scale that takes the largest value
        byte += (most > MOST * 2.0 ** (s - 127)).long()
    byte = torch.where(finite, byte, 255)
    v = torch.where(finite[..., None], clean / torch.exp2(byte.double() - 127)[..., None], 0.0)
    m = v.abs()
    code = torch.searchsorted(middle, m.contiguous(), right=False)  # middles below m
    at = (code < 126) & (m == middle[code.clamp(max=125)])
    code = torch.where(at & (code % 2 == 1), code + 1, code)
    code = code + 128 * (torch.signbit(v) & finite[..., None])
    return code.reshape(x.shape).to(torch.uint8), byte.to(torch.uint8)


def values8(q, s):
    """Code and scale bytes on the CPU -> the values they stand for, in 64 bits."""
    lv = torch.cat((levels(), torch.tensor([float("nan")], dtype=torch.float64)))
    v = torch.where(q >= 128, -1.0, 1.0).double() * lv[(q & 127).long()]
    scale = torch.where(s == 255, float("nan"), torch.exp2(s.double() - 127))
    return v * scale.repeat_interleave(32, dim=-1)


def silu_and_gradient(g, u, dh):
    """(h, dg, du) in 64 bits."""
    y, rest = torch.sigmoid(g), torch.sigmoid(-g)
    silu = g * y
    return silu * u, dh * u * (y + silu * rest), dh * silu
