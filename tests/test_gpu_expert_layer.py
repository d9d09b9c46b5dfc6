"""A training step of the experts' layer from its parts: rows to their experts, two products around the gated activation
with its 8-bit checkpoint, rows back, and every gradient, against 64-bit autograd with bounds carried from part to part."""
import os
import re

import pytest
import torch

import w4a16_grouped_gemm_amd as w
from _gpu import say
from _grouped import SUM_STEP, TYPES, Routing, half_step, quantize8, values8

pytestmark = pytest.mark.gpu


class Layer:
    """The layer on the GPU. `gather`: the first product reads token rows through the routing, else permuted ones."""

    def __init__(self, r: Routing, H, I, dtype, gather):
        self.r, self.H, self.I, self.dtype, self.gather = r, H, I, dtype, gather
        new = lambda *shape, t=dtype: torch.full(shape, 77, dtype=t, device="cuda")  # noqa: E731
        rows, T, E = r.capacity, r.T, r.E
        self.xp, self.gu, self.h, self.y = new(rows, H), new(rows, 2 * I), new(rows, I), new(rows, H)
        self.slot_rows = new(T, r.topk, t=torch.int32)
        self.q, self.s = new(rows, 2 * I, t=torch.uint8), new(rows, I // 16, t=torch.uint8)
        self.out, self.dx = new(T, H), new(T, H)
        self.dy, self.dh, self.again, self.dgu, self.dxp = (new(rows, n) for n in (H, I, I, 2 * I, H))
        self.dw1, self.dw2 = new(E, 2 * I, H, t=torch.float32), new(E, H, I, t=torch.float32)
        self.dweights = new(T, r.topk, t=torch.float32)
        self.ws = [torch.empty(max(1, w.moe_grouped_gemm_wgrad_workspace_bytes(*d.shape, rows)), dtype=torch.uint8,
                               device="cuda") for d in (self.dw1, self.dw2)]

    def forward(self, x, w1, w2, weights):
        r, route = self.r, self.r.args()
        w.moe_permute(x, r.sorted, r.ntpp, r.topk, self.xp, self.slot_rows)
        w.moe_grouped_gemm(x if self.gather else self.xp, *route, w1, self.gu, gather=self.gather)
        w.mxfp8_silu_mul(self.gu, self.h, self.q, self.s, num_rows=r.ntpp)
        w.moe_grouped_gemm(self.h, *route, w2, self.y)
        w.moe_unpermute(self.y, self.slot_rows, self.out, weights)

    def backward(self, x, w1, w2, weights, dout):
        r, route = self.r, self.r.args()
        w.moe_unpermute_backward(dout, self.y, self.slot_rows, weights, r.sorted, r.ntpp, self.dy, self.dweights)
        w.moe_grouped_gemm(self.dy, *route, w2, self.dh, transposed=True)
        w.mxfp8_silu_mul_backward(self.q, self.s, self.dh, self.dgu, h=self.again, num_rows=r.ntpp)
        w.moe_grouped_gemm_wgrad(self.dy, self.again, *route, self.dw2, workspace=self.ws[1])
        w.moe_grouped_gemm_wgrad(self.dgu, x if self.gather else self.xp, *route, self.dw1, gather=self.gather,
                                 workspace=self.ws[0])
        w.moe_grouped_gemm(self.dgu, *route, w1, self.dxp, transposed=True)
        w.moe_permute_backward(self.dxp, self.slot_rows, self.dx)

    def results(self):
        n = self.r.rows  # rows behind the last block are nobody's
        return {"out": self.out, "y": self.y[:n], "q": self.q[:n], "s": self.s[:n], "dx": self.dx, "dw1": self.dw1,
                "dw2": self.dw2, "dweights": self.dweights}


def inputs(r, H, I, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(r.T, H, generator=g).to(dtype)
    w1 = (torch.randn(r.E, 2 * I, H, generator=g) * 2 * H**-0.5).to(dtype)
    w2 = (torch.randn(r.E, H, I, generator=g) * I**-0.5).to(dtype)
    weights = torch.rand(r.T, r.topk, generator=g)
    return x, w1, w2, weights, torch.randn(r.T, H, generator=g).to(dtype)


def rounded(err, ref, dtype):
    """The bound err and one rounding of what it bounds."""
    tiny = 2.0**-25 if dtype == torch.float16 else 2.0**-133
    return err + half_step(dtype) * (ref.abs() + err) + tiny


def matmul(a, ea, m, terms):
    """(a m, bound): a off by at most ea, `terms` fp32 additions, each off by SUM_STEP of at most the magnitudes' sum."""
    size = (a.abs() + ea) @ m.abs()
    return a @ m, ea @ m.abs() + terms * SUM_STEP * size


def within(got, ref, bound, what):
    err = (got.cpu().double() - ref).abs()
    say(f"  {what}: max err/tol {float((err / bound.clamp(min=1e-300)).max()):.4f}")
    assert bool((err <= bound).all()), f"{what}: {int((err > bound).sum())} of {err.numel()} off"


SHAPES = [  # T, topk, resident, routed, block_m, H, I
    (1, 2, 3, 4, 16, 64, 32),
    (97, 3, 5, 8, 16, 200, 96),
    (300, 2, 4, 4, 64, 328, 160),
    (700, 2, 3, 5, 128, 512, 256),
]


@pytest.mark.parametrize("gather", [False, True], ids=["permuted", "gathered"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_a_training_step(shape, dtype, gather):
    T, topk, E, G, bm, H, I = shape
    say("layer", shape, dtype, "gathered" if gather else "permuted")
    t = TYPES[dtype]
    r = Routing(T, topk, E, G, bm, seed=31)
    host = inputs(r, H, I, t, 32)
    x, w1, w2, weights, dout = (v.cuda() for v in host)
    layer = Layer(r, H, I, t, gather)
    layer.forward(x, w1, w2, weights)
    layer.backward(x, w1, w2, weights, dout)
    torch.cuda.synchronize()

    # Per slot in 64 bits. What the backward pass starts from are the codes that were kept, so these are compared with
    # their definition first, and are inputs from there on.
    n = r.rows
    gu_seen = layer.gu[:n].cpu()
    code, scale = quantize8(gu_seen)
    assert torch.equal(layer.q[:n].cpu(), code) and torch.equal(layer.s[:n].cpu(), scale)
    kept = values8(code, scale)
    rows_of = layer.slot_rows.cpu().long()
    hx, h1, h2, hw, hd = (v.double() for v in host)
    leaves = [v.clone().requires_grad_() for v in (hx, h1, h2)]
    out, out_err = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    loss = torch.zeros((), dtype=torch.float64)
    bound = {"dx": torch.zeros(T, H, dtype=torch.float64), "dw1": torch.zeros_like(h1), "dw2": torch.zeros_like(h2)}
    size_dx = torch.zeros(T, H, dtype=torch.float64)
    dweights, dweights_err = torch.zeros(T, topk, dtype=torch.float64), torch.zeros(T, topk, dtype=torch.float64)
    live = [(tk, j, int(rows_of[tk, j])) for tk in range(T) for j in range(topk) if rows_of[tk, j] >= 0]
    assert len(live) == r.live.numel()
    expert = dict(zip(r.live.tolist(), r.expert.tolist()))
    for e in sorted(set(expert.values())):
        mine = [(tk, j, p) for tk, j, p in live if expert[p] == e]
        tk, j, p = (torch.tensor(v) for v in zip(*mine))
        none = torch.zeros(len(mine), H, dtype=torch.float64)
        gu, egu = matmul(hx[tk], none, h1[e].T, H)
        egu = rounded(egu, gu, t)
        within(layer.gu[p], gu, egu, f"gu of expert {e}")
        g, u, eg, eu = gu[:, :I], gu[:, I:], egu[:, :I], egu[:, I:]
        h = torch.nn.functional.silu(g) * u
        # |silu| grows by at most 1.1 a unit; the activation's own arithmetic is good to 16 roundings of 2^-24
        eh = 1.1 * eg * (u.abs() + eu) + torch.nn.functional.silu(g).abs() * eu
        eh = rounded(eh + 16 * 2.0**-24 * (h.abs() + eh), h, t)
        y, ey = matmul(h, eh, h2[e].T, I)
        ey = rounded(ey, y, t)
        out.index_add_(0, tk, hw[tk, j, None] * y)
        out_err.index_add_(0, tk, hw[tk, j, None] * (ey + 2 * topk * SUM_STEP * (y.abs() + ey)))
        dweights[tk, j] = (hd[tk] * y).sum(1)
        dweights_err[tk, j] = (hd[tk].abs() * (ey + H * SUM_STEP * (y.abs() + ey))).sum(1)
        # backward: autograd's own graph of the same formula, of the values that were kept
        lx, l1, l2 = leaves
        gu_l = lx[tk] @ l1[e].T
        gu_l = gu_l + (kept[p] - gu_l).detach()
        h_l = torch.nn.functional.silu(gu_l[:, :I]) * gu_l[:, I:]
        loss = loss + (hw[tk, j, None] * (h_l @ l2[e].T) * hd[tk]).sum()
        # and the bounds
        dy = hw[tk, j, None] * hd[tk]
        edy = rounded(2.0**-24 * dy.abs(), dy, t)
        dh, edh = matmul(dy, edy, h2[e], H)
        edh = rounded(edh, dh, t)
        g, u = kept[p, :I], kept[p, I:]
        sig = torch.sigmoid(g)
        silu, slope = g * sig, sig + g * sig * torch.sigmoid(-g)
        parts = sig + (g * sig * torch.sigmoid(-g)).abs()
        again = silu * u
        eagain = rounded(16 * 2.0**-24 * again.abs(), again, t)
        dgu = torch.cat((dh * u * slope, dh * silu), 1)
        size = torch.cat(((dh.abs() + edh) * u.abs() * parts, (dh.abs() + edh) * silu.abs()), 1)
        edgu = torch.cat((edh * (u * slope).abs(), edh * silu.abs()), 1) + 16 * 2.0**-24 * size
        edgu = rounded(edgu, dgu, t)
        dxp, edxp = matmul(dgu, edgu, h1[e], 2 * I)
        edxp = rounded(edxp, dxp, t)
        bound["dx"].index_add_(0, tk, edxp)
        size_dx.index_add_(0, tk, dxp.abs() + edxp)
        # sums over the expert's rows, both factors off
        terms = len(mine) + 32
        a, ea = dy.abs(), edy
        bound["dw2"][e] = ea.T @ (again.abs() + eagain) + a.T @ eagain + terms * SUM_STEP * (
            (a + ea).T @ (again.abs() + eagain))
        bound["dw1"][e] = edgu.T @ hx[tk].abs() + terms * SUM_STEP * ((dgu.abs() + edgu).T @ hx[tk].abs())
    if live:
        loss.backward()
    grads = {k: v.grad if v.grad is not None else torch.zeros_like(v) for k, v in zip(("dx", "dw1", "dw2"), leaves)}
    bound["dx"] = rounded(bound["dx"] + topk * SUM_STEP * size_dx, grads["dx"], t)
    within(layer.out, out, rounded(out_err, out, t), "out")
    within(layer.dweights, dweights, dweights_err, "dweights")
    for k in ("dx", "dw1", "dw2"):
        # autograd's own sums in 64 bits are off by far less than 2^-40 of what they add up
        within(getattr(layer, k), grads[k], bound[k] + 2.0**-40 * grads[k].abs() + 2.0**-60, k)


def test_steps_in_a_graph():
    """The step captured once and replayed on new tokens and weights, with eager steps of another layer in between."""
    T, topk, E, G, bm, H, I = SHAPES[2]
    r = Routing(T, topk, E, G, bm, seed=33)
    t = torch.bfloat16
    graphed, eager = Layer(r, H, I, t, True), Layer(r, H, I, t, True)
    static = [v.cuda() for v in inputs(r, H, I, t, 34)]

    def step(layer, given):
        layer.forward(*given[:4])
        layer.backward(*given)

    step(graphed, static)  # loads what a first call loads
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(graphed, static)
    for seed in (35, 36, 37):
        given = [v.cuda() for v in inputs(r, H, I, t, seed)]
        for s, v in zip(static, given):
            s.copy_(v)
        graph.replay()
        step(eager, given)
        torch.cuda.synchronize()
        for k, v in graphed.results().items():
            assert torch.equal(v, eager.results()[k]), (seed, k)


def test_two_layers_at_once():
    """Two layers on two streams, each with its own buffers and workspace: the bits of each alone."""
    t = torch.bfloat16
    cases = []
    for shape, seed in ((SHAPES[1], 41), (SHAPES[3], 42)):
        T, topk, E, G, bm, H, I = shape
        r = Routing(T, topk, E, G, bm, seed=seed)
        given = [v.cuda() for v in inputs(r, H, I, t, seed)]
        alone, beside = Layer(r, H, I, t, False), Layer(r, H, I, t, False)
        alone.forward(*given[:4])
        alone.backward(*given)
        cases.append((given, alone, beside, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(3):
        for given, _, beside, stream in cases:
            with torch.cuda.stream(stream):
                beside.forward(*given[:4])
                beside.backward(*given)
    torch.cuda.synchronize()
    for _, alone, beside, _ in cases:
        for k, v in beside.results().items():
            assert torch.equal(v, alone.results()[k]), k


def test_readme_step():
    """The README's training step on buffers of its names: the bits of Layer's calls."""
    with open(os.path.join(os.path.dirname(__file__), "..", "README.md")) as f:
        code, = [c for c in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "moe_grouped_gemm_wgrad" in c]
    T, topk, E, G, bm, H, I = SHAPES[1]
    t = torch.bfloat16
    r = Routing(T, topk, E, G, bm, seed=51)
    given = [v.cuda() for v in inputs(r, H, I, t, 52)]
    layer, own = Layer(r, H, I, t, True), Layer(r, H, I, t, True)
    layer.forward(*given[:4])
    layer.backward(*given)
    x, w1, w2, weights, dout = given
    exec(code, {"w": w, "T": T, "topk": topk, "srt": r.sorted, "eid": r.expert_ids, "ntpp": r.ntpp, "bm": bm, "x": x,
                "w1": w1, "w2": w2, "topk_weights": weights, "dout": dout, "xp": own.xp, "slot_rows": own.slot_rows,
                "gu": own.gu, "h": own.h, "q": own.q, "s": own.s, "y": own.y, "out": own.out, "dy": own.dy, "dh": own.dh,
                "dgu": own.dgu, "dw1": own.dw1, "dw2": own.dw2, "ws1": own.ws[0], "ws2": own.ws[1], "dxp": own.dxp,
                "dx": own.dx, "dtopk_weights": own.dweights})
    torch.cuda.synchronize()
    for k, v in own.results().items():
        assert torch.equal(v, layer.results()[k]), k
