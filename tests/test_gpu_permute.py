"""moe_permute, moe_unpermute and their gradients against plain 64-bit numpy,
and a run of them with the alignment and the contiguous layout as a program uses them."""
import numpy as np
import pytest
import torch

import w4a16_grouped_gemm_amd as w
from _fp4 import dev, floor_of, half_step, routing, slot_rows, wide
from _gpu import say

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# T, topk, resident experts, routed experts, hidden, block_m
SHAPES = [
    (1, 1, 1, 1, 1, 16),
    (1, 8, 48, 384, 7168, 16),
    (5, 2, 3, 4, 65, 16),
    (7, 3, 8, 8, 64, 32),
    (33, 8, 16, 16, 1000, 64),
    (129, 4, 6, 24, 513, 128),
    (257, 2, 64, 64, 72, 128),
    (300, 32, 40, 64, 40, 16),
    (2100, 8, 16, 32, 200, 128),
    (1200, 12, 13, 13, 2056, 32),
    (1100, 8, 12, 15, 1001, 64),
    (40, 4, 160, 160, 77, 128),
    (2050, 5, 9, 9, 4101, 128),
]


class Plan:
    def __init__(self, T, topk, E, G, bm, seed=0, ids=None):
        import oracle

        rng = np.random.default_rng(seed)
        self.ids = routing(rng, T, topk, E, G) if ids is None else ids
        srt, eid, self.rows, _ = oracle.moe_align(self.ids, E, bm)
        self.n = T * topk
        self.srt = srt
        self.slot_rows = slot_rows(srt, self.rows, self.n).reshape(T, topk)
        self.sorted, self.expert_ids = dev(srt), dev(eid)
        self.ntpp = dev(np.array([self.rows], np.int32))
        self.live = np.nonzero(srt[: self.rows] < self.n)[0]
        self.slots = srt[self.live]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_permute(shape, dtype):
    T, topk, E, G, H, bm = shape
    say("permute", shape, dtype)
    plan = Plan(T, topk, E, G, bm)
    x = torch.randn(T, H, device="cuda").to(TYPES[dtype])
    xp = torch.full((len(plan.srt), H), 7.0, dtype=TYPES[dtype], device="cuda")
    rows = torch.full((T, topk), -9, dtype=torch.int32, device="cuda")
    w.moe_permute(x, plan.sorted, plan.ntpp, topk, xp, rows)
    torch.cuda.synchronize()
    want = np.full(xp.shape, 7.0)  # rows behind the last block stay as they were
    want[: plan.rows] = 0
    want[plan.live] = wide(x)[plan.slots // topk]
    assert np.array_equal(wide(xp), want)
    assert np.array_equal(rows.cpu().numpy(), plan.slot_rows)


@pytest.mark.parametrize("types", ["bf16-bf16", "fp16-fp16", "fp32-fp32", "fp32-bf16", "fp32-fp16"])
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_unpermute_and_gradients(shape, weighted, types):
    T, topk, E, G, H, bm = shape
    ty, to = (TYPES[t] for t in types.split("-"))
    say("unpermute", shape, weighted, types)
    plan = Plan(T, topk, E, G, bm, seed=1)
    gen = torch.Generator(device="cuda").manual_seed(3)
    y = torch.randn(len(plan.srt), H, device="cuda", generator=gen).to(ty)
    dout = torch.randn(T, H, device="cuda", generator=gen).to(to)
    wt = torch.rand(T, topk, device="cuda", generator=gen)
    # what no slot points to is never read: padding rows of y and weights without a row hold NaN
    dead = np.setdiff1d(np.arange(len(plan.srt)), plan.live)
    y[dev(dead)] = float("nan")
    wt[dev(plan.slot_rows < 0)] = float("nan")
    weights = wt if weighted else None
    rows = dev(plan.slot_rows)

    out = torch.full((T, H), 7.0, dtype=to, device="cuda")
    w.moe_unpermute(y, rows, out, topk_weights=weights)
    dy = torch.full_like(y, 7.0)
    dw = torch.full((T, topk), 7.0, device="cuda")
    w.moe_unpermute_backward(dout, y, rows, weights, plan.sorted, plan.ntpp, dy, dw)
    only_dy = torch.full_like(y, 7.0)
    w.moe_unpermute_backward(dout, None, rows, weights, plan.sorted, plan.ntpp, only_dy, None)
    only_dw = torch.full_like(dw, 7.0)
    w.moe_unpermute_backward(dout, y, rows, weights, None, None, None, only_dw)
    torch.cuda.synchronize()
    assert torch.equal(only_dy, dy) and torch.equal(only_dw, dw)

    y64, d64 = wide(y), wide(dout)
    w64 = wide(wt) if weighted else np.ones((T, topk))
    slot_w = w64.reshape(-1)[plan.slots][:, None]
    ref, size = np.zeros((T, H)), np.zeros((T, H))
    np.add.at(ref, plan.slots // topk, slot_w * y64[plan.live])
    np.add.at(size, plan.slots // topk, np.abs(slot_w * y64[plan.live]))
    # topk products and sums in fp32, each off by at most 2^-24 of the terms' size, then one rounding
    off = 2 * topk * 2.0**-24 * size
    assert np.all(np.abs(wide(out) - ref) <= off + half_step(to) * (np.abs(ref) + off) + floor_of(to))

    want = np.full(dy.shape, 7.0)
    want[: plan.rows] = 0
    want[plan.live] = slot_w * d64[plan.slots // topk]
    # one product in fp32 and one rounding
    assert np.all(np.abs(wide(dy) - want) <= (2.0**-23 + half_step(ty)) * np.abs(want) + floor_of(ty))

    ref_w, size_w = np.zeros(plan.n), np.zeros(plan.n)
    ref_w[plan.slots] = (d64[plan.slots // topk] * y64[plan.live]).sum(1)
    size_w[plan.slots] = np.abs(d64[plan.slots // topk] * y64[plan.live]).sum(1)
    got = wide(dw).reshape(-1)
    # H products and sums in fp32
    assert np.all(np.abs(got - ref_w) <= (H + 1) * 2.0**-24 * size_w)
    none = np.ones(plan.n, bool)
    none[plan.slots] = False
    assert np.all(got[none] == 0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_permute_backward(shape, dtype):
    T, topk, E, G, H, bm = shape
    plan = Plan(T, topk, E, G, bm, seed=2)
    dxp = torch.randn(len(plan.srt), H, device="cuda").to(TYPES[dtype])
    dx = torch.full((T, H), 7.0, dtype=TYPES[dtype], device="cuda")
    w.moe_permute_backward(dxp, dev(plan.slot_rows), dx)
    torch.cuda.synchronize()
    ref, size = np.zeros((T, H)), np.zeros((T, H))
    np.add.at(ref, plan.slots // topk, wide(dxp)[plan.live])
    np.add.at(size, plan.slots // topk, np.abs(wide(dxp)[plan.live]))
    off = topk * 2.0**-24 * size
    half = half_step(TYPES[dtype])
    assert np.all(np.abs(wide(dx) - ref) <= off + half * (np.abs(ref) + off) + floor_of(TYPES[dtype]))


def test_gradients_against_differences():
    """L = <c, unpermute(f(permute(x)), w)> with f doubling a row: dL/dx and dL/dw by the operators
    against central differences of the operators' own forward pass (fp32; L is bilinear, so a
    difference is exact but for the rounding of L, about 2^-22 of the terms' size over a step of 1/4)."""
    T, topk, E, H, bm = 6, 2, 3, 24, 16
    plan = Plan(T, topk, E, 4, bm, seed=5)
    gen = torch.Generator(device="cuda").manual_seed(9)
    x, c = (torch.randn(T, H, device="cuda", generator=gen) for _ in range(2))
    wt = torch.rand(T, topk, device="cuda", generator=gen)
    xp = torch.zeros(len(plan.srt), H, device="cuda")
    rows = torch.zeros(T, topk, dtype=torch.int32, device="cuda")

    def forward(x, wt):
        w.moe_permute(x, plan.sorted, plan.ntpp, topk, xp, rows)
        out = torch.zeros(T, H, device="cuda")
        w.moe_unpermute(2 * xp, rows, out, topk_weights=wt)
        return float((out.double() * c.double()).sum())

    forward(x, wt)
    y = 2 * xp
    dy, dw, dx = torch.zeros_like(xp), torch.zeros_like(wt), torch.zeros_like(x)
    w.moe_unpermute_backward(c, y, rows, wt, plan.sorted, plan.ntpp, dy, dw)
    w.moe_permute_backward(2 * dy, rows, dx)
    size = float((c.abs().double() * 2 * topk * (x.abs().double() + 0.25)).sum())
    for t, h in [(0, 0), (1, 5), (3, 23), (5, 11)]:
        step = torch.zeros_like(x)
        step[t, h] = 0.125
        diff = (forward(x + step, wt) - forward(x - step, wt)) / 0.25
        assert abs(diff - float(dx[t, h])) <= 2 * 4 * 2.0**-22 * size
    for t, j in [(0, 0), (2, 1), (4, 0), (5, 1)]:
        step = torch.zeros_like(wt)
        step[t, j] = 0.125
        diff = (forward(x, wt + step) - forward(x, wt - step)) / 0.25
        assert abs(diff - float(dw[t, j])) <= 2 * 4 * 2.0**-22 * size


def test_no_tokens_and_nothing_resident():
    x = torch.zeros(0, 64, device="cuda")
    out = torch.zeros(0, 64, device="cuda")
    rows = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    plan = Plan(0, 2, 4, 4, 16)
    xp = torch.full((len(plan.srt), 64), 7.0, device="cuda")
    w.moe_permute(x, plan.sorted, plan.ntpp, 2, xp, rows)
    w.moe_unpermute(xp, rows, out)
    torch.cuda.synchronize()
    assert bool((xp == 7).all())
    ids = np.full((5, 2), 9, np.int32)  # experts of another GPU
    plan = Plan(5, 2, 4, 4, 16, ids=ids)
    x = torch.randn(5, 64, device="cuda")
    xp = torch.full((len(plan.srt), 64), 7.0, device="cuda")
    rows = torch.zeros(5, 2, dtype=torch.int32, device="cuda")
    w.moe_permute(x, plan.sorted, plan.ntpp, 2, xp, rows)
    out = torch.full((5, 64), 7.0, device="cuda")
    w.moe_unpermute(xp, rows, out)
    torch.cuda.synchronize()
    assert bool((rows == -1).all()) and bool((out == 0).all()) and bool((xp == 7).all())


def test_same_expert_twice_and_filtered():
    """A token may name an expert twice; experts that moe_align_filtered leaves out have no rows."""
    ids = np.array([[1, 1], [0, 1], [2, 2], [1, 0]], np.int32)
    d = dev(ids)
    E, bm, H = 3, 16, 40
    buf = w.align_buffers(4, 2, E, bm)
    w.moe_align_filtered(d, E, bm, 3, 100, buf["sorted_token_ids"], buf["expert_ids"], buf["num_tokens_post_padded"])
    x = torch.randn(4, H, device="cuda")
    xp = torch.zeros(buf["sorted_token_ids"].numel(), H, device="cuda")
    rows = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    w.moe_permute(x, buf["sorted_token_ids"], buf["num_tokens_post_padded"], 2, xp, rows)
    torch.cuda.synchronize()
    assert rows.cpu().tolist() == [[0, 1], [-1, 2], [-1, -1], [3, -1]]
    for p, t in enumerate([0, 0, 1, 3]):
        assert torch.equal(xp[p], x[t])
    out = torch.zeros(4, H, device="cuda")
    w.moe_unpermute(xp, rows, out)
    torch.cuda.synchronize()
    assert torch.equal(out, x * torch.tensor([2.0, 1.0, 0.0, 1.0], device="cuda")[:, None])


def test_unaligned_buffers():
    """Rows and buffers that start at any element, as slices of larger buffers do."""
    T, topk, E, H, bm = 9, 2, 4, 31, 16
    plan = Plan(T, topk, E, 4, bm, seed=4)
    for dtype in TYPES.values():
        x = torch.randn(T * H + 1, device="cuda").to(dtype)[1:].view(T, H)
        xp = torch.zeros(len(plan.srt) * H + 3, device="cuda", dtype=dtype)[3:].view(-1, H)
        rows = torch.zeros(T, topk, dtype=torch.int32, device="cuda")
        w.moe_permute(x, plan.sorted, plan.ntpp, topk, xp, rows)
        out = torch.zeros(T * H + 1, device="cuda", dtype=dtype)[1:].view(T, H)
        w.moe_unpermute(xp, rows, out)
        torch.cuda.synchronize()
        assert torch.equal(out, 2 * x)  # exact: the same value twice


def test_shorter_sorted_list_stays_in_bounds():
    """Only the first `capacity` rows are the call's: no row past them is read or written."""
    T, topk, E, H, bm = 12, 2, 3, 48, 16
    plan = Plan(T, topk, E, 3, bm, seed=8)
    cap = 20  # inside the second block
    x = torch.randn(T, H, device="cuda")
    xp = torch.full((40, H), 7.0, device="cuda")
    rows = torch.zeros(T, topk, dtype=torch.int32, device="cuda")
    w.moe_permute(x, plan.sorted[:cap], plan.ntpp, topk, xp, rows)
    torch.cuda.synchronize()
    assert bool((xp[cap:] == 7).all())
    assert np.array_equal(rows.cpu().numpy(), np.where(plan.slot_rows < cap, plan.slot_rows, -1))
    # rows beyond y count as no row
    out = torch.zeros(T, H, device="cuda")
    w.moe_unpermute(xp[:10], dev(plan.slot_rows), out)
    torch.cuda.synchronize()
    want = np.zeros((T, H))
    for t in range(T):
        for r in plan.slot_rows[t]:
            if 0 <= r < 10:
                want[t] += wide(xp)[r]
    assert np.allclose(wide(out), want, rtol=2.0**-22, atol=0)


def test_graph_and_streams():
    """Captured and replayed with eager work of the same buffers between the replays, and on another stream."""
    T, topk, E, H, bm = 70, 4, 8, 520, 32
    plan = Plan(T, topk, E, 8, bm, seed=6)
    x = torch.randn(T, H, device="cuda")
    wt = torch.rand(T, topk, device="cuda")
    xp = torch.zeros(len(plan.srt), H, device="cuda")
    rows = torch.zeros(T, topk, dtype=torch.int32, device="cuda")
    out, dy = torch.zeros(T, H, device="cuda"), torch.zeros_like(xp)
    dw = torch.zeros_like(wt)

    def step():
        w.moe_permute(x, plan.sorted, plan.ntpp, topk, xp, rows)
        w.moe_unpermute(xp, rows, out, topk_weights=wt)
        w.moe_unpermute_backward(out, xp, rows, wt, plan.sorted, plan.ntpp, dy, dw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(4):
        x.copy_(torch.randn(T, H, device="cuda"))
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (xp, rows, out, dy, dw)]
        for t in (xp, rows, out, dy, dw):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, (xp, rows, out, dy, dw)):
            assert torch.equal(a, b), k


def test_contiguous_layer_from_tokens():
    """Tokens permuted into the contiguous layout, the INT4 layer on it, and its rows brought back weighted
    equal the routed layer: the rows are the same but for the bf16 rounding of each row's output before
    the weighted sum."""
    import synthetic
    from _gpu import DeviceCase

    c = synthetic.random_case("permuted", T=64, H=256, I=128, E=8, topk=2, block_m=128, seed=77)
    d = DeviceCase(c)
    buf = d.align(128)
    M = int(buf["num_tokens_post_padded"].item())
    srt = buf["sorted_token_ids"]
    x = d.x.view(torch.bfloat16)
    xp = torch.empty(M, c.H, dtype=torch.bfloat16, device="cuda")
    rows = torch.empty(c.T, c.topk, dtype=torch.int32, device="cuda")
    w.moe_permute(x, srt[:M], buf["num_tokens_post_padded"], c.topk, xp, rows)
    expert = buf["expert_ids"][: M // 128].repeat_interleave(128)
    expert = torch.where(srt[:M] < c.T * c.topk, expert, -1).int()
    ws = torch.empty(w.w4a16_moe_contiguous_workspace_bytes(d.shape, M), dtype=torch.uint8, device="cuda")
    y = torch.empty(M, c.H, dtype=torch.bfloat16, device="cuda")
    w.w4a16_moe_contiguous_forward(d.shape, xp, expert, d.w13p, d.w2p, y, ws)
    out = torch.empty(c.T, c.H, dtype=torch.bfloat16, device="cuda")
    w.moe_unpermute(y, rows, out, topk_weights=d.wts)
    torch.cuda.synchronize()
    routed = torch.from_numpy(d.forward(128).view(np.int16)).view(torch.bfloat16)
    y64 = np.abs(wide(y))[rows.cpu().numpy()]
    # each row and both outputs are off by at most half a bf16 step; the fp32 sums of the same terms by far less
    size = (wide(d.wts)[..., None] * y64).sum(1)
    assert np.all(np.abs(wide(out) - wide(routed)) <= 3.05 * 2.0**-8 * size)


def test_offsets_past_32_bits():
    """320000 rows of 7168: more elements than 2^31. Exact on the device: rows are copied, and with weights of
    1/8 the weighted sum of eight equal rows is the row."""
    T, topk, E, H, bm = 40000, 8, 16, 7168, 128
    say("far offsets")
    ids = torch.rand(T, E, device="cuda").topk(topk, dim=1)[1].int()
    buf = w.align_buffers(T, topk, E, bm)
    w.moe_align(ids, E, bm, buf["sorted_token_ids"], buf["expert_ids"], buf["num_tokens_post_padded"],
                workspace=buf["workspace"])
    srt, ntpp = buf["sorted_token_ids"], buf["num_tokens_post_padded"]
    M = int(ntpp.item())
    assert M * H > 2**31
    x = torch.randn(T, H, device="cuda").bfloat16()
    xp = torch.full((M, H), 7.0, dtype=torch.bfloat16, device="cuda")
    rows = torch.zeros(T, topk, dtype=torch.int32, device="cuda")
    w.moe_permute(x, srt[:M], ntpp, topk, xp, rows)
    real = srt[:M] < T * topk
    at = torch.nonzero(real).flatten()[:: 997]
    at = torch.cat([at, torch.nonzero(real).flatten()[-64:]])
    assert torch.equal(xp[at], x[(srt[at] // topk).long()])
    assert not bool(xp[torch.nonzero(~real).flatten()].any())
    assert torch.equal(srt[rows.flatten().long()], torch.arange(T * topk, dtype=torch.int32, device="cuda"))
    wt = torch.full((T, topk), 0.125, device="cuda")
    out, dy, dw = torch.zeros_like(x), torch.full_like(xp, 7.0), torch.zeros_like(wt)
    w.moe_unpermute(xp, rows, out, topk_weights=wt)
    assert torch.equal(out, x)
    w.moe_unpermute_backward(x, xp, rows, wt, srt[:M], ntpp, dy, dw)
    assert torch.equal(dy[at], x[(srt[at] // topk).long()] / 8)
    dot = (x[-64:].double() ** 2).sum(1, keepdim=True)
    assert bool(((dw[-64:] - dot).abs() <= (H + 1) * 2.0**-24 * dot).all())


def test_more_column_passes_than_a_launch_has_workgroups():
    """4 Mi tokens of two passes of 2048 columns each: a workgroup takes a whole row. Exact: one slot a token, weight 1."""
    T, H = (1 << 22) + 5, 2057
    say("many tokens")
    y = torch.randn(7, H, device="cuda").bfloat16()
    rows = torch.full((T, 1), -1, dtype=torch.int32, device="cuda")
    at = torch.tensor([0, 1, 1 << 20, (1 << 21) - 1, 1 << 21, T - 2, T - 1], device="cuda")
    rows[at, 0] = torch.arange(7, dtype=torch.int32, device="cuda")
    out = torch.full((T, H), 7.0, dtype=torch.bfloat16, device="cuda")
    w.moe_unpermute(y, rows, out)
    assert torch.equal(out[at], y)
    out[at] = 0
    for part in out.split(1 << 19):
        assert not bool(part.any())


@pytest.mark.parametrize("T", [70, 2100])
def test_the_stream_that_is_given(T):
    """Each row operator on a stream given by argument, behind work there that makes its inputs, while another stream
    is current: the small permutes' one launch and the three of many slots."""
    topk, E, H, bm = 8, 16, 264, 32
    plan = Plan(T, topk, E, 16, bm, seed=10)
    x0, x1 = (torch.randn(T, H, device="cuda") for _ in range(2))
    x = x0.clone()
    wt = torch.rand(T, topk, device="cuda")
    xp = torch.zeros(len(plan.srt), H, device="cuda")
    rows = torch.full((T, topk), -1, dtype=torch.int32, device="cuda")
    out, dx, dy, dw = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(xp), torch.zeros_like(wt)

    def step(stream=None):
        w.moe_permute(x, plan.sorted, plan.ntpp, topk, xp, rows, stream=stream)
        w.moe_unpermute(xp, rows, out, topk_weights=wt, stream=stream)
        w.moe_unpermute_backward(out, xp, rows, wt, plan.sorted, plan.ntpp, dy, dw, stream=stream)
        w.moe_permute_backward(dy, rows, dx, stream=stream)

    x.copy_(x1)
    step()
    torch.cuda.synchronize()
    outputs = (xp, rows, out, dy, dw, dx)
    want = [t.clone() for t in outputs]
    x.copy_(x0)
    for t in outputs:
        t.zero_()
    big = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(20):
            big = (big @ big).clamp(-1, 1)
        x.copy_(x1)
    step(side)
    side.synchronize()
    for a, b in zip(want, outputs):
        assert torch.equal(a, b)
