"""4-bit floating point rows and the experts' product on them against plain 64-bit numpy.

Quantisation is exact by definition (a division by a power of two and one
rounding), so codes and scales are compared bit for bit. The product's inputs in
the exact tests have few enough bits that every partial sum is an fp32 value:
there the output is the rounded 64-bit result, bit for bit, in any order of summation."""
import numpy as np
import pytest
import torch

import w4a16_grouped_gemm_amd as w
from _fp4 import dev, floor_of, half_step, pack, quantize, rounded, routing, values, wide
from _gpu import say

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def run_quantize(x: torch.Tensor, num_rows=None):
    rows, K = x.shape
    q = torch.full((rows, K // 2), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((rows, K // 32), 0x55, dtype=torch.uint8, device="cuda")
    w.mxfp4_quantize(x, q, s, num_rows=num_rows)
    torch.cuda.synchronize()
    return q, s


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(1, 32), (3, 64), (1, 7168), (129, 96), (1000, 1056), (70, 20000 // 32 * 32)], ids=str)
def test_quantize_is_exact(shape, dtype):
    rng = np.random.default_rng(1)
    say("quantize", shape, dtype)
    x = rng.standard_normal(shape) * np.exp2(rng.integers(-6, 7, (shape[0], shape[1] // 32)).repeat(32, 1))
    t = dev(x, TYPES[dtype])
    q, s = run_quantize(t)
    code, scale = quantize(wide(t))
    assert np.array_equal(s.cpu().numpy(), scale)
    assert np.array_equal(q.cpu().numpy(), pack(code))
    back = torch.zeros(shape, dtype=TYPES[dtype], device="cuda")
    w.mxfp4_dequantize(q, s, back)
    torch.cuda.synchronize()
    assert np.array_equal(wide(back), rounded(values(pack(code), scale), TYPES[dtype]))


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_every_border(dtype):
    """Every halfway point, its two neighbours in the type, and every magnitude, in both signs, at scales
    from the smallest to the largest of the type."""
    t = TYPES[dtype]
    top = {"bf16": 125, "fp16": 13, "fp32": 125}[dtype]
    low = {"bf16": -120, "fp16": -10, "fp32": -140}[dtype]
    points = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, 7.75, 0.0]
    rows = []
    for e in range(low, top + 1):
        p = torch.tensor(points, dtype=torch.float64) * 2.0**e
        p = p.to(t)
        near = torch.cat([p, torch.nextafter(p.float(), torch.tensor(float("inf"))).to(t) if t == torch.float32 else
                          (p.view(torch.int16) + 1).view(t)])
        rows.append(torch.cat([near, near]))  # 64 values: two blocks
        less = (p.view(torch.int32) - 1).view(t) if t == torch.float32 else (p.view(torch.int16) - 1).view(t)
        less[-1] = 0
        rows.append(-torch.cat([p, less, less, p]))
    x = torch.stack(rows).cuda()
    ok = torch.isfinite(x.float()).all()
    assert bool(ok)
    q, s = run_quantize(x)
    code, scale = quantize(wide(x))
    assert np.array_equal(s.cpu().numpy(), scale)
    assert np.array_equal(q.cpu().numpy(), pack(code))


def test_quantize_specials():
    inf, nan = float("inf"), float("nan")
    x = np.zeros((10, 64))
    x[1, :32] = np.arange(32) - 16
    x[1, 5] = inf
    x[2, 40] = -inf
    x[3, 63] = nan
    x[3, :32] = 1e-30
    x[4] = 2.0**-126
    x[4, 3] = -(2.0**-149)
    x[5] = 2.0**-149 * np.arange(64)  # below the normal numbers: the scale stays 2^-127
    x[6] = 3.4e38 * np.sin(np.arange(64))
    x[7] = -0.0
    x[8, 0] = 1.0
    x[8, 1] = -1e-20  # rounds to zero, sign kept
    x[9] = 2.0**-127 * np.linspace(-1, 7.9, 64)
    t = dev(x, torch.float32)
    q, s = run_quantize(t)
    code, scale = quantize(wide(t))
    assert np.array_equal(s.cpu().numpy(), scale)
    assert scale[1, 0] == 255 and scale[2, 1] == 255 and scale[3, 1] == 255 and scale[0, 0] == 0
    assert np.array_equal(q.cpu().numpy(), pack(code))
    for dtype in TYPES.values():
        out = torch.zeros(10, 64, dtype=dtype, device="cuda")
        w.mxfp4_dequantize(q, s, out)
        torch.cuda.synchronize()
        assert np.array_equal(wide(out), rounded(values(pack(code), scale), dtype), equal_nan=True)
    t = dev(np.array([[nan] + [1.0] * 31, [inf] + [1.0] * 31]), torch.bfloat16)
    q, s = run_quantize(t)
    assert s.cpu().tolist() == [[255], [255]] and not bool(q.any())


def test_dequantize_every_code_and_scale():
    q = np.tile(np.arange(256, dtype=np.uint8)[None], (256, 1))
    s = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, 1)
    for dtype in TYPES.values():
        out = torch.zeros(256, 512, dtype=dtype, device="cuda")
        w.mxfp4_dequantize(dev(q), dev(s), out)
        torch.cuda.synchronize()
        with np.errstate(over="ignore"):
            want = rounded(values(q, s), dtype)
        assert np.array_equal(wide(out), want, equal_nan=True)


@pytest.mark.parametrize("live", [0, 1, 13, 64, 100])
def test_num_rows_limits_all_three(live):
    x = torch.randn(64, 128, device="cuda")
    n = dev(np.array([live], np.int32))
    q, s = run_quantize(x, n)
    code, scale = quantize(wide(x))
    k = min(live, 64)
    assert np.array_equal(q.cpu().numpy()[:k], pack(code)[:k]) and bool((q[k:] == 0x55).all())
    assert np.array_equal(s.cpu().numpy()[:k], scale[:k]) and bool((s[k:] == 0x55).all())
    out = torch.full((64, 128), 7.0, device="cuda")
    w.mxfp4_dequantize(dev(pack(code)), dev(scale), out, num_rows=n)
    hq, hs = torch.full((64, 32), 0x55, dtype=torch.uint8, device="cuda"), torch.full((64, 2), 0x55, dtype=torch.uint8, device="cuda")
    w.mxfp4_silu_mul_quantize(x, hq, hs, num_rows=n)
    torch.cuda.synchronize()
    assert bool((out[k:] == 7).all()) and bool((hq[k:] == 0x55).all()) and bool((hs[k:] == 0x55).all())
    assert np.array_equal(wide(out)[:k], values(pack(code), scale)[:k])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(1, 32), (5, 96), (67, 2048)], ids=str)
def test_silu_mul_quantize(shape, dtype):
    """a = silu(g) u in fp32 is off by a few steps of fp32 (exp, reciprocal and three products: 8 * 2^-24 of a,
    plus exp's argument error 2^-24 |g| where g < 0), so where a lies that near a rounding border (or the
    block's largest that near a power of two) either neighbour is right; everywhere else codes are equal."""
    rows, I = shape
    gen = torch.Generator(device="cuda").manual_seed(2)
    gu = (3 * torch.randn(rows, 2 * I, device="cuda", generator=gen)).to(TYPES[dtype])
    q = torch.zeros(rows, I // 2, dtype=torch.uint8, device="cuda")
    s = torch.zeros(rows, I // 32, dtype=torch.uint8, device="cuda")
    w.mxfp4_silu_mul_quantize(gu, q, s)
    torch.cuda.synchronize()
    g, u = wide(gu)[:, :I], wide(gu)[:, I:]
    a = g / (1 + np.exp(-g)) * u
    rel = (8 + 2 * np.abs(g)) * 2.0**-24
    got_s, got_q = s.cpu().numpy(), q.cpu().numpy()
    low = quantize(a * (1 - rel))
    high = quantize(a * (1 + rel))
    assert np.all((got_s == low[1]) | (got_s == high[1]))
    sure = np.repeat(low[1] == high[1], 32, axis=1) & (low[0] == high[0])
    code = np.stack((got_q & 15, got_q >> 4), -1).reshape(rows, I)
    assert np.all((code == low[0])[sure])
    either = (code == low[0]) | (code == high[0])
    assert np.all(either[np.repeat(low[1] == high[1], 32, axis=1)])
    assert sure.mean() > 0.999


# ------------------------------------------------------------------ the product


class Product:
    """Quantised operands and the alignment of one product."""

    def __init__(self, T, topk, E, G, N, K, bm, gather, seed=0, spread=1, ids=None, counts=None):
        import oracle

        rng = np.random.default_rng(seed)
        self.ids = routing(rng, T, topk, E, G) if ids is None else ids
        self.T, self.topk, self.E, self.N, self.K, self.bm, self.gather = T, topk, E, N, K, bm, gather
        self.srt, self.eid, self.rows, _ = oracle.moe_align(self.ids, E, bm)
        self.capacity = len(self.srt)
        a_rows = T if gather else self.capacity
        draw = lambda *shape: rng.integers(0, 256, shape, dtype=np.uint8)  # noqa: E731
        scales = lambda *shape: rng.integers(127, 127 + spread + 1, shape).astype(np.uint8)  # noqa: E731
        self.a_q, self.a_s = draw(a_rows, K // 2), scales(a_rows, K // 32)
        self.w_q, self.w_s = draw(E, N, K // 2), scales(E, N, K // 32)

    def reference(self):
        """64-bit rows [capacity, N]: real rows' products, zeros for padding; rows past the last block are 7."""
        out = np.full((self.capacity, self.N), 7.0)
        out[: self.rows] = 0
        a, size = values(self.a_q, self.a_s), np.zeros_like(out)
        p = np.arange(self.rows)
        p = p[self.srt[: self.rows] < self.T * self.topk]
        e = self.eid[p // self.bm]
        src = self.srt[p] // self.topk if self.gather else p
        for x in np.unique(e):
            m = e == x
            wt = values(self.w_q[x], self.w_s[x]).T
            out[p[m]] = a[src[m]] @ wt
            size[p[m]] = np.abs(a[src[m]]) @ np.abs(wt)
        return out, size

    def upload(self):
        self.d = {k: dev(getattr(self, k)) for k in ("a_q", "a_s", "w_q", "w_s", "srt", "eid")}
        self.d["ntpp"] = dev(np.array([self.rows], np.int32))
        self.d["packed"] = torch.full((w.mxfp4_packed_bytes(self.E, self.N, self.K),), 0xAA, dtype=torch.uint8, device="cuda")
        w.mxfp4_repack(self.d["w_q"], self.d["w_s"], self.d["packed"])
        return self.d

    def run(self, dtype, out=None):
        d = self.d if hasattr(self, "d") else self.upload()
        out = torch.full((self.capacity, self.N), 7.0, dtype=dtype, device="cuda") if out is None else out
        w.mxfp4_moe_gemm(d["a_q"], d["a_s"], self.T, self.topk, d["srt"], d["eid"], d["ntpp"], self.bm, self.E,
                         d["packed"], out, gather=self.gather)
        torch.cuda.synchronize()
        return out


# T, topk, resident experts, routed experts, N, K
GEMMS = [
    (1, 1, 1, 1, 16, 32),
    (1, 8, 48, 384, 64, 128),
    (1, 8, 16, 16, 4096, 512),
    (3, 2, 4, 4, 80, 96),
    (17, 1, 1, 1, 256, 160),
    (40, 2, 3, 4, 144, 288),
    (64, 8, 8, 8, 512, 1024),
    (130, 4, 5, 10, 272, 416),
    (300, 2, 2, 2, 528, 544),
    (700, 2, 4, 4, 1024, 512),
    (1100, 1, 1, 1, 768, 2048),
    (90, 6, 40, 64, 320, 7168),
    # enough tiles of 256 columns for the tile kernel at block_m 64 and 128: K of one step, of odd
    # and even numbers of steps, of whole groups of four; weights read by one row block and by several
    (130, 8, 48, 96, 512, 128),
    (900, 2, 6, 6, 1040, 384),
    (640, 4, 20, 20, 272, 640),
    (2100, 1, 1, 1, 1024, 7168),
    (2000, 2, 4, 4, 1040, 96),  # as many, and K ends inside a step
]


@pytest.mark.parametrize("bm", [16, 32, 64, 128])
@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("shape", GEMMS, ids=str)
def test_gemm_is_exact(shape, gather, bm):
    """Scales of two neighbouring powers of two on each side: a product is a multiple of 1/4 of at most 144,
    and 7168 of them stay below 2^24 quarters, so every partial sum is exact in fp32."""
    T, topk, E, G, N, K = shape
    say("gemm", shape, gather, bm)
    c = Product(T, topk, E, G, N, K, bm, gather, seed=3)
    ref, _ = c.reference()
    for dtype in TYPES.values():
        if dtype == torch.float16 and K > 2048:
            continue  # may pass fp16's largest value
        got = wide(c.run(dtype))
        assert np.array_equal(got, rounded(ref, dtype)), (dtype, np.argwhere(got != rounded(ref, dtype))[:5])


@pytest.mark.parametrize("shape", [(150, 2, 4, 4, 208, 672), (1000, 2, 4, 4, 1024, 1152)], ids=str)
@pytest.mark.parametrize("bm", [16, 32, 64, 128])
def test_gemm_wide_scales(shape, bm):
    """Scales over 40 powers of two: each of the K additions is off by at most one fp32 step of the terms' size."""
    c = Product(*shape, bm, True, seed=5, spread=40)
    ref, size = c.reference()
    got = wide(c.run(torch.float32))
    assert np.all(np.abs(got - ref) <= c.K * 2.0**-23 * size)


@pytest.mark.parametrize("shape", [(40, 2, 3, 3, 96, 320), (900, 2, 3, 3, 1024, 640), (900, 2, 3, 3, 1024, 512)], ids=str)
@pytest.mark.parametrize("bm", [16, 64, 128])
def test_gemm_scale_of_nan(shape, bm):
    """A scale byte of 255 makes NaN of exactly the outputs it enters: of a row, and of a column."""
    c = Product(*shape, bm, True, seed=6)
    c.a_s[7, 3] = 255
    c.a_s[9, -1] = 255
    c.w_s[1, 17, 9] = 255
    c.w_s[2, 95, -1] = 255
    ref, _ = c.reference()
    got = wide(c.run(torch.float32))
    assert np.isnan(ref).any() and np.array_equal(got, ref, equal_nan=True)


@pytest.mark.parametrize("bm", [16, 128])
def test_gemm_small_and_large_scales(bm):
    """Products whose scales multiply to both ends of fp32's normal range are exact."""
    for a_scale, w_scale in [(127 - 90, 127 - 30), (127 + 80, 127 + 30), (1, 127 + 100), (254, 20)]:
        c = Product(20, 1, 2, 2, 64, 128, bm, False, seed=7)
        c.a_s[:] = a_scale
        c.w_s[:] = w_scale
        ref, _ = c.reference()
        assert np.array_equal(wide(c.run(torch.float32)), rounded(ref, torch.float32)), (a_scale, w_scale)


def test_gemm_one_expert_is_a_plain_product():
    """One expert and one slot per token: a linear layer, quantised on the way."""
    x = torch.randn(200, 256, device="cuda").bfloat16()
    q, s = run_quantize(x)
    c = Product(200, 1, 1, 1, 320, 256, 128, True, seed=8)
    c.upload()
    c.d["a_q"], c.d["a_s"] = q, s
    code, scale = quantize(wide(x))
    c.a_q, c.a_s = pack(code), scale
    ref, size = c.reference()
    got = wide(c.run(torch.float32))
    assert np.all(np.abs(got - ref) <= c.K * 2.0**-23 * size)


@pytest.mark.parametrize("T, N, bm", [(60, 64, 16), (900, 1024, 64), (900, 1024, 128)])
def test_gemm_unknown_blocks_and_rows(T, N, bm):
    """Blocks whose expert id is outside the resident ones, and slots past T * topk, give zero rows."""
    c = Product(T, 2, 4, 4, N, 128, bm, True, seed=9)
    c.eid[1] = -1
    c.eid[2] = 4
    c.srt[3] = T * 2 + 5
    c.srt[3 * bm + 2] = -1
    got = wide(c.run(torch.float32))
    a, wt = values(c.a_q, c.a_s), [values(c.w_q[e], c.w_s[e]).T for e in range(4)]
    for p in range(c.rows):
        s, e = c.srt[p], c.eid[p // bm]
        ok = 0 <= s < 2 * T and 0 <= e < 4
        want = a[s // 2] @ wt[e] if ok else np.zeros(N)
        assert np.array_equal(got[p], want), p
    assert np.all(got[c.rows :] == 7)


@pytest.mark.parametrize("shape", [(300, 4, 8, 8, 448, 1056), (900, 2, 6, 6, 1040, 640)], ids=str)
@pytest.mark.parametrize("bm", [16, 32, 64, 128])
def test_gemm_runs_agree(shape, bm):
    c = Product(*shape, bm, True, seed=10, spread=30)
    first = c.run(torch.float32)
    for _ in range(5):
        assert torch.equal(c.run(torch.float32), first)


def test_expert_layer_in_four_bits():
    """Routing to output as a program runs it, captured in a graph and replayed: logits -> alignment, token
    rows to 4 bits, gate_up, SiLU-and-mul to 4 bits, down in fp32, and the weighted sum per token. Each stage
    is checked on the very operands it was given."""
    T, topk, E, H, I, bm = 90, 4, 8, 512, 192, 32
    rng = np.random.default_rng(11)
    w13 = Product(T, topk, E, E, 2 * I, H, bm, True, seed=12)
    w2 = Product(T, topk, E, E, H, I, bm, False, seed=13)
    p13, p2 = w13.upload()["packed"], w2.upload()["packed"]
    logits = dev(rng.standard_normal((T, E)).astype(np.float32))
    x = torch.randn(T, H, device="cuda").bfloat16()
    buf = w.align_buffers(T, topk, E, bm)
    srt, eid, ntpp = buf["sorted_token_ids"], buf["expert_ids"], buf["num_tokens_post_padded"]
    cap = srt.numel()
    ids = torch.zeros(T, topk, dtype=torch.int32, device="cuda")
    wts = torch.zeros(T, topk, device="cuda")
    byte = lambda *shape: torch.zeros(*shape, dtype=torch.uint8, device="cuda")  # noqa: E731
    xq, xs, hq, hs = byte(T, H // 2), byte(T, H // 32), byte(cap, I // 2), byte(cap, I // 32)
    gu = torch.zeros(cap, 2 * I, device="cuda")
    y = torch.zeros(cap, H, device="cuda")
    xp = torch.zeros(cap, H, dtype=torch.bfloat16, device="cuda")
    rows = torch.zeros(T, topk, dtype=torch.int32, device="cuda")
    out = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")

    def step():
        w.moe_route_align(logits, topk, E, bm, ids, wts, srt, eid, ntpp, workspace=buf["workspace"])
        w.moe_permute(x, srt, ntpp, topk, xp, rows)
        w.mxfp4_quantize(x, xq, xs)
        w.mxfp4_moe_gemm(xq, xs, T, topk, srt, eid, ntpp, bm, E, p13, gu, gather=True)
        w.mxfp4_silu_mul_quantize(gu, hq, hs, num_rows=ntpp)
        w.mxfp4_moe_gemm(hq, hs, T, topk, srt, eid, ntpp, bm, E, p2, y)
        w.moe_unpermute(y, rows, out, topk_weights=wts)

    step()
    torch.cuda.synchronize()
    M = int(ntpp.item())
    srt_h, eid_h = srt.cpu().numpy(), eid.cpu().numpy()
    p = np.nonzero(srt_h[:M] < T * topk)[0]
    e = eid_h[p // bm]
    a = values(xq.cpu().numpy(), xs.cpu().numpy())
    h = values(hq.cpu().numpy(), hs.cpu().numpy())
    assert np.array_equal(wide(xp)[p], wide(x)[srt_h[p] // topk])
    for ex in range(E):
        m = e == ex
        w1, w2v = values(w13.w_q[ex], w13.w_s[ex]).T, values(w2.w_q[ex], w2.w_s[ex]).T
        rows_in = a[srt_h[p[m]] // topk]
        assert np.all(np.abs(wide(gu)[p[m]] - rows_in @ w1) <= H * 2.0**-23 * (np.abs(rows_in) @ np.abs(w1)))
        assert np.all(np.abs(wide(y)[p[m]] - h[p[m]] @ w2v) <= I * 2.0**-23 * (np.abs(h[p[m]]) @ np.abs(w2v)))
    y64, r = wide(y), rows.cpu().numpy()
    terms = wide(wts)[..., None] * y64[r]
    off = 2 * topk * 2.0**-24 * np.abs(terms).sum(1)
    ref = terms.sum(1)
    half = half_step(torch.bfloat16)
    assert np.all(np.abs(wide(out) - ref) <= off + half * (np.abs(ref) + off) + floor_of(torch.bfloat16))

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
        logits.copy_(torch.randn(T, E, device="cuda"))
        step()
        torch.cuda.synchronize()
        want, M = out.clone(), int(ntpp.item())
        want_y = y[:M].clone()
        out.zero_(), y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(y[:M], want_y), k


def test_offsets_past_32_bits():
    """More than 2^32 values quantised and back, and a product whose rows are more than 4 GiB of codes: the
    last rows against the same rows alone."""
    say("far offsets")
    rows, K = 600064, 7168
    x = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda").normal_()
    assert rows * K > 2**32
    q, s = torch.zeros(rows, K // 2, dtype=torch.uint8, device="cuda"), torch.zeros(rows, K // 32, dtype=torch.uint8, device="cuda")
    w.mxfp4_quantize(x, q, s)
    tail = x[-96:].clone()
    tq, ts = run_quantize(tail)
    assert torch.equal(q[-96:], tq) and torch.equal(s[-96:], ts)
    w.mxfp4_dequantize(q, s, x)
    back = torch.zeros_like(tail)
    w.mxfp4_dequantize(tq, ts, back)
    assert torch.equal(x[-96:], back)
    h = torch.zeros(rows, K // 4, dtype=torch.uint8, device="cuda")
    hs = torch.zeros(rows, K // 64, dtype=torch.uint8, device="cuda")
    w.mxfp4_silu_mul_quantize(x, h, hs)
    th, ths = torch.zeros(96, K // 4, dtype=torch.uint8, device="cuda"), torch.zeros(96, K // 64, dtype=torch.uint8, device="cuda")
    w.mxfp4_silu_mul_quantize(back, th, ths)
    assert torch.equal(h[-96:], th) and torch.equal(hs[-96:], ths)
    del x, h, hs
    # as a product's rows: twice as many, so that the codes pass 4 GiB
    q, s = torch.cat([q, q]), torch.cat([s, s])
    T = 2 * rows
    assert T * K // 2 > 2**32
    N, bm = 64, 128
    c = Product(96, 1, 1, 1, N, K, bm, True, seed=14)
    d = c.upload()
    c.a_q, c.a_s = tq.cpu().numpy(), ts.cpu().numpy()
    ref, size = c.reference()  # one expert, one slot a token: aligned row p is token p
    srt = torch.arange(T + bm - 1, dtype=torch.int32, device="cuda").clamp(max=T)
    eid = torch.zeros((T + bm - 1) // bm, dtype=torch.int32, device="cuda")
    ntpp = dev(np.array([T], np.int32))
    for gather in (True, False):
        out = torch.full((T + bm - 1, N), 7.0, device="cuda")
        a_q, a_s = (q, s) if gather else (torch.cat([q, q[: bm - 1]]), torch.cat([s, s[: bm - 1]]))
        w.mxfp4_moe_gemm(a_q, a_s, T, 1, srt, eid, ntpp, bm, 1, d["packed"], out, gather=gather)
        torch.cuda.synchronize()
        assert np.all(np.abs(wide(out[T - 96 : T]) - ref[:96]) <= K * 2.0**-23 * size[:96])
        assert torch.equal(out[rows - 96 : rows], out[T - 96 : T]) and bool((out[T:] == 7).all())
        del a_q, a_s


@pytest.mark.parametrize("dtype", TYPES)
def test_silu_mul_quantize_at_the_ends(dtype):
    """Blocks of one g each, from the flush below exp(g) = 2^-126 to infinities and NaN, against rows of u over the
    type's range. Tolerance of what stays finite: as in test_silu_mul_quantize; g of -87 is 126 halvings, an argument
    of exp2 rounded by 2^-18 and a constant by 2^-25 of it, together within 2 * 87 * 2^-24 of the result."""
    t = TYPES[dtype]
    inf, nan = float("inf"), float("nan")
    gs = torch.tensor([-inf, -1000, -100, -88, -87.5, -87, -50, -1, -0.0, 0, 1, 50, 87, 88, 100, 1000, inf, nan]).to(t)
    gen = torch.Generator().manual_seed(15)
    top = 14 if dtype == "fp16" else 120
    us = [torch.randn(32, generator=gen) * 2.0**e for e in (0, top, -top, 5, -5)]
    us += [torch.where(torch.arange(32) == 7, torch.tensor(v), torch.randn(32, generator=gen)) for v in (inf, -inf, nan)]
    us = torch.stack(us).to(t)  # one row of the operator each
    rows, I = len(us), 32 * len(gs)
    gu = torch.cat([gs.repeat_interleave(32).expand(rows, I), us.repeat(1, len(gs))], 1).contiguous().cuda()
    q = torch.full((rows, I // 2), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((rows, I // 32), 0x55, dtype=torch.uint8, device="cuda")
    w.mxfp4_silu_mul_quantize(gu, q, s)
    torch.cuda.synchronize()
    g, u = wide(gu)[:, :I], wide(gu)[:, I:]
    with np.errstate(over="ignore", invalid="ignore"):
        flushed = np.exp(g) < 2.0**-126
        a = np.where(flushed & np.isfinite(g), 0 * u, g / (1 + np.exp(-g)) * u)
        a = np.where(np.abs(a) > 3.4028235e38, np.inf * a, a)  # none lies near fp32's largest value
    blocks = a.reshape(rows, -1, 32)
    assert not np.any(np.isfinite(blocks) & (np.abs(blocks) > 3.3e38))
    finite = np.isfinite(blocks).all(-1)
    got_s, got_q = s.cpu().numpy(), q.cpu().numpy()
    code = np.stack((got_q & 15, got_q >> 4), -1).reshape(rows, I)
    assert np.array_equal(got_s == 255, ~finite)
    assert not finite[:, [0, -1, -2]].any() and finite[0, 1:-2].all() and not finite[5:].any()
    assert not code.reshape(rows, -1, 32)[~finite].any()
    zero = (np.abs(blocks) == 0).all(-1)
    assert not got_s[zero].any() and not (code.reshape(rows, -1, 32)[zero] & 7).any()
    rel = (8 + 2 * np.where(np.isfinite(g), np.abs(g), 0)) * 2.0**-24
    kept = np.where(np.repeat(finite, 32, axis=1), a, 0)
    low, high = quantize(kept * (1 - rel)), quantize(kept * (1 + rel))
    live = finite & ~zero
    assert np.all(((got_s == low[1]) | (got_s == high[1]))[live])
    same = np.repeat(live & (low[1] == high[1]), 32, axis=1)
    assert np.all(((code == low[0]) | (code == high[0]))[same])


@pytest.mark.parametrize("bm", [16, 32, 64, 128])
@pytest.mark.parametrize("shape", [(90, 6, 40, 64, 320, 7168), (2100, 1, 1, 1, 1024, 7168)], ids=str)
def test_gemm_long_rows_in_fp16(shape, bm):
    """As test_gemm_is_exact, with rows 2^6 smaller: 7168 products of at most 144 / 64 stay below fp16's largest value."""
    c = Product(*shape, bm, True, seed=16)
    c.a_s -= 6
    ref, _ = c.reference()
    assert np.array_equal(wide(c.run(torch.float16)), rounded(ref, torch.float16))


@pytest.mark.parametrize("bm", [16, 64, 128])
def test_gemm_smallest_scales(bm):
    """The scale byte 0 is 2^-127. Products below 2^-126 may count as zero, each and each partial sum then off by that."""
    for a_scale, w_scale in [(0, 227), (227, 0), (0, 0), (37, 90), (0, 120)]:
        c = Product(900, 1, 2, 2, 1024, 128, bm, False, seed=17)
        c.a_s[:], c.w_s[:] = a_scale, w_scale
        ref, _ = c.reference()
        got = wide(c.run(torch.float32))
        if a_scale + w_scale == 227:
            assert np.array_equal(got, rounded(ref, torch.float32)), (a_scale, w_scale)
        assert np.all(np.abs(got - ref) <= 2 * c.K * 2.0**-126), (a_scale, w_scale)


@pytest.mark.parametrize("bm", [16, 32, 64, 128])
@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("shape", [(64, 8, 8, 8, 512, 1024), (900, 2, 6, 6, 1040, 384), (2100, 1, 1, 1, 1024, 512)], ids=str)
def test_gemm_scales_at_any_byte(shape, gather, bm):
    """Row scales that start one byte into their buffer, with K of whole steps."""
    c = Product(*shape, bm, gather, seed=18)
    ref, _ = c.reference()
    d = c.upload()
    d["a_s"] = torch.cat([d["a_s"].flatten()[:1], d["a_s"].flatten()])[1:].view(c.a_s.shape)
    assert d["a_s"].data_ptr() % 4 == 1
    assert np.array_equal(wide(c.run(torch.float32)), ref)


@pytest.mark.parametrize("bm", [64, 128])
def test_tile_kernel_offsets_past_31_bits(bm):
    """Just under 4 GiB of row codes, the most that the tile kernel's 32-bit offsets take: the rows on both sides of
    2 GiB, the last ones, and the slot order turned round, exactly."""
    say("tile kernel, far offsets", bm)
    T, N, K = 1198200, 64, 7168
    rows = T + bm - 1
    assert 2**32 - 2**20 < rows * (K // 2) < 2**32
    gen = torch.Generator(device="cuda").manual_seed(19)
    a_q = torch.randint(0, 256, (rows, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    a_s = torch.randint(127, 129, (rows, K // 32), dtype=torch.uint8, device="cuda", generator=gen)
    c = Product(96, 1, 1, 1, N, K, bm, True, seed=20)
    packed, wt = c.upload()["packed"], values(c.w_q[0], c.w_s[0]).T
    srt = torch.arange(rows, dtype=torch.int32, device="cuda").clamp(max=T)
    turned = torch.where(srt < T, T - 1 - srt, srt)
    eid = torch.zeros((rows + bm - 1) // bm, dtype=torch.int32, device="cuda")
    used = (T + bm - 1) // bm * bm
    ntpp = dev(np.array([used], np.int32))
    half = 2**31 // (K // 2)
    at = torch.tensor([0, 1, half - 1, half, half + 1, T // 2, T - 65, T - 2, T - 1], device="cuda")
    ref = values(a_q[at].cpu().numpy(), a_s[at].cpu().numpy()) @ wt
    for gather, order in ((True, srt), (False, srt), (True, turned)):
        out = torch.full((rows, N), 7.0, device="cuda")
        w.mxfp4_moe_gemm(a_q, a_s, T, 1, order, eid, ntpp, bm, 1, packed, out, gather=gather)
        torch.cuda.synchronize()
        where = at if order is srt else T - 1 - at
        assert np.array_equal(wide(out[where]), ref)
        assert not bool(out[T:used].any()) and bool((out[used:] == 7).all())


def test_the_stream_that_is_given():
    """Each operator on a stream given by argument, behind work there that makes its inputs, while another stream is
    current; a stream of another GPU is refused."""
    from types import SimpleNamespace

    c = Product(130, 4, 5, 10, 272, 416, 32, True, seed=21)
    d = c.upload()
    x0, x1 = (torch.randn(c.T, 2 * c.K, device="cuda").bfloat16() for _ in range(2))
    x = x0.clone()
    byte = lambda *shape: torch.zeros(*shape, dtype=torch.uint8, device="cuda")  # noqa: E731
    q, s, hq, hs = byte(c.T, c.K), byte(c.T, c.K // 16), byte(c.T, c.K // 2), byte(c.T, c.K // 32)
    back, out = torch.zeros_like(x), torch.zeros(c.capacity, c.N, device="cuda")
    packed = torch.zeros_like(d["packed"])
    w_q = torch.zeros_like(d["w_q"])

    def step(stream=None):
        w.mxfp4_quantize(x, q, s, stream=stream)
        w.mxfp4_dequantize(q, s, back, stream=stream)
        w.mxfp4_silu_mul_quantize(back, hq, hs, stream=stream)
        w.mxfp4_repack(w_q, d["w_s"], packed, stream=stream)
        w.mxfp4_moe_gemm(hq, hs, c.T, c.topk, d["srt"], d["eid"], d["ntpp"], c.bm, c.E, packed, out, gather=True,
                         stream=stream)

    x.copy_(x1), w_q.copy_(d["w_q"])
    step()
    torch.cuda.synchronize()
    outputs = (q, s, back, hq, hs, packed, out)
    want = [t.clone() for t in outputs]
    x.copy_(x0), w_q.zero_()
    for t in outputs:
        t.zero_()
    big = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(20):
            big = (big @ big).clamp(-1, 1)
        x.copy_(x1), w_q.copy_(d["w_q"])
    step(side)
    side.synchronize()
    for a, b in zip(want, outputs):
        assert torch.equal(a, b)
    other = SimpleNamespace(device_index=torch.cuda.current_device() + 1, cuda_stream=0)
    with pytest.raises(w.W4A16Error) as e:
        w.mxfp4_quantize(x, q, s, stream=other)
    assert e.value.status == w.INVALID_ARG


@pytest.mark.parametrize("T, N, bm", [(60, 64, 16), (900, 1024, 64), (900, 1024, 128)])
def test_gemm_shorter_sorted_list(T, N, bm):
    """A list that ends inside a block: the whole blocks before its end are computed, nothing behind them is written."""
    c = Product(T, 2, 4, 4, N, 128, bm, True, seed=22)
    ref, _ = c.reference()
    d = c.upload()
    assert c.rows >= 4 * bm
    cap = c.rows - bm - bm // 2
    out = torch.full((c.capacity, N), 7.0, device="cuda")
    w.mxfp4_moe_gemm(d["a_q"], d["a_s"], T, 2, d["srt"][:cap], d["eid"], d["ntpp"], bm, 4, d["packed"], out[:cap],
                     gather=True)
    torch.cuda.synchronize()
    whole = cap // bm * bm
    assert np.array_equal(wide(out)[:whole], ref[:whole]) and bool((out[whole:] == 7).all())
