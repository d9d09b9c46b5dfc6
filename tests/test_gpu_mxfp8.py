"""8-bit checkpoints and the activation that keeps and reads them, against plain 64-bit torch.

Quantisation is exact by definition, so codes and scales are compared bit for bit."""
import pytest
import torch

import w4a16_grouped_gemm_amd as w
from _grouped import TYPES, half_step, levels, quantize8, silu_and_gradient, values8
from _gpu import say

pytestmark = pytest.mark.gpu


def run_quantize(x, num_rows=None):
    q = torch.full(x.shape, 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((x.shape[0], x.shape[1] // 32), 0x55, dtype=torch.uint8, device="cuda")
    w.mxfp8_quantize(x, q, s, num_rows=num_rows)
    torch.cuda.synchronize()
    return q, s


def run_dequantize(q, s, dtype, num_rows=None):
    out = torch.full(q.shape, 77.0, dtype=dtype, device="cuda")
    w.mxfp8_dequantize(q, s, out, num_rows=num_rows)
    torch.cuda.synchronize()
    return out


def same(a, b):
    return torch.equal(a.nan_to_num(nan=-7.25, posinf=1e300, neginf=-1e300), b.nan_to_num(nan=-7.25, posinf=1e300, neginf=-1e300))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(1, 32), (3, 64), (1, 7168), (129, 96), (1000, 1056), (17, 20000)], ids=str)
def test_quantize_is_exact(shape, dtype):
    say("quantize", shape, dtype)
    g = torch.Generator().manual_seed(1)
    size = torch.exp2(torch.randint(-6, 7, (shape[0], shape[1] // 32), generator=g).float()).repeat_interleave(32, 1)
    x = (torch.randn(*shape, generator=g) * size).to(TYPES[dtype])
    q, s = run_quantize(x.cuda())
    code, scale = quantize8(x)
    assert torch.equal(s.cpu(), scale) and torch.equal(q.cpu(), code)
    got = run_dequantize(q, s, TYPES[dtype])
    assert same(got.cpu().double(), values8(code, scale).to(TYPES[dtype]).double())


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_every_border(dtype):
    """Every code's value, every halfway point and the type's neighbours of both, in both signs, in blocks whose largest
    value is a power of two, 448 times one, and the type's next value above that."""
    t = TYPES[dtype]
    lv = levels()
    points = torch.cat((lv, (lv[1:] + lv[:-1]) / 2))
    for e in {"bf16": (-140, -100, 0, 110), "fp16": (-20, -6, 0, 6), "fp32": (-149, -120, 0, 110)}[dtype]:
        for most in (256.0, 448.0, 449.0, 511.0):
            p = (points * 2.0**e).to(t)
            bits = torch.int32 if t == torch.float32 else torch.int16
            near = torch.cat((p, (p.view(bits) + 1).view(t), (p.view(bits) - 1).view(t)))
            near = torch.where(torch.isfinite(near), near, 0).to(t)
            near = near[near.double().abs() <= 448 * 2.0**e]
            near = torch.cat((near, -near))
            near = torch.cat((near, torch.zeros((-near.numel()) % 31, dtype=t))).view(-1, 31)
            x = torch.cat((near, torch.full((near.shape[0], 1), most * 2.0**e, dtype=torch.float64).to(t)), dim=1)
            q, s = run_quantize(x.cuda())
            code, scale = quantize8(x)
            assert torch.equal(s.cpu(), scale), (e, most)
            assert torch.equal(q.cpu(), code), (e, most)


def test_quantize_specials():
    inf, nan = float("inf"), float("nan")
    x = torch.zeros(9, 64, dtype=torch.float64)
    x[1, :32] = torch.arange(32) - 16
    x[1, 5] = inf
    x[2, 40] = -inf
    x[3, 63] = nan
    x[3, :32] = 1e-30
    x[4] = 2.0**-126
    x[4, 3] = -(2.0**-149)
    x[5] = 2.0**-149 * torch.arange(64)  # below the normal numbers: the scale stays 2^-127
    x[6] = 3.4e38 * torch.sin(torch.arange(64).double())
    x[7] = -0.0
    x[8, 0], x[8, 1] = 1.0, -1e-20  # rounds to zero, sign kept
    x = x.float()
    q, s = run_quantize(x.cuda())
    code, scale = quantize8(x)
    assert torch.equal(s.cpu(), scale) and torch.equal(q.cpu(), code)
    assert scale[1, 0] == 255 and scale[2, 1] == 255 and scale[3, 1] == 255 and scale[0, 0] == 0
    for t in TYPES.values():
        assert same(run_dequantize(q, s, t).cpu().double(), values8(code, scale).to(t).double())
    x = torch.tensor([[nan] + [1.0] * 31, [inf] + [1.0] * 31]).bfloat16().cuda()
    q, s = run_quantize(x)
    assert s.cpu().tolist() == [[255], [255]] and not bool(q.any())


@pytest.mark.parametrize("dtype", TYPES)
def test_dequantize_every_code_and_scale(dtype):
    q = torch.arange(256, dtype=torch.uint8).repeat(256, 1)
    s = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 8)
    got = run_dequantize(q.cuda(), s.cuda(), TYPES[dtype]).cpu().double()
    assert same(got, values8(q, s).to(TYPES[dtype]).double())


def test_rows_behind_the_count_stay():
    x = torch.randn(70, 96).cuda()
    for n, live in [(0, 0), (-3, 0), (41, 41), (70, 70), (1000, 70)]:
        count = torch.tensor([n], dtype=torch.int32, device="cuda")
        q, s = run_quantize(x, num_rows=count)
        code, scale = quantize8(x.cpu())
        assert torch.equal(q[:live].cpu(), code[:live]) and torch.equal(s[:live].cpu(), scale[:live])
        assert bool((q[live:] == 0x55).all()) and bool((s[live:] == 0x55).all())
        out = run_dequantize(code.cuda(), scale.cuda(), torch.float32, num_rows=count)
        assert bool((out[live:] == 77).all()) and same(out[:live].cpu().double(), values8(code, scale)[:live])
        h, q, s, dgu, again = run_silu(torch.cat((x, x), 1)[:, :128].contiguous(), x[:, :64].contiguous(), num_rows=count)
        for t in (h, dgu, again):
            assert bool((t[live:] == 77).all()) and not bool((t[:live] == 77).any())
        assert bool((q[live:] == 0x55).all()) and bool((s[live:] == 0x55).all())


def run_silu(gu, dh, num_rows=None, keep=True):
    rows, I = dh.shape
    h, again = (torch.full_like(dh, 77.0) for _ in range(2))
    dgu = torch.full_like(gu, 77.0)
    q = torch.full(gu.shape, 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((rows, I // 16), 0x55, dtype=torch.uint8, device="cuda")
    w.mxfp8_silu_mul(gu, h, q, s, num_rows=num_rows)
    w.mxfp8_silu_mul_backward(q, s, dh, dgu, h=again if keep else None, num_rows=num_rows)
    torch.cuda.synchronize()
    return h, q, s, dgu, again


def close(got, ref, parts, far, what):
    """One rounding to the type, and fp32 arithmetic: `parts` bounds the magnitudes that are added up, each good to 16
    roundings of 2^-24 (a dozen operations, of which the exponential's and the reciprocal's few units). `far`: by
    definition exp(-|gate|) below 2^-126 counts as zero; the result is that exponential over 1 + itself, times factors
    of at most `far` in all, so leaving it out changes the result by less than 2^-126 far."""
    dtype = got.dtype
    err = (got.cpu().double() - ref).abs()
    fp32 = 16 * 2.0**-24 * parts
    tiny = {torch.float16: 2.0**-25, torch.bfloat16: 2.0**-134, torch.float32: 0.0}[dtype] + 2.0**-126 * (1 + far)
    tol = fp32 + (half_step(dtype) * (ref.abs() + fp32) if dtype != torch.float32 else 0) + tiny
    bad = ~(err <= tol)
    say(f"  {what}: max err/tol {float((err / tol).max()):.4f}")
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} off, e.g. {torch.nonzero(bad)[:4].tolist()}"


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(1, 32), (5, 96), (33, 2048), (300, 416), (2, 8192)], ids=str)
def test_silu_and_its_gradient(shape, dtype):
    g = torch.Generator().manual_seed(2)
    rows, I = shape
    t = TYPES[dtype]
    gu = (torch.randn(rows, 2 * I, generator=g) * torch.exp2(2 * torch.randn(2 * I, generator=g))).clamp(-200, 200).to(t)
    dh = torch.randn(rows, I, generator=g).to(t)
    h, q, s, dgu, again = run_silu(gu.cuda(), dh.cuda())
    code, scale = quantize8(gu)
    assert torch.equal(q.cpu(), code) and torch.equal(s.cpu(), scale)
    wide = gu.double()
    ref = silu_and_gradient(wide[:, :I], wide[:, I:], dh.double())[0]
    close(h, ref, ref.abs(), (wide[:, :I] * wide[:, I:]).abs(), "h")
    kept = values8(code, scale)
    gate, up, grad = kept[:, :I], kept[:, I:], dh.double()
    ref_h, ref_dg, ref_du = silu_and_gradient(gate, up, grad)
    close(again, ref_h, ref_h.abs(), (gate * up).abs(), "h again")
    # the slope is a sum of two terms that may cancel
    y = torch.sigmoid(gate)
    parts = (grad * up).abs() * (y + (gate * y * torch.sigmoid(-gate)).abs())
    close(dgu[:, :I], ref_dg, parts, (grad * up).abs() * (1 + gate.abs()), "dgate")
    close(dgu[:, I:], ref_du, ref_du.abs(), (grad * gate).abs(), "dup")
    without = run_silu(gu.cuda(), dh.cuda(), keep=False)
    assert torch.equal(without[3], dgu) and bool((without[4] == 77).all())


def test_silu_far_gates():
    """Gates out to where exp leaves fp32's numbers, and past it."""
    gate = torch.cat((torch.linspace(-120, 120, 961), torch.tensor([-1e30, 1e30, 0.0, -0.0, 1e-30, -1e-30, 88.7, -88.8, -87.3])))
    gate = torch.cat((gate, torch.zeros((-gate.numel()) % 32)))
    gu = torch.cat((gate, torch.full_like(gate, 3.0)))[None]
    dh = torch.ones(1, gate.numel())
    h, q, s, dgu, again = run_silu(gu.cuda(), dh.cuda())
    ref = silu_and_gradient(gate.double(), gu[:, gate.numel() :].double(), dh.double())[0]
    # fp32's smallest normal number stands for exp's, times gate and up
    err = (h.cpu().double() - ref).abs()
    assert bool((err <= 16 * 2.0**-24 * ref.abs() + 2.0**-126 * 400).all())
    kept = values8(q.cpu(), s.cpu())
    n = gate.numel()
    _, dg, du = silu_and_gradient(kept[:, :n], kept[:, n:], dh.double())
    y = torch.sigmoid(kept[:, :n])
    parts = 3.0 * (y + (kept[:, :n] * y * torch.sigmoid(-kept[:, :n])).abs())
    assert bool(((dgu[:, :n].cpu().double() - dg).abs() <= 16 * 2.0**-24 * parts + 2.0**-126 * 400).all())
    assert bool(((dgu[:, n:].cpu().double() - du).abs() <= 16 * 2.0**-24 * du.abs() + 2.0**-126 * 400).all())


def test_silu_not_finite():
    """An infinity or a NaN marks its block in the checkpoint; h follows the values as given."""
    inf, nan = float("inf"), float("nan")
    I = 64
    gu = torch.ones(4, 2 * I)
    gu[0, 3], gu[1, 40], gu[2, I + 5], gu[3, 9] = inf, nan, -inf, -inf
    dh = torch.ones(4, I)
    h, q, s, dgu, again = (t.cpu() for t in run_silu(gu.cuda(), dh.cuda()))
    assert h[0, 3] == inf and h[1, 40].isnan() and h[2, 5] == -inf and h[3, 9].isnan()
    assert int((~torch.isfinite(h)).sum()) == 4
    assert s.tolist() == [[255 if (r, b) in ((0, 0), (1, 1), (2, 2), (3, 0)) else s[0, 1].item() for b in range(4)]
                          for r in range(4)]
    for r, block in [(0, 0), (1, 1), (2, 0), (3, 0)]:  # a marked block of gate or up reaches its 32 columns
        for t in (dgu[:, :I], again):
            marked = torch.zeros(I, dtype=torch.bool)
            marked[32 * block : 32 * block + 32] = True
            assert torch.equal(t[r].isnan(), marked)


def test_gradient_against_differences():
    """fp32, values that 8 bits hold exactly, so that the checkpoint is the input: central differences in 64 bits of the
    formula, and the returned gradient at those points."""
    g = torch.Generator().manual_seed(3)
    rows, I = 4, 64
    gu = torch.randint(-15, 16, (rows, 2 * I), generator=g).double() / 4
    dh = torch.randn(rows, I, generator=g)
    h, q, s, dgu, again = run_silu(gu.float().cuda(), dh.cuda())
    assert torch.equal(values8(q.cpu(), s.cpu()), gu) and torch.equal(h, again)
    f = lambda x: (torch.nn.functional.silu(x[:, :I]) * x[:, I:] * dh.double()).sum()  # noqa: E731
    step = 2.0**-12
    for r, c in [(0, 0), (1, 7), (3, 63), (2, 64), (0, 127), (3, 100)]:
        up, down = gu.clone(), gu.clone()
        up[r, c] += step
        down[r, c] -= step
        slope = float((f(up) - f(down)) / (2 * step))
        # the third derivative of silu is below 1, of gate below 4: step^2 / 6 * |up dh|
        tol = step**2 * 4 * float(dh[r, c % I].abs()) + 1e-6 * (1 + abs(slope))
        assert abs(float(dgu[r, c]) - slope) <= tol


def test_streams_and_replays():
    x, dh = torch.randn(200, 512).bfloat16().cuda(), torch.randn(200, 256).bfloat16().cuda()
    ref = run_silu(x, dh)
    stream = torch.cuda.Stream()
    q, s = torch.empty_like(ref[1]), torch.empty_like(ref[2])
    h, dgu, again, back = torch.empty_like(dh), torch.empty_like(x), torch.empty_like(dh), torch.empty_like(x)
    torch.cuda.synchronize()
    w.mxfp8_silu_mul(x, h, q, s, stream=stream)
    w.mxfp8_silu_mul_backward(q, s, dh, dgu, h=again, stream=stream)
    w.mxfp8_dequantize(q, s, back, stream=stream)
    stream.synchronize()
    for a, b in zip((h, q, s, dgu, again), ref):
        assert torch.equal(a, b)
    assert torch.equal(run_quantize(x)[0], q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w.mxfp8_silu_mul(x, h, q, s)
        w.mxfp8_silu_mul_backward(q, s, dh, dgu, h=again)
        w.mxfp8_quantize(dgu, q, s)
        w.mxfp8_dequantize(q, s, back)
    for _ in range(3):
        x.copy_(torch.randn_like(x))
        graph.replay()
        torch.cuda.synchronize()
        ref = run_silu(x, dh)
        assert torch.equal(h, ref[0]) and torch.equal(dgu, ref[3]) and torch.equal(again, ref[4])
        assert torch.equal(back, run_dequantize(*run_quantize(dgu), torch.bfloat16))
