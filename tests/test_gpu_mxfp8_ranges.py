"""The activation and its gradient where a factor leaves fp32's numbers and the result does not: exp(-|gate|) down to
e^-290 beside large other factors, and products of those that pass 2^128 before the exponential brings them back."""
import pytest
import torch

import w4a16_grouped_gemm_amd as w
from _gpu import say
from _grouped import TYPES, half_step, silu_and_gradient, values8

pytestmark = pytest.mark.gpu


def run(gu, dh):
    rows, I = dh.shape
    gu, dh = gu.cuda(), dh.cuda()
    h, again, dgu = torch.full_like(dh, 77.0), torch.full_like(dh, 77.0), torch.full_like(gu, 77.0)
    q = torch.zeros(gu.shape, dtype=torch.uint8, device="cuda")
    s = torch.zeros(rows, I // 16, dtype=torch.uint8, device="cuda")
    w.mxfp8_silu_mul(gu, h, q, s)
    w.mxfp8_silu_mul_backward(q, s, dh, dgu, h=again)
    torch.cuda.synchronize()
    return [t.cpu() for t in (h, q, s, dgu, again)]


def close(got, ref, parts, what):
    """Relative to `parts`, the magnitudes that are added up: 16 roundings of 2^-24 (about ten operations, the exponential's
    and the reciprocal's good to a few units) and one rounding to the type; half a step of the type below its normal
    numbers, of fp32 once more where the type is narrower. What passes the type's largest value by a hundredth is infinite."""
    t = got.dtype
    got, most = got.double(), torch.finfo(t).max
    tiny = {torch.float32: 0.0, torch.bfloat16: 2.0**-134, torch.float16: 2.0**-25}[t] + 2.0**-149
    fp32 = 16 * 2.0**-24 * parts
    tol = fp32 + (half_step(t) * (ref.abs() + fp32) if t != torch.float32 else 0) + tiny
    inside, past = ref.abs() < 0.99 * most, ref.abs() > 1.01 * most
    err = (got - ref).abs()
    say(f"  {what}: {int(inside.sum())} inside, max err/tol {float((err / tol)[inside].max()):.3f}, {int(past.sum())} past")
    bad = inside & ~(err <= tol)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} off, e.g. {torch.nonzero(bad)[:4].tolist()}"
    assert torch.equal(got[past], torch.sign(ref[past]) * float("inf")), what


def magnitudes(g, shape, each, low, high):
    """Random values whose sizes are spread over 2^low .. 2^high, the same for `each` neighbours."""
    size = torch.rand(shape[0], shape[1] // each, generator=g, dtype=torch.float64) * (high - low) + low
    return torch.exp2(size).repeat_interleave(each, 1) * (0.75 + 0.25 * torch.rand(*shape, generator=g)) * (
        torch.randint(0, 2, shape, generator=g) * 2 - 1)


def compare(gu, dh):
    I = dh.shape[1]
    h, q, s, dgu, again = run(gu, dh)
    wide, grad = gu.double(), dh.double()
    ref = silu_and_gradient(wide[:, :I], wide[:, I:], grad)[0]
    close(h, ref, ref.abs(), "h")
    kept = values8(q, s)
    gate, up = kept[:, :I], kept[:, I:]
    ref_h, ref_dg, ref_du = silu_and_gradient(gate, up, grad)
    y = torch.sigmoid(gate)
    close(again, ref_h, ref_h.abs(), "h again")
    close(dgu[:, :I], ref_dg, (grad * up).abs() * (y + (gate * y * torch.sigmoid(-gate)).abs()), "dgate")
    close(dgu[:, I:], ref_du, ref_du.abs(), "dup")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("far", [56, 64, 100, 200, 290])
def test_gates_of_any_size_beside_factors_of_any_size(far, dtype):
    """Blocks of gates up to +-far; up and dh of sizes up to the type's range, each product of the two among them."""
    say("activation", far, dtype)
    g = torch.Generator().manual_seed(61)
    t = TYPES[dtype]
    rows, I = 64, 512
    low, high = (-14, 15) if dtype == "fp16" else (-110, 127)
    gate = (torch.rand(rows, I, generator=g, dtype=torch.float64) * 2 - 1) * far
    gate[0] = torch.linspace(-far, far, I)
    up, dh = magnitudes(g, (rows, I), 32, low, high), magnitudes(g, (rows, I), 1, low, high)
    compare(torch.cat((gate, up), 1).to(t), dh.to(t))


def test_results_that_only_the_exponential_would_lose():
    """fp32, single values: past 2^-126 of exp alone (-88), of both factors' product past 2^128 (-150), and the reverse, a
    slope of two that cancel among large factors (-1.2785)."""
    cases = torch.tensor([[-88.0, 100.0, 1.0], [-100.0, 2.0**60, 2.0**10], [-150.0, 1e38, 1e3], [-150.0, 1e38, 1e38],
                          [-60.0, 2.0**-60, 2.0**120], [-280.0, 3e38, 3e38], [-1.25, 1e30, 1e30], [150.0, 1e30, 1e-30],
                          [-96.0, 2.0**-100, 2.0**-100], [-1e30, 3e38, 3e38], [1e30, 1e-30, 1e-30], [0.0, 3e38, 3e38]])
    n = cases.shape[0]
    gu = torch.cat((cases[:, :1].expand(n, 32), cases[:, 1:2].expand(n, 32)), 1).contiguous()
    compare(gu, cases[:, 2:].expand(n, 32).contiguous())


@pytest.mark.parametrize("dtype", TYPES)
def test_not_finite_beside_far_gates(dtype):
    """Infinities and NaN of the values as given, in blocks whose gates are far: g = -infinity gives NaN, what is 0 times
    infinity gives NaN, and the others in the block are as ever."""
    inf, nan = float("inf"), float("nan")
    t = TYPES[dtype]
    gate = torch.linspace(-60000, 60000, 32)[None].repeat(6, 1)
    up, dh = torch.ones(6, 32), torch.ones(6, 32)
    gate[1, 3], gate[2, 4], gate[3, 5], up[4, 31], dh[5, 31] = inf, -inf, nan, inf, -inf
    up[4, 0] = inf
    h, _, _, dgu, again = run(torch.cat((gate, up), 1).to(t), dh.to(t))
    plain = torch.nn.functional.silu(gate) * up
    assert h[1, 3] == inf and h[2, 4].isnan() and h[3, 5].isnan() and h[4, 31] == inf and h[4, 0].isnan()
    special = ~torch.isfinite(plain)
    assert int(special.sum()) == 5 and torch.equal(~torch.isfinite(h.float()), special)
    assert bool(dgu[1:4, :32].isnan().all()) and bool(again[1:5].isnan().all()) and bool(dgu[4, :32].isnan().all())
    assert dgu[5, 31] == -inf and dgu[5, 63] == -inf
    assert bool(torch.isfinite(dgu[0]).all()) and bool(torch.isfinite(dgu[5, :31]).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_far_neighbours_change_no_bits(dtype):
    """A wave goes by mantissas and exponents where one of its factors is far: rows of ordinary values have the same bits beside
    far rows as without them. 32 columns: a wave holds sixteen rows."""
    g = torch.Generator().manual_seed(62)
    t = TYPES[dtype]
    rows, I = 512, 32
    gu = (torch.randn(rows, 2 * I, generator=g) * torch.exp2(torch.randn(rows, 1, generator=g))).clamp(-30, 30).to(t)
    dh = torch.randn(rows, I, generator=g).to(t)
    alone = run(gu, dh)
    mixed_gu, mixed_dh = gu.clone(), dh.clone()
    mixed_gu[::7, 3], mixed_gu[::7, 5] = -200.0, 300.0
    if dtype != "fp16":
        mixed_dh[::11, 9] = 2.0**90
    mixed = run(mixed_gu, mixed_dh)
    same = (torch.arange(rows) % 7 != 0) & (torch.arange(rows) % 11 != 0)
    for a, b in zip(alone, mixed):
        assert torch.equal(a[same], b[same])
