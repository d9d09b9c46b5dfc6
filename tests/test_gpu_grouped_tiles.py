"""The experts' products at each of their tiles with 16-bit outputs, and the parts that only large tiles go through.

Which tile a call goes by is a rule on its sizes; each test says which it is there for, and the rule is asked. Inputs of
small whole numbers make every sum an fp32 value, so an output is the 64-bit result rounded once, bit for bit."""
import ctypes
import os

import pytest
import torch

import w4a16_grouped_gemm_amd as w
from _gpu import say
from _grouped import TYPES, Routing, product, weight_gradient
from test_gpu_grouped_gemm import POISON, run, run_wgrad, whole


@pytest.fixture(scope="module", autouse=True)
def library():
    if not os.path.exists(w.LIB_PATH):
        from w4a16_grouped_gemm_amd import build

        build.build()


class Pair(ctypes.Structure):
    _fields_ = [("first", ctypes.c_int32), ("second", ctypes.c_int32)]


def tile_of(E, N, n_slots, transposed):
    """(rows, columns) of the product's tiles."""
    rule = w.load()._ZN5w4a1612grouped_tileEiiib
    rule.argtypes, rule.restype = [ctypes.c_int32] * 3 + [ctypes.c_bool], Pair
    pair = rule(E, N, n_slots, transposed)
    return pair.first, pair.second


def cut_of(E, N, K, capacity):
    """(rows and columns of the weights' gradient's tiles, workgroups that share an expert's rows)."""
    rule = w.load()._ZN5w4a169wgrad_cutEiiii
    rule.argtypes, rule.restype = [ctypes.c_int32] * 4, Pair
    pair = rule(E, N, K, capacity)
    return pair.first, pair.second


# T, topk, E, N, K, bm; the tile that both ways of reading the weights go by, or one each (K last, transposed)
PRODUCTS = [
    ((1200, 2, 8, 4104, 136, 128), (256, 256), (256, 256)),
    ((1200, 2, 8, 3848, 328, 16), (256, 256), (256, 256)),
    ((1200, 1, 8, 1544, 264, 16), (128, 128), (128, 128)),
    ((600, 2, 8, 1544, 192, 64), (128, 128), (128, 128)),
    ((240, 2, 16, 520, 328, 16), (32, 64), (64, 128)),
    ((240, 2, 16, 520, 136, 128), (32, 64), (64, 128)),
    ((60, 2, 4, 264, 328, 16), (32, 32), (32, 64)),
]
# T, topk, E, N, K, bm; the cut
GRADIENTS = [
    ((600, 1, 8, 1032, 776, 64), (256, 1)),
    ((200, 2, 4, 520, 528, 128), (128, 1)),
    ((2300, 2, 4, 520, 528, 64), (128, 2)),
    ((300, 2, 4, 136, 264, 32), (64, 1)),
    ((1500, 2, 2, 136, 264, 128), (64, 3)),
]


def test_each_tile_is_reached():
    for (T, topk, E, N, K, bm), last, transposed in PRODUCTS:
        assert tile_of(E, N, T * topk, False) == last and tile_of(E, N, T * topk, True) == transposed
    for (T, topk, E, N, K, bm), cut in GRADIENTS:
        assert cut_of(E, N, K, w.moe_align_capacity(T, topk, E, bm)) == cut, (E, N, K)
    assert {p[1] for p in PRODUCTS} == {(256, 256), (128, 128), (32, 64), (32, 32)}  # all that the rule has
    assert {p[2] for p in PRODUCTS} == {(256, 256), (128, 128), (64, 128), (32, 64)}


def both_halves(r: Routing, rows):
    """Whether some tile has its first half of rows alone and some more than that, by the blocks that the experts have."""
    blocks = torch.bincount(r.expert_ids[: r.rows // r.bm].cpu().long(), minlength=r.E) * r.bm
    rest = blocks[blocks % rows > 0] % rows
    return bool((rest <= rows // 2).any()) and bool((blocks >= rows).any() or (rest > rows // 2).any())


@pytest.mark.gpu
@pytest.mark.parametrize("gather", [False, True], ids=["aligned", "gathered"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("transposed", [False, True], ids=["K last", "transposed"])
@pytest.mark.parametrize("case", PRODUCTS, ids=str)
def test_16_bit_outputs(case, transposed, dtype, gather):
    (T, topk, E, N, K, bm), *tiles = case
    tile = tile_of(E, N, T * topk, transposed)
    say("16-bit output", case, transposed, dtype, gather, "tile", tile)
    assert tile == tiles[transposed]
    t = TYPES[dtype]
    g = torch.Generator().manual_seed(71)
    r = Routing(T, topk, E, E, bm, seed=72)
    if tile[0] >= 128 and bm <= tile[0] // 2:
        assert both_halves(r, tile[0])
    a, weights = whole(g, T if gather else r.capacity, K), whole(g, *((E, K, N) if transposed else (E, N, K)))
    ref, _ = product(r, a, weights, gather, transposed)
    filled = a.clone()
    if not gather:
        pad = torch.ones(r.capacity, dtype=torch.bool)
        pad[r.live] = False
        filled[pad] = float("nan")
    out = run(r, filled.to(t).cuda(), weights.to(t).cuda(), t, gather, transposed).cpu()
    assert torch.equal(out[: r.rows], ref.to(t))
    assert bool((out[r.rows :] == POISON).all())


@pytest.mark.gpu
@pytest.mark.parametrize("gather", [False, True], ids=["aligned", "gathered"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("case", GRADIENTS, ids=str)
def test_16_bit_weight_gradients(case, dtype, gather):
    (T, topk, E, N, K, bm), cut = case
    say("16-bit weight gradient", case, dtype, gather)
    t = TYPES[dtype]
    g = torch.Generator().manual_seed(73)
    r = Routing(T, topk, E, E, bm, seed=74)
    assert cut_of(E, N, K, r.capacity) == cut
    a, dout = whole(g, T if gather else r.capacity, K), whole(g, r.capacity, N)
    ref, _ = weight_gradient(r, dout, a, E, gather)
    pad = torch.ones(r.capacity, dtype=torch.bool)
    pad[r.live] = False
    dout[pad] = float("nan")
    dout, a = dout.to(t).cuda(), a.to(t).cuda()
    assert torch.equal(run_wgrad(r, dout, a, E, t, gather).cpu(), ref.to(t))
    old = whole(g, E, N, K, most=200).to(t)
    got = run_wgrad(r, dout, a, E, t, gather, accumulate=old.cuda())
    assert torch.equal(got.cpu(), (ref + old.double()).to(t))
    got = run_wgrad(r, dout, a, E, torch.float32, gather, accumulate=old.float().cuda())
    assert torch.equal(got.cpu().double(), ref + old.double())


@pytest.mark.gpu
@pytest.mark.parametrize("case", [PRODUCTS[0], PRODUCTS[2], PRODUCTS[5], PRODUCTS[6]], ids=str)
def test_values_below_the_types_normal_numbers(case):
    """fp16 values down to 2^-24, normal numbers of fp32, count in full: products of two of them are multiples of 2^-48, their sums
    below 2^24 of those, so fp32 outputs are exact."""
    (T, topk, E, N, K, bm), *_ = case
    g = torch.Generator().manual_seed(75)
    r = Routing(T, topk, E, E, bm, seed=76)
    a, weights, dout = whole(g, T, K) * 2.0**-24, whole(g, E, N, K) * 2.0**-24, whole(g, r.capacity, N) * 2.0**-24
    a16, w16, d16 = (x.half().cuda() for x in (a, weights, dout))
    out = run(r, a16, w16, torch.float32, True, False)
    assert torch.equal(out[: r.rows].cpu().double(), product(r, a, weights, True, False)[0])
    out = run(r, d16, w16, torch.float32, False, True)
    assert torch.equal(out[: r.rows].cpu().double(), product(r, dout, weights, False, True)[0])
    dw = run_wgrad(r, d16, a16, E, torch.float32, True)
    assert torch.equal(dw.cpu().double(), weight_gradient(r, dout, a, E, True)[0])


@pytest.mark.gpu
@pytest.mark.parametrize("sizes", [(-70, -60), (-133, 10), (10, -133), (-133, -10)], ids=str)
@pytest.mark.parametrize("case", [PRODUCTS[0], PRODUCTS[2], PRODUCTS[5], PRODUCTS[6]], ids=str)
def test_sums_below_fp32s_normal_numbers(case, sizes):
    """bf16 values of which either or the products lie below 2^-126, the products multiples of 2^-143 and their sums below 2^24
    of those: fp32 values, so the outputs are exact."""
    (T, topk, E, N, K, bm), *_ = case
    rows, columns = 2.0 ** sizes[0], 2.0 ** sizes[1]
    g = torch.Generator().manual_seed(82)
    r = Routing(T, topk, E, E, bm, seed=83)
    a, dout = whole(g, T, K).double() * rows, whole(g, r.capacity, N).double() * rows
    weights, dout2 = whole(g, E, N, K).double() * columns, whole(g, r.capacity, N).double() * columns
    a16, w16, d16 = (x.bfloat16().cuda() for x in (a, weights, dout))
    out = run(r, a16, w16, torch.float32, True, False)
    assert torch.equal(out[: r.rows].cpu().double(), product(r, a, weights, True, False)[0])
    out = run(r, d16, w16, torch.float32, False, True)
    assert torch.equal(out[: r.rows].cpu().double(), product(r, dout, weights, False, True)[0])
    dw = run_wgrad(r, dout2.bfloat16().cuda(), a16, E, torch.float32, True)
    assert torch.equal(dw.cpu().double(), weight_gradient(r, dout2, a, E, True)[0])


@pytest.mark.gpu
@pytest.mark.parametrize("case", PRODUCTS[:4], ids=str)
def test_infinities_stay_in_their_sums(case):
    (T, topk, E, N, K, bm), *_ = case
    g = torch.Generator().manual_seed(77)
    r = Routing(T, topk, E, E, bm, seed=78)
    same = lambda got, ref: torch.equal(got.cpu().double().nan_to_num(nan=-5e5), ref.nan_to_num(nan=-5e5))  # noqa: E731
    a, weights, dout = whole(g, T, K), whole(g, E, N, K), whole(g, r.capacity, N)
    a[3, 5], a[T - 1, K - 1], weights[1, 17, 2], weights[E - 1, N - 1, 0] = float("inf"), float("nan"), float("-inf"), float("nan")
    dout[r.live[7], 11], dout[r.live[-1], N - 1] = float("-inf"), float("nan")
    a16, w16, d16 = a.bfloat16().cuda(), weights.bfloat16().cuda(), dout.bfloat16().cuda()
    out = run(r, a16, w16, torch.float32, True, False)
    assert same(out[: r.rows], product(r, a, weights, True, False)[0])
    out = run(r, d16, w16, torch.float32, False, True)
    assert same(out[: r.rows], product(r, dout, weights, False, True)[0])
    dw = run_wgrad(r, d16, a16, E, torch.float32, True)
    assert same(dw, weight_gradient(r, dout, a, E, True)[0])


T, TOPK, E, BM, H, I = 1360, 2, 16, 64, 1544, 800  # a layer whose products go by 256 and by 128 rows


def test_a_large_layer_goes_by_large_tiles():
    assert tile_of(E, 2 * I, T * TOPK, False) == (256, 256) and tile_of(E, H, T * TOPK, False) == (256, 256)
    assert tile_of(E, H, T * TOPK, True) == (256, 256) and tile_of(E, I, T * TOPK, True) == (128, 128)
    capacity = w.moe_align_capacity(T, TOPK, E, BM)
    assert cut_of(E, 2 * I, H, capacity) == (256, 1) and cut_of(E, H, I, capacity) == (256, 1)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype, gather", [("bf16", True), ("fp16", False)])
def test_a_training_step_of_a_large_layer(dtype, gather):
    import test_gpu_expert_layer as layer

    layer.test_a_training_step((T, TOPK, E, E, BM, H, I), dtype, gather)


@pytest.mark.gpu
def test_large_tiles_captured_and_replayed():
    """As the small ones: other inputs and another routing of the same buffers between the replays."""
    g = torch.Generator().manual_seed(79)
    r = Routing(T, TOPK, E, E, BM, seed=80)
    a, weights = torch.randn(T, H, generator=g).bfloat16().cuda(), torch.randn(E, 2 * I, H, generator=g).bfloat16().cuda()
    dout = torch.randn(r.capacity, 2 * I, generator=g).bfloat16().cuda()
    out = torch.full((r.capacity, 2 * I), POISON, dtype=torch.bfloat16, device="cuda")
    da = torch.full((r.capacity, H), POISON, dtype=torch.bfloat16, device="cuda")
    dw = torch.zeros(E, 2 * I, H, dtype=torch.bfloat16, device="cuda")
    w.moe_grouped_gemm(a, *r.args(), weights, out, gather=True)  # loads what a first call loads
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w.moe_grouped_gemm(a, *r.args(), weights, out, gather=True)
        w.moe_grouped_gemm(dout, *r.args(), weights, da, transposed=True)
        w.moe_grouped_gemm_wgrad(dout, a, *r.args(), dw, gather=True)
    for i in range(3):
        a.copy_(torch.randn_like(a.float()))
        other = Routing(T, TOPK, E, E, BM, seed=81 + i)
        for name in ("sorted", "expert_ids", "ntpp"):
            getattr(r, name).copy_(getattr(other, name))
        graph.replay()
        torch.cuda.synchronize()
        n, got = other.rows, (out.clone(), da.clone(), dw.clone())
        assert torch.equal(got[0][:n], run(r, a, weights, torch.bfloat16, True, False)[:n])
        assert torch.equal(got[1][:n], run(r, dout, weights, torch.bfloat16, False, True)[:n])
        assert torch.equal(got[2], run_wgrad(r, dout, a, E, torch.bfloat16, True))
