"""The experts' product on 16-bit weights and its gradients against plain 64-bit sums.

Inputs of small whole numbers make every product and every partial sum an fp32 value, so in the
exact tests the fp32 output equals the 64-bit result, bit for bit, in any order of summation. The others
allow the error of their fp32 sums and one rounding of the output."""
import pytest
import torch

import w4a16_grouped_gemm_amd as w
from _grouped import TYPES, Routing, check, product, weight_gradient
from _gpu import say

pytestmark = pytest.mark.gpu

POISON = 77.0  # fits every type


def whole(g, *shape, most=4):
    return torch.randint(-most, most + 1, shape, generator=g).float()


def run(r, a, weights, out_dtype, gather, transposed, stream=None):
    N = weights.shape[2] if transposed else weights.shape[1]
    out = torch.full((r.capacity, N), POISON, dtype=out_dtype, device="cuda")
    w.moe_grouped_gemm(a, *r.args(), weights, out, gather=gather, transposed=transposed, stream=stream)
    torch.cuda.synchronize()
    return out


def run_wgrad(r, dout, a, E, dtype, gather, accumulate=None):
    N, K = dout.shape[1], a.shape[1]
    dw = torch.full((E, N, K), POISON, dtype=dtype, device="cuda") if accumulate is None else accumulate.clone()
    nbytes = w.moe_grouped_gemm_wgrad_workspace_bytes(E, N, K, r.capacity)
    ws = torch.full((max(nbytes, 1),), 0xFF, dtype=torch.uint8, device="cuda") if nbytes else None  # NaN
    w.moe_grouped_gemm_wgrad(dout, a, *r.args(), dw, gather=gather, accumulate=accumulate is not None, workspace=ws)
    torch.cuda.synchronize()
    return dw


# T, topk, E, G, N, K, bm
SHAPES = [
    (1, 1, 1, 1, 8, 8, 16), (1, 2, 3, 4, 16, 40, 16), (2, 2, 2, 2, 8, 1024, 128), (5, 3, 7, 7, 72, 64, 16),
    (17, 2, 3, 5, 264, 136, 32), (40, 1, 2, 2, 512, 72, 64), (33, 4, 5, 9, 248, 200, 64), (130, 2, 2, 3, 256, 64, 128),
    (200, 3, 4, 4, 264, 328, 128), (600, 1, 1, 1, 520, 192, 128), (700, 2, 3, 3, 136, 712, 128),
    (64, 8, 60, 64, 64, 512, 16), (520, 1, 2, 2, 1000, 88, 16), (260, 1, 1, 1, 96, 264, 32),
    (1000, 2, 6, 8, 384, 96, 64),
    # large tiles, with full, half and nearly empty ones, and blocks larger and smaller than a tile
    (300, 1, 1, 1, 28928, 72, 128), (500, 2, 3, 3, 10248, 136, 16), (900, 2, 8, 9, 4104, 64, 64), (700, 1, 3, 3, 2056, 136, 128),
    (40, 2, 8, 8, 1032, 200, 128), (40, 2, 8, 8, 1032, 200, 16), (150, 2, 5, 5, 4104, 2056, 32), (130, 1, 2, 2, 1032, 1160, 128),
    (1300, 1, 1, 1, 1032, 1160, 64), (5000, 1, 1, 1, 8, 24, 128), (6000, 2, 2, 2, 200, 136, 16),
]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_product_is_exact_on_whole_numbers(shape, transposed, gather):
    T, topk, E, G, N, K, bm = shape
    g = torch.Generator().manual_seed(5)
    dtype = torch.bfloat16 if (N + K) % 16 else torch.float16
    say("product", shape, transposed, gather)
    r = Routing(T, topk, E, G, bm, seed=T)
    a = whole(g, T if gather else r.capacity, K)
    weights = whole(g, *((E, K, N) if transposed else (E, N, K)))
    ref, _ = product(r, a, weights, gather, transposed)
    filled = a.clone()
    if not gather:  # what padding rows hold is not read into anything
        pad = torch.ones(r.capacity, dtype=torch.bool)
        pad[r.live] = False
        filled[pad] = float("nan")
    for e in set(range(E)) - set(r.expert.tolist()):  # neither are the weights of an expert without a row
        weights[e] = float("inf")
    out = run(r, filled.to(dtype).cuda(), weights.to(dtype).cuda(), torch.float32, gather, transposed).cpu()
    assert torch.equal(out[: r.rows].double(), ref)
    assert bool((out[r.rows :] == POISON).all())


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_weight_gradient_is_exact_on_whole_numbers(shape, gather):
    T, topk, E, G, N, K, bm = shape
    g = torch.Generator().manual_seed(6)
    dtype = torch.bfloat16 if (N + K) % 16 else torch.float16
    say("weight gradient", shape, gather)
    r = Routing(T, topk, E, G, bm, seed=T + 1)
    a, dout = whole(g, T if gather else r.capacity, K), whole(g, r.capacity, N)
    ref, _ = weight_gradient(r, dout, a, E, gather)
    pad = torch.ones(r.capacity, dtype=torch.bool)
    pad[r.live] = False
    dout[pad] = float("nan")
    if not gather:
        a[pad] = float("inf")
    dout, a = dout.to(dtype).cuda(), a.to(dtype).cuda()
    dw = run_wgrad(r, dout, a, E, torch.float32, gather)
    assert torch.equal(dw.cpu().double(), ref)
    old = whole(g, E, N, K).cuda()
    assert torch.equal(run_wgrad(r, dout, a, E, torch.float32, gather, accumulate=old).cpu().double(),
                       ref + old.cpu().double())


@pytest.mark.parametrize("out", ["same", "fp32"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("shape", [(3, 2, 4, 4, 40, 2048, 16), (96, 4, 8, 8, 320, 1000, 64), (600, 2, 3, 4, 520, 456, 128)],
                         ids=str)
def test_product_of_random_numbers(shape, transposed, dtype, out):
    T, topk, E, G, N, K, bm = shape
    g = torch.Generator().manual_seed(7)
    t = TYPES[dtype]
    r = Routing(T, topk, E, G, bm, seed=3)
    a = torch.randn(T, K, generator=g).to(t)
    weights = (torch.randn(*((E, K, N) if transposed else (E, N, K)), generator=g) * K**-0.5).to(t)
    ref, size = product(r, a, weights, True, transposed)
    got = run(r, a.cuda(), weights.cuda(), t if out == "same" else torch.float32, True, transposed)
    check(got[: r.rows], ref, size, K, f"{shape} {dtype} {out}")


@pytest.mark.parametrize("out", ["same", "fp32"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", [(3, 2, 4, 4, 40, 264, 16), (600, 2, 3, 4, 520, 456, 128), (3000, 1, 1, 1, 64, 136, 128)],
                         ids=str)
def test_weight_gradient_of_random_numbers(shape, dtype, out):
    T, topk, E, G, N, K, bm = shape
    g = torch.Generator().manual_seed(8)
    t = TYPES[dtype]
    r = Routing(T, topk, E, G, bm, seed=4)
    a, dout = torch.randn(T, K, generator=g).to(t), torch.randn(r.capacity, N, generator=g).to(t)
    ref, size = weight_gradient(r, dout, a, E, True)
    o = t if out == "same" else torch.float32
    rows = int(torch.bincount(r.expert, minlength=1).max())
    check(run_wgrad(r, dout.cuda(), a.cuda(), E, o, True), ref, size, rows, f"{shape} {dtype} {out}")
    old = torch.randn(E, N, K, generator=g).to(o)
    got = run_wgrad(r, dout.cuda(), a.cuda(), E, o, True, accumulate=old.cuda())
    check(got, ref + old.double(), size + old.double().abs(), rows + 1, f"{shape} {dtype} {out} added")


def test_gradients_against_differences():
    """loss = sum(out * c): the rows' and weights' gradients against central differences. The loss is linear in
    each, so a difference over a step is the derivative up to the fp32 outputs' error."""
    T, topk, E, N, K, bm = 12, 2, 3, 24, 32, 16
    g = torch.Generator().manual_seed(9)
    r = Routing(T, topk, E, E, bm, seed=2)
    a, weights = whole(g, r.capacity, K).bfloat16().cuda(), whole(g, E, N, K).bfloat16().cuda()
    c = whole(g, r.capacity, N).bfloat16().cuda()
    live = torch.zeros(r.capacity, 1, dtype=torch.float64)
    live[r.live] = 1

    def loss(a, weights):
        return float((run(r, a, weights, torch.float32, False, False).cpu().double()[: r.rows] * (c.cpu().double() * live)[: r.rows]).sum())

    da = run(r, c, weights, torch.float32, False, True)  # [E, N, K] read the other way
    dw = run_wgrad(r, c, a, E, torch.float32, False)
    for row, k in [(int(r.live[0]), 0), (int(r.live[-1]), K - 1), (int(r.live[5]), 7)]:
        up, down = a.clone(), a.clone()
        up[row, k] += 1
        down[row, k] -= 1
        assert (loss(up, weights) - loss(down, weights)) / 2 == float(da[row, k])  # whole numbers: exact
    for e, n, k in [(0, 0, 0), (2, N - 1, K - 1), (1, 5, 9)]:
        up, down = weights.clone(), weights.clone()
        up[e, n, k] += 1
        down[e, n, k] -= 1
        assert (loss(a, up) - loss(a, down)) / 2 == float(dw[e, n, k])


@pytest.mark.parametrize("bm", [16, 32, 64, 128])
def test_all_rows_on_few_experts(bm):
    """Long runs of one expert's blocks beside experts without any."""
    g = torch.Generator().manual_seed(10)
    T, topk, E, N, K = 400, 2, 9, 264, 72
    r = Routing(T, topk, E, E, bm, seed=5, only=[2, 7, 7, 7])
    a, weights = whole(g, T, K), whole(g, E, N, K)
    ref, _ = product(r, a, weights, True, False)
    a16 = a.bfloat16().cuda()
    out = run(r, a16, weights.bfloat16().cuda(), torch.float32, True, False)
    assert torch.equal(out[: r.rows].cpu().double(), ref)
    dout = whole(g, r.capacity, N)
    ref, _ = weight_gradient(r, dout, a, E, True)
    dw = run_wgrad(r, dout.bfloat16().cuda(), a16, E, torch.float32, True)
    assert torch.equal(dw.cpu().double(), ref)


@pytest.mark.parametrize("bm", [16, 64])
def test_blocks_in_any_order_and_of_no_expert(bm):
    """Expert ids that moe_align would not write: an expert's blocks apart, ids outside the experts."""
    g = torch.Generator().manual_seed(11)
    T, topk, E, N, K = 80, 2, 4, 136, 104
    r = Routing(T, topk, E, E, bm, seed=6)
    blocks = r.rows // bm
    order = torch.randperm(blocks, generator=g)
    ids = r.expert_ids[:blocks].cpu()[order]
    ids[1], ids[blocks - 1] = -1, E
    r.expert_ids[:blocks] = ids.cuda()
    r.expert = ids[r.live // bm].long()
    a, weights, dout = whole(g, r.capacity, K), whole(g, E, N, K), whole(g, r.capacity, N)
    ref, _ = product(r, a, weights, False, False)
    out = run(r, a.bfloat16().cuda(), weights.bfloat16().cuda(), torch.float32, False, False).cpu()
    assert torch.equal(out[: r.rows].double(), ref) and bool((out[r.rows :] == POISON).all())
    ref, _ = weight_gradient(r, dout, a, E, False)
    dw = run_wgrad(r, dout.bfloat16().cuda(), a.bfloat16().cuda(), E, torch.float32, False)
    assert torch.equal(dw.cpu().double(), ref)


@pytest.mark.parametrize("bm", [16, 64])
@pytest.mark.parametrize("shape", [(4096, 2, 2, 1024, 72), (2048, 2, 4, 384, 136), (256, 2, 8, 1024, 1024),
                                   (500, 2, 4, 512, 768)], ids=str)
def test_many_blocks_in_any_order(shape, bm):
    """The same with more runs of blocks than experts, so that workgroups take tile after tile, at each tile's size."""
    T, topk, E, N, K = shape
    g = torch.Generator().manual_seed(22)
    r = Routing(T, topk, E, E, bm, seed=23)
    blocks = r.rows // bm
    ids = r.expert_ids[:blocks].cpu()[torch.randperm(blocks, generator=g)]
    ids[blocks // 2], ids[blocks // 3] = -1, E
    r.expert_ids[:blocks] = ids.cuda()
    r.expert = ids[r.live // bm].long()
    a, weights, dout = whole(g, T, K), whole(g, E, N, K), whole(g, r.capacity, N)
    a16, w16, d16 = a.bfloat16().cuda(), weights.bfloat16().cuda(), dout.bfloat16().cuda()
    out = run(r, a16, w16, torch.float32, True, False).cpu()
    assert torch.equal(out[: r.rows].double(), product(r, a, weights, True, False)[0])
    assert bool((out[r.rows :] == POISON).all())
    out = run(r, d16, w16, torch.float32, False, True).cpu()
    assert torch.equal(out[: r.rows].double(), product(r, dout, weights, False, True)[0])
    dw = run_wgrad(r, d16, a16, E, torch.float32, True)
    assert torch.equal(dw.cpu().double(), weight_gradient(r, dout, a, E, True)[0])


@pytest.mark.parametrize("blocks", [64, 65, 512, 513, 1025, 8192, 8193, 20000])
@pytest.mark.parametrize("N", [8, 136])
def test_many_blocks(N, blocks):
    """Blocks of 16 rows on both sides of what is searched at once, runs of all lengths, experts without a block."""
    E, K, bm = 40, 16, 16
    g = torch.Generator().manual_seed(24)
    r = Routing(blocks * bm, 1, E, E, bm, seed=25)
    r.expert_ids[:blocks] = torch.randint(1, E - 1, (blocks,), generator=g).sort()[0].int().cuda()
    slots = torch.randperm(blocks * bm, generator=g)
    slots[torch.rand(blocks * bm, generator=g) < 0.1] = r.n  # padding anywhere
    r.sorted[: blocks * bm] = slots.int().cuda()
    r.ntpp.fill_(blocks * bm)
    r.rows = blocks * bm
    r.live = torch.nonzero(slots < r.n).flatten()
    r.token = slots[r.live]
    r.expert = r.expert_ids.cpu()[r.live // bm].long()
    a, weights = whole(g, r.T, K), whole(g, E, N, K)
    out = run(r, a.bfloat16().cuda(), weights.bfloat16().cuda(), torch.float32, True, False).cpu()
    assert torch.equal(out[: r.rows].double(), product(r, a, weights, True, False)[0])
    assert bool((out[r.rows :] == POISON).all())
    dout = whole(g, r.capacity, N)
    dw = run_wgrad(r, dout.bfloat16().cuda(), a.bfloat16().cuda(), E, torch.float32, True)
    assert torch.equal(dw.cpu().double(), weight_gradient(r, dout, a, E, True)[0])


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("shape", [(8, 1024, 1024), (4, 512, 768), (2, 136, 264)], ids=str)
def test_padding_anywhere(shape, gather):
    """Rows without a slot between real ones, NaN in them, at each tile size of the weights' gradient: a few blocks whole, then
    one hole in a wave's eight rows, then many."""
    E, N, K = shape
    T, bm = 400 * E, 128
    g = torch.Generator().manual_seed(30)
    r = Routing(T, 1, E, E, bm, seed=31)
    slots = r.sorted[: r.rows].cpu()
    hole = (torch.rand(r.rows, generator=g) < 0.2) & (torch.arange(r.rows) % 384 >= 256)
    hole[torch.arange(0, r.rows, 389)] = True
    slots[hole] = r.n + 5
    r.sorted[: r.rows] = slots.cuda()
    r.live = torch.nonzero(slots < r.n).flatten()
    r.token = slots[r.live].long()
    r.expert = r.expert_ids.cpu()[r.live // bm].long()
    a, dout = whole(g, T if gather else r.capacity, K), whole(g, r.capacity, N)
    pad = torch.ones(r.capacity, dtype=torch.bool)
    pad[r.live] = False
    a16, d16 = a.bfloat16(), dout.bfloat16()
    d16[pad] = float("nan")
    if not gather:
        a16[pad] = float("inf")
    dw = run_wgrad(r, d16.cuda(), a16.cuda(), E, torch.float32, gather)
    assert torch.equal(dw.cpu().double(), weight_gradient(r, dout, a, E, gather)[0])
    weights = whole(g, E, N, K)
    out = run(r, a16.cuda(), weights.bfloat16().cuda(), torch.float32, gather, False)
    assert torch.equal(out[: r.rows].cpu().double(), product(r, a, weights, gather, False)[0])


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("K", [8, 64, 128, 192, 256, 320, 328, 1024])
def test_many_experts_of_few_rows(K, gather):
    """Tiles that begin K at a stage of their expert's: numbers of stages below and above what is copied ahead."""
    T, topk, E, N, bm = 1800, 2, 60, 304, 64
    g = torch.Generator().manual_seed(28)
    r = Routing(T, topk, E, E, bm, seed=29)
    a, weights = whole(g, T if gather else r.capacity, K), whole(g, E, N, K)
    out = run(r, a.bfloat16().cuda(), weights.bfloat16().cuda(), torch.float32, gather, False)
    assert torch.equal(out[: r.rows].cpu().double(), product(r, a, weights, gather, False)[0])
    assert bool((out[r.rows :] == POISON).all())


@pytest.mark.parametrize("T", [0, 4])
def test_no_rows(T):
    """No tokens, and tokens without a resident expert: zeros, or what was there with accumulate; no row written."""
    E, N, K, bm = 3, 24, 40, 16
    r = Routing(T, 2, E, 8, bm, only=[5, 6] if T else None)
    assert r.rows == 0
    a, dout = torch.ones(max(T, 1), K).bfloat16().cuda(), torch.ones(r.capacity, N).bfloat16().cuda()
    weights = torch.ones(E, N, K).bfloat16().cuda()
    assert bool((run(r, a, weights, torch.float32, True, False) == POISON).all())
    assert not bool(run_wgrad(r, dout, a, E, torch.bfloat16, True).any())
    old = torch.randn(E, N, K).cuda()
    assert torch.equal(run_wgrad(r, dout, a, E, torch.float32, True, accumulate=old), old)


def test_infinities_stay_in_their_sums():
    T, topk, E, N, K, bm = 20, 1, 2, 40, 72, 16
    g = torch.Generator().manual_seed(12)
    r = Routing(T, topk, E, E, bm, seed=7)
    a, weights = whole(g, T, K), whole(g, E, N, K)
    a[3, 5], a[9, 71] = float("inf"), float("nan")
    weights[1, 17, 2] = float("-inf")
    ref, _ = product(r, a, weights, True, False)
    out = run(r, a.bfloat16().cuda(), weights.bfloat16().cuda(), torch.float32, True, False)
    assert torch.equal(out[: r.rows].cpu().double().nan_to_num(nan=-5e5), ref.nan_to_num(nan=-5e5))
    dout = whole(g, r.capacity, N)
    ref, _ = weight_gradient(r, dout, a, E, True)
    dw = run_wgrad(r, dout.bfloat16().cuda(), a.bfloat16().cuda(), E, torch.float32, True)
    assert torch.equal(dw.cpu().double().nan_to_num(nan=-5e5), ref.nan_to_num(nan=-5e5))


def test_weights_and_rows_past_32_bits():
    """Weights of more than 2^32 bytes, rows read and written past that, the last expert's among them."""
    E, N, K, bm = 70, 8192, 4096, 16
    r = Routing(40, 2, E, E, bm, only=[0, 69])
    weights = torch.zeros(E, N, K, dtype=torch.bfloat16, device="cuda")  # 4.7 GB
    g = torch.Generator().manual_seed(13)
    weights[0], weights[69] = whole(g, N, K).cuda(), whole(g, N, K).cuda()
    a = whole(g, 40, K)
    pair = torch.stack((weights[0], weights[69])).cpu()
    r.expert = (r.expert == 69).long()
    ref, _ = product(r, a, pair, True, False)
    out = run(r, a.bfloat16().cuda(), weights, torch.float32, True, False)
    assert torch.equal(out[: r.rows].cpu().double(), ref)
    dout = whole(g, r.capacity, N)
    da = run(r, dout.bfloat16().cuda(), weights, torch.float32, False, True)
    ref, _ = product(r, dout, pair, False, True)
    assert torch.equal(da[: r.rows].cpu().double(), ref)
    dw = run_wgrad(r, dout.bfloat16().cuda(), a.bfloat16().cuda(), E, torch.bfloat16, True)
    ref, _ = weight_gradient(r, dout, a, 2, True)
    assert torch.equal(dw[[0, 69]].cpu(), ref.bfloat16()) and not bool(dw[1:69].any())


@pytest.mark.parametrize("bm", [16, 128])
def test_rows_past_32_bits(bm):
    """Token rows and aligned rows of more than 2^32 bytes."""
    K, N, E = 1 << 20, 8, 2
    T = 2100
    r = Routing(T, 1, E, E, bm, seed=8)
    g = torch.Generator().manual_seed(14)
    a = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")  # 4.4 GB
    weights = torch.zeros(E, N, K, dtype=torch.bfloat16, device="cuda")
    at = torch.randint(0, K, (24,), generator=g).unique()
    part, wpart = whole(g, T, at.numel()), whole(g, E, N, at.numel())
    a[:, at.cuda()], weights[:, :, at.cuda()] = part.bfloat16().cuda(), wpart.bfloat16().cuda()
    ref, _ = product(r, part, wpart, True, False)
    out = run(r, a, weights, torch.float32, True, False)
    assert torch.equal(out[: r.rows].cpu().double(), ref)
    dout = whole(g, r.capacity, N)
    ref, _ = product(r, dout, wpart, False, True)
    da = run(r, dout.bfloat16().cuda(), weights, torch.bfloat16, False, True)
    assert torch.equal(da[: r.rows, at.cuda()].cpu(), ref.bfloat16())
    ref, _ = weight_gradient(r, dout, part, E, True)
    dw = run_wgrad(r, dout.bfloat16().cuda(), a, E, torch.float32, True)
    assert torch.equal(dw[:, :, at.cuda()].cpu().double(), ref) and int((dw != 0).any(0).any(0).sum()) <= at.numel()


@pytest.mark.parametrize("E, N", [(64, 8), (3, 904), (2, 4096)])
def test_token_rows_past_32_bits_at_each_tile(E, N):
    """The same gathered rows by the small tiles, the ones of 128 rows, and those of 256 with a shorter last one."""
    K, T, bm = 1 << 20, 2100, 16
    r = Routing(T, 1, E, E, bm, seed=26)
    g = torch.Generator().manual_seed(27)
    a = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")  # 4.4 GB
    weights = torch.zeros(E, N, K, dtype=torch.bfloat16, device="cuda")
    at = torch.randint(0, K, (24,), generator=g).unique()
    part, wpart = whole(g, T, at.numel()), whole(g, E, N, at.numel())
    a[:, at.cuda()], weights[:, :, at.cuda()] = part.bfloat16().cuda(), wpart.bfloat16().cuda()
    ref, _ = product(r, part, wpart, True, False)
    out = run(r, a, weights, torch.float32, True, False)
    assert torch.equal(out[: r.rows].cpu().double(), ref)


def _case(T=300, topk=2, E=4, N=264, K=328, bm=64, seed=15):
    g = torch.Generator().manual_seed(seed)
    r = Routing(T, topk, E, E, bm, seed=seed)
    a, weights = torch.randn(T, K, generator=g).bfloat16().cuda(), torch.randn(E, N, K, generator=g).bfloat16().cuda()
    dout = torch.randn(r.capacity, N, generator=g).bfloat16().cuda()
    return r, a, weights, dout


def test_same_bits_again_and_on_two_streams():
    r, a, weights, dout = _case(T=3000, bm=128)
    E, N, K = weights.shape
    first, grad = run(r, a, weights, torch.bfloat16, True, False), run_wgrad(r, dout, a, E, torch.float32, True)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [torch.empty_like(first).fill_(POISON) for _ in streams]
    grads = [torch.empty_like(grad) for _ in streams]
    nbytes = w.moe_grouped_gemm_wgrad_workspace_bytes(E, N, K, r.capacity)
    assert nbytes > 0
    spaces = [torch.empty(nbytes, dtype=torch.uint8, device="cuda") for _ in streams]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, o, d, ws in zip(streams, outs, grads, spaces):
            w.moe_grouped_gemm(a, *r.args(), weights, o, gather=True, stream=s)
            w.moe_grouped_gemm_wgrad(dout, a, *r.args(), d, gather=True, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for o, d in zip(outs, grads):
        assert torch.equal(o[: r.rows], first[: r.rows]) and torch.equal(d, grad)


def test_captured_and_replayed():
    r, a, weights, dout = _case(T=1500, bm=128)
    E, N, K = weights.shape
    out = torch.full((r.capacity, N), POISON, dtype=torch.bfloat16, device="cuda")
    da = torch.full((r.capacity, K), POISON, dtype=torch.bfloat16, device="cuda")
    dw = torch.zeros(E, N, K, device="cuda")
    nbytes = w.moe_grouped_gemm_wgrad_workspace_bytes(E, N, K, r.capacity)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda") if nbytes else None
    w.moe_grouped_gemm(a, *r.args(), weights, out, gather=True)  # loads the library before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w.moe_grouped_gemm(a, *r.args(), weights, out, gather=True)
        w.moe_grouped_gemm(dout, *r.args(), weights, da, transposed=True)
        w.moe_grouped_gemm_wgrad(dout, a, *r.args(), dw, gather=True, workspace=ws)
    for i in range(4):  # other inputs, and another routing of the same buffers, between the replays
        a.copy_(torch.randn_like(a.float()))
        other = Routing(r.T, r.topk, E, E, r.bm, seed=40 + i)
        for name in ("sorted", "expert_ids", "ntpp"):
            getattr(r, name).copy_(getattr(other, name))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), da.clone(), dw.clone()
        eager = run(r, a, weights, torch.bfloat16, True, False), run(r, dout, weights, torch.bfloat16, False, True)
        n = other.rows
        assert torch.equal(got[0][:n], eager[0][:n]) and torch.equal(got[1][:n], eager[1][:n])
        assert torch.equal(got[2], run_wgrad(r, dout, a, E, torch.float32, True))
