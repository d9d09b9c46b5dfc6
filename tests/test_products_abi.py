"""Refusals of the 16-bit products' and 8-bit checkpoints' entry points, on the host (no GPU needed: validation runs
before any launch), by the C ABI and by the Python binding."""
import ctypes

import pytest
import torch

import w4a16_grouped_gemm_amd as w

OK, INVALID, UNSUPPORTED, CAPACITY, WORKSPACE = 0, 1, 2, 3, 4
FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: every call below fails validation first
ODD = ctypes.c_void_p(0x1008)
BF16, FP16, FP32 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    import os

    if not os.path.exists(w.LIB_PATH):
        from w4a16_grouped_gemm_amd import build

        build.build()
    return w.load()


def gemm(lib, E=4, N=64, K=72, a=FAKE, dtype=BF16, a_rows=64, gather=0, T=4, topk=2, srt=FAKE, cap=64, eid=FAKE,
         ntpp=FAKE, bm=16, weights=FAKE, transposed=0, out=FAKE, ot=BF16):
    return lib.moe_grouped_gemm(E, N, K, a, dtype, a_rows, gather, T, topk, srt, cap, eid, ntpp, bm, weights, transposed,
                                out, ot, None)


def wgrad(lib, E=4, N=64, K=72, dout=FAKE, a=FAKE, dtype=BF16, a_rows=64, gather=0, T=4, topk=2, srt=FAKE, cap=64,
          eid=FAKE, ntpp=FAKE, bm=16, dw=FAKE, ot=BF16, accumulate=0, ws=None, ws_bytes=0):
    return lib.moe_grouped_gemm_wgrad(E, N, K, dout, a, dtype, a_rows, gather, T, topk, srt, cap, eid, ntpp, bm, dw, ot,
                                      accumulate, ws, ws_bytes, None)


SHARED = [
    (dict(E=0), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(K=-8), INVALID), (dict(E=513), UNSUPPORTED),
    (dict(N=60), UNSUPPORTED), (dict(K=68), UNSUPPORTED), (dict(N=(1 << 20) + 8), UNSUPPORTED),
    (dict(K=(1 << 20) + 8), UNSUPPORTED), (dict(dtype=3), INVALID), (dict(ot=-1), INVALID), (dict(dtype=FP32, ot=FP32), UNSUPPORTED),
    (dict(ot=FP16), UNSUPPORTED), (dict(dtype=FP16), UNSUPPORTED), (dict(T=-1), INVALID), (dict(topk=0), INVALID),
    (dict(topk=33), UNSUPPORTED), (dict(bm=48), UNSUPPORTED), (dict(bm=0), UNSUPPORTED), (dict(bm=256), UNSUPPORTED),
    (dict(T=1 << 29), UNSUPPORTED), (dict(cap=-1), INVALID), (dict(a_rows=63), INVALID), (dict(gather=1, a_rows=3), INVALID),
    (dict(a=None), INVALID), (dict(srt=None), INVALID), (dict(eid=None), INVALID), (dict(ntpp=None), INVALID),
    (dict(a=ODD), INVALID), (dict(cap=(1 << 21) + 16, a_rows=1 << 22), UNSUPPORTED),
]


@pytest.mark.parametrize("change, status", SHARED + [
    (dict(weights=None), INVALID), (dict(out=None), INVALID), (dict(weights=ODD), INVALID), (dict(out=ODD), INVALID),
])
def test_product_refusals(lib, change, status):
    assert gemm(lib, **change) == status
    assert gemm(lib, transposed=1, **change) == status


@pytest.mark.parametrize("change, status", SHARED + [
    (dict(dout=None), INVALID), (dict(dw=None), INVALID), (dict(dout=ODD), INVALID), (dict(dw=ODD), INVALID),
    (dict(E=512, N=1 << 20, K=1 << 14), UNSUPPORTED), (dict(ws=ODD), INVALID), (dict(T=0, dw=None), INVALID),
    (dict(E=1, cap=1 << 16, a_rows=1 << 16), WORKSPACE), (dict(E=1, cap=1 << 16, a_rows=1 << 16, ws=FAKE, ws_bytes=1000), WORKSPACE),
])
def test_weight_gradient_refusals(lib, change, status):
    assert wgrad(lib, **change) == status


def test_weight_gradient_workspace():
    """The shares' sums, where few weights have many rows; none where the tiles fill the card."""
    need = w.moe_grouped_gemm_wgrad_workspace_bytes(1, 64, 72, 1 << 16)
    assert need > 0 and need % (4 * 64 * 72) == 0
    assert w.moe_grouped_gemm_wgrad_workspace_bytes(16, 4096, 7168, 1 << 16) == 0
    assert w.moe_grouped_gemm_wgrad_workspace_bytes(4, 64, 72, 64) == 0
    for bad in [(0, 64, 64, 64), (4, 63, 64, 64), (4, 64, 0, 64), (4, 64, 64, -1), (600, 64, 64, 64)]:
        assert w.moe_grouped_gemm_wgrad_workspace_bytes(*bad) == 0


def quantize(lib, x=FAKE, dtype=BF16, rows=4, K=64, n=None, q=FAKE, s=FAKE):
    return lib.mxfp8_quantize(x, dtype, rows, K, n, q, s, None)


def dequantize(lib, x=FAKE, dtype=BF16, rows=4, K=64, n=None, q=FAKE, s=FAKE):
    return lib.mxfp8_dequantize(q, s, rows, K, n, x, dtype, None)


def silu(lib, x=FAKE, dtype=BF16, rows=4, K=64, n=None, q=FAKE, s=FAKE, h=FAKE):
    return lib.mxfp8_silu_mul(x, dtype, rows, K, n, h, q, s, None)


def backward(lib, x=FAKE, dtype=BF16, rows=4, K=64, n=None, q=FAKE, s=FAKE, h=FAKE):
    return lib.mxfp8_silu_mul_backward(q, s, h, dtype, rows, K, n, x, None, None)


@pytest.mark.parametrize("call", [quantize, dequantize, silu, backward])
@pytest.mark.parametrize("change, status", [
    (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID), (dict(rows=-1), INVALID), (dict(K=0), INVALID),
    (dict(K=48), UNSUPPORTED), (dict(K=(1 << 20) + 32), UNSUPPORTED), (dict(x=None), INVALID), (dict(q=None), INVALID),
    (dict(s=None), INVALID), (dict(x=ODD), INVALID), (dict(q=ODD), INVALID),
])
def test_checkpoint_refusals(lib, call, change, status):
    assert call(lib, **change) == status


def test_activation_refusals(lib):
    for call in (silu, backward):
        assert call(lib, h=None) == INVALID and call(lib, h=ODD) == INVALID
    assert lib.mxfp8_silu_mul_backward(FAKE, FAKE, FAKE, BF16, 4, 64, None, FAKE, ODD, None) == INVALID


def test_nothing_to_do_is_ok(lib):
    assert gemm(lib, T=0, a=None, out=None, weights=None) == OK
    assert gemm(lib, cap=0, a_rows=0, srt=None, eid=None) == OK
    for call in (quantize, dequantize, silu, backward):
        assert call(lib, rows=0, x=None, q=None, s=None) == OK


def refused(status, f, *args, **kw):
    with pytest.raises(w.W4A16Error) as e:
        f(*args, **kw)
    assert e.value.status == status, e.value


def i32(*shape, device="cpu"):
    return torch.zeros(*shape, dtype=torch.int32, device=device)


def test_binding_refuses_what_pointers_hide(lib):
    """Host tensors, strides, types and shapes that do not fit."""
    bf = lambda *shape: torch.zeros(*shape, dtype=torch.bfloat16)  # noqa: E731
    u8 = lambda *shape: torch.zeros(*shape, dtype=torch.uint8)  # noqa: E731
    good = dict(a=bf(32, 64), T=4, topk=2, sorted_token_ids=i32(32), expert_ids=i32(2), num_tokens_post_padded=i32(1),
                block_m=16, w=bf(2, 24, 64), out=bf(32, 24))
    refused(INVALID, w.moe_grouped_gemm, **good)  # on no GPU
    for status, change in [
            (INVALID, dict(w=bf(2, 64, 24))), (INVALID, dict(transposed=True)), (INVALID, dict(w=bf(2, 24, 64).half())),
            (INVALID, dict(out=bf(32, 32))), (CAPACITY, dict(out=bf(31, 24))), (INVALID, dict(expert_ids=i32(1))),
            (INVALID, dict(sorted_token_ids=i32(32).long())), (INVALID, dict(num_tokens_post_padded=i32(0))),
            (UNSUPPORTED, dict(out=bf(32, 24).double()))]:
        refused(status, w.moe_grouped_gemm, **{**good, **change})
    good = dict(dout=bf(32, 24), a=bf(32, 64), T=4, topk=2, sorted_token_ids=i32(32), expert_ids=i32(2),
                num_tokens_post_padded=i32(1), block_m=16, dw=bf(2, 24, 64))
    refused(INVALID, w.moe_grouped_gemm_wgrad, **good)
    for status, change in [
            (INVALID, dict(dout=bf(32, 32))), (INVALID, dict(a=bf(32, 32))), (INVALID, dict(dout=bf(32, 24).half())),
            (CAPACITY, dict(dout=bf(31, 24))), (INVALID, dict(expert_ids=i32(1))), (INVALID, dict(dout=bf(24))),
            (INVALID, dict(expert_ids=i32(2).long())), (UNSUPPORTED, dict(dw=bf(2, 24, 64).double()))]:
        refused(status, w.moe_grouped_gemm_wgrad, **{**good, **change})
    x = bf(4, 64)
    refused(INVALID, w.mxfp8_quantize, x, u8(4, 64), u8(4, 2))
    refused(INVALID, w.mxfp8_quantize, x, u8(4, 32), u8(4, 2))
    refused(INVALID, w.mxfp8_quantize, x, u8(4, 64).int(), u8(4, 2))
    refused(INVALID, w.mxfp8_quantize, x, u8(4, 64), u8(4, 2), num_rows=i32(0))
    refused(UNSUPPORTED, w.mxfp8_quantize, x[:, :40], u8(4, 40), u8(4, 1))
    refused(UNSUPPORTED, w.mxfp8_dequantize, u8(4, 64), u8(4, 2), x.double())
    refused(INVALID, w.mxfp8_dequantize, u8(4, 64), u8(4, 3), x)
    h, gu = bf(4, 32), x
    refused(INVALID, w.mxfp8_silu_mul, gu, h, u8(4, 64), u8(4, 2))
    refused(INVALID, w.mxfp8_silu_mul, gu, h.half(), u8(4, 64), u8(4, 2))
    refused(INVALID, w.mxfp8_silu_mul, gu, x, u8(4, 64), u8(4, 2))
    refused(UNSUPPORTED, w.mxfp8_silu_mul, bf(4, 32), bf(4, 16), u8(4, 32), u8(4, 1))
    refused(INVALID, w.mxfp8_silu_mul_backward, u8(4, 64), u8(4, 2), h, gu)
    refused(INVALID, w.mxfp8_silu_mul_backward, u8(4, 64), u8(4, 2), h, h)
    refused(INVALID, w.mxfp8_silu_mul_backward, u8(4, 64), u8(4, 2), h, gu, h=gu)
    refused(UNSUPPORTED, w.mxfp8_silu_mul_backward, u8(4, 32), u8(4, 1), bf(4, 16), bf(4, 32))


BIG = 1 << 32  # a size of 2^32 + n is n in 32 bits


def test_binding_refuses_sizes_past_32_bits(lib):
    """Tensors of the meta device have shapes only; a call that gets past the sizes says that they are on no GPU."""
    def meta(*shape, dtype=torch.bfloat16):
        return torch.empty(*shape, dtype=dtype, device="meta")

    u8 = lambda *shape: meta(*shape, dtype=torch.uint8)  # noqa: E731
    far, wide = BIG + 32, BIG + 64
    good = dict(a=meta(32, 64), T=4, topk=2, sorted_token_ids=i32(32, device="meta"), expert_ids=i32(2, device="meta"),
                num_tokens_post_padded=i32(1, device="meta"), block_m=16)
    product = dict(w=meta(2, 24, 64), out=meta(32, 24))
    gradient = dict(dout=meta(32, 24), dw=meta(2, 24, 64))
    long = dict(sorted_token_ids=i32(far, device="meta"), expert_ids=i32(far // 16, device="meta"))
    refused(INVALID, w.moe_grouped_gemm, **good, **product)  # on no GPU
    refused(INVALID, w.moe_grouped_gemm_wgrad, **good, **gradient)
    for change in (dict(T=BIG + 4), dict(topk=BIG + 2), dict(block_m=BIG + 16), dict(a=meta(far, 64))):
        refused(UNSUPPORTED, w.moe_grouped_gemm, **{**good, **product, **change})
        refused(UNSUPPORTED, w.moe_grouped_gemm_wgrad, **{**good, **gradient, **change})
    for change in (dict(a=meta(32, wide), w=meta(2, 24, wide)), dict(w=meta(2, BIG + 24, 64), out=meta(32, BIG + 24)),
                   dict(w=meta(BIG + 2, 24, 64)), dict(out=meta(far, 24), **long)):
        refused(UNSUPPORTED, w.moe_grouped_gemm, **{**good, **product, **change})
    for change in (dict(a=meta(32, wide), dw=meta(2, 24, wide)), dict(dout=meta(32, BIG + 24), dw=meta(2, BIG + 24, 64)),
                   dict(dw=meta(BIG + 2, 24, 64)), dict(dout=meta(far, 24), **long)):
        refused(UNSUPPORTED, w.moe_grouped_gemm_wgrad, **{**good, **gradient, **change})
    for change in (dict(T=-BIG + 4), dict(topk=-BIG + 2)):
        refused(INVALID, w.moe_grouped_gemm, **{**good, **product, **change})
        refused(INVALID, w.moe_grouped_gemm_wgrad, **{**good, **gradient, **change})
    for sizes in [(BIG + 2, 64, 64, 64), (2, BIG + 64, 64, 64), (2, 64, BIG + 64, 64), (2, 64, 64, BIG + 64)]:
        refused(UNSUPPORTED, w.moe_grouped_gemm_wgrad_workspace_bytes, *sizes)
    for rows, K in [(far, 64), (4, wide)]:
        q, s, x, half = u8(rows, K), u8(rows, K // 32), meta(rows, K), meta(rows, K // 2)
        refused(UNSUPPORTED, w.mxfp8_quantize, x, q, s)
        refused(UNSUPPORTED, w.mxfp8_dequantize, q, s, x)
        refused(UNSUPPORTED, w.mxfp8_silu_mul, x, half, q, s)
        refused(UNSUPPORTED, w.mxfp8_silu_mul_backward, q, s, half, x)
