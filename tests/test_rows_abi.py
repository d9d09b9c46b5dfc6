"""Refusals of the row and 4-bit floating point entry points, on the host (no GPU needed: validation
runs before any launch), by the C ABI and by the Python binding."""
import ctypes

import pytest
import torch

import w4a16_grouped_gemm_amd as w

OK, INVALID, UNSUPPORTED, CAPACITY = 0, 1, 2, 3
FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: every call below fails validation first
ODD = ctypes.c_void_p(0x1001)
BF16, FP16, FP32 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    import os

    if not os.path.exists(w.LIB_PATH):
        from w4a16_grouped_gemm_amd import build

        build.build()
    return w.load()


def permute(lib, x=FAKE, dtype=BF16, T=4, topk=2, H=64, srt=FAKE, cap=32, ntpp=FAKE, xp=FAKE, rows=FAKE):
    return lib.moe_permute(x, dtype, T, topk, H, srt, cap, ntpp, xp, rows, None)


def unpermute(lib, y=FAKE, yt=BF16, rows=32, T=4, topk=2, H=64, slots=FAKE, wts=FAKE, out=FAKE, ot=BF16):
    return lib.moe_unpermute(y, yt, rows, T, topk, H, slots, wts, out, ot, None)


def backward(lib, dout=FAKE, ot=BF16, y=FAKE, yt=BF16, rows=32, T=4, topk=2, H=64, slots=FAKE, wts=FAKE, srt=FAKE,
             cap=32, ntpp=FAKE, dy=FAKE, dw=FAKE):
    return lib.moe_unpermute_backward(dout, ot, y, yt, rows, T, topk, H, slots, wts, srt, cap, ntpp, dy, dw, None)


def quantize(lib, x=FAKE, dtype=BF16, rows=4, K=64, n=None, q=FAKE, s=FAKE, f="mxfp4_quantize"):
    return getattr(lib, f)(x, dtype, rows, K, n, q, s, None)


def dequantize(lib, q=FAKE, s=FAKE, rows=4, K=64, n=None, out=FAKE, dtype=BF16):
    return lib.mxfp4_dequantize(q, s, rows, K, n, out, dtype, None)


def gemm(lib, E=4, N=64, K=64, a=FAKE, s=FAKE, a_rows=64, gather=0, T=4, topk=2, srt=FAKE, cap=64, eid=FAKE,
         ntpp=FAKE, bm=16, packed=FAKE, out=FAKE, dtype=BF16):
    return lib.mxfp4_moe_gemm(E, N, K, a, s, a_rows, gather, T, topk, srt, cap, eid, ntpp, bm, packed, out, dtype, None)


@pytest.mark.parametrize("change, status", [
    (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID), (dict(T=-1), INVALID), (dict(topk=0), INVALID),
    (dict(H=0), INVALID), (dict(cap=-1), INVALID), (dict(topk=33), UNSUPPORTED), (dict(H=(1 << 20) + 1), UNSUPPORTED),
    (dict(T=1 << 30, topk=2), UNSUPPORTED), (dict(cap=1 << 30), UNSUPPORTED), (dict(cap=1 << 28), UNSUPPORTED),
    (dict(T=1 << 23), UNSUPPORTED), (dict(x=None), INVALID),
    (dict(srt=None), INVALID), (dict(ntpp=None), INVALID), (dict(xp=None), INVALID), (dict(rows=None), INVALID),
    (dict(x=ODD), INVALID), (dict(xp=ODD), INVALID), (dict(dtype=FP32, x=ctypes.c_void_p(0x1002)), INVALID),
])
def test_permute_refusals(lib, change, status):
    assert permute(lib, **change) == status


@pytest.mark.parametrize("change, status", [
    (dict(yt=5), INVALID), (dict(ot=5), INVALID), (dict(yt=BF16, ot=FP32), UNSUPPORTED),
    (dict(yt=BF16, ot=FP16), UNSUPPORTED), (dict(rows=-1), INVALID), (dict(T=-2), INVALID), (dict(topk=40), UNSUPPORTED),
    (dict(H=0), INVALID), (dict(y=None), INVALID), (dict(slots=None), INVALID), (dict(out=None), INVALID),
    (dict(y=ODD), INVALID), (dict(out=ODD), INVALID), (dict(yt=FP32, y=ctypes.c_void_p(0x1002)), INVALID),
])
def test_unpermute_refusals(lib, change, status):
    assert unpermute(lib, **change) == status
    shared = {k: v for k, v in change.items() if k in ("yt", "ot", "rows", "T", "topk", "H", "y", "slots")}
    if shared == change and "y" not in change:
        assert backward(lib, **{**change, "rows": change.get("rows", 64)}) == status


@pytest.mark.parametrize("change, status", [
    (dict(dout=None), INVALID), (dict(y=None), INVALID), (dict(slots=None), INVALID), (dict(dy=None, dw=None), INVALID),
    (dict(srt=None), INVALID), (dict(ntpp=None), INVALID), (dict(cap=-1), INVALID), (dict(cap=33), CAPACITY),
    (dict(dy=ODD), INVALID), (dict(dout=ODD), INVALID),
])
def test_unpermute_backward_refusals(lib, change, status):
    assert backward(lib, **change) == status


@pytest.mark.parametrize("f", ["mxfp4_quantize", "mxfp4_silu_mul_quantize"])
@pytest.mark.parametrize("change, status", [
    (dict(dtype=3), INVALID), (dict(rows=-1), INVALID), (dict(K=0), INVALID), (dict(K=48), UNSUPPORTED),
    (dict(K=(1 << 20) + 32), UNSUPPORTED), (dict(x=None), INVALID), (dict(q=None), INVALID), (dict(s=None), INVALID),
    (dict(x=ctypes.c_void_p(0x1008)), INVALID), (dict(q=ctypes.c_void_p(0x1002)), INVALID),
])
def test_quantize_refusals(lib, f, change, status):
    assert quantize(lib, f=f, **change) == status


@pytest.mark.parametrize("change, status", [
    (dict(dtype=3), INVALID), (dict(rows=-1), INVALID), (dict(K=31), UNSUPPORTED), (dict(q=None), INVALID),
    (dict(s=None), INVALID), (dict(out=None), INVALID), (dict(out=ctypes.c_void_p(0x1008)), INVALID),
    (dict(q=ctypes.c_void_p(0x1002)), INVALID),
])
def test_dequantize_refusals(lib, change, status):
    assert dequantize(lib, **change) == status


@pytest.mark.parametrize("change, status", [
    (dict(E=0), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(E=513), UNSUPPORTED), (dict(N=40), UNSUPPORTED),
    (dict(K=48), UNSUPPORTED), (dict(N=(1 << 20) + 16), UNSUPPORTED), (dict(K=(1 << 20) + 32), UNSUPPORTED),
    (dict(dtype=7), INVALID), (dict(T=-1), INVALID), (dict(topk=0), INVALID), (dict(topk=33), UNSUPPORTED),
    (dict(bm=48), UNSUPPORTED), (dict(bm=0), UNSUPPORTED), (dict(cap=-1), INVALID), (dict(a_rows=63), INVALID),
    (dict(gather=1, a_rows=3), INVALID), (dict(a=None), INVALID), (dict(s=None), INVALID), (dict(srt=None), INVALID),
    (dict(eid=None), INVALID), (dict(ntpp=None), INVALID), (dict(packed=None), INVALID), (dict(out=None), INVALID),
    (dict(a=ctypes.c_void_p(0x1008)), INVALID), (dict(out=ctypes.c_void_p(0x1008)), INVALID),
    (dict(packed=ctypes.c_void_p(0x1008)), INVALID),
])
def test_gemm_refusals(lib, change, status):
    assert gemm(lib, **change) == status


def test_packed_bytes_and_repack_refusals(lib):
    # 64 columns by K = 128 are 4096 bytes of codes and 256 of scales; N rounds up to 64, K to 128
    assert w.mxfp4_packed_bytes(3, 64, 128) == 3 * 4352
    assert w.mxfp4_packed_bytes(3, 80, 160) == 3 * 2 * 2 * 4352
    for E, N, K, status in [(0, 64, 64, INVALID), (1, 8, 64, UNSUPPORTED), (1, 64, 16, UNSUPPORTED), (513, 64, 64, UNSUPPORTED)]:
        with pytest.raises(w.W4A16Error) as e:
            w.mxfp4_packed_bytes(E, N, K)
        assert e.value.status == status
        assert lib.mxfp4_repack(E, N, K, FAKE, FAKE, FAKE, None) == status
    assert lib.mxfp4_packed_bytes(1, 64, 64, None) == INVALID
    for args in [(None, FAKE, FAKE), (FAKE, None, FAKE), (FAKE, FAKE, None), (ctypes.c_void_p(0x1008), FAKE, FAKE)]:
        assert lib.mxfp4_repack(1, 64, 64, *args, None) == INVALID


def test_nothing_to_do_is_ok(lib):
    assert permute(lib, T=0, x=None, srt=None, ntpp=None, xp=None, rows=None) == OK
    assert unpermute(lib, T=0, y=None, slots=None, out=None) == OK
    assert quantize(lib, rows=0, x=None, q=None, s=None) == OK
    assert dequantize(lib, rows=0, q=None, s=None, out=None) == OK
    assert gemm(lib, T=0) == OK


def refused(status, f, *args, **kw):
    with pytest.raises(w.W4A16Error) as e:
        f(*args, **kw)
    assert e.value.status == status, e.value


def test_binding_refuses_what_pointers_hide(lib):
    """Host tensors, strides, types and shapes that do not fit."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    i32 = lambda *shape: torch.zeros(*shape, dtype=torch.int32)  # noqa: E731
    u8 = lambda *shape: torch.zeros(*shape, dtype=torch.uint8)  # noqa: E731
    xp = torch.zeros(32, 64, dtype=torch.bfloat16)
    refused(INVALID, w.moe_permute, x, i32(32), i32(1), 2, xp, i32(4, 2))  # not on a GPU
    refused(INVALID, w.moe_permute, x, i32(32), i32(1), 2, xp, i32(4, 3))
    refused(CAPACITY, w.moe_permute, x, i32(33), i32(1), 2, xp, i32(4, 2))
    refused(INVALID, w.moe_permute, x, i32(32), i32(1), 2, xp.float(), i32(4, 2))
    refused(INVALID, w.moe_permute, x, i32(32).long(), i32(1), 2, xp, i32(4, 2))
    refused(UNSUPPORTED, w.moe_permute, x.double(), i32(32), i32(1), 2, xp.double(), i32(4, 2))
    refused(INVALID, w.moe_permute_backward, xp, i32(4, 2), x)
    refused(INVALID, w.moe_permute_backward, xp, i32(5, 2), x)
    refused(INVALID, w.moe_unpermute, xp, i32(4, 2), x, topk_weights=torch.zeros(4, 3))
    refused(INVALID, w.moe_unpermute, xp, i32(4, 2), x, topk_weights=torch.zeros(4, 2, dtype=torch.bfloat16))
    refused(INVALID, w.moe_unpermute_backward, x, None, i32(4, 2), None, i32(32), i32(1), None, None)
    refused(INVALID, w.moe_unpermute_backward, x, None, i32(4, 2), None, i32(32), i32(1), xp, torch.zeros(4, 2))
    refused(INVALID, w.moe_unpermute_backward, x, xp, i32(4, 2), None, None, i32(1), xp, None)
    refused(INVALID, w.mxfp4_quantize, x, u8(4, 32), u8(4, 2))
    refused(INVALID, w.mxfp4_quantize, x, u8(4, 31), u8(4, 2))
    refused(UNSUPPORTED, w.mxfp4_quantize, x[:, :40], u8(4, 20), u8(4, 1))
    refused(INVALID, w.mxfp4_silu_mul_quantize, x, u8(4, 32), u8(4, 2))
    refused(INVALID, w.mxfp4_quantize, x, u8(4, 32), u8(4, 2), num_rows=i32(0))  # not "all rows"
    refused(INVALID, w.moe_permute, x, i32(32), i32(0), 2, xp, i32(4, 2))
    refused(INVALID, w.mxfp4_dequantize, u8(4, 32), u8(4, 3), x)
    refused(INVALID, w.mxfp4_repack, u8(2, 64, 32), u8(2, 64, 2), u8(10))
    packed = u8(w.mxfp4_packed_bytes(2, 64, 64))
    out = torch.zeros(32, 64)
    args = (u8(32, 32), u8(32, 2), 4, 2, i32(32), i32(2), i32(1), 16, 2)
    refused(INVALID, w.mxfp4_moe_gemm, *args, packed, out)
    refused(INVALID, w.mxfp4_moe_gemm, *args, packed[1:], out)
    refused(CAPACITY, w.mxfp4_moe_gemm, *args, packed, out[:31])
    refused(UNSUPPORTED, w.mxfp4_moe_gemm, *args, packed, out.double())
    refused(INVALID, w.mxfp4_moe_gemm, u8(32, 32), u8(32, 2), 4, 2, i32(32), i32(1), i32(1), 16, 2, packed, out)


BIG = 1 << 32  # a size of 2^32 + n is n in 32 bits


def test_binding_refuses_sizes_past_32_bits(lib):
    """A size that 32 bits do not hold is refused as the C ABI refuses one past its limits, not cut to its low
    bits. Tensors of the meta device have shapes only; a call that gets past the sizes says that they are on no GPU."""
    def meta(*shape, dtype=torch.bfloat16):
        return torch.empty(*shape, dtype=dtype, device="meta")

    i32 = lambda *shape: meta(*shape, dtype=torch.int32)  # noqa: E731
    u8 = lambda *shape: meta(*shape, dtype=torch.uint8)  # noqa: E731
    f32 = lambda *shape: meta(*shape, dtype=torch.float32)  # noqa: E731
    far, wide = BIG + 4, BIG + 64
    # hidden, tokens, capacity
    refused(UNSUPPORTED, w.moe_permute, meta(4, wide), i32(32), i32(1), 2, meta(32, wide), i32(4, 2))
    refused(UNSUPPORTED, w.moe_permute, meta(far, 64), i32(32), i32(1), 2, meta(32, 64), i32(far, 2))
    refused(UNSUPPORTED, w.moe_permute, meta(4, 64), i32(BIG + 32), i32(1), 2, meta(BIG + 32, 64), i32(4, 2))
    refused(UNSUPPORTED, w.moe_permute, meta(4, 64), i32(32), i32(1), BIG + 2, meta(32, 64), i32(4, BIG + 2))
    refused(UNSUPPORTED, w.moe_permute_backward, meta(BIG + 32, 64), i32(4, 2), meta(4, 64))
    refused(UNSUPPORTED, w.moe_permute_backward, meta(32, wide), i32(4, 2), meta(4, wide))
    refused(UNSUPPORTED, w.moe_unpermute, meta(BIG + 32, 64), i32(4, 2), meta(4, 64))
    refused(UNSUPPORTED, w.moe_unpermute, meta(32, 64), i32(far, 2), meta(far, 64))
    refused(UNSUPPORTED, w.moe_unpermute_backward, meta(4, 64), meta(BIG + 32, 64), i32(4, 2), None, i32(32), i32(1),
            meta(BIG + 32, 64), f32(4, 2))
    refused(UNSUPPORTED, w.moe_unpermute_backward, meta(4, wide), meta(32, wide), i32(4, 2), None, i32(32), i32(1),
            meta(32, wide), f32(4, 2))
    refused(UNSUPPORTED, w.moe_unpermute_backward, meta(4, 64), meta(32, 64), i32(4, 2), None, i32(BIG + 32), i32(1),
            meta(32, 64), f32(4, 2))
    for rows, K in [(far, 64), (4, wide)]:
        q, s = u8(rows, K // 2), u8(rows, K // 32)
        refused(UNSUPPORTED, w.mxfp4_quantize, meta(rows, K), q, s)
        refused(UNSUPPORTED, w.mxfp4_silu_mul_quantize, meta(rows, 2 * K), q, s)
        refused(UNSUPPORTED, w.mxfp4_dequantize, q, s, meta(rows, K))
    for E, N, K in [(BIG + 1, 64, 64), (1, wide, 64), (1, 64, wide)]:
        refused(UNSUPPORTED, w.mxfp4_packed_bytes, E, N, K)
        refused(UNSUPPORTED, w.mxfp4_repack, u8(E, N, K // 2), u8(E, N, K // 32), u8(1 << 40))
    good = dict(a_q=u8(32, 32), a_s=u8(32, 2), T=4, topk=2, sorted_token_ids=i32(32), expert_ids=i32(2),
                num_tokens_post_padded=i32(1), block_m=16, num_experts=2, packed=u8(1 << 40), out=f32(32, 64))
    refused(INVALID, w.mxfp4_moe_gemm, **good)  # on no GPU
    for change in (dict(a_q=u8(far, 32), a_s=u8(far, 2)), dict(a_q=u8(32, wide // 2), a_s=u8(32, wide // 32)),
                   dict(T=far), dict(topk=BIG + 2), dict(block_m=BIG + 16), dict(num_experts=BIG + 2),
                   dict(out=f32(32, wide)),
                   dict(sorted_token_ids=i32(BIG + 32), expert_ids=i32(BIG // 16 + 2), out=f32(BIG + 32, 64))):
        refused(UNSUPPORTED, w.mxfp4_moe_gemm, **{**good, **change})
    # what is too small stays an invalid argument
    for change in (dict(T=-BIG + 4), dict(topk=-BIG + 2), dict(num_experts=-BIG + 2)):
        refused(INVALID, w.mxfp4_moe_gemm, **{**good, **change})


def test_readme_example_makes_what_it_reads():
    """The README's 4-bit layer, with calls that only note their buffers: each buffer is the program's input or was
    written by an earlier call."""
    import os
    import re

    with open(os.path.join(os.path.dirname(__file__), "..", "README.md")) as f:
        code, = [c for c in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "mxfp4_moe_gemm" in c]
    made = {"topk_ids", "topk_weights", "x", "w13_packed", "w2_packed"}
    writes = {"moe_align": ("sorted_token_ids", "expert_ids", "num_tokens_post_padded", "workspace"),
              "moe_permute": ("xp", "slot_rows"), "mxfp4_quantize": ("q", "s"), "mxfp4_silu_mul_quantize": ("q", "s"),
              "mxfp4_moe_gemm": ("out",), "moe_unpermute": ("out",)}
    sizes = {"T": 4, "topk": 2, "E": 8, "bm": 16}

    class Calls:
        def __getattr__(self, name):
            import inspect

            def call(*args, **kw):
                given = inspect.signature(getattr(w, name)).bind(*args, **kw).arguments
                for k, v in given.items():
                    if isinstance(v, str) and k not in writes[name]:
                        assert v in made, f"{name} reads {v}, which no earlier call has written"
                made.update(given[k] for k in writes[name] if k in given)
            return call

    class Names(dict):
        def __missing__(self, name):
            return name

    exec(code, {}, Names(w=Calls(), **sizes))
    assert "out" in made
