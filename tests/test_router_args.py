"""Refusals of the router calls, the MXFP4 quantizer and TQ_FP4, on made-up addresses: every call
made here is refused, or has nothing to do, before the library's first HIP call, so it is safe
with a GPU too."""

import ctypes
import math

import pytest

tq = pytest.importorskip("trellis_quantized_moe_amd")
from trellis_quantized_moe_amd import _lib  # noqa: E402

P = 0x10000
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def router(**kw):
    f = dict(E=64, topk=4, score=0, groups=1, group_topk=1, group_top=1, renorm=1, scale=1.0, bias=None)
    f.update(kw)
    return _lib.RouterC(**f)


def route(lib, R, logits=P, T=3, ids=P, w=P, flags=0):
    return lib.expert_route(ctypes.byref(R) if R else None, logits, T, ids, w, flags, None)


def backward(lib, R, logits=P, T=3, ids=P, dw=P, dx=P, flags=0):
    return lib.expert_route_backward(ctypes.byref(R) if R else None, logits, T, ids, dw, dx, flags, None)


BAD = [dict(E=0), dict(E=4097), dict(topk=0), dict(topk=65, E=128), dict(topk=65), dict(score=2),
       dict(score=-1), dict(groups=0), dict(groups=3), dict(groups=128, E=128), dict(groups=4, group_topk=0),
       dict(groups=4, group_topk=5), dict(group_topk=2), dict(group_top=0), dict(group_top=3), dict(renorm=2),
       dict(groups=16, group_topk=1, topk=5), dict(scale=math.inf), dict(scale=math.nan)]


@pytest.mark.parametrize("kw", BAD)
@pytest.mark.parametrize("T", [0, 3])
def test_routers(lib, kw, T):
    for fn in (route, backward):
        assert fn(lib, router(**kw), T=T) == _lib.TQ_EINVAL
        assert lib.tq_last_error()


@pytest.mark.parametrize("fn", [route, backward])
def test_calls(lib, fn):
    R = router()
    assert fn(lib, None) == _lib.TQ_EINVAL
    assert fn(lib, R, T=-1) == _lib.TQ_EINVAL
    assert fn(lib, R, T=(1 << 33) // 64 + 1) == _lib.TQ_EINVAL
    assert fn(lib, R, logits=None) == _lib.TQ_EINVAL
    assert fn(lib, R, logits=P + 2) == _lib.TQ_EALIGN
    assert fn(lib, R, logits=P + 1, flags=_lib.TQ_LOGITS_BF16) == _lib.TQ_EALIGN
    assert fn(lib, R, ids=None) == _lib.TQ_EINVAL
    assert fn(lib, R, ids=P + 2) == _lib.TQ_EALIGN
    assert fn(lib, router(bias=P + 2)) == _lib.TQ_EALIGN
    for flags in (2, 4, 16, 64, 3):
        assert fn(lib, R, flags=flags) == _lib.TQ_EINVAL
    assert fn(lib, R, T=0, logits=None, ids=None) == _lib.TQ_OK


def test_outputs(lib):
    R = router()
    assert route(lib, R, w=None) == _lib.TQ_EINVAL
    assert route(lib, R, w=P + 2) == _lib.TQ_EALIGN
    assert backward(lib, R, dw=None) == _lib.TQ_EINVAL
    assert backward(lib, R, dw=P + 1) == _lib.TQ_EALIGN
    assert backward(lib, R, dx=None) == _lib.TQ_EINVAL
    assert backward(lib, R, dx=P + 2) == _lib.TQ_EALIGN
    assert backward(lib, R, dx=P + 1, flags=_lib.TQ_LOGITS_BF16) == _lib.TQ_EALIGN


def test_quantize(lib):
    def call(x=P, rows=3, n=64, codes=P, scales=P):
        return lib.mxfp4_quantize(x, rows, n, codes, scales, None)
    for kw in (dict(rows=-1), dict(n=0), dict(n=48), dict(n=-32), dict(n=(1 << 20) + 32),
               dict(rows=(1 << 33) // 64 + 1), dict(x=None), dict(codes=None), dict(scales=None)):
        assert call(**kw) == _lib.TQ_EINVAL, kw
    for kw in (dict(x=P + 8), dict(codes=P + 8)):
        assert call(**kw) == _lib.TQ_EALIGN, kw
    assert call(rows=0, x=None, codes=None, scales=None) == _lib.TQ_OK


FP4 = _lib.TQ_FP4


def experts(lib, fn="mxfp4_expert_gemm", E=4, out=128, in_=1024, flags=FP4, T=3, topk=2, ws=P, ws_bytes=BIG,
            ids=P, x=P, y=P):
    L = _lib.Mxfp4LayerC(E, out, in_, 0, P)
    return getattr(lib, fn)(ctypes.byref(L), x, T, ids, None, topk, y, flags, ws, ws_bytes, None)


def test_fp4_flags(lib):
    assert experts(lib, flags=FP4 | _lib.TQ_FP8) == _lib.TQ_EINVAL
    assert experts(lib, flags=FP4 | _lib.TQ_ROTATE) == _lib.TQ_EINVAL
    assert experts(lib, flags=FP4 | 3) == _lib.TQ_EINVAL
    assert experts(lib, flags=FP4 | 32) == _lib.TQ_EINVAL
    assert experts(lib, flags=FP4 | 128) == _lib.TQ_EINVAL
    assert experts(lib, fn="fp8b32_expert_gemm") == _lib.TQ_EINVAL
    T = _lib.TrellisLayerC(4, 128, 1024, 0, P, P, P, P, None, 1 << 30, None, 0)
    assert lib.trellis_expert_gemm(ctypes.byref(T), P, 3, P, None, 2, P, FP4, P, BIG, None) == _lib.TQ_EINVAL
    assert b"TQ_FP4" in lib.tq_last_error()
    assert lib.trellis_expert_ffn(ctypes.byref(T), ctypes.byref(T), P, 3, P, None, 2, P, FP4, P, BIG,
                                  None) == _lib.TQ_EINVAL


def test_fp4_sizes(lib):
    assert experts(lib, in_=768) == _lib.TQ_EINVAL
    assert experts(lib, out=24) == _lib.TQ_EINVAL
    assert experts(lib, T=1 << 24, topk=1) == _lib.TQ_EINVAL
    for mode in (0, _lib.TQ_GEMM):
        assert experts(lib, T=1 << 20, topk=1, flags=FP4 | mode) == _lib.TQ_EINVAL
        assert b"2^30" in lib.tq_last_error()
    assert experts(lib, topk=65) == _lib.TQ_EINVAL
    assert experts(lib, ids=None) == _lib.TQ_EINVAL
    assert experts(lib, x=P + 8) == _lib.TQ_EALIGN
    assert experts(lib, y=P + 8) == _lib.TQ_EALIGN
    assert experts(lib, T=0, x=None, y=None, ids=None, ws=None) == _lib.TQ_OK


def test_fp4_decode_batches_are_small(lib):
    assert experts(lib, T=513, topk=2, flags=FP4 | _lib.TQ_GEMV) == _lib.TQ_EINVAL
    assert b"1024" in lib.tq_last_error()
    assert lib.tq_workspace_bytes(512, 2, 4, 128, 1024, FP4 | _lib.TQ_GEMV) == 256
    assert experts(lib, T=512, topk=2, flags=FP4 | _lib.TQ_GEMV, ws_bytes=255) == _lib.TQ_EWORKSPACE


@pytest.mark.parametrize("mode", [0, _lib.TQ_GEMM])
def test_fp4_workspace(lib, mode):
    for extra in (0, _lib.TQ_COMBINE):
        flags = FP4 | mode | extra
        need = lib.tq_workspace_bytes(300, 2, 4, 128, 1024, flags)
        assert need >= 300 * (512 + 32)
        assert experts(lib, T=300, flags=flags, ws_bytes=need - 1) == _lib.TQ_EWORKSPACE
        assert experts(lib, T=300, flags=flags, ws=None) == _lib.TQ_EWORKSPACE
        assert experts(lib, T=300, flags=flags, ws=P + 128) == _lib.TQ_EALIGN


def test_python_refusals():
    torch = pytest.importorskip("torch")
    from trellis_quantized_moe_amd import ops
    with pytest.raises(ValueError, match="softmax"):
        ops.Router(8, 2, score="tanh")
    with pytest.raises(ValueError, match="GPU"):
        ops.Router(8, 2, bias=torch.zeros(8))
    with pytest.raises(ValueError, match="GPU"):
        ops.expert_route(ops.Router(8, 2), torch.zeros(3, 8))
    with pytest.raises(ValueError, match="GPU"):
        ops.mxfp4_quantize(torch.zeros(3, 64, dtype=torch.bfloat16))
