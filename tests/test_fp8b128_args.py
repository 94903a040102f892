"""Refusals of the fp8b128 calls (FORMAT F22-F26) on the host: the C ABI's argument checks, all
of which come before the first HIP call, and the Python wrappers' checks of tensors."""

import ctypes

import pytest

tq = pytest.importorskip("trellis_quantized_moe_amd")
from trellis_quantized_moe_amd import _lib  # noqa: E402

P = 0x10000
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def layer(out=256, inp=512, codes=P, scales=P):
    return _lib.Fp8b128LayerC(out, inp, codes, scales)


def calls(lib, L, T=3, xq=P, xs=P, y=P, d=P, dx=P, dw=P, ws=P, ws_bytes=BIG, flags=0):
    """Each products call with the same arguments, by name."""
    r = ctypes.byref(L) if L is not None else None
    return {
        "gemm": lib.fp8b128_gemm(r, xq, xs, T, y, flags, None),
        "gated": lib.fp8b128_gated(r, xq, xs, T, y, None),
        "gemm_backward": lib.fp8b128_gemm_backward(r, xq, xs, T, d, dx, dw, ws, ws_bytes, None),
        "gated_backward": lib.fp8b128_gated_backward(r, xq, xs, T, d, dx, dw, ws, ws_bytes, None),
    }


@pytest.mark.parametrize("bad,code", [
    (None, _lib.TQ_EINVAL),
    (layer(out=0), _lib.TQ_EINVAL), (layer(out=-16), _lib.TQ_EINVAL), (layer(out=24), _lib.TQ_EINVAL),
    (layer(out=(1 << 20) + 16, inp=16), _lib.TQ_EINVAL),
    (layer(inp=0), _lib.TQ_EINVAL), (layer(inp=520), _lib.TQ_EINVAL),
    (layer(out=16, inp=(1 << 20) + 16), _lib.TQ_EINVAL),
    (layer(out=1 << 16, inp=1 << 15), _lib.TQ_EINVAL),      # out * in = 2^31
    (layer(codes=0), _lib.TQ_EINVAL), (layer(scales=0), _lib.TQ_EINVAL),
    (layer(codes=P + 8), _lib.TQ_EALIGN), (layer(scales=P + 2), _lib.TQ_EALIGN),
])
def test_bad_layers(lib, bad, code):
    for name, rc in calls(lib, bad).items():
        assert rc == code, name


@pytest.mark.parametrize("kw,code", [
    ({"T": -1}, _lib.TQ_EINVAL), ({"T": 1 << 33}, _lib.TQ_EINVAL), ({"T": (1 << 24) + 1}, _lib.TQ_EINVAL),
    ({"xq": 0}, _lib.TQ_EINVAL), ({"xs": 0}, _lib.TQ_EINVAL),
    ({"xq": P + 8}, _lib.TQ_EALIGN), ({"xs": P + 1}, _lib.TQ_EALIGN),
    ({"y": 0, "d": 0}, _lib.TQ_EINVAL), ({"y": P + 8, "d": P + 8}, _lib.TQ_EALIGN),
])
def test_bad_arguments(lib, kw, code):
    for name, rc in calls(lib, layer(), **kw).items():
        assert rc == code, name


def test_bad_flags_and_shapes(lib):
    for flags in (1, 2, 4, 16, 64, 33):
        assert calls(lib, layer(), flags=flags)["gemm"] == _lib.TQ_EINVAL
    odd = layer(out=48)  # I = 24 is not a multiple of 16
    got = calls(lib, odd, T=0, xq=0, xs=0, y=0, d=0, dx=0, ws=0)
    assert got["gated"] == got["gated_backward"] == _lib.TQ_EINVAL
    assert got["gemm"] == _lib.TQ_OK


def test_backward_arguments(lib):
    for name in ("gemm_backward", "gated_backward"):
        assert calls(lib, layer(), dx=0, dw=0)[name] == _lib.TQ_EINVAL
        assert calls(lib, layer(), dx=P + 8)[name] == _lib.TQ_EALIGN
        assert calls(lib, layer(), dw=P + 4)[name] == _lib.TQ_EALIGN
        assert calls(lib, layer(), ws=0)[name] == _lib.TQ_EWORKSPACE
        assert calls(lib, layer(), ws=P + 64)[name] == _lib.TQ_EALIGN
        need = lib.tq_fp8b128_workspace_bytes(3, 256, 512)
        assert calls(lib, layer(), ws_bytes=need - 1)[name] == _lib.TQ_EWORKSPACE
    assert lib.tq_fp8b128_workspace_bytes(-1, 256, 512) == 0
    assert lib.tq_fp8b128_workspace_bytes(3, 0, 512) == 0
    assert lib.tq_fp8b128_workspace_bytes(3, 256, 8) == 0


def test_no_tokens_is_a_no_op(lib):
    got = calls(lib, layer(), T=0, xq=0, xs=0, y=0, d=0, dx=P, dw=0, ws=0, ws_bytes=0)
    assert set(got.values()) == {_lib.TQ_OK}
    assert lib.fp8b128_quantize(0, 0, 128, 0, 0, None) == _lib.TQ_OK
    g, d = layer(), layer(out=512, inp=128)
    assert lib.fp8b128_ffn(ctypes.byref(g), ctypes.byref(d), 0, 0, 0, 0, 0, 0, None) == _lib.TQ_OK


def test_quantize_arguments(lib):
    q = lib.fp8b128_quantize
    for rows, n in ((-1, 128), (4, 0), (4, -16), (4, 24), (4, (1 << 20) + 16), (1 << 24, 1 << 10),
                    # a block of 128 has its threads however few inputs it holds
                    ((1 << 26) + 1, 16), ((1 << 25) + 1, 144)):
        assert q(P, rows, n, P, P, None) == _lib.TQ_EINVAL, (rows, n)
    assert q(0, 4, 128, P, P, None) == _lib.TQ_EINVAL
    assert q(P, 4, 128, 0, P, None) == _lib.TQ_EINVAL
    assert q(P, 4, 128, P, 0, None) == _lib.TQ_EINVAL
    assert q(P + 8, 4, 128, P, P, None) == _lib.TQ_EALIGN
    assert q(P, 4, 128, P + 8, P, None) == _lib.TQ_EALIGN
    assert q(P, 4, 128, P, P + 2, None) == _lib.TQ_EALIGN


def test_ffn_arguments(lib):
    def ffn(g, d, x=P, T=2, y=P, flags=0, ws=P, nbytes=BIG):
        return lib.fp8b128_ffn(ctypes.byref(g), ctypes.byref(d), x, T, y, flags, ws, nbytes, None)
    g, d = layer(), layer(out=512, inp=128)
    assert ffn(layer(out=48), layer(out=512, inp=32)) == _lib.TQ_EINVAL
    assert ffn(g, layer(out=512, inp=256)) == _lib.TQ_EINVAL
    assert ffn(g, layer(out=256, inp=128)) == _lib.TQ_EINVAL
    assert ffn(g, d, flags=4) == _lib.TQ_EINVAL
    assert ffn(g, d, x=0) == _lib.TQ_EINVAL and ffn(g, d, y=0) == _lib.TQ_EINVAL
    assert ffn(g, d, x=P + 2) == _lib.TQ_EALIGN
    assert ffn(g, d, T=-1) == _lib.TQ_EINVAL
    assert ffn(g, d, ws=0) == _lib.TQ_EWORKSPACE
    need = lib.tq_fp8b128_ffn_workspace_bytes(2, 512, 128)
    assert ffn(g, d, nbytes=need - 1) == _lib.TQ_EWORKSPACE
    assert lib.tq_fp8b128_ffn_workspace_bytes(-1, 512, 128) == 0
    for T in ((1 << 24) + 1, 1 << 62):  # more than a call takes
        assert lib.tq_fp8b128_ffn_workspace_bytes(T, 512, 128) == 0
        assert lib.tq_fp8b128_workspace_bytes(T, 512, 128) == 0
    assert lib.tq_fp8b128_workspace_bytes(4, 512, 1 << 21) == 0


def test_wrappers_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    from trellis_quantized_moe_amd import ops
    with pytest.raises(ValueError, match="on the GPU"):
        ops.fp8b128_quantize(torch.zeros((2, 128), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="on the GPU"):
        ops.Fp8b128Layer(torch.zeros((16, 128), dtype=torch.uint8), torch.ones((1, 1)))
