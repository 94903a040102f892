"""Fp8b128Layer through the calls, after its tensors have been changed in place: what the call
gives is what a new layer over the same tensors gives, or it is refused."""

import pytest

from gpu_helpers import dev, gpu, needs_gpu, ops, to_dev, torch
from workloads import bf16_from_normal, fp8b128_layer, rng_for

pytestmark = [gpu, needs_gpu]


def tensors(seed, out, in_):
    host = fp8b128_layer(seed, out, in_)
    return to_dev(host["codes"]), to_dev(host["scales"])


def activations(T, in_):
    x = to_dev(bf16_from_normal(rng_for(1000, 3, T, in_), (T, in_)).view("int16")).view(torch.bfloat16)
    return ops().fp8b128_quantize(x)


def all_calls(L, x, dy):
    o = ops()
    return (o.fp8b128_gemm(L, *x), o.fp8b128_gated(L, *x), *o.fp8b128_gemm_backward(L, *x, dy),
            *o.fp8b128_gated_backward(L, *x, dy[:, :L.codes.shape[0] // 2].contiguous()))


def check_follows(L, T):
    """Every call over L gives what it gives over a new layer of the same tensors."""
    out, in_ = L.codes.shape
    x = activations(T, in_)
    dy = torch.randn((T, out), device=dev()).bfloat16()
    for a, b in zip(all_calls(L, x, dy), all_calls(ops().Fp8b128Layer(L.codes, L.scales), x, dy)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [1, 5, 300])
def test_changes_at_the_same_address_are_followed(T):
    L = ops().Fp8b128Layer(*tensors(1001, 96, 272))
    check_follows(L, T)
    at = L.codes.data_ptr()
    L.codes.data = L.codes.data[:64]
    check_follows(L, T)
    L.codes.resize_(32, 272)
    check_follows(L, T)
    L.codes.data, L.scales.data = L.codes.data.view(544, 16), torch.ones((5, 1), device=dev())
    check_follows(L, T)
    assert L.codes.data_ptr() == at


def test_a_smaller_tensor_in_freed_memory_is_followed():
    o = ops()
    codes, scales = tensors(1002, 512, 2048)
    L = o.Fp8b128Layer(codes, scales)
    x = activations(4, 2048)
    o.fp8b128_gemm(L, *x)
    at = codes.data_ptr()
    empty = torch.empty(0, dtype=torch.uint8, device=dev())
    small, small_scales = tensors(1003, 64, 400)
    L.codes.data, L.scales.data = empty, torch.empty(0, device=dev())  # frees the old memory
    del codes, scales
    for _ in range(64):  # the caching allocator gives a block of the freed size back
        again = torch.empty((512, 2048), dtype=torch.uint8, device=dev())
        if again.data_ptr() == at:
            break
    L.codes.data = again.view(-1)[:64 * 400].view(64, 400)
    L.codes.copy_(small)
    L.scales.data = small_scales
    check_follows(L, 4)
    with pytest.raises(ValueError):
        o.fp8b128_gemm(L, *x)  # fitted the old tensors


def test_transposed_in_place_is_refused_by_every_call():
    o = ops()
    L = o.Fp8b128Layer(*tensors(1004, 128, 128))
    x, dy = activations(3, 128), torch.zeros((3, 128), dtype=torch.bfloat16, device=dev())
    down = o.Fp8b128Layer(*tensors(1005, 128, 64))
    all_calls(L, x, dy)
    L.codes.t_()
    for call in (lambda: o.fp8b128_gemm(L, *x), lambda: o.fp8b128_gated(L, *x),
                 lambda: o.fp8b128_gemm_backward(L, *x, dy),
                 lambda: o.fp8b128_gated_backward(L, *x, dy[:, :64].contiguous()),
                 lambda: o.fp8b128_ffn(L, down, dy)):
        with pytest.raises(ValueError):
            call()
    L.codes.t_()
    check_follows(L, 3)
