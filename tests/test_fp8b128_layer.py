"""Fp8b128Layer keeps what it found out about its two tensors between calls. A tensor that has
been changed in place (resize_, t_, set_, an assignment to .data), also where its memory stays
where it was, has to be followed or refused. On the host: the tensors only say that they are on
the GPU, and nothing is launched."""

import pytest

torch = pytest.importorskip("torch")
from trellis_quantized_moe_amd import ops  # noqa: E402


class OnGpu(torch.Tensor):
    is_cuda = True


def layer(out=96, in_=272):
    codes = torch.zeros((out, in_), dtype=torch.uint8).as_subclass(OnGpu)
    scales = torch.ones((-(-out // 128), -(-in_ // 128))).as_subclass(OnGpu)
    return ops.Fp8b128Layer(codes, scales)


def found(L):
    """What the next call uses."""
    L.renew()
    assert (L._c.out, L._c.in_) == (L.out, L.in_) and L.blocks == -(-L.in_ // 128)
    assert L._c.codes == L.codes.data_ptr() and L._c.scales == L.scales.data_ptr()
    return L.out, L.in_


def resized(L):
    L.codes.resize_(64, 272)


def sliced(L):
    L.codes.data = L.codes.data[:64]


def smaller_at_the_same_address(L):  # as when the old memory is freed and allocated again
    L.codes.set_(L.codes.untyped_storage(), 0, (64, 272), (272, 1))


@pytest.mark.parametrize("change", [resized, sliced, smaller_at_the_same_address])
def test_fewer_outputs_are_followed(change):
    L = layer()
    at = L.codes.data_ptr()
    assert found(L) == (96, 272)
    change(L)
    assert L.codes.data_ptr() == at
    assert found(L) == (64, 272)


def test_another_shape_of_the_same_memory_is_followed():
    L = layer()
    L.codes.data, L.scales.data = L.codes.data.view(272, 96), L.scales.data.view(3, 1)
    assert found(L) == (272, 96)


@pytest.mark.parametrize("change", [
    lambda L: L.codes.t_(),
    lambda L: L.codes.resize_(96, 256),                              # two blocks, three scales
    lambda L: setattr(L.codes, "data", L.codes.data.view(272, 96)),
    lambda L: setattr(L.codes, "data", L.codes.data[:, :256]),       # rows with gaps
    lambda L: setattr(L.codes, "data", L.codes.data.view(torch.float8_e5m2)),
    lambda L: setattr(L.codes, "data", L.codes.data.view(-1)),
    lambda L: L.scales.t_(),
    lambda L: L.scales.resize_(1, 2),
    lambda L: setattr(L.scales, "data", L.scales.data.view(torch.int32)),
])
def test_what_no_longer_fits_is_refused(change):
    L = layer()
    at = L.codes.data_ptr(), L.scales.data_ptr()
    change(L)
    assert (L.codes.data_ptr(), L.scales.data_ptr()) == at
    for _ in range(2):  # not only once
        with pytest.raises(ValueError):
            L.renew()


def test_square_codes_transposed_in_place_are_refused():
    L = layer(128, 128)  # the same shape afterwards
    L.codes.t_()
    with pytest.raises(ValueError):
        L.renew()


def test_a_tensor_on_another_device_is_found(monkeypatch):
    L = layer()
    monkeypatch.setattr(OnGpu, "device", torch.device("cuda", 1), raising=False)
    L.renew()
    assert L.device == torch.device("cuda", 1)
