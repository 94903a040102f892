"""mxfp4_quantize on the GPU (FORMAT F29): codes and scales bit for bit as the oracle's, the unit
they make, and the memory around it."""

import numpy as np
import pytest

import oracle
from gpu_helpers import dev, gpu, needs_gpu, ops, to_dev, torch
from workloads import bf16_from_normal, rng_for

pytestmark = [gpu, needs_gpu]


def check(x):
    codes, scales = ops().mxfp4_quantize(to_dev(x, np.int16))
    want_codes, want_scales = oracle.mxfp4_quantize(x)
    assert np.array_equal(scales.cpu().numpy(), want_scales)
    assert np.array_equal(codes.cpu().numpy(), oracle.mxfp4_pack(want_codes))


@pytest.mark.parametrize("rows,n", [(1, 32), (1, 96), (3, 64), (7, 544), (64, 5120), (129, 1056), (1000, 32),
                                    (2, 1 << 20)])
def test_rows(rows, n):
    check(bf16_from_normal(rng_for(920, rows), (rows, n)))


def test_every_bf16_pattern_in_blocks_of_every_exponent():
    """Each pattern is the largest of a block, and a small one beside a larger one."""
    p = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    x = np.zeros((65536, 32), dtype=np.uint16)
    x[:, 7] = p
    x[:, 20] = p ^ 0x8000
    x[:, 31] = np.where(p & 0x7F80, p - 0x80, p)
    with np.errstate(invalid="ignore"):
        check(x)
    y = np.zeros((65536, 32), dtype=np.uint16)
    y[:, 0] = p
    y[:, 31] = np.random.default_rng(3).integers(0, 0x7F80, 65536).astype(np.uint16)
    check(y)


def test_ties_and_borders():
    borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0], dtype=np.float32)
    rows = []
    for k in (-126, -100, -3, 0, 5, 100, 120):
        v = np.zeros(32, dtype=np.float32)
        v[0] = 7.0
        v[1:10], v[10:19] = borders, -borders
        v[20] = -0.0
        rows.append(np.ldexp(v, k).astype(np.float32).view(np.uint32) >> 16)
    check(np.array(rows).astype(np.uint16))


def test_the_unit_reads_back():
    o = ops()
    x = bf16_from_normal(rng_for(921, 0), (48, 512))
    size = 48 * 256
    unit = torch.full((size + 48 * 16 + 64,), 0xAB, dtype=torch.uint8, device=dev())
    o.mxfp4_quantize(to_dev(x, np.int16), codes=unit[:size].view(48, 256), scales=unit[size:size + 48 * 16].view(48, 16))
    assert torch.all(unit[-64:] == 0xAB)
    w = o.mxfp4_decode(unit[:size + 48 * 16], 48, 512).cpu().numpy().view(np.uint16)
    want = oracle.mxfp4_values(*oracle.mxfp4_quantize(x))
    assert np.array_equal(oracle.bf16_bits_to_f64(w), want)


def test_wrapper_refusals():
    o = ops()
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device=dev())
    for bad in (x.float(), x.t(), x[:, ::2], x[0]):
        with pytest.raises(ValueError):
            o.mxfp4_quantize(bad)
    with pytest.raises(ValueError):
        o.mxfp4_quantize(x, codes=torch.zeros((4, 64), dtype=torch.uint8, device=dev()))
    with pytest.raises(ValueError):
        o.mxfp4_quantize(x, scales=torch.zeros((4, 2), dtype=torch.int8, device=dev()))
    with pytest.raises(Exception, match="multiple of 32"):
        o.mxfp4_quantize(x[:, :48].contiguous())


def test_no_rows():
    codes, scales = ops().mxfp4_quantize(torch.zeros((0, 64), dtype=torch.bfloat16, device=dev()))
    assert codes.shape == (0, 32) and scales.shape == (0, 2)


def test_offsets_past_32_bits():
    rows = (1 << 31) // 8192 + 3
    x = torch.zeros((rows, 8192), dtype=torch.bfloat16, device=dev())
    x[-1, -32:] = 3.0
    codes, scales = ops().mxfp4_quantize(x)
    assert codes[-1, -16:].tolist() == [0x77] * 16 and scales[-1, -1].item() == 126
    assert codes[:-1].max().item() == 0 and codes[-1, :-16].max().item() == 0
    assert torch.all(scales[:-1] == 127) and torch.all(scales[-1, :-1] == 127)


def test_replayed_graph():
    x = to_dev(bf16_from_normal(rng_for(922, 0), (33, 256)), np.int16).view(torch.bfloat16)
    codes, scales = ops().mxfp4_quantize(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops().mxfp4_quantize(x, codes=codes, scales=scales)
    for k in range(3):
        x.mul_(1.37)
        graph.replay()
        torch.cuda.synchronize()
        c, s = ops().mxfp4_quantize(x)
        assert torch.equal(c, codes) and torch.equal(s, scales)
