"""The operators as they are used together: a layer encoded from bf16 weights (mxfp4_quantize), a
router's choice (expert_route), the routed 4-bit product over it (mxfp4_expert_gemm, TQ_FP4), and the
gradient of a loss of the outputs with respect to the router's logits (expert_route_backward)."""

import numpy as np
import pytest

import oracle
from gpu_helpers import dev, gpu, needs_gpu, ops, to_dev, torch
from workloads import bf16_from_normal, rng_for

pytestmark = [gpu, needs_gpu]


def encode(o, w_bits):
    """An expert layer from bf16 weights [E, out, in]: each expert's codes, then its scales."""
    E, out, in_ = w_bits.shape
    size = out * in_ // 2
    units = torch.empty((E, size + out * in_ // 32), dtype=torch.uint8, device=dev())
    for e in range(E):
        o.mxfp4_quantize(to_dev(w_bits[e], np.int16), codes=units[e, :size].view(out, in_ // 2),
                         scales=units[e, size:].view(out, in_ // 32))
    return o.Mxfp4Layer(E, out, in_, units.view(-1))


@pytest.mark.parametrize("T,score,renorm", [(1, "softmax", True), (48, "sigmoid", True), (48, "softmax", False),
                                            (300, "sigmoid", True)])
def test_router_to_experts_and_back(T, score, renorm):
    o = ops()
    E, topk, out, in_ = 12, 3, 144, 512
    w_bits = bf16_from_normal(rng_for(950, 0), (E, out, in_))
    x_bits = bf16_from_normal(rng_for(950, 1), (T, in_))
    logits = torch.from_numpy(rng_for(950, 2).standard_normal((T, E)).astype(np.float32))
    if T > 8:
        logits[-3:] = -float("inf")  # padded tokens
    layer = encode(o, w_bits)
    R = o.Router(E, topk, score=score, renorm=renorm, scale=1.5)
    flags = o.TQ_FP4
    ws = o.workspace(T, topk, E, out, in_, flags)
    x, z = to_dev(x_bits, np.int16), logits.to(dev())
    dy_h = rng_for(950, 3).standard_normal((T, out)).astype(np.float32)
    dy = to_dev(dy_h)
    ids, w = o.expert_route(R, z)
    dz = torch.empty_like(z)
    slots = torch.empty((T, topk, out), device=dev())

    def step():
        o.expert_route(R, z, ids=ids, w=w)
        o.mxfp4_expert_gemm(layer, x, ids, None, flags=flags, out=slots, ws=ws)
        y = (slots * w[:, :, None]).sum(1)
        dw = (slots * dy[:, None]).sum(2)
        o.expert_route_backward(R, z, ids, dw, dlogits=dz)
        return y

    y = step()
    xq = oracle.mxfp4_values(*oracle.mxfp4_quantize(x_bits))
    wq = [oracle.mxfp4_values(*oracle.mxfp4_quantize(w_bits[e])) for e in range(E)]
    kw = dict(score=score, renorm=renorm, scale=1.5)
    want_ids, want_w = oracle.expert_route(logits.numpy(), topk, **kw)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    s = oracle.expert_gemm_values(xq, want_ids, None, E, lambda e: wq[e])
    want_y = (s * want_w[:, :, None]).sum(1)
    want_dz = oracle.expert_route_backward(logits.numpy(), want_ids, (s * dy_h[:, None]).sum(2), **kw)
    # sums of at most 512 fp32 terms of both signs, each off by some 2^-24: far within 1e-5 in the 2-norm
    for got, want in ((y, want_y), (dz, want_dz)):
        assert np.linalg.norm(got.cpu().numpy() - want) <= 1e-5 * np.linalg.norm(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o.expert_route(R, z, ids=ids, w=w)
        o.mxfp4_expert_gemm(layer, x, ids, w, flags=flags, out=slots, ws=ws)
    for k in range(3):  # replays with other logits, the program's own work between them
        z.copy_(torch.from_numpy(rng_for(951, k).standard_normal((T, E)).astype(np.float32)))
        graph.replay()
        i, v = o.expert_route(R, z)
        want = o.mxfp4_expert_gemm(layer, x, i, v, flags=flags)
        torch.cuda.synchronize()
        assert torch.equal(slots, want) and torch.equal(ids, i)


def test_routes_of_more_slots_than_fit_one_grid():
    """2^29 slots and more: the placement's workgroups of 32 slots would be more than 2^32 threads."""
    o = ops()
    T, topk, E = (1 << 23) + 3, 64, 5
    N = T * topk
    ids = (torch.arange(N, device=dev()) % E).int()
    ids[N - 7] = -1
    counts, offsets, pairs = o.route_bucket(ids.view(T, topk), E)
    gone = (N - 7) % E
    for e in range(E):
        want = torch.arange(e, N, E, device=dev(), dtype=torch.int32)
        want = want[want != N - 7] if e == gone else want
        assert int(counts[e]) == want.numel()
        assert torch.equal(pairs[int(offsets[e]):int(offsets[e + 1])], want)
