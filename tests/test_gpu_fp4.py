"""mxfp4_expert_gemm with TQ_FP4 (FORMAT F30) against the FP64 product of the oracle's MXFP4 values.

Tolerance, per output: a block's sum is exact; each of the in / 32 sums added, and each of the
partial sums that a split of the inputs adds (fewer than those), is rounded or cut, so off by at
most 2^-23 of the sum of magnitudes A = |X| |W|^T; the gate rounds by 2^-24, and the combine adds
topk such values: (in / 16 + topk + 2) * 2^-23 * A, gates applied."""

import numpy as np
import pytest

import oracle
from gpu_helpers import dev, gpu, mxfp4_weight_fn, needs_gpu, ops, to_dev, torch
from workloads import bf16_from_normal, mxfp4_layer, rng_for, softmax_gates, uniform_routes

pytestmark = [gpu, needs_gpu]


def reference(layer, x_bits, ids, gates):
    """(outputs, sums of magnitudes) [T, topk, out] in FP64."""
    xq = oracle.mxfp4_values(*oracle.mxfp4_quantize(x_bits))
    w = mxfp4_weight_fn(layer)
    g = None if gates is None else np.abs(gates)
    y = oracle.expert_gemm_values(xq, ids, gates, layer["E"], w)
    a = oracle.expert_gemm_values(np.abs(xq), ids, g, layer["E"], lambda e: np.abs(w(e)))
    return y, a


def compare(got, y, a, in_, topk, combine):
    got = got.cpu().numpy().astype(np.float64)
    if combine:
        y, a = y.sum(1), a.sum(1)
    bad = np.isnan(y)
    assert np.array_equal(np.isnan(got), bad)
    bound = (in_ / 16 + topk + 2) * 2.0 ** -23 * a
    assert np.all(np.abs(got - y)[~bad] <= bound[~bad])


def case(seed, E, T, topk, out, in_, empty=True):
    layer = mxfp4_layer(seed, E, out, in_)
    x = bf16_from_normal(rng_for(seed, 1), (T, in_))
    ids = uniform_routes(rng_for(seed, 2), T, E, topk)
    if empty and T > 2:
        ids[1, :] = -1
        ids[2, -1] = -1
    return layer, x, ids, softmax_gates(rng_for(seed, 3), T, topk)


# (E, T, topk, out, in): one token to more rows than an item of every kernel, out below, at and past
# a group of 128, rows and channels that end inside tiles, few and many experts
SIZES = [(1, 1, 1, 16, 512), (1, 1, 1, 128, 5120), (8, 1, 4, 144, 1024), (8, 1, 8, 1536, 2560), (5, 2, 3, 48, 512),
         (60, 3, 6, 1424, 512), (4, 7, 2, 128, 1536), (7, 17, 3, 272, 1024), (3, 31, 2, 400, 512),
         (16, 33, 4, 128, 2560), (6, 64, 6, 96, 1024), (64, 64, 8, 128, 1024), (2, 65, 1, 112, 512),
         (1, 129, 1, 256, 1024), (5, 130, 5, 384, 512), (2, 257, 2, 144, 1536), (3, 300, 2, 528, 1024),
         (1, 513, 1, 1040, 512), (4, 700, 3, 256, 512), (9, 1100, 4, 160, 512), (40, 600, 8, 128, 512)]


@pytest.mark.parametrize("E,T,topk,out,in_", SIZES)
@pytest.mark.parametrize("repack", [False, True])
def test_sizes(E, T, topk, out, in_, repack):
    o = ops()
    layer, x, ids, gates = case(930 + T, E, T, topk, out, in_)
    L = o.Mxfp4Layer.from_host(layer)
    L = L.repacked() if repack else L
    y, a = reference(layer, x, ids, gates)
    xd, idd, gd = to_dev(x, np.int16), to_dev(ids), to_dev(gates)
    for mode in (o.TQ_AUTO, o.TQ_GEMM, o.TQ_GEMV):
        if mode == o.TQ_GEMV and T * topk > 1024:
            continue
        for combine in (0, o.TQ_COMBINE):
            flags = o.TQ_FP4 | mode | combine
            guard = torch.full((T + 2,) + ((out,) if combine else (topk, out)), 7.0, device=dev())
            o.mxfp4_expert_gemm(L, xd, idd, gd, flags=flags, out=guard[1:-1])
            compare(guard[1:-1], y, a, in_, topk, combine)
            assert torch.all(guard[0] == 7) and torch.all(guard[-1] == 7)


def test_no_gates_bad_ids_and_no_experts():
    o = ops()
    layer, x, ids, _ = case(931, 6, 40, 3, 144, 512)
    ids[5, 1], ids[6, 0] = 6, -2
    L = o.Mxfp4Layer.from_host(layer)
    y, a = reference(layer, x, ids, None)
    for mode in (o.TQ_GEMV, o.TQ_GEMM):
        ws = o.workspace(40, 3, 6, 144, 512, o.TQ_FP4 | mode)
        got = o.mxfp4_expert_gemm(L, to_dev(x, np.int16), to_dev(ids), flags=o.TQ_FP4 | mode, ws=ws)
        compare(got, y, a, 512, 3, 0)
        assert o.device_status(ws) == 1 and o.device_status(ws) == 0
        none = torch.full((40, 3), -1, dtype=torch.int32, device=dev())
        for combine in (0, o.TQ_COMBINE):
            w2 = o.workspace(40, 3, 6, 144, 512, o.TQ_FP4 | mode | combine)
            got = o.mxfp4_expert_gemm(L, to_dev(x, np.int16), none, flags=o.TQ_FP4 | mode | combine, ws=w2)
            assert torch.all(got == 0) and o.device_status(w2) == 0


@pytest.mark.parametrize("T", [1, 5, 200])
def test_special_activations_and_scales(T):
    """Zero rows, rows with an infinity or NaN (their slots alone are NaN), the ends of bf16's range,
    and weights' scales at the ends of theirs."""
    o = ops()
    E, topk, out, in_ = 3, 2, 80, 1024
    layer, x, ids, gates = case(932, E, T, topk, out, in_, empty=False)
    units = layer["units"].reshape(E, -1)
    scales = units[:, out * in_ // 2:]
    scales[1] = np.where(rng_for(932, 9).random(scales[1].shape) < 0.5, 120, 0)  # 2^-127 beside 2^-7
    scales[2, ::40] = 230
    L = o.Mxfp4Layer.from_host(layer)
    x[0, :] = (oracle.f32_to_bf16_bits_rne(oracle.bf16_bits_to_f64(x[0]).astype(np.float32) * np.float32(2.0 ** -100)))
    if T > 4:
        x[1] = 0
        x[2, 700] = 0x7F80
        x[3, 5] = 0x7FC0
        x[4, ::3] = 0x0001  # the smallest subnormal
    y, a = reference(layer, x, ids, gates)
    for mode in (o.TQ_GEMV, o.TQ_GEMM):
        got = o.mxfp4_expert_gemm(L, to_dev(x, np.int16), to_dev(ids), to_dev(gates), flags=o.TQ_FP4 | mode)
        got = got.cpu().numpy().astype(np.float64)
        assert np.array_equal(np.isnan(got), np.isnan(y))
        ok = ~np.isnan(y)
        # products below fp32's smallest normal number keep fewer bits, or none
        assert np.all(np.abs(got - y)[ok] <= (in_ / 16 + 4) * 2.0 ** -23 * a[ok] + in_ * 2.0 ** -126)


def test_a_nan_scale_of_the_weights_reaches_its_channel():
    o = ops()
    layer, x, ids, gates = case(933, 2, 50, 1, 48, 512, empty=False)
    units = layer["units"].reshape(2, -1)
    units[1, 48 * 256 + 16 * 7 + 3] = 255
    L = o.Mxfp4Layer.from_host(layer)
    y, a = reference(layer, x, ids, gates)
    for mode in (o.TQ_GEMV, o.TQ_GEMM):
        got = o.mxfp4_expert_gemm(L, to_dev(x, np.int16), to_dev(ids), to_dev(gates), flags=o.TQ_FP4 | mode)
        compare(got, y, a, 512, 1, 0)


# (E, T, topk, out, in): items of 256 rows and channels, full and with 1
# to 255 rows, channels that end in and past the second half; more slots than one launch routes
@pytest.mark.parametrize("E,T,topk,out,in_", [(2, 1025, 1, 8208, 512), (3, 1500, 1, 6800, 512), (4, 2100, 2, 2448, 1024),
                                              (1, 4200, 1, 2576, 512), (20, 2049, 2, 2064, 512)])
@pytest.mark.parametrize("repack", [False, True])
def test_large_items(E, T, topk, out, in_, repack):
    """Outputs of some rows (all experts, the ends of their lists) against FP64, every output against
    the call of the token alone."""
    o = ops()
    layer, x, ids, gates = case(950 + E, E, T, topk, out, in_)
    L = o.Mxfp4Layer.from_host(layer)
    L = L.repacked() if repack else L
    xd, idd, gd = to_dev(x, np.int16), to_dev(ids), to_dev(gates)
    got = o.mxfp4_expert_gemm(L, xd, idd, gd, flags=o.TQ_FP4 | o.TQ_GEMM)
    pick = sorted({0, 1, 2, T - 1, T - 2} | {int(t) for e in range(E) for t in (lambda r: (r[0], r[-1], r[len(r) // 2]))(
        np.nonzero((ids == e).any(1))[0])})
    y, a = reference(layer, x[pick], ids[pick], gates[pick])
    compare(got[torch.tensor(pick, device=dev())], y, a, in_, topk, 0)
    # other tiles hold the same rows: the sums are in the same order
    for t0 in range(0, T, 512):
        part = slice(t0, t0 + 512)
        same = o.mxfp4_expert_gemm(L, xd[part], idd[part], gd[part], flags=o.TQ_FP4 | o.TQ_GEMM)
        assert torch.equal(got[part], same)


@pytest.mark.parametrize("E,T,topk", [(1500, 300, 4), (4096, 130, 8), (4096, 1200, 4), (1025, 1, 6), (300, 2, 64)])
def test_many_experts(E, T, topk):
    """Units of few channels, so that thousands of experts fit."""
    o = ops()
    layer, x, ids, gates = case(960 + T, E, T, topk, 16, 512)
    if T > 4:
        ids[3, :2] = E - 1, E
    L = o.Mxfp4Layer.from_host(layer)
    y, a = reference(layer, x, ids, gates)
    for mode in (o.TQ_AUTO, o.TQ_GEMM, o.TQ_GEMV):
        if mode == o.TQ_GEMV and T * topk > 1024:
            continue
        ws = o.workspace(T, topk, E, 16, 512, o.TQ_FP4 | mode)
        got = o.mxfp4_expert_gemm(L, to_dev(x, np.int16), to_dev(ids), to_dev(gates), flags=o.TQ_FP4 | mode, ws=ws)
        compare(got, y, a, 512, topk, 0)
        assert o.device_status(ws) == (1 if T > 4 else 0)


@pytest.mark.parametrize("T,mode", [(1, 0), (40, 1), (256, 1), (400, 0), (40, 2)])
def test_the_same_bits_again_and_in_any_order_of_tokens(T, mode):
    o = ops()
    layer, x, ids, gates = case(934, 12, T, 4, 144, 1024)
    L = o.Mxfp4Layer.from_host(layer).repacked()
    flags = o.TQ_FP4 | mode
    ws = o.workspace(T, 4, 12, 144, 1024, flags)
    args = to_dev(x, np.int16), to_dev(ids), to_dev(gates)
    first = o.mxfp4_expert_gemm(L, *args, flags=flags, ws=ws)
    for _ in range(3):
        assert torch.equal(o.mxfp4_expert_gemm(L, *args, flags=flags, ws=ws), first)
    order = torch.randperm(T, generator=torch.Generator().manual_seed(1)).to(dev())
    moved = o.mxfp4_expert_gemm(L, *(a[order].contiguous() for a in args), flags=flags, ws=ws)
    assert torch.equal(moved, first[order])


@pytest.mark.parametrize("T,mode", [(1, 0), (24, 1), (24, 2), (300, 0)])
def test_replayed_graph_with_changing_routes(T, mode):
    o = ops()
    E, topk, out, in_ = 10, 3, 272, 1024
    layer, x, ids, gates = case(935, E, T, topk, out, in_)
    L = o.Mxfp4Layer.from_host(layer).repacked()
    flags = o.TQ_FP4 | mode | o.TQ_COMBINE
    ws = o.workspace(T, topk, E, out, in_, flags)
    xd, idd, gd = to_dev(x, np.int16), to_dev(ids), to_dev(gates)
    got = torch.empty((T, out), device=dev())
    o.mxfp4_expert_gemm(L, xd, idd, gd, flags=flags, out=got, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o.mxfp4_expert_gemm(L, xd, idd, gd, flags=flags, out=got, ws=ws)
    for k in range(4):
        x = bf16_from_normal(rng_for(936, k), (T, in_))
        ids = uniform_routes(rng_for(937, k), T, E, topk)
        ids[0, 0] = -1 if k % 2 else ids[0, 0]
        xd.copy_(torch.from_numpy(x.view(np.int16)))
        idd.copy_(torch.from_numpy(ids))
        got.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        want = o.mxfp4_expert_gemm(L, xd, idd, gd, flags=flags)
        assert torch.equal(got, want)
        y, a = reference(layer, x, ids, gates)
        compare(got, y, a, in_, topk, 1)


def test_two_streams_at_once():
    o = ops()
    layer, x, ids, gates = case(938, 8, 96, 4, 528, 2560)
    L = o.Mxfp4Layer.from_host(layer).repacked()
    args = [(to_dev(x, np.int16), to_dev(ids), to_dev(gates)),
            (to_dev(x[::-1], np.int16), to_dev(ids), to_dev(gates))]
    want = [o.mxfp4_expert_gemm(L, *a, flags=o.TQ_FP4) for a in args]
    ws = [o.workspace(96, 4, 8, 528, 2560, o.TQ_FP4) for _ in args]
    streams = [torch.cuda.Stream() for _ in args]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i].append(o.mxfp4_expert_gemm(L, *args[i], flags=o.TQ_FP4, ws=ws[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i]) for i in (0, 1) for g in got[i])


def test_one_workspace_for_calls_of_other_sizes():
    """A workspace of the largest call serves smaller ones, in both modes and with other flags."""
    o = ops()
    layer, x, ids, gates = case(939, 6, 200, 4, 144, 1024)
    L = o.Mxfp4Layer.from_host(layer)
    ws = torch.zeros(max(o.workspace_bytes(200, 4, 6, 144, 1024, f) for f in (0, 1, 2, o.TQ_FP4, o.TQ_FP4 | 2)),
                     dtype=torch.uint8, device=dev())
    y, a = reference(layer, x, ids, gates)
    for T, flags in ((200, o.TQ_FP4), (3, o.TQ_FP4), (200, o.TQ_GEMM), (1, o.TQ_FP4), (50, o.TQ_GEMV),
                     (200, o.TQ_FP4 | o.TQ_GEMM), (7, o.TQ_FP4)):
        got = o.mxfp4_expert_gemm(L, to_dev(x[:T], np.int16), to_dev(ids[:T]), to_dev(gates[:T]), flags=flags, ws=ws)
        if flags & o.TQ_FP4:
            compare(got, y[:T], a[:T], 1024, 4, 0)
    assert o.device_status(ws) == 0


def test_what_ran_before_keeps_its_results():
    """The bf16 and fp8 products are what they were beside the new flag."""
    o = ops()
    layer, x, ids, gates = case(941, 5, 60, 2, 128, 1024)
    L = o.Mxfp4Layer.from_host(layer)
    w = mxfp4_weight_fn(layer)
    ref = oracle.expert_gemm(x, ids, gates, 5, w)
    for flags in (o.TQ_GEMV, o.TQ_GEMM):
        got = o.mxfp4_expert_gemm(L, to_dev(x, np.int16), to_dev(ids), to_dev(gates), flags=flags).cpu().numpy()
        assert np.linalg.norm(got - ref) <= 1e-3 * np.linalg.norm(ref)


def test_refusals():
    """Arguments whose memory the kernels would read as something else; nothing is launched."""
    o = ops()
    layer, x, ids, gates = case(942, 4, 6, 2, 48, 512)
    L = o.Mxfp4Layer.from_host(layer)
    x, ids, gates = to_dev(x, np.int16), to_dev(ids), to_dev(gates)
    flags = o.TQ_FP4
    good = o.mxfp4_expert_gemm(L, x, ids, gates, flags=flags)
    bad = [dict(x=x.float()), dict(x=x[:, :256]), dict(x=x[:5]), dict(x=x.t().contiguous().t()), dict(x=x.cpu()),
           dict(topk_ids=ids.long()), dict(topk_ids=ids[0]), dict(topk_ids=ids.t().contiguous().t()),
           dict(topk_w=gates.double()), dict(topk_w=gates[:, :1]), dict(topk_w=gates.bfloat16()),
           dict(out=torch.empty((6, 2, 48), device=dev(), dtype=torch.bfloat16)), dict(out=torch.empty((6, 48), device=dev())),
           dict(out=torch.empty((6, 2, 64), device=dev())[:, :, :48]),
           dict(out=torch.empty((6, 2, 48), device=dev()), flags=flags | o.TQ_COMBINE),
           dict(ws=torch.empty(1 << 20, device=dev())), dict(ws=torch.empty(1 << 20, dtype=torch.uint8))]
    for b in bad:
        args = dict(x=x, topk_ids=ids, topk_w=gates, flags=flags)
        args.update(b)
        with pytest.raises(ValueError):
            o.mxfp4_expert_gemm(L, **args)
    small = torch.zeros(256, dtype=torch.uint8, device=dev())
    for b in (dict(ws=small, flags=flags | o.TQ_GEMM), dict(flags=flags | o.TQ_FP8), dict(flags=flags | 3)):
        args = dict(x=x, topk_ids=ids, topk_w=gates, flags=flags)
        args.update(b)
        with pytest.raises(RuntimeError):
            o.mxfp4_expert_gemm(L, **args)
    assert torch.equal(o.mxfp4_expert_gemm(L, x, ids, gates, flags=flags), good)


def random_units(E, out, in_, seed):
    g = torch.Generator(device=dev()).manual_seed(seed)
    units = torch.randint(0, 256, (E, out * in_ // 2 + out * in_ // 32), dtype=torch.uint8, device=dev(), generator=g)
    units[:, out * in_ // 2:] %= 8
    units[:, out * in_ // 2:] += 118
    return units


def test_offsets_past_32_bits():
    """Activations of nearly 2^30 elements, results and units past 2^32 bytes: the last rows and
    experts against small calls of them alone."""
    o = ops()
    g = torch.Generator(device=dev()).manual_seed(7)

    def rows(T, in_, n):  # the last n tokens are random, the others zero (padding)
        x = torch.zeros((T, in_), dtype=torch.bfloat16, device=dev())
        x[-n:] = torch.randn((n, in_), dtype=torch.bfloat16, device=dev(), generator=g)
        return x

    # (the last: more outputs than a launch has threads, combined)
    for T, E, out, in_, flags in (((1 << 20) - 1, 3, 16, 1024, 0), (135001, 1, 8208, 512, 0),
                                  (525001, 1, 8208, 512, o.TQ_COMBINE)):
        L = o.Mxfp4Layer(E, out, in_, random_units(E, out, in_, T).reshape(-1))
        x = rows(T, in_, 300)
        ids = (torch.arange(T, device=dev(), dtype=torch.int32) % E).view(T, 1)
        got = o.mxfp4_expert_gemm(L, x, ids, flags=o.TQ_FP4 | flags)
        want = o.mxfp4_expert_gemm(L, x[-300:], ids[-300:], flags=o.TQ_FP4 | o.TQ_GEMM | flags)
        assert torch.equal(got[-300:], want) and bool(want.any())
        assert not bool(got[:-300].any())
        del x, got, want
        torch.cuda.empty_cache()

    E, out, in_ = 800, 2048, 5120
    units = random_units(E, out, in_, 3)
    L = o.Mxfp4Layer(E, out, in_, units.view(-1))
    last = o.Mxfp4Layer(1, out, in_, units[-1])
    for T, mode in ((3, o.TQ_GEMV), (3, o.TQ_GEMM), (40, o.TQ_AUTO)):
        x = rows(T, in_, T)
        got = o.mxfp4_expert_gemm(L, x, torch.full((T, 1), E - 1, dtype=torch.int32, device=dev()), flags=o.TQ_FP4 | mode)
        want = o.mxfp4_expert_gemm(last, x, torch.zeros((T, 1), dtype=torch.int32, device=dev()),
                                   flags=o.TQ_FP4 | (mode or o.TQ_GEMM))
        assert torch.equal(got, want) and bool(want.any())


@pytest.mark.parametrize("repack", [False, True])
def test_fp8_products_beside_the_flag(repack):
    """TQ_FP8 over the same layer and workspace as TQ_FP4: the product of MXFP8 activations, before and
    after, and the same bits both times."""
    o = ops()
    layer, x, ids, gates = case(943, 5, 60, 2, 128, 1024)
    L = o.Mxfp4Layer.from_host(layer)
    L = L.repacked() if repack else L
    xq = oracle.dequantize_mxfp8_rows(*oracle.quantize_mxfp8_rows(oracle.bf16_bits_to_f64(x)))
    ref = oracle.expert_gemm_values(xq, ids, gates, 5, mxfp4_weight_fn(layer))
    ws = torch.zeros(max(o.workspace_bytes(60, 2, 5, 128, 1024, f) for f in (o.TQ_FP8, o.TQ_FP4)), dtype=torch.uint8,
                     device=dev())
    args = to_dev(x, np.int16), to_dev(ids), to_dev(gates)
    first = o.mxfp4_expert_gemm(L, *args, flags=o.TQ_FP8, ws=ws)
    o.mxfp4_expert_gemm(L, *args, flags=o.TQ_FP4, ws=ws)
    assert torch.equal(o.mxfp4_expert_gemm(L, *args, flags=o.TQ_FP8, ws=ws), first)
    assert np.linalg.norm(first.cpu().numpy() - ref) <= 1e-3 * np.linalg.norm(ref)


@pytest.mark.parametrize("T", [3, 64, 300])
@pytest.mark.parametrize("places", [(0,), (5,), (0, 2), tuple(range(0, 16, 2))])
@pytest.mark.parametrize("ratio", [2, 9, 16, 18, 21, 25, 28])
def test_large_blocks_that_cancel(T, places, ratio):
    """Blocks whose products cancel, 2^ratio times as large as those of the others: the sum that is left
    keeps to the bound of fp32 additions, and at a ratio whose sums all have 24 bits it is exact."""
    o = ops()
    out, in_ = 48, 512
    rng = rng_for(944, ratio)
    values = np.array([0.5, 1, 1.5, 2, 3, 4, 6])
    codes = rng.integers(0, 16, (out, in_)).astype(np.uint8)
    x = rng.choice(values, (T, in_)) * rng.choice([-1, 1], (T, in_))
    for b in places:
        s, h = slice(32 * b, 32 * b + 16), slice(32 * b + 16, 32 * b + 32)
        x[:, s] = 2.0 ** ratio * rng.choice(values, (T, 16))
        codes[:, s] = rng.integers(1, 8, (out, 16))
        x[:, h], codes[:, h] = -x[:, s], codes[:, s]
    bits = oracle.f32_to_bf16_bits_rne(x.astype(np.float32))
    scales = np.full((out, in_ // 32), 127, np.uint8)
    unit = np.concatenate([oracle.mxfp4_pack(codes).reshape(-1), scales.reshape(-1)])
    layer = dict(E=1, out=out, units=unit, **{"in": in_})
    L = o.Mxfp4Layer.from_host(layer)
    ids = np.zeros((T, 1), np.int32)
    y, a = reference(layer, bits, ids, None)
    for mode in (o.TQ_GEMV, o.TQ_GEMM):
        for l in (L, L.repacked()):
            got = o.mxfp4_expert_gemm(l, to_dev(bits, np.int16), to_dev(ids), flags=o.TQ_FP4 | mode)
            compare(got, y, a, in_, 1, 0)
            if ratio <= 9:  # sums are multiples of 2^-2 below 16 * 36 * 32 * 2^9 = 2^23.2: exact up to 2^22
                exact = a[:, 0] <= 2.0 ** 22
                assert exact.any() and np.array_equal(got.cpu().numpy()[:, 0][exact], y[:, 0][exact])
