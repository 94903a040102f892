"""expert_route and expert_route_backward on the GPU (FORMAT F27, F28) against the FP64 oracle.

Choices have to be equal. Tolerances: a weight is a product and quotient of exponentials and sums
of them. An exponential is off by two steps of fp32 (2^-22) and by its argument's rounding, 2^-24 of
the distance of the logit from the row's largest; sums (six adds in a row's lanes, six and up to 64
values a lane) are off by 2^-21 and less; so a weight is off by 2^-20 plus 2^-22 times that distance
at most, relative to it. A gradient is a difference of such terms, two or three of them multiplied,
at distances up to 8: 2^-18 of the sum of their magnitudes, and half a step of bf16, 2^-8, where it
is rounded to it. Results below 2^-126 keep fewer bits: 2^-140 on top."""

import copy
import pickle

import numpy as np
import pytest

import oracle
from gpu_helpers import dev, gpu, needs_gpu, ops, torch

pytestmark = [gpu, needs_gpu]

W_TOL, G_TOL, BF16 = 2.0 ** -20, 2.0 ** -18, 2.0 ** -8


def logits_for(seed, T, E, dtype, spread=1.0):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy((spread * rng.standard_normal((T, E))).astype(np.float32))
    return x.to(dtype)


def bias_for(seed, E, step=0.001):
    return torch.from_numpy((step * np.round(20 * np.random.default_rng(seed).standard_normal(E))).astype(np.float32))


def options(kw):
    kw = dict(kw)
    if kw.get("bias") is not None:
        kw["bias"] = kw["bias"].numpy()
    return {k: v for k, v in kw.items() if k != "topk"}


def router_of(E, kw):
    kw = dict(kw)
    if kw.get("bias") is not None:
        kw["bias"] = kw["bias"].to(dev())
    return ops().Router(E, **kw)


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def check_route(x, **kw):
    R = router_of(x.shape[1], kw)
    ids, w = ops().expert_route(R, x.to(dev()))
    want_ids, want_w = oracle.expert_route(f64(x), kw["topk"], **options(kw))
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    got = f64(w)
    assert np.array_equal(np.isnan(got), np.isnan(want_w))
    ok = ~np.isnan(want_w)
    v = f64(x)
    top = np.max(np.where(v < np.inf, v, -np.inf), axis=1, keepdims=True)
    far = top - np.take_along_axis(v, np.maximum(want_ids, 0), 1)
    far = np.where(np.isfinite(far), far, 0.0)
    bound = (W_TOL + 2.0 ** -22 * far) * np.abs(want_w) + 2.0 ** -140
    assert np.all(np.abs(got - want_w)[ok] <= bound[ok])
    return R, ids, w


def check_backward(R, x, ids, seed, **kw):
    dw = torch.from_numpy(np.random.default_rng(seed).standard_normal(tuple(ids.shape)).astype(np.float32))
    got = ops().expert_route_backward(R, x.to(dev()), ids, dw.to(dev()))
    assert got.dtype == x.dtype and got.shape == x.shape
    i, o = ids.cpu().numpy(), options(kw)
    want = oracle.expert_route_backward(f64(x), i, f64(dw), **o)
    # the sum of the magnitudes of a gradient's terms
    s = np.array([oracle.router_scores(r, o.get("score", "softmax")) for r in f64(x)])
    c = np.where(i >= 0, np.take_along_axis(s, np.maximum(i, 0), 1), 0.0)
    total = c.sum(1, keepdims=True) if o.get("renorm", True) else np.ones((len(c), 1))
    c = c / np.where(total > 0, total, 1)
    mean = (c * np.abs(f64(dw))).sum(1, keepdims=True)
    size = np.zeros_like(s)
    for t in range(len(i)):
        for k, e in enumerate(i[t]):
            if e >= 0:
                size[t, e] += c[t, k] * (abs(f64(dw)[t, k]) + mean[t, 0])
    if not o.get("renorm", True) and o.get("score", "softmax") == "softmax":
        size += s * mean
    bound = abs(o.get("scale", 1.0)) * G_TOL * size + 2.0 ** -140
    if x.dtype == torch.bfloat16:
        bound = bound * (1 + BF16) + BF16 * np.abs(want)
    assert np.all(np.abs(f64(got) - want) <= bound)
    return got


PLAIN = [dict(topk=1), dict(topk=2, renorm=False), dict(topk=4, score="sigmoid", scale=2.5),
         dict(topk=3, score="sigmoid", renorm=False)]


@pytest.mark.parametrize("E", [4, 7, 64, 65, 100, 200, 384, 500, 1000, 4096])
@pytest.mark.parametrize("kw", PLAIN, ids=str)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("biased", [False, True])
def test_sizes(E, kw, dtype, biased):
    x = logits_for(E, 37, E, dtype)
    kw = dict(kw, bias=bias_for(E, E) if biased else None)
    R, ids, _ = check_route(x, **kw)
    check_backward(R, x, ids, 3, **kw)


@pytest.mark.parametrize("T", [1, 2, 3, 5, 64, 1000])
def test_tokens(T):
    x = logits_for(T, T, 96, torch.float32)
    kw = dict(topk=6, score="sigmoid", bias=bias_for(1, 96))
    R, ids, _ = check_route(x, **kw)
    check_backward(R, x, ids, 4, **kw)


@pytest.mark.parametrize("topk", [16, 33, 63, 64])
def test_many_slots(topk):
    for score in ("softmax", "sigmoid"):
        kw = dict(topk=topk, score=score, renorm=score == "softmax")
        x = logits_for(topk, 9, 80, torch.bfloat16)
        R, ids, _ = check_route(x, **kw)
        check_backward(R, x, ids, 5, **kw)
    x = logits_for(topk, 5, topk, torch.float32)  # every expert is chosen
    check_route(x, topk=topk)


@pytest.mark.parametrize("E,groups", [(8, 2), (8, 8), (96, 3), (96, 4), (256, 8), (65, 5), (384, 64), (320, 40),
                                      (64, 64), (4096, 16), (2048, 1)])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("biased", [False, True])
def test_groups(E, groups, group_top, biased):
    for group_topk in sorted({1, max(1, groups // 2), groups}):
        for score, dtype in (("softmax", torch.float32), ("sigmoid", torch.bfloat16)):
            topk = min(8, E // groups * group_topk)
            check_route(logits_for(E + groups, 21, E, dtype), topk=topk, score=score, groups=groups,
                        group_topk=group_topk, group_top=group_top, bias=bias_for(2, E) if biased else None)


@pytest.mark.parametrize("biased", [False, True])
def test_ties_go_to_the_lowest_index(biased):
    rng = np.random.default_rng(11)
    for E in (5, 64, 130, 384):
        x = torch.from_numpy(rng.integers(0, 3, (40, E)).astype(np.float32))
        x[0] = 1.5
        b = torch.from_numpy(rng.integers(0, 2, E).astype(np.float32) * 0.25) if biased else None
        for score in ("softmax", "sigmoid"):
            check_route(x, topk=min(8, E), score=score, bias=b)
            if E % 2 == 0:
                check_route(x, topk=4, score=score, bias=b, groups=2, group_topk=1, group_top=2)


def test_keys_that_fp32_cannot_tell_apart():
    """Scores plus biases that differ by 1e-9: the bias takes back what a logit adds, up to that."""
    rng = np.random.default_rng(12)
    E, T = 64, 50
    x = rng.standard_normal(E).astype(np.float32)
    s = 1 / (1 + np.exp(-x.astype(np.float64)))
    b = (0.75 - s).astype(np.float32)  # every key is 0.75 up to the bias's rounding, about 2^-25
    rows = torch.from_numpy(np.tile(x, (T, 1)) + np.float32(2.0 ** -20) * rng.integers(0, 3, (T, E)).astype(np.float32))
    check_route(rows, topk=8, score="sigmoid", bias=torch.from_numpy(b))
    check_route(rows, topk=8, score="sigmoid", bias=torch.from_numpy(b), groups=8, group_topk=2, group_top=2)
    check_route(rows, topk=8, score="sigmoid", bias=torch.from_numpy(b), groups=8, group_topk=2, group_top=1)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("biased", [False, True])
def test_experts_out_of_the_choice(score, renorm, biased):
    x = logits_for(13, 30, 24, torch.float32)
    x[:10, 3::4] = -float("inf")
    x[10:14] = -float("inf")
    x[14, :] = -float("inf")
    x[14, 5] = 0.5
    x[15, 2:] = torch.finfo(torch.float32).min  # the type's lowest value is a logit like any other
    b = bias_for(3, 24) if biased else None
    if biased:
        b[7] = -float("inf")
    kw = dict(topk=6, score=score, renorm=renorm, bias=b)
    R, ids, w = check_route(x, **kw)
    i = ids.cpu().numpy()
    assert np.all(i[10:14] == -1) and list(i[14]) == [5, -1, -1, -1, -1, -1]
    assert np.all(w[10:14].cpu().numpy() == 0)
    got = check_backward(R, x, ids, 6, **kw)
    assert torch.all(got[10:14] == 0) and torch.isfinite(got).all()
    check_route(x, topk=4, score=score, renorm=renorm, bias=b, groups=4, group_topk=2, group_top=2)


@pytest.mark.parametrize("groups", [1, 4])
def test_undefined_rows(groups):
    x = logits_for(14, 12, 16, torch.float32)
    x[1, 4] = float("nan")
    x[2, 9] = float("inf")
    x[3] = float("nan")
    x[4, 0], x[4, 1] = float("inf"), -float("inf")
    for score in ("softmax", "sigmoid"):
        for dtype in (torch.float32, torch.bfloat16):
            _, ids, w = check_route(x.to(dtype), topk=4, score=score, groups=groups, group_topk=groups)
            assert list(ids[1].tolist()) == [0, 1, 2, 3] and torch.isnan(w[1]).all()
    b = bias_for(4, 16)
    b[6] = float("nan")
    _, ids, w = check_route(x, topk=4, bias=b, groups=groups, group_topk=groups)
    assert torch.isnan(w).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_extreme_logits(score):
    x = 40 * logits_for(15, 20, 48, torch.float32)
    x[0] = -1e30
    x[1] = 1e30
    x[2, ::2] = -3e38
    x[3] = torch.linspace(-150, -100, 48)
    for renorm in (True, False):
        kw = dict(topk=5, score=score, renorm=renorm)
        R, ids, w = check_route(x, **kw)
        assert torch.isfinite(ops().expert_route_backward(R, x.to(dev()), ids, torch.ones_like(w))).all()


def test_backward_of_given_slots():
    """The same expert twice, empty slots between others, and ids that name no expert."""
    x = logits_for(16, 6, 20, torch.float32)
    ids = torch.tensor([[3, 3, 5], [7, 7, 7], [-1, 4, -1], [-1, -1, -1], [0, 20, 1], [-2, 1, 2]], dtype=torch.int32)
    for kw in (dict(topk=3), dict(topk=3, renorm=False), dict(topk=3, score="sigmoid"),
               dict(topk=3, score="sigmoid", renorm=False)):
        R = router_of(20, kw)
        good = ids.clone()
        good[4:] = -1
        check_backward(R, x, good.to(dev()), 8, **kw)
        got = ops().expert_route_backward(R, x.to(dev()), ids.to(dev()), torch.ones(6, 3, device=dev()))
        assert torch.isnan(got[4:]).all() and torch.isfinite(got[:4]).all()


@pytest.mark.parametrize("kw", PLAIN, ids=str)
def test_gradient_against_differences(kw):
    """Differences of the kernel's own weights: a step of 2^-6 (truncation h^2 / 6 times a third
    derivative below 8 times the scale), over weights off by 2^-20."""
    E, topk, scale = 12, kw["topk"], kw.get("scale", 1.0)
    x = logits_for(17, 1, E, torch.float32)
    R = router_of(E, kw)
    ids, _ = ops().expert_route(R, x.to(dev()))
    h = 2.0 ** -6
    dw = torch.tensor([np.random.default_rng(18).standard_normal(topk)], dtype=torch.float32, device=dev())
    got = ops().expert_route_backward(R, x.to(dev()), ids, dw).cpu().numpy()[0]

    def weights(z):  # by expert, as the order of the slots may change
        i, w = ops().expert_route(R, z.to(dev()))
        by = dict(zip(i[0].tolist(), w[0].tolist()))
        return [by[e] for e in ids[0].tolist()] if set(by) == set(ids[0].tolist()) else None

    tried = 0
    for e in range(E):
        up, down = x.clone(), x.clone()
        up[0, e] += h
        down[0, e] -= h
        a, b = weights(up), weights(down)
        if a is None or b is None:
            continue  # the step changes the choice
        tried += 1
        size = dw.abs().sum().item() * scale
        d = sum((p - q) * g for p, q, g in zip(a, b, dw[0].tolist())) / (2 * h)
        assert abs(d - got[e]) <= size * (8 * h * h / 6 + 2.0 ** -19 / h)
    assert tried >= E // 2


def test_rows_around_the_outputs_stay():
    x = logits_for(19, 7, 33, torch.bfloat16).to(dev())
    R = ops().Router(33, 5)
    ids = torch.full((9, 5), 77, dtype=torch.int32, device=dev())
    w = torch.full((9, 5), 7.0, device=dev())
    ops().expert_route(R, x, ids=ids[1:8], w=w[1:8])
    assert torch.all(ids[[0, 8]] == 77) and torch.all(w[[0, 8]] == 7.0)
    grad = torch.full((9, 33), 7.0, dtype=torch.bfloat16, device=dev())
    ops().expert_route_backward(R, x, ids[1:8], w[1:8], dlogits=grad[1:8])
    assert torch.all(grad[[0, 8]] == 7.0)


def test_gradients_may_replace_the_logits():
    for kw in PLAIN:
        x = logits_for(20, 50, 70, torch.float32).to(dev())
        R = router_of(70, kw)
        ids, w = ops().expert_route(R, x)
        want = ops().expert_route_backward(R, x, ids, w)
        ops().expert_route_backward(R, x, ids, w, dlogits=x)
        assert torch.equal(x, want)


def test_no_tokens():
    R = ops().Router(8, 2)
    x = torch.zeros((0, 8), device=dev())
    ids, w = ops().expert_route(R, x)
    assert ids.shape == (0, 2) and ops().expert_route_backward(R, x, ids, w).shape == (0, 8)


def test_wrapper_refusals():
    R = ops().Router(16, 4)
    x = torch.zeros((3, 16), device=dev())
    for bad in (x.double(), x.t().contiguous(), x.t(), x[:, ::2], x[0], x.half()):
        with pytest.raises(ValueError):
            ops().expert_route(R, bad)
    with pytest.raises(ValueError):
        ops().expert_route(R, x, ids=torch.zeros((3, 4), dtype=torch.int64, device=dev()))
    with pytest.raises(ValueError):
        ops().expert_route(R, x, w=torch.zeros((2, 4), device=dev()))
    ids, w = ops().expert_route(R, x)
    for bad in ((ids.long(), w), (ids, w.double()), (ids[:2], w), (ids, w[:, :3])):
        with pytest.raises(ValueError):
            ops().expert_route_backward(R, x, *bad)
    with pytest.raises(ValueError):
        ops().expert_route_backward(R, x, ids, w, dlogits=torch.zeros_like(x).bfloat16())
    for bias in (torch.zeros(15, device=dev()), torch.zeros(16, device=dev()).double(),
                 torch.zeros(32, device=dev())[::2]):
        with pytest.raises(ValueError):
            ops().Router(16, 4, bias=bias)
    with pytest.raises(Exception, match="topk"):
        ops().expert_route(ops().Router(16, 17), x)


def test_a_router_follows_its_bias():
    x = logits_for(21, 9, 16, torch.float32).to(dev())
    b = torch.zeros(16, device=dev())
    R = ops().Router(16, 3, score="sigmoid", bias=b)
    plain, _ = ops().expert_route(R, x)
    b[11] = 5.0  # updated in place, as a balancing step does
    assert torch.all(ops().expert_route(R, x)[0][:, 0] == 11)
    b.set_(torch.zeros(16, device=dev()).index_fill_(0, torch.tensor([2], device=dev()), 9.0))
    assert torch.all(ops().expert_route(R, x)[0][:, 0] == 2)
    b.resize_(8)
    with pytest.raises(ValueError, match="bias"):
        ops().expert_route(R, x)
    R = ops().Router(16, 3, score="sigmoid", bias=torch.zeros(16, device=dev()))
    for other in (copy.copy(R), copy.deepcopy(R), pickle.loads(pickle.dumps(R))):
        assert torch.equal(ops().expert_route(other, x)[0], plain)


def test_replayed_graph_and_another_stream():
    T, E = 40, 96
    kw = dict(topk=8, score="sigmoid", bias=bias_for(5, E), groups=4, group_topk=2, group_top=2)
    R = router_of(E, kw)
    x = logits_for(22, T, E, torch.float32).to(dev())
    ids, w = ops().expert_route(R, x)
    grad = ops().expert_route_backward(R, x, ids, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops().expert_route(R, x, ids=ids, w=w)
        ops().expert_route_backward(R, x, ids, w, dlogits=grad)
    side = torch.cuda.Stream()
    for seed in range(4):
        x.copy_(logits_for(30 + seed, T, E, torch.float32))
        graph.replay()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.default_stream())
            i, v = ops().expert_route(R, x)
            g = ops().expert_route_backward(R, x, i, v)
        side.synchronize()
        assert torch.equal(i, ids) and torch.equal(v, w) and torch.equal(g, grad)


def test_offsets_past_32_bits():
    """2^31 bf16 logits and more: the last rows are read and written where they are."""
    E = 4096
    T = (1 << 31) // E + 5
    x = torch.zeros((T, E), dtype=torch.bfloat16, device=dev())
    x[-1, 4000], x[-1, 17], x[0, 9] = 3.0, 2.0, 1.0
    R = ops().Router(E, 2)
    ids, w = ops().expert_route(R, x)
    assert ids[-1].tolist() == [4000, 17] and ids[0].tolist() == [9, 0] and ids[-2].tolist() == [0, 1]
    dw = torch.zeros_like(w)
    dw[-1, 0] = 1.0
    ops().expert_route_backward(R, x, ids, dw, dlogits=x)
    r = w[-1, 0].item()
    want = torch.tensor([r * (1 - r), -r * (1 - r)])
    assert torch.allclose(x[-1, [4000, 17]].float().cpu(), want, rtol=BF16 * 1.01, atol=0)
    assert x[:-1].abs().max().item() == 0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,group_top", [(1, 1), (4, 1), (4, 2)])
def test_huge_and_infinite_biases(score, groups, group_top):
    """Keys that round together (a bias far above every score), infinite ones, and none at all."""
    x = logits_for(391, 40, 64, torch.float32)
    for values in ([float("inf")], [1e30, -1e30], [float("inf"), float("-inf"), 3e38, -3e38, 0.0], [65536.0]):
        bias = torch.tensor([values[(5 * e) % len(values)] for e in range(64)], dtype=torch.float32)
        for some in (1, 3):
            b = torch.where(torch.arange(64) % some == 0, bias, torch.zeros(64))
            check_route(x, topk=6, score=score, bias=b, groups=groups, group_topk=max(1, groups // 2), group_top=group_top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_top", [1, 2])
def test_groups_whose_scores_round_together(score, group_top):
    """Logits whose scores are equal in 64 bits (all 1, or all 0), in groups: by one score the groups go
    by their logits, by two they tie."""
    rng = np.random.default_rng(400)
    x = np.empty((30, 96), dtype=np.float32)
    x[:] = rng.permuted(np.tile(np.arange(96, dtype=np.float32), (30, 1)), axis=1)
    x = x + 40 if score == "sigmoid" else -900 - x  # one expert of softmax has the whole of it
    if score == "softmax":
        x[:, 50] = 0.0
    for groups, group_topk in ((2, 1), (8, 3), (24, 5)):
        for renorm in (True, False):
            check_route(torch.from_numpy(x), topk=4, score=score, groups=groups, group_topk=group_topk, group_top=group_top,
                        renorm=renorm)


@pytest.mark.parametrize("E", [1, 5, 8, 33, 63, 65, 100])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_an_infinite_bias_closes_the_choice(E, score):
    """The last key chosen is +inf: no lane past the last expert takes part, and equal ones go by index."""
    x = logits_for(401, 9, E, torch.float32)
    for many in sorted({1, min(3, E), E}):
        b = torch.zeros(E)
        b[torch.arange(many) * E // many] = float("inf")
        b[E // 2] = -1e30 if many < E else b[E // 2]
        for topk in sorted({1, min(2, E), min(many, 64), min(many + 1, E, 64)}):
            check_route(x, topk=topk, score=score, bias=b)
            if E % 5 == 0 and topk <= E // 5 * 2:
                check_route(x, topk=topk, score=score, bias=b, groups=5, group_topk=2, group_top=2)


@pytest.mark.parametrize("group_topk", [1, 2, 3])
@pytest.mark.parametrize("big", [3e38, 1.7014118e38, 1.8e38])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_sums_of_two_keys_past_fp32(score, big, group_topk):
    """Finite biases whose sums are beyond fp32, in groups before and behind ones without experts."""
    x = logits_for(410, 20, 16, torch.float32)
    low = float(torch.finfo(torch.float32).min)
    lists = [[0.0, -big, -0.9 * big, -0.99 * big], [0.0, big, 0.9 * big, 0.99 * big],
             [-big, -0.99 * big, low, 0.0], [0.0, low, -0.97 * big, low], [low] * 4]
    for values in lists:
        b = torch.tensor(values, dtype=torch.float32).repeat_interleave(4)
        check_route(x, topk=4, score=score, bias=b, groups=4, group_topk=group_topk, group_top=2)
        y = x.clone()
        y[:, :4] = -float("inf")  # a group without experts before one masked by the lowest value
        check_route(y, topk=4, score=score, bias=b, groups=4, group_topk=group_topk, group_top=2)
        y[::2, 4:8] = -float("inf")
        check_route(y, topk=4, score=score, bias=b, groups=4, group_topk=group_topk, group_top=2)
        b[9] = -float("inf")
        check_route(y, topk=4, score=score, bias=b, groups=4, group_topk=group_topk, group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_a_masked_expert_costs_no_certainty(score):
    """One expert taken out by its bias leaves the groups as sure as before: a chunk is not chosen in 64
    bits throughout (twice the time), which the largest magnitude among all keys had asked for. The least
    times of calls in turn, sixteen at a time."""
    o = ops()
    T, E = 8192, 384
    x = logits_for(420, T, E, torch.float32).to(dev())
    routers = []
    for value in (None, -float("inf"), -1e9, torch.finfo(torch.float32).min):
        b = bias_for(1, E)
        if value is not None:
            b[100] = value
        routers.append(o.Router(E, 8, score=score, bias=b.to(dev()), groups=8, group_topk=4, group_top=2))
    ids, w = o.expert_route(routers[0], x)
    best = [1e9] * len(routers)
    for _ in range(20):
        for i, R in enumerate(routers):
            e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
            torch.cuda.synchronize()
            o.expert_route(R, x, ids=ids, w=w)
            e[0].record()
            for _ in range(16):
                o.expert_route(R, x, ids=ids, w=w)
            e[1].record()
            torch.cuda.synchronize()
            best[i] = min(best[i], e[0].elapsed_time(e[1]) / 16 * 1e3)
    print(" ".join("%.1f" % t for t in best))
    assert max(best[1:]) <= 1.4 * best[0], best


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("value", [-float("inf"), -1e9, -65536.0, 1e9])
def test_masked_experts_in_groups(score, group_top, value):
    """Some experts of every group, whole groups, and all but one expert of a group masked by the bias."""
    x = logits_for(430, 40, 96, torch.float32)
    b = bias_for(7, 96)
    b[::7] = value
    for groups in (4, 8, 32):
        size = 96 // groups
        for m in (b, torch.where(torch.arange(96) // size == 1, torch.full((96,), value), b),
                  torch.where((torch.arange(96) // size == 2) & (torch.arange(96) % size > 0), torch.full((96,), value), b)):
            for group_topk in (1, groups // 2, groups - 1):
                check_route(x, topk=min(6, size * group_topk), score=score, bias=m, groups=groups, group_topk=group_topk,
                            group_top=group_top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E", [16, 65, 400, 1100])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients_of_undefined_rows(score, renorm, E, dtype):
    """NaN and infinities at experts that slots name and at ones that none does, among -inf alone, and in
    rows without slots; the gradients may replace the logits."""
    inf, nan = float("inf"), float("nan")
    x = logits_for(440, 13, E, dtype)
    x[1, E - 1], x[2, 0], x[3, E - 1], x[4, 1], x[5, E - 1] = nan, nan, inf, inf, -inf
    x[6] = -inf
    x[6, E - 2] = nan
    x[7], x[8], x[9] = nan, inf, -inf
    x[10, 5] = nan
    x[11] = -inf
    x[11, 0] = nan
    ids = torch.tensor([[0, 1, 2]] * 13, dtype=torch.int32)
    ids[9:11] = -1
    ids[12] = torch.tensor([2, -1, 2])
    kw = dict(topk=3, score=score, renorm=renorm, scale=1.5)
    R = router_of(E, kw)
    dw = torch.from_numpy(np.random.default_rng(9).standard_normal((13, 3)).astype(np.float32))
    want = oracle.expert_route_backward(f64(x), ids.numpy(), f64(dw), **options(kw))
    for target in (None, x.to(dev())):
        z = x.to(dev()) if target is None else target
        got = f64(ops().expert_route_backward(R, z, ids.to(dev()), dw.to(dev()), dlogits=target))
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert np.all(got[9:11] == 0)
    rows = torch.from_numpy(~np.isnan(want).any(1))
    rows[8] = False  # (infinities: no distance from a largest logit)
    if renorm or score == "sigmoid":
        assert rows[[0, 1, 3, 5, 9, 10, 12]].all()
        x = torch.where(torch.isfinite(x), x, torch.zeros_like(x))  # logits that no slot of these rows names
    else:
        rows[9:11] = False
    check_backward(R, x[rows], ids[rows].to(dev()), 10, **kw)


def near_ties(score, E, T, shape, spread, seed):
    """Logits [T, E] and a bias that takes back the score of a base row, so that the keys of rows which
    repeat it up to a few steps of fp32 are 0.75 up to about `spread` and the bias's rounding, 2^-25.
    shape: scores that are alike (flat: a sum of softmax near E), of one or two dominant experts (a sum
    near 1), or spread as logits are."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal(E).astype(np.float32)
    if shape == "flat":
        x *= np.float32(2.0 ** -6)
    if shape == "dominant":
        x[E // 3] += np.float32(12.0)
        x[E // 2] += np.float32(11.0)
    s = oracle.router_scores(x, score)
    b = (0.75 - s + spread * rng.standard_normal(E)).astype(np.float32)
    rows = np.tile(x, (T, 1)) + np.float32(2.0 ** -22) * rng.integers(-1, 2, (T, E)).astype(np.float32)
    return torch.from_numpy(rows), torch.from_numpy(b)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [60, 64, 384, 1000, 4096])
@pytest.mark.parametrize("shape", ["flat", "dominant", "normal"])
@pytest.mark.parametrize("spread", [0.0, 2.0 ** -24, 2.0 ** -21])
def test_keys_within_the_errors_of_each_other(score, E, shape, spread):
    """All keys within some steps of fp32 of each other (more than 64 of them where E is larger), and a
    spread at which some are told apart; without groups and in groups by one and two."""
    rows, b = near_ties(score, E, 12, shape, spread, E)
    assert np.ptp(oracle.router_scores(f64(rows)[0], score) + f64(b)) < 2.0 ** -22 + 12 * spread
    for topk in (1, 8):
        check_route(rows, topk=topk, score=score, bias=b)
    for groups in (4, 20):
        if E % groups == 0:
            for group_top in (1, 2):
                check_route(rows, topk=min(6, E // groups), score=score, bias=b, groups=groups, group_topk=3,
                            group_top=group_top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [64, 384, 1000])
def test_pairs_of_keys_a_step_apart(score, E):
    """The last expert chosen and the next differ by less than fp32 shows, on either side of a clear order
    of the others; in the last lanes and values too."""
    rng = np.random.default_rng(E)
    T, topk = 40, 8
    x = rng.standard_normal((T, E)).astype(np.float32)
    x[:, -1] = np.float32(0.5)
    x[:, 5] = np.float32(0.5) + np.float32(2.0 ** -22) * rng.integers(-2, 3, T).astype(np.float32)
    b = rng.uniform(-0.3, 0.3, E).astype(np.float32)
    s = np.array([oracle.router_scores(r, score) for r in x.astype(np.float64)])
    # the pair is put where the choice ends: seven others stay ahead, the rest behind
    b[-1] = b[5] = np.float32(2.0)
    ahead = rng.choice(np.arange(6, E - 1), 7, replace=False)
    b[ahead] = np.float32(4.0) + np.float32(0.25) * np.arange(7, dtype=np.float32)
    c = s + b.astype(np.float64)
    gap = np.abs(c[:, 5] - c[:, -1])
    assert np.median(gap) < 2.0 ** -22 and np.all((gap > 2.0 ** -50) | (x[:, 5] == x[:, -1]))
    check_route(torch.from_numpy(x), topk=topk, score=score, bias=torch.from_numpy(b))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("scale", [1.0, 1e-6, 1e4])
def test_weights_below_the_smallest_normal_number(score, renorm, scale):
    """Logits 80 to 110 below the largest: a weight, or what the scale multiplies, is below 2^-126. Its terms
    are then multiples of 2^-149: off by max(1, |scale|) 2^-147 on top of the relative bound."""
    x = np.full((16, 24), -300.0, dtype=np.float32)
    x[:, 3] = 0.0
    x[:, 5:12] = -np.random.default_rng(450).uniform(80, 110, (16, 7)).astype(np.float32)
    R = router_of(24, dict(topk=8, score=score, renorm=renorm, scale=scale))
    ids, w = ops().expert_route(R, torch.from_numpy(x).to(dev()))
    want_ids, want = oracle.expert_route(x, 8, score=score, renorm=renorm, scale=scale)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    far = -np.take_along_axis(x.astype(np.float64), want_ids, 1)
    assert np.sum(want / scale < 2.0 ** -126) > 40 and np.sum(want / scale > 2.0 ** -126) > 40
    bound = (2.0 ** -18 + 2.0 ** -22 * far) * want + max(1.0, scale) * 2.0 ** -147
    assert np.all(np.abs(f64(w) - want) <= bound)
