"""The fp8b128 operators on the GPU (FORMAT F22-F26) against the FP64 oracle.

Tolerances, per element, from the number formats (a rounding is off by at most half a step):
  - fp32 sums of exact products: every add of the in + blocks + 10 on a sum's path is off by at
    most 2^-23 (rounded or cut) of the sum of magnitudes A = |X| |W|^T;
  - the fp8 matrix cores' sums (results in bf16): 2^-12 of A. An instruction aligns its products
    to the largest, so the error scales with the magnitudes; one block of uniformly drawn codes
    shows up to 2^-13.6 of A;
  - rounding a result to bf16: 2^-8 of it.
The gradients' bounds follow the formulas: errors of g and u times the slopes, dg and du
rounded to bf16, fp32 sums, a last rounding to bf16."""

import copy
import pickle

import numpy as np
import pytest

import oracle
from gpu_helpers import dev, gpu, needs_gpu, ops, rel_l2, to_dev, torch
from workloads import bf16_from_normal, fp8b128_layer, rng_for

pytestmark = [gpu, needs_gpu]

BF16, F32 = 2.0 ** -8, 2.0 ** -23
FP8_SUM = 2.0 ** -12

# (T, out, in): one token to several tiles of every kernel; sides that end inside a block, a
# tile and a 16-byte chunk pair; fewer blocks than waves, and more
FORWARD = [(1, 16, 16), (1, 1536, 5120), (2, 48, 112), (5, 160, 128), (16, 32, 144), (17, 128, 256),
           (33, 272, 400), (64, 144, 1040), (65, 96, 2064), (100, 64, 1168), (129, 256, 128),
           (200, 400, 272), (257, 528, 640), (300, 1040, 96), (513, 288, 1296), (1030, 784, 528), (3000, 2832, 144),
           # strips of each shape, tiles of each shape, more tiles than compute units
           (12, 5120, 272), (60, 5120, 400), (300, 2064, 656), (1000, 3088, 528), (2100, 2064, 400),
           (2100, 4112, 272), (4200, 4112, 144), (265, 10048, 144), (1714, 11680, 144),
           (33, 5984, 2064), (333, 3808, 1040), (273, 3808, 1040), (513, 10880, 144), (3513, 9248, 144),
           (1714, 9248, 400)]
GATED = [(1, 32, 16), (1, 1536, 5120), (3, 96, 144), (16, 288, 272), (31, 64, 400), (64, 1440, 528),
         (130, 160, 1040), (257, 544, 256), (300, 800, 400), (700, 1056, 272), (2900, 2848, 272),
         (60, 5120, 400), (700, 4128, 272), (2100, 2080, 400), (4100, 4096, 144), (4200, 4128, 144),
         (265, 8672, 144), (1971, 10304, 144), (33, 5984, 2064), (33, 8704, 1040), (273, 3808, 1040),
         (513, 10880, 144), (3513, 9248, 144)]
BACKWARD = [(1, 32, 16), (1, 288, 400), (2, 64, 128), (17, 32, 272), (40, 288, 144), (64, 96, 1040),
            (129, 256, 256), (200, 544, 400), (257, 160, 656), (333, 1056, 272), (600, 288, 784), (2100, 352, 2064), (4200, 64, 2320),
            (1000, 3104, 144), (3000, 2848, 144), (2100, 2048, 272),
            (40, 3104, 2064), (33, 5152, 2064), (265, 8672, 144),
            # whole and half tiles of the weight gradient
            (600, 2080, 2064), (420, 2848, 2832),
            # the two gradients in one launch or apart, in each of their kernels
            (580, 1056, 144), (580, 64, 1296), (130, 1600, 2064), (310, 1056, 2832), (400, 160, 1296),
            (580, 160, 2832), (850, 64, 2064), (940, 352, 4112), (4300, 64, 784), (4000, 64, 4112),
            (513, 10880, 144), (1714, 9248, 144)]


def bits_of(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


def f64_of(t):
    if t.dtype == torch.bfloat16:
        return oracle.bf16_bits_to_f64(bits_of(t))
    return t.cpu().numpy().astype(np.float64)


def bf16_dev(bits):
    return to_dev(bits, np.int16).view(torch.bfloat16)


class Inputs:
    """A layer and activations, on the host and on the GPU. Activation codes come from the
    oracle's quantizer; `any_scale` replaces its powers of two by arbitrary fp32 values."""

    def __init__(self, seed, T, out, inp, any_scale=False):
        self.host = fp8b128_layer(seed, out, inp, (T,))
        x = bf16_from_normal(rng_for(seed, 3, T, out, inp), (T, inp))
        if T > 4:
            x[T // 2] = 0  # a padded token
        self.codes, s = oracle.fp8b128_quantize(x)
        if any_scale:
            s = s * rng_for(seed, 6).uniform(0.6, 1.4, size=s.shape)
        self.scales = s.astype(np.float32)
        self.X = oracle.fp8b128_activations(self.codes, self.scales)
        self.W = oracle.fp8b128_weights(self.host["codes"], self.host["scales"])
        self.layer = ops().Fp8b128Layer.from_host(self.host, dev())
        self.xq, self.xs = to_dev(self.codes), to_dev(self.scales)


def guarded(T, width, dtype, fill):
    """(rows to write, whole buffer): rows with 3 guard rows on each side."""
    whole = torch.full((T + 6, width), fill, dtype=dtype, device=dev())
    return whole[3:3 + T], whole


def check_guards(whole, fill):
    w = whole.float()
    assert bool((w[:3] == fill).all()) and bool((w[-3:] == fill).all())


def assert_within(got, ref, tol, what=""):
    bad = np.argwhere(~(np.abs(got - ref) <= tol))
    if bad.size:
        at = tuple(bad[0])
        raise AssertionError("%s %d of %d off, first at %s: %r, not %r within %.3g" % (
            what, len(bad), got.size, at, got[at], ref[at], tol[at]))


# ---- quantizer ------------------------------------------------------------------------------
@pytest.mark.parametrize("T,n", [(1, 16), (1, 128), (3, 144), (7, 5120), (130, 272), (64, 1040)])
def test_quantize_bits(T, n):
    x = bf16_from_normal(rng_for(970, 3, T, n), (T, n))
    if T > 2:
        x[1] = 0
    codes, scales = ops().fp8b128_quantize(bf16_dev(x))
    rc, rs = oracle.fp8b128_quantize(x)
    assert np.array_equal(codes.cpu().numpy(), rc)
    assert np.array_equal(scales.cpu().numpy().astype(np.float64), rs)


def test_quantize_every_bf16_pattern():
    # every finite bf16 pattern, in rows of one magnitude range and in mixed rows; then blocks
    # with an infinity or a NaN
    pats = np.arange(65536, dtype=np.uint16)
    fin = pats[(pats & 0x7F80) != 0x7F80]
    rng = rng_for(971, 0)
    x = np.concatenate([fin, rng.permutation(fin)]).reshape(-1, 510)
    x = np.concatenate([x, x[:, :2]], axis=1)  # 512 wide
    x[5, 100], x[6, 511], x[7, 256] = 0x7F80, 0xFF80, 0x7FC1
    codes, scales = ops().fp8b128_quantize(bf16_dev(x))
    rc, rs = oracle.fp8b128_quantize(x)
    assert np.array_equal(codes.cpu().numpy(), rc)
    assert np.array_equal(scales.cpu().numpy().astype(np.float64), rs, equal_nan=True)


# ---- the product ----------------------------------------------------------------------------
@pytest.mark.parametrize("T,out,inp", FORWARD)
@pytest.mark.parametrize("bf16", [False, True])
def test_gemm(T, out, inp, bf16):
    c = Inputs(972, T, out, inp, any_scale=True)
    y, whole = guarded(T, out, torch.bfloat16 if bf16 else torch.float32, 7.0)
    ops().fp8b128_gemm(c.layer, c.xq, c.xs, flags=ops().TQ_OUT_BF16 if bf16 else 0, out=y)
    got, ref, A = f64_of(y), c.X @ c.W.T, np.abs(c.X) @ np.abs(c.W).T
    adds = (inp + inp / 128 + 10) * F32 * A
    assert_within(got, ref, BF16 * np.abs(ref) + FP8_SUM * A if bf16 else adds)
    # in the 2-norm the roundings do not add up with one sign
    assert rel_l2(got, ref) <= (BF16 if bf16 else np.sqrt(inp + 10) * F32)
    check_guards(whole, 7.0)


def test_gemm_takes_float8_tensors_and_special_scales():
    c = Inputs(973, 9, 144, 272)
    f8 = torch.float8_e4m3fn
    L = ops().Fp8b128Layer(c.layer.codes.view(f8), c.layer.scales)
    assert torch.equal(ops().fp8b128_gemm(L, c.xq.view(f8), c.xs), ops().fp8b128_gemm(c.layer, c.xq, c.xs))
    # zero and negative scales are values like others; a zero weight block adds nothing
    s = c.host["scales"].copy()
    s[0, 0], s[1, 1] = 0.0, -s[1, 1]
    W = oracle.fp8b128_weights(c.host["codes"], s)
    got = f64_of(ops().fp8b128_gemm(ops().Fp8b128Layer(c.layer.codes, to_dev(s)), c.xq, c.xs))
    assert_within(got, c.X @ W.T, 300 * F32 * (np.abs(c.X) @ np.abs(W).T))


@pytest.mark.parametrize("T", [3, 70, 300])
def test_non_finite_values_stay_in_their_rows(T):
    c = Inputs(974, T, 160, 400)
    xs, codes, wc = c.scales.copy(), c.codes.copy(), c.host["codes"].copy()
    xs[0, 1] = np.nan               # a token the quantizer could not represent
    codes[T - 1, 399] = 0x7F        # a NaN code in a token's last input
    wc[37, 200] = 0xFF              # and in one channel
    wc[117, 399] = 0x7F
    L = ops().Fp8b128Layer(to_dev(wc), c.layer.scales)
    good_t = np.arange(1, T - 1)
    for flags in (0, ops().TQ_OUT_BF16):
        y = f64_of(ops().fp8b128_gemm(L, to_dev(codes), to_dev(xs), flags=flags))
        nan = np.isnan(y)
        assert nan[0].all() and nan[T - 1].all() and nan[:, 37].all() and nan[:, 117].all()
        keep = np.setdiff1d(np.arange(160), [37, 117])
        assert not nan[np.ix_(good_t, keep)].any()
    h = f64_of(ops().fp8b128_gated(L, to_dev(codes), to_dev(xs)))
    nan = np.isnan(h)
    assert nan[0].all() and nan[T - 1].all() and nan[:, 37].all()  # channel 117 is up 37
    assert not nan[np.ix_(good_t, np.setdiff1d(np.arange(80), [37]))].any()


# ---- the gated product ----------------------------------------------------------------------
def sums_and_error(c):
    """g, u and the bound of their error on the fp8 matrix cores."""
    gu, A = c.X @ c.W.T, np.abs(c.X) @ np.abs(c.W).T
    half = gu.shape[1] // 2
    return gu[:, :half], gu[:, half:], FP8_SUM * A[:, :half], FP8_SUM * A[:, half:]


@pytest.mark.parametrize("T,out,inp", GATED)
def test_gated(T, out, inp):
    c = Inputs(975, T, out, inp, any_scale=True)
    h, whole = guarded(T, out // 2, torch.bfloat16, 5.0)
    ops().fp8b128_gated(c.layer, c.xq, c.xs, out=h)
    ref = oracle.fp8b128_gated(c.X, c.W)
    g, u, eg, eu = sums_and_error(c)
    # |silu'| <= 1.1; eight fp32 roundings of the activation and its exponential
    tol = BF16 * np.abs(ref) + 1.1 * eg * (np.abs(u) + eu) + np.abs(oracle.silu(g)) * eu + 8 * F32 * np.abs(ref)
    assert_within(f64_of(h), ref, tol + 2.0 ** -133)
    assert rel_l2(f64_of(h), ref) <= BF16
    check_guards(whole, 5.0)


def test_gated_far_arguments():
    # gate sums of +-40000: the exponential overflows or vanishes, silu is its limit
    T, inp = 4, 128
    codes = np.full((32, inp), 0x38, dtype=np.uint8)      # 1.0
    codes[1] |= 0x80                                      # gate 1 negative
    host = {"out": 32, "in": inp, "codes": codes, "scales": np.full((1, 1), 312.5, np.float32)}
    L = ops().Fp8b128Layer.from_host(host, dev())
    x = np.full((T, inp), 0x38, dtype=np.uint8)
    h = f64_of(ops().fp8b128_gated(L, to_dev(x), to_dev(np.ones((T, 1), np.float32))))
    assert np.allclose(h[:, 0], 1.6e9, rtol=BF16) and (h[:, 1] == 0).all()
    dh = bf16_dev(np.full((T, 16), 0x3F80, np.uint16))
    dx, dw = ops().fp8b128_gated_backward(L, to_dev(x), to_dev(np.ones((T, 1), np.float32)), dh)
    assert torch.isfinite(dx.float()).all() and torch.isfinite(dw.float()).all()


# ---- gradients ------------------------------------------------------------------------------
def check_product_grads(dx, dw, D, eD, X, W):
    """dx = D W and dw = D^T X, from D known to within eD (element by element)."""
    aD = np.abs(D) + eD
    T, out = D.shape
    for got, ref, mag, err, n in (
            (dx, D @ W, aD @ np.abs(W), eD @ np.abs(W), out),
            (dw, D.T @ X, aD.T @ np.abs(X), eD.T @ np.abs(X), T)):
        assert_within(got, ref, BF16 * (np.abs(ref) + err) + err + (n + n / 128 + 10) * F32 * mag + 2.0 ** -133)


def grads_of(T, out, width):
    d = 0.25 * rng_for(976, 5, T, out).standard_normal((T, width)).astype(np.float32)
    return oracle.f32_to_bf16_bits_rne(d)


@pytest.mark.parametrize("T,out,inp", BACKWARD)
def test_gemm_backward(T, out, inp):
    c = Inputs(976, T, out, inp)
    db = grads_of(T, out, out)
    D = oracle.bf16_bits_to_f64(db)
    dx, wx = guarded(T, inp, torch.bfloat16, 3.0)
    dw, ww = guarded(out, inp, torch.bfloat16, 3.0)
    ops().fp8b128_gemm_backward(c.layer, c.xq, c.xs, bf16_dev(db), dx=dx, dw=dw)
    check_product_grads(f64_of(dx), f64_of(dw), D, 0 * D, c.X, c.W)
    assert rel_l2(f64_of(dx), D @ c.W) <= BF16 and rel_l2(f64_of(dw), D.T @ c.X) <= BF16
    check_guards(wx, 3.0)
    check_guards(ww, 3.0)


def test_gemm_backward_rounds_general_scales():
    c = Inputs(977, 70, 160, 272, any_scale=True)
    db = grads_of(70, 160, 160)
    D = oracle.bf16_bits_to_f64(db)
    _, dw = ops().fp8b128_gemm_backward(c.layer, c.xq, c.xs, bf16_dev(db), need_dx=False)
    err = BF16 * (np.abs(D).T @ np.abs(c.X))
    ref = D.T @ c.X
    assert_within(f64_of(dw), ref, BF16 * (np.abs(ref) + err) + err + 100 * F32 * (np.abs(D).T @ np.abs(c.X)))


@pytest.mark.parametrize("T,out,inp", BACKWARD)
def test_gated_backward(T, out, inp):
    c = Inputs(978, T, out, inp)
    hb = grads_of(T, out, out // 2)
    dh = oracle.bf16_bits_to_f64(hb)
    dx, wx = guarded(T, inp, torch.bfloat16, 3.0)
    dw, ww = guarded(out, inp, torch.bfloat16, 3.0)
    ops().fp8b128_gated_backward(c.layer, c.xq, c.xs, bf16_dev(hb), dx=dx, dw=dw)
    D = oracle.fp8b128_gated_grads(c.X, c.W, dh)
    g, u, eg, eu = sums_and_error(c)
    # |silu'| <= 1.1, |silu''| <= 0.5; ten fp32 roundings, then one to bf16
    a = np.abs(dh)
    eD = np.concatenate([a * (1.1 * eu + 0.5 * eg * (np.abs(u) + eu)), a * 1.1 * eg], axis=1)
    eD = eD + (BF16 + 10 * F32) * (np.abs(D) + eD)
    check_product_grads(f64_of(dx), f64_of(dw), D, eD, c.X, c.W)
    assert rel_l2(f64_of(dx), D @ c.W) <= 2 * BF16 and rel_l2(f64_of(dw), D.T @ c.X) <= 2 * BF16
    check_guards(wx, 3.0)
    check_guards(ww, 3.0)


@pytest.mark.parametrize("T", [3, 90])
def test_gradients_of_special_scales(T):
    # a block the quantizer could not represent (scale NaN, zero codes) makes its inputs' columns
    # of dw NaN; zero, tiny, huge and negative scales are values like others
    c = Inputs(989, T, 96, 400)
    xs, codes = c.scales.copy(), c.codes.copy()
    xs[1, 2], codes[1, 256:384] = np.nan, 0
    xs[0, 0], xs[2, 0], xs[2, 1] = 0.0, -xs[2, 0], -2.0 ** -3
    xs[0, 1], xs[0, 3] = 2.0 ** -120, 2.0 ** 30
    codes[0, 384:] = 0x38
    X = oracle.fp8b128_activations(codes, xs)
    db = grads_of(T, 96, 96)
    D = oracle.bf16_bits_to_f64(db)
    dx, dw = ops().fp8b128_gemm_backward(c.layer, to_dev(codes), to_dev(xs), bf16_dev(db))
    assert torch.isfinite(dx.float()).all()
    got = f64_of(dw)
    assert np.isnan(got[:, 256:384]).all()
    keep = np.r_[0:256, 384:400]
    mag = np.abs(D).T @ np.abs(X[:, keep])
    ref = D.T @ X[:, keep]
    # one scale is no power of two (the negative ones among them): X rounded to bf16
    assert_within(got[:, keep], ref, BF16 * (np.abs(ref) + mag) + (BF16 + 100 * F32) * mag)


def test_backward_needs():
    c = Inputs(979, 50, 96, 272)
    dh = bf16_dev(grads_of(50, 96, 48))
    o = ops()
    dx, dw = o.fp8b128_gated_backward(c.layer, c.xq, c.xs, dh)
    dx1, none = o.fp8b128_gated_backward(c.layer, c.xq, c.xs, dh, need_dw=False)
    assert none is None and torch.equal(dx, dx1)
    none, dw1 = o.fp8b128_gated_backward(c.layer, c.xq, c.xs, dh, need_dx=False)
    assert none is None and torch.equal(dw, dw1)
    ws = o.fp8b128_workspace(50, 96, 272, dev())
    ws.fill_(255)  # the workspace need not be cleared
    dx2, dw2 = o.fp8b128_gated_backward(c.layer, c.xq, c.xs, dh, ws=ws)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


@pytest.mark.parametrize("T,out,inp", [(70, 96, 272), (333, 1056, 272), (580, 1056, 144), (580, 64, 1296),
                                       (420, 2848, 2832), (850, 64, 2064)])
def test_one_gradient_alone(T, out, inp):
    c = Inputs(995, T, out, inp)
    db = grads_of(T, out, out)
    D = oracle.bf16_bits_to_f64(db)
    o, dy = ops(), bf16_dev(db)
    dx, none = o.fp8b128_gemm_backward(c.layer, c.xq, c.xs, dy, need_dw=False)
    assert none is None
    none, dw = o.fp8b128_gemm_backward(c.layer, c.xq, c.xs, dy, need_dx=False)
    assert none is None
    check_product_grads(f64_of(dx), f64_of(dw), D, 0 * D, c.X, c.W)


def test_no_tokens():
    o = ops()
    c = Inputs(980, 3, 96, 272)
    xq, xs = c.xq[:0], c.xs[:0]
    assert o.fp8b128_gemm(c.layer, xq, xs).shape == (0, 96)
    assert o.fp8b128_gated(c.layer, xq, xs).shape == (0, 48)
    dw = torch.full((96, 272), 9.0, dtype=torch.bfloat16, device=dev())
    for fn, width in ((o.fp8b128_gemm_backward, 96), (o.fp8b128_gated_backward, 48)):
        dw.fill_(9.0)
        dx, _ = fn(c.layer, xq, xs, torch.empty((0, width), dtype=torch.bfloat16, device=dev()), dw=dw)
        assert dx.shape == (0, 272) and bool((dw == 0).all())
    codes, scales = o.fp8b128_quantize(torch.empty((0, 272), dtype=torch.bfloat16, device=dev()))
    assert codes.shape == (0, 272) and scales.shape == (0, 3)


# ---- used together --------------------------------------------------------------------------
def ffn_layers(H, I):
    L = ops().Fp8b128Layer
    return (L.from_host(fp8b128_layer(981, 2 * I, H), dev()), L.from_host(fp8b128_layer(982, H, I), dev()))


@pytest.mark.parametrize("T,H,I", [(1, 5120, 768), (30, 400, 144), (300, 272, 208)])
def test_ffn_is_its_four_calls(T, H, I):
    o = ops()
    gate_up, down = ffn_layers(H, I)
    x = bf16_from_normal(rng_for(981, 3, T), (T, H))
    for flags in (0, o.TQ_OUT_BF16):
        y = o.fp8b128_ffn(gate_up, down, bf16_dev(x), flags=flags)
        h = o.fp8b128_gated(gate_up, *o.fp8b128_quantize(bf16_dev(x)))
        assert torch.equal(y, o.fp8b128_gemm(down, *o.fp8b128_quantize(h), flags=flags))
    # and against the formulas: the codes of h are half a step of E4M3 (2^-4) from h
    X = oracle.fp8b128_activations(*oracle.fp8b128_quantize(x))
    hr = oracle.fp8b128_gated(X, oracle.fp8b128_weights(gate_up.codes.cpu().numpy(), gate_up.scales.cpu().numpy()))
    ref = hr @ oracle.fp8b128_weights(down.codes.cpu().numpy(), down.scales.cpu().numpy()).T
    assert rel_l2(f64_of(y), ref) <= 2.0 ** -4


def training_step(o, gate_up, down, x, dy):
    """Forward with 8-bit activations kept, and every gradient of the block."""
    xc = o.fp8b128_quantize(x)
    h = o.fp8b128_gated(gate_up, *xc)
    hc = o.fp8b128_quantize(h)
    y = o.fp8b128_gemm(down, *hc, flags=o.TQ_OUT_BF16)
    dh, dwd = o.fp8b128_gemm_backward(down, *hc, dy)
    dx, dwg = o.fp8b128_gated_backward(gate_up, *xc, dh)
    return y, dx, dwd, dwg


def test_training_step_against_the_formulas():
    o = ops()
    T, H, I = 140, 400, 208
    gate_up, down = ffn_layers(H, I)
    x = bf16_from_normal(rng_for(983, 3), (T, H))
    db = grads_of(T, H, H)
    y, dx, dwd, dwg = training_step(o, gate_up, down, bf16_dev(x), bf16_dev(db))
    Wg = oracle.fp8b128_weights(gate_up.codes.cpu().numpy(), gate_up.scales.cpu().numpy())
    Wd = oracle.fp8b128_weights(down.codes.cpu().numpy(), down.scales.cpu().numpy())
    X = oracle.fp8b128_activations(*oracle.fp8b128_quantize(x))
    h = oracle.fp8b128_gated(X, Wg)
    dy = oracle.bf16_bits_to_f64(db)
    D = oracle.fp8b128_gated_grads(X, Wg, dy @ Wd)
    # h in 8 bits is the one coarse rounding (2^-4); the others are bf16's
    assert rel_l2(f64_of(y), h @ Wd.T) <= 2.0 ** -4
    assert rel_l2(f64_of(dwd), dy.T @ h) <= 2.0 ** -4
    assert rel_l2(f64_of(dx), D @ Wg) <= 3 * BF16
    assert rel_l2(f64_of(dwg), D.T @ X) <= 3 * BF16


@pytest.mark.parametrize("T", [5, 300])
def test_replayed_graph_equals_eager(T):
    o = ops()
    H, I = 400, 208
    gate_up, down = ffn_layers(H, I)
    x = bf16_dev(bf16_from_normal(rng_for(984, 3), (T, H)))
    dy = bf16_dev(grads_of(T, H, H))
    for _ in range(2):
        training_step(o, gate_up, down, x, dy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = training_step(o, gate_up, down, x, dy)
    for k in range(3):  # other inputs in the same memory, eager work between the replays
        x.copy_(bf16_dev(bf16_from_normal(rng_for(985 + k, 3), (T, H))))
        eager = training_step(o, gate_up, down, x, dy)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, eager):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T,out,inp", [(70, 96, 272), (1100, 64, 272), (500, 1056, 272)])
def test_two_graphs_share_a_workspace(T, out, inp):
    # on one stream, in any order: one range of tokens, several, and X widened first
    o = ops()
    c = Inputs(993, T, out, inp)
    dy, dh = bf16_dev(grads_of(T, out, out)), bf16_dev(grads_of(T, out, out // 2))
    ws = o.fp8b128_workspace(T, out, inp, dev())
    calls = [lambda: o.fp8b128_gemm_backward(c.layer, c.xq, c.xs, dy, ws=ws),
             lambda: o.fp8b128_gated_backward(c.layer, c.xq, c.xs, dh, ws=ws)]
    for call in calls:
        call()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for call in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(call())
    for k in range(3):
        dy.copy_(bf16_dev(grads_of(T, out, out)) * (k + 1))
        dh.copy_(bf16_dev(grads_of(T, out, out // 2)) * (k - 1))
        for g in (0, 1, 0, 1, 1):
            graphs[g].replay()
        eager = [call() for call in calls]
        graphs[0].replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, eager):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_two_streams_and_repeats_give_the_same_bits():
    o = ops()
    T, H, I = 200, 656, 272
    gate_up, down = ffn_layers(H, I)
    xs = [bf16_dev(bf16_from_normal(rng_for(986, 3, k), (T, H))) for k in range(2)]
    dy = bf16_dev(grads_of(T, H, H))
    ref = [training_step(o, gate_up, down, x, dy) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(3):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[k] = training_step(o, gate_up, down, xs[k], dy)
    torch.cuda.synchronize()
    for k in range(2):
        for a, b in zip(ref[k], got[k]):
            assert torch.equal(a, b)


def test_a_layer_follows_its_tensors():
    # tensors given other memory are found and checked again; one that does not fit is refused
    o = ops()
    c, other = Inputs(990, 6, 96, 272), Inputs(991, 6, 64, 400)
    L = o.Fp8b128Layer(c.layer.codes.clone(), c.layer.scales.clone())
    ref = o.fp8b128_gemm(c.layer, c.xq, c.xs)
    assert torch.equal(ref, o.fp8b128_gemm(L, c.xq, c.xs))
    L.codes.data, L.scales.data = other.layer.codes, other.layer.scales
    assert torch.equal(o.fp8b128_gemm(L, other.xq, other.xs),
                       o.fp8b128_gemm(other.layer, other.xq, other.xs))
    dy = bf16_dev(grads_of(6, 64, 64))
    assert torch.equal(o.fp8b128_gemm_backward(L, other.xq, other.xs, dy)[1],
                       o.fp8b128_gemm_backward(other.layer, other.xq, other.xs, dy)[1])
    L.codes.data = c.layer.codes.clone()
    with pytest.raises(ValueError):
        o.fp8b128_gemm(L, c.xq, c.xs)
    L.scales.data = c.layer.scales.clone()
    assert torch.equal(ref, o.fp8b128_gemm(L, c.xq, c.xs))


def test_layers_are_copied_with_their_tensors():
    o = ops()
    c = Inputs(994, 6, 96, 272)
    ref = o.fp8b128_gemm(c.layer, c.xq, c.xs)
    L = copy.deepcopy(c.layer)
    assert L.codes.data_ptr() != c.layer.codes.data_ptr()
    c.layer.codes.zero_()
    assert torch.equal(ref, o.fp8b128_gemm(L, c.xq, c.xs))
    assert torch.equal(ref, o.fp8b128_gemm(pickle.loads(pickle.dumps(L)), c.xq, c.xs))


@pytest.mark.parametrize("out,inp", [(32, 2064), (2080, 16)])
def test_offsets_past_32_bits(out, inp):
    # 2^21 + 37 tokens: the bytes of codes (or of the results), and with 2,064 inputs (2,080
    # outputs) the elements too, pass 2^32. The tokens are zero (padding) up to the last 70.
    o = ops()
    T, n = (1 << 21) + 37, 70
    c, I = Inputs(992, n, out, inp), out // 2
    x = torch.zeros((T, inp), dtype=torch.bfloat16, device=dev())
    x[-n:] = (torch.from_numpy(c.X).to(torch.bfloat16)).to(dev())
    xq, xs = o.fp8b128_quantize(x)
    del x
    xqt, xst = o.fp8b128_quantize(torch.from_numpy(c.X).to(torch.bfloat16).to(dev()))
    assert torch.equal(xq[-n:], xqt) and torch.equal(xs[-n:], xst)
    assert not bool(xq[:-n].any()) and bool((xs[:-n] == 1).all())
    A = np.abs(c.X) @ np.abs(c.W).T
    ref = c.X @ c.W.T
    for flags in (0, o.TQ_OUT_BF16):
        y = o.fp8b128_gemm(c.layer, xq, xs, flags=flags)
        assert_within(f64_of(y[-n:]), ref, BF16 * np.abs(ref) + FP8_SUM * A if flags
                      else (inp + inp / 128 + 10) * F32 * A)
        assert not bool(y[:-n].any())
        del y
    h = o.fp8b128_gated(c.layer, xq, xs)
    assert not bool(h[:-n].any())
    g, u, eg, eu = sums_and_error(c)
    href = oracle.fp8b128_gated(c.X, c.W)
    assert_within(f64_of(h[-n:]), href, BF16 * np.abs(href) + 1.1 * eg * (np.abs(u) + eu)
                  + np.abs(oracle.silu(g)) * eu + 8 * F32 * np.abs(href) + 2.0 ** -133)
    del h
    # padding has no gradient: the sums over the tokens are those of the last ones
    db = grads_of(n, out, out)
    dy = torch.zeros((T, out), dtype=torch.bfloat16, device=dev())
    dy[-n:] = bf16_dev(db)
    D = oracle.bf16_bits_to_f64(db)
    dx, dw = o.fp8b128_gemm_backward(c.layer, xq, xs, dy)
    check_product_grads(f64_of(dx[-n:]), f64_of(dw), D, 0 * D, c.X, c.W)
    assert not bool(dx[:-n].any())
    del dx, dw
    hb = grads_of(n, out, I)
    dh = torch.zeros((T, I), dtype=torch.bfloat16, device=dev())
    dh[-n:] = bf16_dev(hb)
    dx, dw = o.fp8b128_gated_backward(c.layer, xq, xs, dh)
    a = np.abs(oracle.bf16_bits_to_f64(hb))
    D = oracle.fp8b128_gated_grads(c.X, c.W, oracle.bf16_bits_to_f64(hb))
    eD = np.concatenate([a * (1.1 * eu + 0.5 * eg * (np.abs(u) + eu)), a * 1.1 * eg], axis=1)
    check_product_grads(f64_of(dx[-n:]), f64_of(dw), D, eD + (BF16 + 10 * F32) * (np.abs(D) + eD), c.X, c.W)
    assert not bool(dx[:-n].any())


def test_timing_hook_covers_one_product():
    o = ops()
    c = Inputs(987, 40, 288, 400)
    ref = o.fp8b128_gemm(c.layer, c.xq, c.xs)
    start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    stop.record()
    torch.cuda.synchronize()
    o.time_kernel(start, stop)
    assert torch.equal(ref, o.fp8b128_gemm(c.layer, c.xq, c.xs))
    torch.cuda.synchronize()
    first = start.elapsed_time(stop)
    assert 0 < first < 50
    o.fp8b128_gated(c.layer, c.xq, c.xs)  # consumed: the events stay as they were
    torch.cuda.synchronize()
    assert start.elapsed_time(stop) == first


def test_wrappers_refuse_tensors_that_do_not_fit():
    o = ops()
    c = Inputs(988, 6, 96, 272)
    d = dev()
    e = torch.empty
    bad = [
        lambda: o.Fp8b128Layer(c.layer.codes, c.layer.scales[:, :2].contiguous()),
        lambda: o.Fp8b128Layer(c.layer.codes.float(), c.layer.scales),
        lambda: o.Fp8b128Layer(c.layer.codes.t(), c.layer.scales),
        lambda: o.fp8b128_gemm(c.layer, c.xq[:, :256].contiguous(), c.xs),
        lambda: o.fp8b128_gemm(c.layer, c.xq, c.xs[:5]),
        lambda: o.fp8b128_gemm(c.layer, c.xq, c.xs.double()),
        lambda: o.fp8b128_gemm(c.layer, c.xq.t(), c.xs),
        lambda: o.fp8b128_gemm(c.layer, c.xq, c.xs, out=e((6, 96), dtype=torch.bfloat16, device=d)),
        lambda: o.fp8b128_gemm(c.layer, c.xq, c.xs, out=e((5, 96), device=d)),
        lambda: o.fp8b128_gated(c.layer, c.xq, c.xs, out=e((6, 96), dtype=torch.bfloat16, device=d)),
        lambda: o.fp8b128_gemm_backward(c.layer, c.xq, c.xs, e((6, 48), dtype=torch.bfloat16, device=d)),
        lambda: o.fp8b128_gated_backward(c.layer, c.xq, c.xs, e((6, 96), dtype=torch.bfloat16, device=d)),
        lambda: o.fp8b128_gated_backward(c.layer, c.xq, c.xs, e((6, 48), device=d)),
        lambda: o.fp8b128_quantize(e((4, 128), device=d)),
        lambda: o.fp8b128_quantize(e((4, 256), dtype=torch.bfloat16, device=d)[:, ::2]),
        lambda: o.fp8b128_ffn(c.layer, c.layer, e((4, 128), dtype=torch.bfloat16, device=d)),
    ]
    for k, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print("accepted", k)
    with pytest.raises(RuntimeError):  # the library's own check: the workspace is too small
        o.fp8b128_gated_backward(c.layer, c.xq, c.xs, e((6, 48), dtype=torch.bfloat16, device=d),
                                 ws=e((64,), dtype=torch.uint8, device=d))
