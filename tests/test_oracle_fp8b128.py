"""Pins of the fp8b128 oracle (FORMAT F22-F26): the scale's closed form at every border, codes
against torch's float8_e4m3fn cast, block placement by constant blocks, the product against
scalar sums, the gradients against central differences of the forward formulas."""

import math

import numpy as np
import pytest

import oracle
from workloads import bf16_from_normal, fp8b128_layer, rng_for


def bits(values):
    return oracle.f64_to_bf16_bits_exact(np.asarray(values, dtype=np.float64))


def test_scale_borders():
    assert oracle.fp8b128_scale(448.0) == 1.0
    assert oracle.fp8b128_scale(450.0) == 2.0           # the next bf16 value
    assert oracle.fp8b128_scale(224.0) == 0.5
    assert oracle.fp8b128_scale(1.0) == 2.0 ** -8       # 1 <= 448 / 256, > 448 / 512
    assert oracle.fp8b128_scale(0.0) == 1.0
    assert math.isnan(oracle.fp8b128_scale(math.inf)) and math.isnan(oracle.fp8b128_scale(math.nan))
    assert oracle.fp8b128_scale(2.0 ** -133) == 2.0 ** -126   # the smallest scale
    top = (2.0 - 2.0 ** -7) * 2.0 ** 127                      # the largest bf16
    assert oracle.fp8b128_scale(top) == 2.0 ** 120 and top / 2.0 ** 120 <= 448.0
    for m in range(128):  # every bf16 mantissa: the largest code is above 224, at most 448
        v = (1 + m / 128) * 2.0 ** 3
        assert 224.0 < v / oracle.fp8b128_scale(v) <= 448.0


def test_quantize_against_torch_cast():
    torch = pytest.importorskip("torch")
    x = bf16_from_normal(rng_for(960, 3), (5, 300))
    x[2] = 0
    codes, scales = oracle.fp8b128_quantize(x)
    assert scales.shape == (5, 3) and (scales[2] == 1.0).all() and (codes[2] & 0x7F == 0).all()
    v = torch.from_numpy(oracle.bf16_bits_to_f64(x)).float()
    s = torch.from_numpy(np.repeat(scales, 128, 1)[:, :300]).float()
    ref = (v / s).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(codes, ref)
    # the value is within half a step of E4M3: 2^-4 of it, or half the smallest step
    X = oracle.fp8b128_activations(codes, scales)
    err = np.abs(X - v.double().numpy())
    assert (err <= np.maximum(2.0 ** -4 * np.abs(v.double().numpy()), 2.0 ** -10 * s.double().numpy())).all()


def test_quantize_non_finite_block():
    x = bf16_from_normal(rng_for(961, 3), (2, 272))
    x[0, 130] = 0x7F80   # +inf, block 1
    x[1, 271] = 0xFFC1   # NaN, the short last block
    codes, scales = oracle.fp8b128_quantize(x)
    assert np.isnan(scales[0, 1]) and np.isnan(scales[1, 2]) and np.isnan(scales).sum() == 2
    assert (codes[0, 128:256] == 0).all() and (codes[1, 256:] == 0).all()


def test_block_placement():
    out, inp = 272, 144
    scales = np.arange(1, 7, dtype=np.float64).reshape(3, 2)
    W = oracle.fp8b128_weights(np.full((out, inp), 0x38, dtype=np.uint8), scales)  # code 1.0
    for o in (0, 127, 128, 255, 256, 271):
        for i in (0, 127, 128, 143):
            assert W[o, i] == scales[o // 128, i // 128]
    X = oracle.fp8b128_activations(np.full((3, inp), 0xB8, dtype=np.uint8), scales)  # code -1.0
    assert X[2, 0] == -5 and X[2, 127] == -5 and X[2, 128] == -6 and X[0, 143] == -2


def test_gated_and_its_gradients_against_scalars():
    lay = fp8b128_layer(962, 32, 144)
    W = oracle.fp8b128_weights(lay["codes"], lay["scales"])
    X = oracle.bf16_bits_to_f64(bf16_from_normal(rng_for(962, 3), (3, 144)))
    dh = rng_for(962, 5).standard_normal((3, 16))
    h = oracle.fp8b128_gated(X, W)
    d = oracle.fp8b128_gated_grads(X, W, dh)
    for t in range(3):
        for i in range(16):
            g = sum(X[t, k] * W[i, k] for k in range(144))
            u = sum(X[t, k] * W[16 + i, k] for k in range(144))
            f = lambda g, u: g / (1 + math.exp(-g)) * u  # noqa: E731
            assert h[t, i] == pytest.approx(f(g, u), rel=1e-11, abs=1e-13)
            e = 1e-5
            assert d[t, i] == pytest.approx(dh[t, i] * (f(g + e, u) - f(g - e, u)) / (2 * e), rel=1e-7, abs=1e-8)
            assert d[t, 16 + i] == pytest.approx(dh[t, i] * (f(g, u + e) - f(g, u - e)) / (2 * e), rel=1e-7, abs=1e-8)


def test_input_and_weight_gradients_against_differences():
    # L = sum(dh * h); dL/dX = D W and dL/dW = D^T X with D the gradients of the sums
    lay = fp8b128_layer(963, 32, 48)
    W = oracle.fp8b128_weights(lay["codes"], lay["scales"])
    X = oracle.bf16_bits_to_f64(bf16_from_normal(rng_for(963, 3), (2, 48)))
    dh = rng_for(963, 5).standard_normal((2, 16))
    D = oracle.fp8b128_gated_grads(X, W, dh)
    dX, dW = D @ W, D.T @ X
    e = 1e-5
    for t, k in ((0, 0), (1, 47), (0, 17)):
        P, M = X.copy(), X.copy()
        P[t, k] += e
        M[t, k] -= e
        diff = np.sum(dh * (oracle.fp8b128_gated(P, W) - oracle.fp8b128_gated(M, W))) / (2 * e)
        assert dX[t, k] == pytest.approx(diff, rel=1e-6, abs=1e-7)
    for o, k in ((0, 0), (15, 30), (16, 0), (31, 47)):
        P, M = W.copy(), W.copy()
        P[o, k] += e
        M[o, k] -= e
        diff = np.sum(dh * (oracle.fp8b128_gated(X, P) - oracle.fp8b128_gated(X, M))) / (2 * e)
        assert dW[o, k] == pytest.approx(diff, rel=1e-6, abs=1e-7)
