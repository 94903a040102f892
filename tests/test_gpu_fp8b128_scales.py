"""Scales at the ends of fp32 in the fp8b128 products and gradients (FORMAT F22-F26): infinities,
and finite scales whose product is not a normal number. Bounds as stated there: a block's products
are multiplied by the two scales' fp32 product, which is off by 2^-24 of it or 2^-150."""

import numpy as np
import pytest

import oracle
from gpu_helpers import dev, gpu, needs_gpu, ops, to_dev, torch
from workloads import bf16_from_normal, fp8b128_layer, rng_for

pytestmark = [gpu, needs_gpu]

BF16, F32, FP8_SUM = 2.0 ** -8, 2.0 ** -23, 2.0 ** -10
TOKENS = [1, 2, 3, 70, 300, 2100]
OUT = 288
INPUTS = [400, 1200]  # one or two tokens: by strips, by a channel per wave


def host(T, n):
    lay = fp8b128_layer(1020, OUT, n)
    codes, scales = oracle.fp8b128_quantize(bf16_from_normal(rng_for(1020, 3), (T, n)))
    return lay["codes"], lay["scales"].astype(np.float32), codes, scales.astype(np.float32)


def products(wc, ws, xc, xs):
    """The three forward results, and which activations they are of."""
    o = ops()
    L = o.Fp8b128Layer(to_dev(wc), to_dev(ws))
    x = to_dev(xc), to_dev(xs)
    return [f64(o.fp8b128_gemm(L, *x)), f64(o.fp8b128_gemm(L, *x, flags=o.TQ_OUT_BF16)),
            f64(o.fp8b128_gated(L, *x))]


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("n", INPUTS)
@pytest.mark.parametrize("T", TOKENS)
def test_an_infinite_scale_stays_in_its_outputs(T, n):
    wc, ws, xc, xs = host(T, n)
    xs[T // 2, 1] = np.inf
    for y in products(wc, ws, xc, xs):
        assert not np.isfinite(y[T // 2]).any()
        assert np.isfinite(np.delete(y, T // 2, 0)).all()
    wc, ws, xc, xs = host(T, n)
    ws[2, 3] = -np.inf  # channels 256 .. 287
    y32, y16, h = products(wc, ws, xc, xs)
    for y in (y32, y16):
        assert not np.isfinite(y[:, 256:]).any() and np.isfinite(y[:, :256]).all()
    # of the gated product up channels 112 .. 143
    assert not np.isfinite(h[:, 112:]).any() and np.isfinite(h[:, :112]).all()


@pytest.mark.parametrize("n", INPUTS)
@pytest.mark.parametrize("T", TOKENS)
def test_scales_whose_product_is_not_finite(T, n):
    wc, ws, xc, xs = host(T, n)
    xs[T // 2, 0], ws[0, 0] = 2.0 ** 100, 2.0 ** 28  # channels 0 .. 127
    for y in products(wc, ws, xc, xs)[:2]:
        assert not np.isfinite(y[T // 2, :128]).any()
        y[T // 2, :128] = 0
        assert np.isfinite(y).all()


@pytest.mark.parametrize("n", INPUTS)
@pytest.mark.parametrize("T", TOKENS)
def test_scales_whose_product_is_subnormal(T, n):
    wc, ws, xc, xs = host(T, n)
    xs[:], ws[:] = 2.0 ** -126, ws / ws.max() * np.float32(1.3 * 2.0 ** -12)
    X, W = oracle.fp8b128_activations(xc, xs), oracle.fp8b128_weights(wc, ws)
    codes = [oracle.fp8b128_activations(xc, np.ones_like(xs)), oracle.fp8b128_weights(wc, np.ones_like(ws))]
    ref, A = X @ W.T, np.abs(X) @ np.abs(W).T
    lost = 2.0 ** -149 * (np.abs(codes[0]) @ np.abs(codes[1]).T + n)
    y32, y16, _ = products(wc, ws, xc, xs)
    assert (np.abs(y32 - ref) <= (n + n / 128 + 10) * F32 * A + lost).all()
    err = FP8_SUM * A + lost
    assert (np.abs(y16 - ref) <= err + BF16 * (np.abs(ref) + err) + 2.0 ** -133).all()
    assert np.abs(ref).max() > 2.0 ** -126 and bool((y32 != 0).any())


@pytest.mark.parametrize("n", INPUTS)
@pytest.mark.parametrize("T", [1, 3, 300, 2100])
def test_activations_outside_the_range_of_bf16_in_dw(T, n):
    # the largest bf16 rounds to a code of 256 at 2^120, which is 2^128; a gradient of it is not finite
    xb = bf16_from_normal(rng_for(1021, 3), (T, n))
    xb[T // 2, 130] = 0x7F7F
    codes, scales = oracle.fp8b128_quantize(xb)
    assert scales[T // 2, 1] == 2.0 ** 120 and codes[T // 2, 130] == 0x78
    lay = fp8b128_layer(1021, OUT, n)
    o = ops()
    L = o.Fp8b128Layer.from_host(lay, dev())
    db = oracle.f32_to_bf16_bits_rne(rng_for(1021, 5).standard_normal((T, OUT)).astype(np.float32))
    dx, dw = o.fp8b128_gemm_backward(L, to_dev(codes), to_dev(scales.astype(np.float32)),
                                     to_dev(db, np.int16).view(torch.bfloat16))
    dw = f64(dw)
    assert bool(torch.isfinite(dx.float()).all())
    assert not np.isfinite(dw[:, 130]).any() and np.isfinite(np.delete(dw, 130, 1)).all()
