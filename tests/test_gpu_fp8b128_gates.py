"""The gated product and its gradients over the whole range of the gate: sums from -40,000, where the
hardware's exponential overflows, to 40,000, where it vanishes, in every kernel, against the
formulas in FP64. All codes are 0, 1 or -1 and all sums exact in fp32, on the fp8 matrix cores too,
so the bounds are those of the activation's own roundings and of the products of the gradients."""

import numpy as np
import pytest

import oracle
from gpu_helpers import dev, gpu, needs_gpu, ops, to_dev, torch

pytestmark = [gpu, needs_gpu]

BF16, F32 = 2.0 ** -8, 2.0 ** -23
IN = 256


def layer_of(rng, sums):
    """A gated projection of 2 * len(sums) outputs. Its inputs are two blocks with scales 312.5 and
    0.625: for activations of one, the gate sums are `sums`, the up sums random."""
    half = len(sums)
    W = np.zeros((2 * half, IN))
    for o in range(half):
        if abs(sums[o]) == 40000.0:
            W[o, :128] = np.sign(sums[o])
        else:
            n = int(abs(sums[o]) / 0.625)
            assert n <= 128 and n * 0.625 == abs(sums[o])
            W[o, 128:128 + n] = np.sign(sums[o])
    W[half:] = rng.integers(-1, 2, size=(half, IN))
    scales = np.tile(np.array([[312.5, 0.625]], np.float32), (-(-2 * half // 128), 1))
    codes = np.where(W > 0, 0x38, np.where(W < 0, 0xB8, 0)).astype(np.uint8)
    return codes, scales, W * np.repeat(scales[0].astype(np.float64), 128)


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def assert_within(got, ref, tol):
    bad = np.argwhere(~(np.abs(got - ref) <= tol))
    if bad.size:
        at = tuple(bad[0])
        raise AssertionError("%d of %d off, first at %s: %r, not %r within %.3g" % (
            len(bad), got.size, at, got[at], ref[at], tol[at]))


@pytest.mark.parametrize("half", [16, 1040])
@pytest.mark.parametrize("T", [1, 2, 4, 40, 300, 2100])
def test_gate_range(T, half):
    rng = np.random.default_rng(1030)
    values = np.array([-40000.0, 40000.0, 0.0, -80.0, 80.0, -20.0, 20.0, -8.75, -5.0, -2.5, -1.25,
                       -0.625, 0.625, 1.25, 5.0, 8.75])
    codes, scales, W = layer_of(rng, values[np.arange(half) % len(values)])
    o = ops()
    L = o.Fp8b128Layer(to_dev(codes), to_dev(scales))
    # tokens of one, of minus one, and of zeros (padding)
    sign = np.array([1.0, -1.0, 1.0, 0.0])[np.arange(T) % 4]
    X = np.repeat(sign[:, None], IN, 1)
    x = (to_dev(np.where(X > 0, 0x38, np.where(X < 0, 0xB8, 0)).astype(np.uint8)),
         torch.ones((T, 2), device=dev()))
    gu = X @ W.T
    g, u = gu[:, :half], gu[:, half:]
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-g))
    # eight (gradients: ten) fp32 roundings, |g| 2^-24 in the exponent, and a sigmoid below 2^-126,
    # which may be zero
    ref, tiny = oracle.silu(g) * u, 2.0 ** -126 * (1 + np.abs(g)) * (1 + np.abs(u))
    err = (8 + np.minimum(np.abs(g), 128)) * F32 * np.abs(ref) + tiny
    assert_within(f64(o.fp8b128_gated(L, *x)), ref, err + BF16 * (np.abs(ref) + err))

    db = oracle.f32_to_bf16_bits_rne((0.25 * rng.standard_normal((T, half))).astype(np.float32))
    dh = oracle.bf16_bits_to_f64(db)
    a = np.abs(dh)
    with np.errstate(over="ignore"):
        D = oracle.fp8b128_gated_grads(X, W, dh)
    terms = np.concatenate([a * np.abs(u) * s * (1 + np.abs(g) * (1 - s)), a * np.abs(g) * s], axis=1)
    eD = (10 + np.minimum(np.abs(np.tile(g, 2)), 128)) * F32 * terms + np.tile(tiny * a, 2)
    eD = eD + BF16 * (np.abs(D) + eD)
    dx, dw = o.fp8b128_gated_backward(L, *x, to_dev(db, np.int16).view(torch.bfloat16))
    aD = np.abs(D) + eD
    for got, want, mag, e, n in ((dx, D @ W, aD @ np.abs(W), eD @ np.abs(W), 2 * half),
                                 (dw, D.T @ X, aD.T @ np.abs(X), eD.T @ np.abs(X), T)):
        e = e + (n + n / 128 + 10) * F32 * mag
        assert_within(f64(got), want, e + BF16 * (np.abs(want) + e) + 2.0 ** -126)
    # saturated gates pass the up gradient whole or not at all
    dead = g <= -40000
    assert (D[:, :half][dead] == 0).all() and (D[:, half:][dead] == 0).all()
