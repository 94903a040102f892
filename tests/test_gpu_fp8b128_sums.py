"""How far the fp8b128 products are off where a sum's terms cancel (FORMAT F24): rows with pairs of
large products of opposite sign beside small ones, every kernel of the products on the same rows.

Bounds, from the arithmetic stated in FORMAT F24:
  - fp32 results, and every result of one or two tokens: exact products, every add of a sum's
    path off by at most 2^-23 of A = |X| |W|^T;
  - other results (bf16, gated, gradients of gate and up): the fp8 matrix cores add the products
    of 8 consecutive inputs cut at 2^-13 of 2^(e + f), e and f the exponents of the codes with
    the largest e + f among them (a code below the smallest normal counts as 2^-6). That pair's
    own product is whole, so at most 7 are cut: less than 7/8 of 2^-10 of B = |X|+ |W|+^T, |.|+
    the magnitude with codes other than zero raised to 2^-6 at least. The fp32 adds of the
    groups and blocks are off by 2^-23 of A each, (inputs / 8 + inputs / 128 + 10) of them, which is below
    the remaining 2^-13 of B up to 7,000 inputs.
  - rounding to bf16: 2^-8 of the result."""

import numpy as np
import pytest

import oracle
from gpu_helpers import dev, gpu, needs_gpu, ops, to_dev, torch

pytestmark = [gpu, needs_gpu]

BF16, F32, FP8_SUM = 2.0 ** -8, 2.0 ** -23, 2.0 ** -10

# tokens of one, two, a strip, several strips and tiles
TOKENS = [1, 2, 3, 40, 300, 2100]


def e4m3(values):
    """Codes of values that E4M3 holds exactly."""
    codes = oracle.e4m3_round(np.asarray(values, dtype=np.float64))
    assert np.array_equal(oracle.e4m3_all_values()[codes], values)
    return codes


class Rows:
    def __init__(self, x, w):
        """x [T, in], w [out, in]: E4M3 values; all scales are one."""
        self.X, self.W = x, w
        blocks = -(-x.shape[1] // 128)
        self.codes = to_dev(e4m3(x))
        self.scales = torch.ones((x.shape[0], blocks), device=dev())
        self.layer = ops().Fp8b128Layer(to_dev(e4m3(w)), torch.ones((-(-w.shape[0] // 128), blocks), device=dev()))
        raised = [np.where(v != 0, np.maximum(np.abs(v), 2.0 ** -6), 0.0) for v in (x, w)]
        self.B = raised[0] @ raised[1].T
        self.A = np.abs(x) @ np.abs(w).T
        self.ref = x @ w.T

    def first(self, T):
        return self.codes[:T], self.scales[:T]

    def sum_error(self, T, exact):
        n = self.X.shape[1]
        if exact:
            return (n + n / 128 + 10) * F32 * self.A[:T]
        return FP8_SUM * self.B[:T]


def cancelling(T, out, n, small=7.5):
    """In every group of 8 inputs two products of 448 * 448 that cancel, and six small ones, which
    are a little less than what the matrix cores keep beside the two."""
    x, w = np.full((T, n), small), np.ones((out, n))
    x[:, 0::8], x[:, 1::8] = 448.0, -448.0
    w[:, 0::8] = w[:, 1::8] = 448.0
    return x, w


def outliers(T, out, n, seed=1010):
    """Log-uniform magnitudes over all that E4M3 holds, zeros, subnormal codes and pairs of
    outliers that cancel."""
    rng = np.random.default_rng(seed)

    def draw(rows):
        v = np.exp2(rng.integers(-9, 9, size=(rows, n)).astype(np.float64)) * (1 + rng.integers(0, 8, size=(rows, n)) / 8)
        v *= np.where(rng.random((rows, n)) < 0.5, -1.0, 1.0) * (rng.random((rows, n)) < rng.random((rows, 1)))
        return oracle.e4m3_all_values()[oracle.e4m3_round(np.clip(v, -448, 448))]

    x, w = draw(T), draw(out)
    p = rng.integers(0, n // 2, size=n // 32)
    x[:, 2 * p] = np.where(rng.random((T, 1)) < 0.5, 448.0, -256.0)
    x[:, 2 * p + 1] = -x[:, 2 * p]
    w[:, 2 * p] = w[:, 2 * p + 1] = 352.0
    return x, w


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def assert_within(got, ref, tol):
    bad = np.argwhere(~(np.abs(got - ref) <= tol))
    if bad.size:
        at = tuple(bad[0])
        raise AssertionError("%d of %d off, first at %s: %r, not %r within %.3g" % (
            len(bad), got.size, at, got[at], ref[at], tol[at]))


@pytest.mark.parametrize("make", [cancelling, outliers])
@pytest.mark.parametrize("out,n", [(16, 16), (16, 400), (272, 400), (2080, 272)])
def test_products(make, out, n):
    c = Rows(*make(max(TOKENS), out, n))
    for T in TOKENS:
        x, ref = c.first(T), c.ref[:T]
        assert_within(f64(ops().fp8b128_gemm(c.layer, *x)), ref, c.sum_error(T, True))
        err = c.sum_error(T, T <= 2)
        y = f64(ops().fp8b128_gemm(c.layer, *x, flags=ops().TQ_OUT_BF16))
        assert_within(y, ref, err + BF16 * (np.abs(ref) + err))


def test_what_the_fp8_matrix_cores_cut():
    # 7.5 is below 2^-13 of 2^(8 + 8) and beside such a pair nothing of it is kept; 8 is
    for out, small, kept in ((16, 7.5, 0.0), (16, 8.0, 8.0), (96, 7.5, 0.0)):
        c = Rows(*cancelling(300, out, 128, small))
        exact = 96 * small
        assert (c.ref == exact).all()
        for T in (1, 2, 3, 300):
            assert bool((ops().fp8b128_gemm(c.layer, *c.first(T)) == exact).all())
            y = ops().fp8b128_gemm(c.layer, *c.first(T), flags=ops().TQ_OUT_BF16)
            assert bool((y == (exact if T <= 2 else 96 * kept)).all())


def gated_bounds(c, T):
    """g, u and the bounds of their errors."""
    half, err = c.W.shape[0] // 2, c.sum_error(T, T <= 2)
    return c.ref[:T, :half], c.ref[:T, half:], err[:, :half], err[:, half:]


@pytest.mark.parametrize("make", [cancelling, outliers])
@pytest.mark.parametrize("out,n", [(32, 16), (32, 400), (288, 400), (2080, 272)])
def test_gated_and_gradients(make, out, n):
    x, w = make(max(TOKENS), out, n)
    # sums of the order of one, so that the gate is not saturated everywhere
    rng = np.random.default_rng(1011)
    c = Rows(x, w)
    factor = 2.0 ** -int(np.ceil(np.log2(np.median(np.abs(c.ref)) + 1e-30)))
    c.scales *= factor
    c.X, c.ref, c.A, c.B = c.X * factor, c.ref * factor, c.A * factor, c.B * factor
    dh_all = rng.standard_normal((max(TOKENS), out // 2)).astype(np.float32)
    db = oracle.f32_to_bf16_bits_rne(dh_all)
    half = out // 2
    for T in TOKENS:
        g, u, eg, eu = gated_bounds(c, T)
        with np.errstate(over="ignore"):
            ref, s = oracle.silu(g) * u, 1.0 / (1.0 + np.exp(-g))
        # |silu'| <= 1.1; eight fp32 roundings of the activation, and |g| 2^-24 in its exponent; a
        # sigmoid below 2^-126 may be zero
        tiny = 2.0 ** -126 * (1 + np.abs(g))
        tol = 1.1 * eg * (np.abs(u) + eu) + np.abs(oracle.silu(g)) * eu
        tol = tol + (8 + np.abs(g)) * F32 * np.abs(ref) + tiny * (1 + np.abs(u))
        tol = tol + BF16 * (np.abs(ref) + tol)
        assert_within(f64(ops().fp8b128_gated(c.layer, *c.first(T))), ref, tol)

        # the gradients of gate and up, |silu'| <= 1.1 and |silu''| <= 0.5, ten fp32 roundings and
        # the exponent's, one to bf16; then the two products of them, in fp32, and a last rounding
        dh = oracle.bf16_bits_to_f64(db[:T])
        a = np.abs(dh)
        slope = s + g * s * (1.0 - s)
        D = np.concatenate([dh * u * slope, dh * g * s], axis=1)
        # the terms of 1 + g (1 - s) cancel near g = -1.28: roundings of their magnitudes
        rounding = np.concatenate([a * np.abs(u) * s * (1 + np.abs(g) * (1 - s)), a * np.abs(g) * s], axis=1)
        eD = np.concatenate([a * (1.1 * eu + 0.5 * eg * (np.abs(u) + eu)), a * 1.1 * eg], axis=1)
        eD = eD + (10 + np.abs(np.tile(g, 2))) * F32 * rounding + np.tile(tiny * a * (1 + np.abs(u)), 2)
        eD = eD + BF16 * (np.abs(D) + eD) + 2.0 ** -126
        dx, dw = ops().fp8b128_gated_backward(c.layer, *c.first(T), to_dev(db[:T], np.int16).view(torch.bfloat16))
        aD, X = np.abs(D) + eD, c.X[:T]
        for got, want, mag, err, m in (
                (dx, D @ c.W, aD @ np.abs(c.W), eD @ np.abs(c.W), 2 * half),
                (dw, D.T @ X, aD.T @ np.abs(X), eD.T @ np.abs(X), T)):
            err = err + (m + m / 128 + 10) * F32 * mag
            assert_within(f64(got), want, err + BF16 * (np.abs(want) + err) + 2.0 ** -126)
