"""Block-128 FP8 projections and activations, their product, the gated feed-forward product
and the gradients of both (FORMAT F22-F26).

TEST INFRASTRUCTURE (see the package docstring). Written from the definitions: E4M3 values
(OCP "E4M3FN") times one scale per 128 x 128 block of a weight, or per 128 inputs of an
activation row; every sum in FP64. The only roundings are those of the quantizer, which are
its definition.
"""

import math

import numpy as np

from .ffn import silu
from .fpbits import bf16_bits_to_f64
from .mx import e4m3_all_values, e4m3_round

BLOCK = 128


def fp8b128_blocks(n):
    """Scales along a side of n: one per 128, the last for what is left."""
    return -(-n // BLOCK)


def fp8b128_scale(amax):
    """The activation scale of a block whose largest magnitude is amax: 2^k with k the
    smallest integer >= -126 such that amax <= 448 * 2^k; 1 for a zero block; NaN if amax is
    not finite."""
    if not math.isfinite(amax):
        return math.nan
    if amax == 0.0:
        return 1.0
    k = -126
    while amax > math.ldexp(448.0, k):
        k += 1
    return math.ldexp(1.0, k)


def fp8b128_quantize(x_bits):
    """(codes uint8 [rows, n], scales float64 [rows, blocks]) of bf16 patterns [rows, n]."""
    x = bf16_bits_to_f64(x_bits)
    rows, n = x.shape
    nb = fp8b128_blocks(n)
    codes = np.zeros((rows, n), dtype=np.uint8)
    scales = np.zeros((rows, nb))
    for r in range(rows):
        for b in range(nb):
            v = x[r, BLOCK * b:BLOCK * (b + 1)]
            top = np.max(np.abs(v))  # NaN if the block holds one
            s = fp8b128_scale(float(top))
            scales[r, b] = s
            if not math.isnan(s):
                codes[r, BLOCK * b:BLOCK * (b + 1)] = e4m3_round(v / s)
    return codes, scales


def fp8b128_activations(codes, scales):
    """X [T, in] (FP64) of activation codes and their scales."""
    v = e4m3_all_values()[np.asarray(codes, dtype=np.uint8)]
    return v * np.repeat(np.asarray(scales, dtype=np.float64), BLOCK, axis=1)[:, :v.shape[1]]


def fp8b128_weights(codes, scales):
    """W [out, in] (FP64) of a projection's codes and block scales."""
    v = e4m3_all_values()[np.asarray(codes, dtype=np.uint8)]
    s = np.repeat(np.repeat(np.asarray(scales, dtype=np.float64), BLOCK, axis=0), BLOCK, axis=1)
    return v * s[:v.shape[0], :v.shape[1]]


def fp8b128_gated(X, W):
    """h [T, I] = silu(X Wg^T) * (X Wu^T); W [2I, in] is the gate's rows, then the up's."""
    half = W.shape[0] // 2
    return silu(X @ W[:half].T) * (X @ W[half:].T)


def fp8b128_gated_grads(X, W, dh):
    """The gradients [T, 2I] of the gate's and the up's sums, from dh [T, I]."""
    half = W.shape[0] // 2
    g, u = X @ W[:half].T, X @ W[half:].T
    s = 1.0 / (1.0 + np.exp(-g))
    return np.concatenate([dh * u * (s + g * s * (1.0 - s)), dh * g * s], axis=1)
