"""bf16 rows in MXFP4 (FORMAT F29).

TEST INFRASTRUCTURE (see the package docstring). The scale by its defining inequality, the
codes by a search over the sixteen values.
"""

import math

import numpy as np

from .fpbits import bf16_bits_to_f64
from .mxfp4 import E2M1_VALUES, e2m1_value, e8m0_value


def mxfp4_scale_byte(amax):
    """k + 127 for the smallest integer k >= -127 with amax <= 7 * 2^k; 127 for 0, 255 where amax
    is not finite."""
    if not math.isfinite(amax):
        return 255
    if amax == 0.0:
        return 127
    k = -127
    while amax > math.ldexp(7.0, k):
        k += 1
    return k + 127


def e2m1_round(v):
    """Codes of the values nearest to v, ties to the even code, above 6 the code of 6, with the
    sign of v."""
    v = np.asarray(v, dtype=np.float64)
    far = np.abs(np.abs(v)[..., None] - np.array(E2M1_VALUES))
    near = far == far.min(axis=-1, keepdims=True)
    first = np.argmax(near, axis=-1)
    both = near.sum(axis=-1) == 2
    code = np.where(both & (first % 2 == 1), first + 1, first)
    return (code + 8 * np.signbit(v)).astype(np.uint8)


def mxfp4_quantize(x_bits):
    """(codes uint8 [rows, n] one per element, scales uint8 [rows, n / 32]) of bf16 patterns."""
    x = bf16_bits_to_f64(x_bits)
    rows, n = x.shape
    scales = np.zeros((rows, n // 32), dtype=np.uint8)
    codes = np.zeros((rows, n), dtype=np.uint8)
    for r in range(rows):
        for b in range(n // 32):
            v = x[r, 32 * b:32 * b + 32]
            s = mxfp4_scale_byte(float(np.max(np.abs(v))))
            scales[r, b] = s
            if s != 255:
                codes[r, 32 * b:32 * b + 32] = e2m1_round(v / math.ldexp(1.0, s - 127))
    return codes, scales


def mxfp4_pack(codes):
    """Bytes [rows, n / 2] of codes [rows, n]: the even element in the low nibble."""
    return (codes[:, 0::2] | codes[:, 1::2] << 4).astype(np.uint8)


def mxfp4_values(codes, scales):
    """Values [rows, n] (FP64) of codes [rows, n] and their scales; a scale of 255 gives NaN."""
    value = np.array([e2m1_value(c) for c in range(16)])
    scale = np.array([e8m0_value(b) for b in range(256)])
    return value[codes] * np.repeat(scale[scales], 32, axis=1)
