"""The rest of a model's step around its layers in float64: the E4M3 quantiser, the product with an E4M3
matrix in scaled blocks, rotary positions, and sampling.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np

from . import formats as F
from .decoder import FP8_GROUP, activate


def _spread(scale, rows: int, M: int, K: int) -> np.ndarray:
    """Scales per `rows` x 128 values (or per row, one column) -> one per value."""
    s = np.repeat(np.asarray(scale), rows, 0)[:M]
    return np.repeat(s, K if s.shape[1] == 1 else FP8_GROUP, 1)[:, :K]


def quantize_fp8(x, rows: int = 1):
    """BF16 values [M, K] (as float32) -> E4M3 bytes and float32 scales, by the rule's single 32-bit steps:
    scale = amax / 448 (1 when amax is 0), code = e4m3(x * (448 / amax)); below 2^-64 both factors are
    taken times 2^64, which changes no bit of a product that is not subnormal."""
    x = np.asarray(x, np.float32)
    M, K = x.shape
    m, n = -(-M // rows), -(-K // FP8_GROUP)
    b = np.zeros((m * rows, n * FP8_GROUP), np.float32)
    b[:M, :K] = np.abs(x)
    amax = b.reshape(m, rows, n, FP8_GROUP).max((1, 3))
    one = np.float32(1)
    scale = np.where(amax == 0, one, amax / np.float32(448))
    up = np.where(amax < np.float32(2.0 ** -64), np.float32(2.0 ** 64), one)
    inv = np.where(amax == 0, one, np.float32(448) / np.where(amax == 0, one, amax * up))
    return F.e4m3_encode((x * _spread(up, rows, M, K)) * _spread(inv, rows, M, K)), scale


def fp8_linear(x, x_scale, w, w_scale, activation: str = "identity"):
    """x [M, K], w [N, K] values of E4M3 codes, x_scale [M, 1 or ceil(K / 128)], w_scale per 128 x 128: the result,
    the product before the activation, and the sum of its terms' magnitudes, which bounds a 32-bit sum's error."""
    (M, K), N = x.shape, w.shape[0]
    x = np.asarray(x, np.float64) * _spread(np.asarray(x_scale, np.float64), 1, M, K)
    w = np.asarray(w, np.float64) * np.repeat(np.repeat(np.asarray(w_scale, np.float64), FP8_GROUP, 0)[:N], FP8_GROUP, 1)[:, :K]
    y = x @ w.T
    return activate(y, activation), y, np.abs(x) @ np.abs(w).T


def rotary(x, positions, inv_freq, axes=None, adjacent: bool = False):
    """x [N, heads, dim] turned by positions [num_axes, N]: the result, the magnitudes |a| + |b| of each value's
    pair (0 for values that are not turned), and the angles [N, pairs]."""
    x = np.asarray(x, np.float64)
    half = len(inv_freq)
    axes = np.zeros(half, int) if axes is None else np.asarray(axes, int)
    angle = np.asarray(positions, np.float64)[axes].T * np.asarray(inv_freq, np.float64)
    i = np.arange(half)
    first, second = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
    z = (x[..., first] + 1j * x[..., second]) * np.exp(1j * angle)[:, None, :]
    out, size = x.copy(), np.zeros(x.shape)
    out[..., first], out[..., second] = z.real, z.imag
    size[..., first] = size[..., second] = np.abs(x[..., first]) + np.abs(x[..., second])
    return out, size, angle


def _front(w, part: float) -> int:
    """How many of the descending weights reach that part of their sum. Near a border the float64 sums say nothing (two equal
    weights and a 1e-20 make 2.0): there, in rational numbers, a weight that underflowed counting as less than any."""
    sums = np.cumsum(w)
    reached = sums >= part * sums[-1]
    j = int(np.argmax(reached))
    near = np.flatnonzero(np.abs(sums - part * sums[-1]) <= 1e-9 * sums[-1])
    if not len(near):
        return j + 1
    exact = [Fraction(float(v)) if v > 0 else Fraction(1, 10 ** 400) for v in w]
    target = Fraction(part) * sum(exact)
    first = int(near[0])
    upto = sum(exact[:first])
    while True:
        upto += exact[first]
        first += 1
        if upto >= target or first == len(exact):
            return first


def sample(logits, uniform: float, temperature: float = 1.0, top_k: int = 0, top_p: float = 1.0, min_p: float = 0.0) -> int:
    """One row's token, by the filters as they are defined on the sorted tokens."""
    l = np.asarray(logits, np.float64)
    l = np.where(np.isnan(l), -np.inf, l)
    alive = [i for i in range(len(l)) if l[i] > -np.inf]
    if not alive:
        return -1
    order = sorted(alive, key=lambda i: (-l[i], i))
    top = l[order[0]]
    if not temperature >= 2.0 ** -100:
        return order[0]
    with np.errstate(invalid="ignore"):
        z = [0.0 if l[i] == top else (l[i] - top) / min(temperature, 2.0 ** 100) for i in order]
    w = np.exp(z)
    n = len(order) if top_k <= 0 else min(top_k, len(order))
    if top_p < 1.0:
        n = _front(w[:n], max(float(top_p), 0.0))
    if min_p > 0:
        n = max(1, sum(1 for j in range(n) if w[j] >= min_p or z[j] == 0.0))
    kept = sorted(zip(order[:n], w[:n]))
    u = min(max(uniform, 0.0), 1.0 - 2.0 ** -24) if uniform == uniform else 0.0
    sums = np.cumsum([v for _, v in kept])
    return next(i for (i, _), c in zip(kept, sums) if c > u * sums[-1])
