"""The operators around the routed experts in float64: RMS norm with the residual's addition and
its E4M3 output, the product of a few tokens with an NVFP4 matrix, the NVFP4 key/value cache and
the attention over it. Formats and the block rule are those of ``formats`` and ``quantize``.
"""
from __future__ import annotations

import math

import numpy as np

from . import formats as F
from . import quantize as Q

FP8_GROUP = 128


def fp8_groups(H: int, fp8: str) -> list[slice]:
    """Columns of each scale: one per row ("token") or per 128 columns, the last one short ("group")."""
    step = H if fp8 == "token" else FP8_GROUP
    return [slice(i, min(H, i + step)) for i in range(0, H, step)]


def add_rms_norm(x, weight, residual=None, eps: float = 1e-6, fp8: str | None = None) -> dict:
    """h = x + residual, f = h / sqrt(mean(h^2) + eps) * weight; per scale group scale = max|f| / 448
    (1 when it is 0) and the values f / scale that E4M3 rounds. Nothing is rounded here."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    f = h / np.sqrt((h * h).sum(-1, keepdims=True) / h.shape[-1] + eps) * np.asarray(weight, np.float64)
    out = {"residual": h, "y": f}
    if fp8:
        groups = fp8_groups(h.shape[-1], fp8)
        scale = np.stack([np.abs(f[:, g]).max(-1) for g in groups], -1) / F.E4M3_MAX
        scale[scale == 0] = 1.0
        out["scale"] = scale
        out["y8"] = np.concatenate([f[:, g] / scale[:, i:i + 1] for i, g in enumerate(groups)], -1)
    return out


def nvfp4_values(data, sf) -> np.ndarray:
    """Packed codes [..., n/2] and E4M3 bytes [..., n/16] -> float64 [..., n], without a global scale."""
    return F.e2m1_decode(F.unpack_e2m1(data)) * np.repeat(F.e4m3_decode(sf), 16, -1)


def activate(y, activation: str) -> np.ndarray:
    """act(gate) * up over [gate; up] columns for the gated kinds, act(y) for the others."""
    def sig(v):
        return 0.5 * (1.0 + np.tanh(0.5 * v))

    def gelu(v):
        return 0.5 * v * (1.0 + np.vectorize(math.erf, otypes=[float])(v / math.sqrt(2.0)))
    g, u = np.split(y, 2, -1) if activation in ("swiglu", "geglu") else (y, None)
    return {"swiglu": lambda: g * sig(g) * u, "geglu": lambda: gelu(g) * u, "relu2": lambda: np.maximum(g, 0) ** 2,
            "gelu": lambda: gelu(g), "relu": lambda: np.maximum(g, 0), "silu": lambda: g * sig(g),
            "identity": lambda: g}[activation]()


def linear(x, data, sf, alpha: float, activation: str = "identity", x_scale=None):
    """(act(alpha x W^T), alpha x W^T, |alpha| |x| |W|^T): the result, the product before the activation
    and the sum of its terms' magnitudes, which bounds the error of a 32-bit sum."""
    x = np.asarray(x, np.float64)
    if x_scale is not None:
        x = x * np.repeat(np.asarray(x_scale, np.float64), x.shape[1] if x_scale.shape[1] == 1 else FP8_GROUP,
                          -1)[:, :x.shape[1]]
    w = nvfp4_values(data, sf)
    y = x @ w.T * alpha
    return activate(y, activation), y, np.abs(x) @ np.abs(w).T * abs(alpha)


def kv_encode(x, g: float):
    """BF16 values [..., n] (as float32) -> codes [..., n/2], scale bytes [..., n/16], held values [..., n]."""
    x = np.asarray(x, np.float32)
    data, sf = Q.quantize_rows(x.reshape(-1, x.shape[-1]), g)
    data, sf = data.reshape(*x.shape[:-1], -1), sf.reshape(*x.shape[:-1], -1)
    return data, sf, nvfp4_values(data, sf) / g


def attend(q, k, v, scale: float):
    """One sequence and kv head: query rows q [T, G, D] against k, v [n, D]; row t sees the first
    n - (T - 1) + t tokens. Returns out [T, G, D], lse [T, G] and sum_j p_j |v_j| [T, G, D]."""
    T, n = q.shape[0], k.shape[0]
    out, lse = np.zeros(q.shape), np.full(q.shape[:2], -np.inf)
    mass = np.zeros(q.shape)
    for t in range(T):
        seen = n - (T - 1) + t
        if seen <= 0:
            continue
        s = np.asarray(q[t], np.float64) @ k[:seen].T * scale
        top = s.max(-1, keepdims=True)
        p = np.exp(s - top)
        total = p.sum(-1, keepdims=True)
        out[t], mass[t] = p @ v[:seen] / total, p @ np.abs(v[:seen]) / total
        lse[t] = (top + np.log(total))[:, 0]
    return out, lse, mass
