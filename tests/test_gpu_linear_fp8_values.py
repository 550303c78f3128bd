"""Values of the E4M3 product on which its usual tests' bounds say little: gates far from zero, scales whose product leaves
the 32-bit numbers, long sums.
"""
import numpy as np
import pytest
import torch

from gpu_harness import DEV, bf16_np, pkg, to_np
from oracle import formats as F
from oracle import serving as S
from test_gpu_decoder import assert_within, f32_np
from test_gpu_serving import F8, U, up

pytestmark = pytest.mark.gpu


def gates_case(M, N, K, low, gated):
    """x is 1 in its first column, so that a gate is one rounded product of a token's scale and a code of w: the gates, float32
    [M, columns], spread over [low, 1.875 * low] and the mirrored ones."""
    r = np.random.default_rng(M + N + K)
    x = np.zeros((M, K), np.float32)
    x[:, 0] = 1.0
    xs = r.uniform(low, low * 1.0001 if low > 80 else 46.0, (M, 1)).astype(np.float32) * r.choice([1.0, -1.0], (M, 1), p=[0.1, 0.9]).astype(np.float32)
    cols = N // 2 if gated else N
    code = (-1.0 - (np.arange(cols) % 8) / 8 * (low <= 80)).astype(np.float32)
    w = np.zeros((N, K), np.float32)
    w[:cols, 0] = code
    w[cols:, 0] = 1.0
    ws = np.ones((-(-N // 128), -(-K // 128)), np.float32)
    ws[cols // 128:] = 2.0 ** 60
    up_factor = (xs * np.float32(2.0 ** 60)).astype(np.float64) if gated else 1.0
    return (up(x, F8), up(xs), up(w, F8), up(ws)), xs * code, up_factor


SIZES = [(2000, 256, 16), (40, 256, 1024), (40000, 512, 16)]  # whole tiles, K in slices, pairs


@pytest.mark.parametrize("act", ["silu", "swiglu"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_silu_is_rounded_as_the_exact_one(act, M, N, K):
    """The activation's own error is at most 2^-20 and the gate product's 2^-24: where the exact value is 2^-19 of itself away
    from the middle of two BF16 numbers, the result is the exact value's rounding, for gates from 5 to 86 on both sides."""
    c, g, u = gates_case(M, N, K, 5.0, act == "swiglu")
    g = g.astype(np.float64)
    exact = np.where(g < 0, g * np.exp(-np.abs(g)), g) / (1 + np.exp(-np.abs(g))) * u
    low, high = (F.bf16_round((exact * (1 + s)).astype(np.float32)) for s in (-2.0 ** -19, 2.0 ** -19))
    sure = low == high
    got = bf16_np(pkg.fp8_linear(*c, act))
    assert sure.mean() > 0.99 and np.abs(exact).min() > 1e-36
    assert np.array_equal(got[sure], low[sure])
    assert ((got == low) | (got == high)).all()


@pytest.mark.parametrize("act", ["silu", "swiglu"])
@pytest.mark.parametrize("low", [87.4, 88.0, 88.6, 89.5, 91.0])
def test_silu_where_its_exponential_is_not_normal(act, low):
    """e^-|g| is then a multiple of 2^-149, rounded twice: 2^-148 |g|, half a BF16 step (of the smallest normal number at least) and
    the rest's 2^-20."""
    c, g, u = gates_case(300, 256, 16, low, act == "swiglu")
    g = g.astype(np.float64)
    exact = np.where(g < 0, g * np.exp(-np.abs(g)), g) / (1 + np.exp(-np.abs(g))) * u
    got = bf16_np(pkg.fp8_linear(*c, act)).astype(np.float64)
    tol = np.abs(exact) * (2.0 ** -8 + 2.0 ** -19) + np.abs(g * u) * 2.0 ** -148 + 2.0 ** -134
    assert (np.abs(got - exact) <= tol).all()
    assert (got[g < 0] != 0).all()


@pytest.mark.parametrize("act", ["silu", "swiglu"])
def test_silu_of_gates_without_bounds(act):
    """Far on the negative side 0, far on the positive one the gate itself; infinite gates: +inf, and no number for inf times 0."""
    g = np.array([-105.0, -128.0, -1e3, -1e30, 40.0, 128.0, 1e3, 1e30, 0.0, 2.0 ** -130, -2.0 ** -130, np.inf, -np.inf, np.nan], np.float32)
    M = len(g)
    x, w = np.zeros((M, 16), np.float32), np.zeros((256, 16), np.float32)
    x[:, 0] = 1.0
    w[:, 0] = 1.0
    ws = np.ones((2, 1), np.float32)
    got = bf16_np(pkg.fp8_linear(up(x, F8), up(g[:, None]), up(w, F8), up(ws), act))[:, 0].astype(np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        want = F.bf16_round(g.astype(np.float64) / (1 + np.exp(-g.astype(np.float64))) * (g if act == "swiglu" else 1.0))
    assert np.array_equal(got[:11], want[:11])
    assert got[11] == np.inf and np.isnan(got[12:]).all()


@pytest.mark.parametrize("kind", ["high", "low"])
@pytest.mark.parametrize("M,N,K", [(5, 300, 1024), (130, 140, 512), (20000, 300, 512)])  # slices, whole tiles, pairs
def test_scales_at_the_ends_of_their_range(M, N, K, kind):
    """Products of two scales up to 2^126 and down to 2^-126, the scales themselves far beyond: against float64 by the bound of a 32-bit
    sum of 128 + K / 128 terms, half a BF16 step, and half of BF16's smallest step for what is below the normal numbers."""
    r = np.random.default_rng(M + 3 * N + K)
    groups = -(-K // 128)
    xs, ws = r.uniform(1, 2, (M, groups)), r.uniform(1, 2, (-(-N // 128), groups))
    x, w = r.choice([-1.0, 0.0, 1.0], (M, K)), r.choice([-1.0, 0.0, 1.0], (N, K))
    one, other = r.random((1, groups)) < 0.5, np.exp2(np.where(r.random((M, 1)) < 0.5, 0, 3 if kind == "low" else -3))
    if kind == "high":  # codes of 2^-9 and 2^-6
        x, w = x * 2.0 ** -9, w * 2.0 ** -6
        xs, ws = xs * np.where(one, 2.0 ** 120, 2.0 ** 4) * other, ws * np.where(one, 2.0 ** 4, 2.0 ** 120)
    else:
        x, w = x * 448, w * 448
        xs, ws = xs * np.where(one, 2.0 ** -126, 1.0) * other, ws * np.where(one, 1.0, 2.0 ** -126)
    xs, ws = xs.astype(np.float32), ws.astype(np.float32)
    product = xs.astype(np.float64)[:, :, None] * ws.astype(np.float64).T[None]
    assert product.max() < 2.0 ** 127 if kind == "high" else product.min() >= 2.0 ** -126
    c = up(x.astype(np.float32), F8), up(xs), up(w.astype(np.float32), F8), up(ws)
    at = np.unique(np.r_[0:min(M, 200), max(0, M - 60):M])
    out, _, mass = S.fp8_linear(f32_np(c[0][at]), xs[at], f32_np(c[2]), ws)
    tol = np.abs(out) * 2.0 ** -8 + mass * (128 + groups + 8) * U + 2.0 ** -134
    assert_within(bf16_np(pkg.fp8_linear(*c)[torch.from_numpy(at).to(DEV)]), out, tol, kind)


def test_a_layers_status_word():
    """Calls of every kind that end as they should leave it 0, also in a captured graph; a word elsewhere is refused."""
    word = torch.zeros(2, dtype=torch.int32, device=DEV)
    r = np.random.default_rng(3)
    layers = [pkg.FP8Linear.from_bf16(up(r.normal(size=s).astype(np.float32)).bfloat16(), dev_status=word if i else None)
              for i, s in enumerate(((300, 1024), (1024, 300 // 16 * 16), (40, 1024)))]
    inputs = [pkg.quantize_fp8(up(r.normal(size=(M, layer.w.shape[1])).astype(np.float32)).bfloat16()) for M, layer in zip((5, 20000, 200), layers)]
    for layer, x in zip(layers, inputs):
        layer(*x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        results = [layer(*x) for layer, x in zip(layers, inputs)]
    graph.replay()
    assert all(torch.equal(y, layer(*x)) for y, layer, x in zip(results, layers, inputs))
    assert layers[1].dev_status is word and layers[0].dev_status is not word
    assert not word.any() and not layers[0].dev_status.any()
    with pytest.raises(ValueError, match="dev_status must be int32"):
        pkg.FP8Linear(layers[0].w, layers[0].w_scale, dev_status=word.cpu())(*inputs[0])
