"""The E4M3 product's long sums, to the bound of how they are made: 128 terms by the tensor core, then a term for each block of K.

U = 2^-24. Within a block each of at most 128 additions is off by U of the sum of magnitudes, or 2 U if the tensor core cuts instead of
rounding; a block's scaling adds 3 U (the scales' product, the multiply-add's share), the blocks' additions U each, and the
slices' meeting at most 8. So (2 * 128 + ceil(K / 128) + 11) U of the magnitudes' sum, where one chain of K terms would have K: a
block of K = 7168 that is left out shows in some output, whichever it is. At K = 65536 a block of small scales can hide below the
rounding to BF16; the whole numbers of the last test show each one.
"""
import numpy as np
import pytest
import torch

from gpu_harness import DEV, bf16_np, pkg, to_np
from oracle import formats as F
from oracle import serving as S
from test_gpu_decoder import assert_within, f32_np
from test_gpu_serving import F8, SIZES, U, linear_case, up

pytestmark = pytest.mark.gpu


def bound(K):
    return (2 * 128 + -(-K // 128) + 11) * U


@pytest.mark.parametrize("mode", ["token", "group"])
@pytest.mark.parametrize("M,N,K", SIZES + [(1, 128, 7168), (200, 128, 65536), (2048, 256, 16384), (16, 256, 65536)])
def test_sums(M, N, K, mode):
    x, xs, w, ws = linear_case(M, N, K, mode)
    got = pkg.fp8_linear(x, xs, w, ws)
    at = np.unique(np.r_[0:min(M, 150), max(0, M - 40):M])
    out, _, mass = S.fp8_linear(f32_np(x[at]), to_np(xs)[at], f32_np(w), to_np(ws))
    assert_within(bf16_np(got[torch.from_numpy(at).to(DEV)]), out, mass * bound(K) + np.abs(out) * 2.0 ** -8 + 1e-30)


@pytest.mark.parametrize("M,N,K,mode", [(8192, 4096, 512, "group"), (5000, 7001, 400, "token"), (20000, 300, 1024, "group"),
                                        (40, 129021, 256, "group"), (3000, 3000, 2064, "group"), (12, 40000, 4096, "group")])
def test_sums_of_many_tiles(M, N, K, mode):
    x, xs, w, ws = linear_case(M, N, K, mode)
    got = pkg.fp8_linear(x, xs, w, ws)
    r = np.random.default_rng(2)
    rows = np.unique(np.r_[0:min(8, M), max(0, M - 8):M, r.integers(0, M, 150)])
    cols = np.unique(np.r_[0:8, N - 8:N, r.integers(0, N, 150)])
    out, _, mass = S.fp8_linear(f32_np(x)[rows], to_np(xs)[rows], f32_np(w), to_np(ws))
    tol = mass * bound(K) + np.abs(out) * 2.0 ** -8 + 1e-30
    assert_within(bf16_np(got[torch.from_numpy(rows)])[:, cols], out[:, cols], tol[:, cols])


def whole_case(M, N, K, mode, seed=0):
    """Codes of -2 to 2 and scales of 1 to 8 that are powers of two: every sum is a whole number below 2^24 (65536 * 4 * 64), exact in
    32 bits in any order."""
    r = np.random.default_rng(seed + M + N + K)
    groups = -(-K // 128)
    x, w = r.integers(-2, 3, (M, K)).astype(np.float32), r.integers(-2, 3, (N, K)).astype(np.float32)
    xs = np.exp2(r.integers(0, 4, (M, 1 if mode == "token" else groups))).astype(np.float32)
    ws = np.exp2(r.integers(0, 4, (-(-N // 128), groups))).astype(np.float32)
    return up(x, F8), up(xs), up(w, F8), up(ws)


@pytest.mark.parametrize("act", ["identity", "relu"])
@pytest.mark.parametrize("mode", ["token", "group"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 128, 65536), (3, 1000, 65536), (130, 300, 7168), (64, 129, 16384), (5, 40, 1040), (2048, 512, 16384),
                                   (20000, 300, 528), (333, 7001, 2000)])
def test_sums_that_are_exact(M, N, K, mode, act):
    """... so that the result is the exact sum's rounding, bit for bit: no term is lost, taken twice or scaled by another block's scale."""
    x, xs, w, ws = whole_case(M, N, K, mode)
    got = pkg.fp8_linear(x, xs, w, ws, act)
    at = np.unique(np.r_[0:min(M, 300), max(0, M - 60):M])
    out, _, mass = S.fp8_linear(f32_np(x[at]), to_np(xs)[at], f32_np(w), to_np(ws))
    assert mass.max() < 2.0 ** 24
    assert np.array_equal(bf16_np(got[torch.from_numpy(at).to(DEV)]), F.bf16_round(np.maximum(out, 0.0) if act == "relu" else out))
