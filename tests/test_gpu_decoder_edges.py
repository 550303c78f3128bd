"""Edges of the operators around the routed experts on the GPU: scores and activations of extreme size,
numbers that are none, slices, several threads and streams. Tolerances as in test_gpu_decoder.py unless
a test says otherwise.
"""
import numpy as np
import pytest
import torch

from gpu_harness import DEV, bf16_np, pkg, to_np
from oracle import decoder as D
from test_gpu_decoder import (Pool, U, assert_within, bf16, check_attend, check_linear, f32_np, linear_case, queries,
                              run_linear, sequences)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ attention: large scores
def exact_scores_check(out, lse, q, held, Hkv, scale):
    """Against the oracle where every score is exact in 32 bits: only the weights' rounding (2^-10 of the
    mass) and the result's (2^-8 of the value) are left; the log-sum-exp has 8 roundings of its size."""
    B, T, Hq, Dh = q.shape
    G = Hq // Hkv
    qf = f32_np(q).astype(np.float64)
    for b in range(B):
        k, v = held[b]
        for h in range(Hkv):
            hs = slice(h * G, (h + 1) * G)
            o, l, mass = D.attend(qf[b, :, hs], k[:, h], v[:, h], scale)
            assert_within(bf16_np(out)[b, :, hs], o, np.abs(o) * (2.0 ** -8 + 2.0 ** -18) + mass * 2.0 ** -10 + 1e-30, "out")
            assert_within(to_np(lse).astype(np.float64)[b, :, hs], l, np.abs(l) * 8 * U + 2.0 ** -20, "lse")


@pytest.mark.parametrize("B,Hkv,G,T,Dh,page,n", [(2, 2, 4, 1, 128, 64, 700), (3, 1, 6, 4, 64, 16, 500), (1, 4, 8, 1, 128, 32, 30000),
                                               (40, 8, 4, 1, 128, 64, 3000), (1, 1, 16, 1, 128, 16, 5000), (1, 1, 30, 1, 64, 64, 4000)])
def test_attend_scores_past_24_bits(B, Hkv, G, T, Dh, page, n):
    """Finite queries whose scores are up to 2^36: a difference of two scores is 0 (several tokens share the
    maximum) or far above the exponential's range. A row has one dimension, so its scores are exact."""
    lens = [n - 7 * b for b in range(B)]
    p = Pool(sum(-(-m // page) for m in lens), page, Hkv, Dh)
    table, ln, held = sequences(p, lens, seed=n)
    r = np.random.default_rng(n)
    q = np.zeros((B, T, Hkv * G, Dh), np.float32)
    for i in np.ndindex(*q.shape[:3]):
        q[i][r.integers(0, Dh)] = (-1.0) ** r.integers(0, 2) * 2.0 ** r.integers(21, 36)
    q = bf16(q)
    out, lse = p.kv.attend(q, table, ln, softmax_scale=1.0)
    exact_scores_check(out, lse, q, held, Hkv, 1.0)


def test_attend_large_queries_along_one_key():
    """Queries along one token's key, scaled until scores pass 1e7 to 1e12: that token's values come out."""
    lens, page, Dh = [900, 2500], 64, 128
    p = Pool(60, page, 2, Dh)
    table, ln, held = sequences(p, lens, seed=3, spread=100.0)
    r = np.random.default_rng(5)
    q, want = np.zeros((2, 1, 8, Dh), np.float32), np.zeros((2, 1, 8, Dh))
    for b in range(2):
        for h in range(8):
            k, v = held[b][0][:, h // 4], held[b][1][:, h // 4]
            j = int(r.integers(0, lens[b]))
            q[b, 0, h] = k[j] * 10.0 ** h
            q[b, 0, h] = torch.from_numpy(q[b, 0, h]).bfloat16().float().numpy()
            s = k @ q[b, 0, h].astype(np.float64) * Dh ** -0.5
            top = int(s.argmax())
            gap = np.sort(s)[-1] - np.sort(s)[-2]
            # the score's own error in 32 bits stays far below the gap to the next token
            assert gap > 40 + 4 * (Dh + 16) * U * float(np.abs(k[top]) @ np.abs(q[b, 0, h])) * Dh ** -0.5
            want[b, 0, h] = v[top]
    out, _ = p.kv.attend(bf16(q), table, ln)
    assert_within(bf16_np(out), want, np.abs(want) * (2.0 ** -8 + 2.0 ** -18), "out")
