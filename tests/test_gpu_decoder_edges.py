"""Edges of the operators around the routed experts on the GPU: scores and activations of extreme size,
numbers that are none, slices, several threads and streams. Tolerances as in test_gpu_decoder.py unless
a test says otherwise.
"""
import threading

import numpy as np
import pytest
import torch

from gpu_harness import DEV, F, bf16_np, pkg, to_np
from oracle import decoder as D
from test_gpu_decoder import (Pool, U, assert_within, bf16, check_attend, check_linear, f32_np, linear_case, queries,
                              run_linear, sequences)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ attention: large scores
def exact_scores_check(out, lse, q, held, Hkv, scale, smallest=0.0):
    """Against the oracle where every score is exact in 32 bits: only the weights' rounding (2^-10 of the
    mass) and the result's (2^-8 of the value) are left; the log-sum-exp has 8 roundings of its size. `smallest`: the
    error of a weight of any size, of the largest one: FP16 ends at 2^-24, the largest weight is above 2^14, so 2^-39."""
    B, T, Hq, Dh = q.shape
    G = Hq // Hkv
    qf = f32_np(q).astype(np.float64)
    for b in range(B):
        k, v = held[b]
        for h in range(Hkv):
            hs = slice(h * G, (h + 1) * G)
            o, l, mass = D.attend(qf[b, :, hs], k[:, h], v[:, h], scale)
            assert_within(bf16_np(out)[b, :, hs], o, np.abs(o) * (2.0 ** -8 + 2.0 ** -18) + mass * 2.0 ** -10 + 1e-30
                          + smallest * np.abs(v[:, h]).sum(0), "out")
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


# -------------------------------------------------------------- linear: range of activations
def zero_weights(data, ks, rows):
    """Codes of zero at columns ks of the given rows of packed weights."""
    for k in ks:
        data[rows, k // 2] &= 0xF0 if k % 2 == 0 else 0x0F


@pytest.mark.parametrize("act", ["identity", "swiglu"])
@pytest.mark.parametrize("M,N,K", [(1, 32, 128), (3, 50, 144), (5, 1000, 512), (12, 300, 2000), (16, 4096, 1024), (8, 100, 2080),
                                   (2, 4096, 7168), (16, 40006, 528), (12, 60000, 256), (33, 70, 256), (9, 40, 65520)])
def test_linear_small_values_beside_an_outlier(M, N, K, act):
    """One value of each 128 is 2^40 (for every other token 2^90, or 1), and half of the rows have zero for its
    weight: their results are made of the small values alone."""
    x, _, data, sf, alpha = linear_case(M, N, K, None)
    r = np.random.default_rng(K)
    ks = [min(c + int(r.integers(0, 128)), K - 1) for c in range(0, K, 128)]
    rows = np.arange(0, N // 2 if act == "swiglu" else N, 2)
    if act == "swiglu":
        rows = np.r_[rows, rows + N // 2]
    zero_weights(data, ks, rows)
    x[::3, ks] = 2.0 ** 40
    x[1::3, ks] = 2.0 ** 90
    if act == "swiglu":
        x[1::3, ks] = -(2.0 ** 50)                          # products of two sums stay in BF16's range
    got = run_linear(x, None, data, sf, alpha, act)
    n_out = N // 2 if act == "swiglu" else N
    cols = np.unique(np.r_[0:min(n_out, 150), max(n_out - 150, 0):n_out, r.integers(0, n_out, 100)])
    if K > 60000:
        cols = cols[::4]
    at = np.r_[cols, cols + n_out] if act == "swiglu" else cols
    check_linear(got[:, torch.from_numpy(cols).to(DEV)], x, None, data[at], sf[at], alpha, act)


@pytest.mark.parametrize("size,outlier,alpha", [(2.0 ** -100, 1.0, 2.0 ** 100), (2.0 ** -60, 2.0 ** 60, 2.0 ** 60), (1.0, 2.0 ** 110, 1.0)])
@pytest.mark.parametrize("K", [256, 400])
def test_linear_far_ranges(K, size, outlier, alpha):
    x, _, data, sf, _ = linear_case(4, 64, K, None)
    zero_weights(data, [5, K - 3], np.arange(64))
    x *= size
    x[:, 5], x[2:, K - 3] = outlier, -outlier
    x[3, :128] = outlier
    x[3, 5:100] = size
    data[:, : 128 // 2][:, ::2] &= 0x0F                    # and zero weights for every fourth of the first 128
    data[:, : 128 // 2][:, ::2] &= 0xF0
    got = bf16_np(run_linear(x, None, data, sf, np.float32(alpha)))
    want, _, mass = D.linear(f32_np(x), data, sf, alpha)
    over = np.abs(want) > 3.4e38                             # past BF16's range: infinity is its rounding
    assert np.array_equal(got[over], np.copysign(np.inf, want[over]))
    got[over], tol = want[over], (K + 16) * U * mass + np.abs(want) * (2.0 ** -8 + 2.0 ** -18) + 1e-30
    assert_within(got, want, tol)


# ------------------------------------------------------------- attention: range of queries
@pytest.mark.parametrize("scale", [0.2, -0.2])
@pytest.mark.parametrize("B,Hkv,G,T,Dh,page,n", [(2, 2, 4, 1, 128, 64, 300), (3, 1, 6, 4, 64, 16, 500), (1, 1, 8, 1, 128, 32, 20000),
                                               (20, 8, 4, 1, 128, 64, 3000), (1, 1, 16, 1, 128, 16, 5000), (1, 1, 24, 1, 64, 64, 4000),
                                               (1, 1, 12, 1, 64, 64, 900)])
def test_attend_small_queries_beside_an_outlier(B, Hkv, G, T, Dh, page, n, scale):
    """Queries with one dimension of 2^40 (or 2^-90 of its size elsewhere) that every key has a zero in: the
    scores are made of the small values alone."""
    lens = [n - 7 * b for b in range(B)]
    p = Pool(sum(-(-m // page) for m in lens), page, Hkv, Dh, 1.0 if G % 8 else 2.5)
    table, ln, held = sequences(p, lens, seed=n)
    r = np.random.default_rng(n)
    d = r.integers(0, Dh, Hkv)
    for b in range(B):                                      # the stored codes of dimension d, and the oracle's values
        for h in range(Hkv):
            held[b][0][:, h, d[h]] = 0.0
            p.t[0][table[b][table[b] >= 0].long(), h, :, int(d[h]) // 2] &= 0xF0 if d[h] % 2 == 0 else 0x0F
    q = queries(B, T, Hkv * G, Dh)
    for h in range(Hkv * G):
        if h % 3 != 1:
            q[:, :, h, int(d[h // G])] = 2.0 ** (40 if h % 3 else 100)
    out, lse = p.kv.attend(q, table, ln, softmax_scale=scale)
    check_attend(out, lse, q, held, Hkv, scale)
    again, lse2 = p.kv.attend(q, table, ln, softmax_scale=scale)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("Hkv,G,T,Dh,page,lens", [(2, 4, 4, 128, 64, (300, 65, 64, 4)), (1, 8, 5, 128, 16, (1000, 17, 3)),
                                                 (2, 6, 3, 64, 16, (130, 2)), (1, 2, 16, 64, 64, (90, 16)), (1, 4, 2, 128, 32, (20000, 9000))])
def test_attend_no_number_of_a_later_token_reaches_an_earlier_row(Hkv, G, T, Dh, page, lens):
    """Scales that are no numbers at the place of a step's second new token, for one block of 16 values: the rows
    before it keep their results bit for bit, those from it on have NaN there and nowhere else."""
    p = Pool(sum(-(-m // page) for m in lens), page, Hkv, Dh)
    table, ln, _ = sequences(p, list(lens), seed=T)
    q = queries(len(lens), T, Hkv * G, Dh)
    ref, ref_lse = (t.clone() for t in p.kv.attend(q, table, ln))
    want = ref.clone()
    for b, n in enumerate(lens):
        at = n - T + 1                                      # the second new token: row 0 does not see it
        if at < 0:
            continue
        p.t[3][int(table[b, at // page]), Hkv - 1, at % page, 1] = 0x7F if b % 2 else 0xFF
        want[b, 1:, (Hkv - 1) * G:, 16:32] = float("nan")
    out, lse = p.kv.attend(q, table, ln)
    assert torch.equal(torch.isnan(out), torch.isnan(want)) and torch.equal(lse, ref_lse)
    assert torch.equal(out.nan_to_num(7.0), want.nan_to_num(7.0))


# ------------------------------------------------------------------- linear: slices
def test_linear_of_one_of_several_matrices_and_of_some_of_the_tokens():
    """alpha, x and its scales as slices of what quantize_weights and add_rms_norm give for several."""
    r = np.random.default_rng(12)
    w = bf16(r.normal(size=(5, 96, 256)) * (1 + np.arange(5))[:, None, None])
    data, sf, alpha = pkg.quantize_weights(w)
    _, _, x8, scale = pkg.add_rms_norm(bf16(r.normal(size=(7, 256))), bf16(np.ones(256)), fp8="group")
    for e in range(5):
        lin = pkg.NVFP4Linear(data[e], sf[e], alpha[e:e + 1])
        for m in range(7):
            check_linear(lin(x8[m:], scale[m:]), x8[m:], to_np(scale[m:]), to_np(data[e]), to_np(sf[e]), float(alpha[e]))


# ------------------------------------------------------------- several threads and streams
@pytest.mark.parametrize("shared", [False, True])
def test_attend_from_several_threads_at_once(shared):
    """Threads with a stream each, or all on one: every call needs scratch for its parts, and none takes
    another's while it is in use."""
    lens, page = [9000, 4000], 64
    p = Pool(300, page, 2, 128)
    table, ln, _ = sequences(p, lens)
    qs = [queries(2, 1, 8, 128, seed=s) for s in range(4)]
    want = [tuple(t.clone() for t in p.kv.attend(q, table, ln)) for q in qs]
    torch.cuda.synchronize()
    one, bad, go = torch.cuda.Stream(), [], threading.Barrier(4)

    def work(i):
        with torch.cuda.stream(one if shared else torch.cuda.Stream()):
            go.wait(timeout=30)
            for _ in range(60):
                got = p.kv.attend(qs[i], table, ln)
                torch.cuda.current_stream().synchronize()
                if not (torch.equal(got[0], want[i][0]) and torch.equal(got[1], want[i][1])):
                    bad.append(i)
            torch.cuda.current_stream().synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


@pytest.mark.parametrize("act", ["identity", "swiglu", "geglu", "relu2", "gelu", "relu", "silu"])
@pytest.mark.parametrize("M,K", [(3, 512), (12, 4096)])
def test_linear_activations_let_a_nan_through(act, M, K):
    x, _, data, sf, alpha = linear_case(M, 64, K, None)
    ref = run_linear(x, None, data, sf, alpha, act).clone()
    x[1, 77] = float("nan")
    got = run_linear(x, None, data, sf, alpha, act)
    rows = [m for m in range(M) if m != 1]
    assert torch.equal(got[rows], ref[rows]) and torch.isnan(got[1].float()).all()


# ------------------------------------------------------------------- append: no numbers
@pytest.mark.parametrize("g", [1.0, 2.5])
@pytest.mark.parametrize("Dh", [64, 128])
def test_append_stores_only_numbers(Dh, g):
    """An infinity becomes the largest value of its block's largest scale, a NaN some finite value within its block's;
    every other value and every other block is what it is without them."""
    r = np.random.default_rng(Dh)
    x = torch.from_numpy(r.normal(size=(4, 2, Dh)).astype(np.float32)).bfloat16().float().numpy()
    bad = x.copy()
    bad[0, 0, 3], bad[1, 1, 17], bad[2, 0, 40], bad[2, 1, 5] = np.inf, -np.inf, np.nan, np.nan
    bad[3, 0, 16:32] = np.nan
    p, slots = Pool(2, 16, 2, Dh, g), torch.tensor([3, 30, 17, 0], device=DEV)
    seen = tuple(torch.empty(4, 2, Dh, dtype=torch.bfloat16, device=DEV) for _ in "kv")
    p.kv.append(bf16(bad), bf16(-bad), slots, seen=seen)
    for sign, s, data, sf in ((1, seen[0], p.t[0], p.t[1]), (-1, seen[1], p.t[2], p.t[3])):
        got = bf16_np(s)
        codes, scales = (to_np(a)[slots.cpu().numpy() // 16, :, slots.cpu().numpy() % 16] for a in (data, sf))
        stored = D.nvfp4_values(codes, scales) / g
        assert np.isfinite(got).all() and np.isfinite(stored).all()
        assert_within(got, stored, np.abs(stored) * (2.0 ** -8 + 4 * U) + 1e-37)
        filled = np.where(np.isnan(bad), 0, bad)
        want = D.kv_encode(sign * np.where(np.isinf(filled), np.sign(filled) * 3e38, filled), g)[2]
        same = np.isfinite(bad)
        assert np.array_equal(stored[same], want[same])
        assert stored[0, 0, 3] == sign * 6 * 448 / g and stored[1, 1, 17] == -sign * 6 * 448 / g
        scale = np.repeat(F.e4m3_decode(scales), 16, -1)
        assert (np.abs(stored) <= 6 * scale / g).all()


@pytest.mark.parametrize("Hkv,G,T,Dh,page,lens", [(2, 4, 1, 128, 64, (700, 90)), (1, 6, 4, 64, 16, (500, 33)), (1, 8, 1, 128, 32, (20000, 100)),
                                                 (1, 16, 1, 128, 16, (3000, 1)), (8, 4, 1, 128, 64, (3000,) * 40)])
def test_attend_scores_of_every_size_in_one_block(Hkv, G, T, Dh, page, lens):
    """Rows whose possible scores lie below, around and above the size where the weights' reference changes, some of
    them in one block. Every query value is the same power of two and every key's values share a quantum, so the
    scores are exact in 32 bits; keys of 500 times a normal value reach a score of 0.3 of the possible."""
    p = Pool(sum(-(-m // page) for m in lens), page, Hkv, Dh)
    table, ln, held = sequences(p, list(lens), seed=Dh + T, spread=500.0)
    r = np.random.default_rng(T)
    for span in ((-6, -3), (-2, 5), (-14, 18)):
        sign = r.choice([-1.0, 1.0], size=(len(lens), T, Hkv * G, Dh))
        q = bf16(sign * 2.0 ** r.integers(*span, size=(len(lens), T, Hkv * G, 1)))
        out, lse = p.kv.attend(q, table, ln, softmax_scale=1.0)
        for b in range(len(lens)):                          # the sums' terms are whole multiples of a quantum
            assert np.abs(held[b][0]).sum(-1).max(initial=0.0) < 2 ** 24 * np.abs(held[b][0][held[b][0] != 0]).min()
        exact_scores_check(out, lse, q, held, Hkv, 1.0, 2.0 ** -39)


@pytest.mark.parametrize("n,B", [(30000, 1), (9000, 3)])
def test_attend_no_number_shows_however_small_its_weight(n, B):
    """A value that is no number at a token whose weight is 0 in 32 bits, in another part of the sequence than the
    token that has all of the weight."""
    p = Pool(-(-n // 64) * B, 64, 1, 128)
    table, ln, held = sequences(p, [n] * B, seed=n)
    q = bf16(np.stack([np.tile(100.0 * held[b][0][n - 5], (1, 4, 1)) for b in range(B)]))
    out, lse = (t.clone() for t in p.kv.attend(q, table, ln))
    assert torch.isfinite(out.float()).all()
    p.t[3][int(table[0, 0]), 0, 7, 2] = 0x7F
    got, got_lse = p.kv.attend(q, table, ln)
    want = out.clone()
    want[0, :, :, 32:48] = float("nan")
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got_lse, lse)
    assert torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))
