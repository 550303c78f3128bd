"""The E4M3 quantiser and product, the rotary positions and the sampling on the GPU against the float64 oracle.

Tolerances (none depends on a run), U = 2^-24:
* the quantiser and the sampled tokens are exact;
* a BF16 result: half a step, 2^-8 of the value, plus the error of the 32-bit arithmetic before it;
* a product of K terms in 32 bits: (K + 16) U of the sum of their magnitudes, each block's scaling included;
* a rotation: the turn's fraction is rounded to 24 bits (2 pi U of at most half a turn: 4 U of an angle), sine and
  cosine are within 2 steps of theirs (4 U), two products and a sum add 3 U: 12 U of |a| + |b|, and the
  float64 angles' own error, 2^-51 of the angle.
"""
import numpy as np
import pytest
import torch

from gpu_harness import DEV, bf16_np, pkg, to_np
from oracle import formats as F
from oracle import serving as S
from test_gpu_decoder import assert_within, bf16, f32_np
from test_gpu_guard_bands import Guarded

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F8 = torch.float8_e4m3fn


def up(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


def same(a, b):
    return a.dtype == b.dtype and a.shape == b.shape and torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ------------------------------------------------------------------------- quantiser
def quantize_case(M, K, seed=0):
    r = np.random.default_rng(seed * 1000 + M * 7 + K)
    x = r.normal(size=(M, K)) * np.exp2(r.integers(-20, 20, (M, 1)))
    x[r.random((M, K)) < 0.1] = 0.0
    return bf16(x)


def check_quantize(got, x, rows):
    codes, scale = S.quantize_fp8(f32_np(x), rows)
    assert np.array_equal(to_np(got[1]), scale)
    assert np.array_equal(to_np(got[0].view(torch.uint8)), codes)


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 128), (3, 127), (5, 129), (2, 2048), (130, 264), (129, 1531), (300, 72), (128, 128),
                                 (1, 65536), (700, 1000), (9, 7160), (257, 8)])
def test_quantize(M, K, rows):
    x = quantize_case(M, K)
    got = pkg.quantize_fp8(x, rows=rows)
    check_quantize(got, x, rows)


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("K", [256, 131])
def test_quantize_zeros_tiny_huge_and_bad_values(K, rows):
    x = torch.zeros(140, K, dtype=torch.bfloat16, device=DEV)
    x[1], x[2, 0], x[3, 1] = 1e-38, 3e38, -9.2e-41  # the smallest subnormal
    x[135, -1] = 1e-30
    if rows == 1:
        check_quantize(pkg.quantize_fp8(x), x, 1)
    else:
        check_quantize(pkg.quantize_fp8(x[:2].contiguous(), rows=128), x[:2], 128)
        check_quantize(pkg.quantize_fp8(x, rows=128), x, 128)
    ref = [t.clone() for t in pkg.quantize_fp8(x, rows=rows)]
    x[5, 3], x[7, K - 1] = float("nan"), float("inf")
    got = pkg.quantize_fp8(x, rows=rows)
    assert torch.isnan(got[1][5 // rows, 0]) and torch.isinf(got[1][7 // rows, -1] if rows == 1 else torch.tensor(np.inf))
    assert torch.isnan(got[0][5, 3].float())
    clean = [i for i in range(140) if (i not in (5, 7) if rows == 1 else i >= 128)]
    assert same(ref[0][clean], got[0][clean]) and same(ref[1][[i // rows for i in clean]], got[1][[i // rows for i in clean]])


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("K", [256, 260, 1531])
def test_quantize_strides_places_and_nothing_else(K, rows):
    x = quantize_case(133, K)
    ref = pkg.quantize_fp8(x, rows=rows)
    for pad in (24, 5):
        wide = torch.zeros(133, K + pad, dtype=torch.bfloat16, device=DEV)
        for at in (0, 3):
            wide[:, at:at + K] = x
            assert all(same(a, b) for a, b in zip(ref, pkg.quantize_fp8(wide[:, at:at + K], rows=rows)))
    g = Guarded(16)
    out = g((133, K), F8), g(tuple(ref[1].shape), torch.float32)
    pkg.quantize_fp8(x, rows=rows, out=out)
    assert g.intact() and all(same(a, b) for a, b in zip(ref, out))
    flat = torch.zeros(133 * K + 1, dtype=F8, device=DEV)  # rows that start at odd addresses
    pkg.quantize_fp8(x, rows=rows, out=(flat[1:].view(133, K), ref[1]))
    assert same(flat[1:].view(133, K), ref[0])
    assert pkg.quantize_fp8(x[:0], rows=rows)[0].shape == (0, K)


def test_quantize_many_rows():
    x = torch.randn(70000, 136, device=DEV).bfloat16()
    y, s = pkg.quantize_fp8(x)
    one = torch.arange(0, 70000, 997)
    check_quantize((y[one], s[one]), x[one], 1)
    y, s = pkg.quantize_fp8(x, rows=128)
    last = 70000 // 128 * 128
    check_quantize((y[last:], s[-1:]), x[last:], 128)


# ---------------------------------------------------------------------------- product
def linear_case(M, N, K, mode="group", seed=0):
    r = np.random.default_rng(seed * 7919 + M * 31 + N * 3 + K)
    x = r.normal(size=(M, K)) * np.where(r.random((1, K)) < 0.02, 20.0, 1.0) * 8
    w = r.normal(size=(N, K)) * np.exp(r.normal(size=(N, 1))) * 30
    groups = -(-K // 128)
    xs = (r.random((M, 1 if mode == "token" else groups)) + 0.1).astype(np.float32)
    ws = (np.exp2(r.integers(-6, 2, (-(-N // 128), groups))) * (1 + r.random((-(-N // 128), groups)))).astype(np.float32)
    return up(x.clip(-448, 448).astype(np.float32), F8), up(xs), up(w.clip(-448, 448).astype(np.float32), F8), up(ws)


def check_linear(got, x, xs, w, ws, act="identity"):
    K = x.shape[1]
    out, y, mass = S.fp8_linear(f32_np(x), to_np(xs), f32_np(w), to_np(ws), act)
    # the product's own error; an activation passes at most 1.2 of it on, a gate product both factors'
    err = (K + 16) * U * mass
    if act in ("swiglu", "geglu"):
        g, u = np.split(y, 2, -1)
        eg, eu = np.split(err, 2, -1)
        gate = S.activate(np.concatenate((g, np.ones_like(g)), -1), act)
        tol = 1.2 * eg * (np.abs(u) + eu) + np.abs(gate) * eu
    elif act == "relu2":
        tol = 2 * np.abs(y) * err + err * err
    else:
        tol = 1.2 * err
    assert_within(bf16_np(got), out, tol + np.abs(out) * (2.0 ** -8 + 2.0 ** -18) + 1e-30, act)


SIZES = [(1, 1, 16), (1, 15, 32), (2, 16, 48), (7, 17, 128), (8, 100, 144), (9, 513, 272), (16, 64, 2000), (3, 1000, 512),
         (13, 70, 4096), (17, 33, 256), (33, 129, 1040), (1, 4096, 7168), (48, 2050, 1024), (64, 300, 528), (65, 300, 528),
         (100, 257, 640), (127, 128, 384), (128, 256, 128), (129, 255, 144), (130, 1000, 2000), (250, 383, 4096),
         (256, 512, 1024), (257, 40, 256), (300, 2049, 272), (1, 128, 65536), (600, 700, 912), (1111, 500, 400)]


@pytest.mark.parametrize("mode", ["token", "group"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_linear(M, N, K, mode):
    c = linear_case(M, N, K, mode)
    check_linear(pkg.fp8_linear(*c), *c)


@pytest.mark.parametrize("act", ["swiglu", "geglu", "relu2", "gelu", "relu", "silu"])
@pytest.mark.parametrize("M,N,K", [(1, 256, 16), (5, 512, 208), (40, 1024, 1024), (130, 768, 528), (300, 256, 272)])
def test_linear_activations(act, M, N, K):
    c = linear_case(M, N, K)
    c = (c[0], c[1] / 4000 / K ** 0.5, *c[2:])  # products of the size where activations bend
    check_linear(pkg.fp8_linear(*c, act), *c, act)


@pytest.mark.parametrize("M,N,K,mode", [(8192, 4096, 512, "group"), (5000, 7001, 400, "token"), (20000, 300, 1024, "group"),
                                        (40, 129021, 256, "group"), (3000, 3000, 2064, "group"), (12, 40000, 4096, "group")])
def test_linear_many_tiles(M, N, K, mode):
    """Products of many tiles a multiprocessor; a sample of rows and columns is compared, the ends among them."""
    c = linear_case(M, N, K, mode)
    got = pkg.fp8_linear(*c)
    r = np.random.default_rng(1)
    rows = np.unique(np.r_[0:min(8, M), max(0, M - 8):M, r.integers(0, M, 150)])
    cols = np.unique(np.r_[0:8, N - 8:N, r.integers(0, N, 150)])
    out, _, mass = S.fp8_linear(f32_np(c[0])[rows], to_np(c[1])[rows], f32_np(c[2]), to_np(c[3]))
    tol = (K + 16) * U * mass + np.abs(out) * (2.0 ** -8 + 2.0 ** -18) + 1e-30
    assert_within(bf16_np(got[torch.from_numpy(rows)])[:, cols], out[:, cols], tol[:, cols])


@pytest.mark.parametrize("M,K,columns", [(40, 128, range(113, 147)), (5, 1024, (113, 127, 129, 130, 132, 136, 145)),
                                         (2600, 128, (898, 1025, 1026, 1028, 1037, 1039, 1041, 1042, 1151))])
def test_linear_rows_at_every_place(M, K, columns):
    """Rows of out that begin anywhere within a sector, and last tiles of any width."""
    for N in columns:
        c = linear_case(M, N, K)
        g = Guarded(16)
        out = g((M, N), torch.bfloat16)
        pkg.fp8_linear(*c, out=out)
        assert g.intact(), N
        check_linear(out, *c)


@pytest.mark.parametrize("M", [5, 200])
def test_linear_slices_and_nothing_else(M):
    N, K = 300, 400
    x, xs, w, ws = linear_case(M, N, K)
    ref = pkg.fp8_linear(x, xs, w, ws)
    wide = torch.zeros(M, K + 32, dtype=torch.uint8, device=DEV)
    wide[:, K:] = 0x7F  # no number
    wide[:, :K] = x.view(torch.uint8)
    assert same(pkg.fp8_linear(wide.view(F8)[:, :K], xs, w, ws), ref)
    wide = wide.roll(16, 1)
    assert same(pkg.fp8_linear(wide.view(F8)[:, 16:K + 16], xs, w, ws), ref)
    g = Guarded(16)
    out = g((M, N), torch.bfloat16)
    pkg.fp8_linear(x, xs, w, ws, out=out)
    assert g.intact() and same(out, ref)
    assert pkg.fp8_linear(x[:0], xs[:0], w, ws).shape == (0, N)
    # results repeat bit for bit
    assert all(same(pkg.fp8_linear(x, xs, w, ws), ref) for _ in range(3))


@pytest.mark.parametrize("act", ["identity", "swiglu", "relu"])
@pytest.mark.parametrize("M", [6, 200])
def test_linear_keeps_a_nan_to_its_row_and_column(M, act):
    N, K = 512, 272
    x, xs, w, ws = linear_case(M, N, K)
    ref = pkg.fp8_linear(x, xs, w, ws, act)
    xb, wb = x.view(torch.uint8).clone(), w.view(torch.uint8).clone()
    xb[3, 100], wb[7, 270] = 0x7F, 0xFF
    got = pkg.fp8_linear(xb.view(F8), xs, wb.view(F8), ws, act)
    bad = torch.isnan(got)
    want = torch.zeros_like(bad)
    want[3], want[:, 7] = True, True
    assert torch.equal(bad, want) and torch.equal(got[~want], ref[~want])


def test_linear_scales_of_any_size():
    """The sums' scales span the whole range of 32 bits: each block's is applied to that block alone."""
    M, N, K = 130, 140, 512
    x, xs, w, ws = linear_case(M, N, K)
    for factor in ((1e-15, 1.0, 1e15, 1.0), (0.0, 1.0, 0.0, 1.0), (1.0, -1.0, 1.0, -2.0)):
        c = x, xs * torch.tensor(factor, device=DEV), w, ws
        check_linear(pkg.fp8_linear(*c), *c)
        c = x[:9], c[1][:9].contiguous(), w, ws
        check_linear(pkg.fp8_linear(*c), *c)


def test_linear_from_norm_and_quantizer():
    """A norm's grouped rows and a BF16 matrix through the quantiser: the product that a model computes."""
    M, H, N = 37, 1040, 640
    r = np.random.default_rng(5)
    x, weight, w = bf16(r.normal(size=(M, H))), bf16(1 + 0.1 * r.normal(size=H)), bf16(r.normal(size=(N, H)) / 32)
    y, _, y8, scale = pkg.add_rms_norm(x, weight, fp8="group")
    layer = pkg.FP8Linear.from_bf16(w)
    got = layer(y8, scale)
    check_linear(got, y8, scale, layer.w, layer.w_scale)
    exact = f32_np(y).astype(np.float64) @ f32_np(w).astype(np.float64).T
    # two roundings to 4 significant bits of each term: 2 x 2^-4 of the magnitudes, far less on the whole
    assert np.abs(bf16_np(got) - exact).max() <= (2.0 ** -3 + 2.0 ** -7) * (np.abs(f32_np(y)) @ np.abs(f32_np(w)).T).max()
    q8, q_scale = pkg.quantize_fp8(y)
    check_linear(layer(q8, q_scale), q8, q_scale, layer.w, layer.w_scale)


# ---------------------------------------------------------------------------- rotary
def rotary_case(N, Hq, Hk, D, rot, axes, seed=0, far=1 << 20, dtype=np.int64):
    r = np.random.default_rng(seed * 101 + N * 7 + Hq * 3 + D + rot)
    half = rot // 2
    q, k = bf16(r.normal(size=(N, Hq, D))), bf16(r.normal(size=(N, Hk, D)))
    pos = r.integers(-far, far, (axes, N)).astype(dtype)
    freq = 500000.0 ** (-np.arange(half) / half)
    which = r.integers(0, axes, half).astype(np.uint8)
    return q, k, pos, freq, which


def check_rotary(got, x, pos, freq, which, adjacent):
    want, size, angle = S.rotary(f32_np(x), pos, freq, which, adjacent)
    assert_within(bf16_np(got), want, np.abs(want) * 2.0 ** -8 + size * (12 * U + 2.0 ** -51 * np.abs(angle).max()) + 1e-38)


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("N,Hq,Hk,D,rot,axes", [(1, 1, 1, 2, 2, 1), (1, 16, 4, 128, 128, 1), (3, 4, 2, 64, 32, 2), (8, 5, 1, 80, 80, 3),
                                                (7, 3, 3, 96, 30, 4), (33, 28, 4, 128, 96, 3), (5, 7, 2, 15, 14, 2), (2, 2, 1, 1024, 1024, 1),
                                                (130, 64, 8, 128, 128, 1), (9, 40, 8, 72, 16, 1), (1, 3, 1, 192, 64, 2),
                                                (1000, 2, 1, 256, 256, 3), (300, 9, 9, 40, 40, 1)])
def test_rotary(N, Hq, Hk, D, rot, axes, adjacent):
    q, k, pos, freq, which = rotary_case(N, Hq, Hk, D, rot, axes)
    kw = dict(axes=up(which), adjacent=adjacent)
    got = pkg.rotary(q, up(pos), up(freq), k=k, **kw)
    check_rotary(got[0], q, pos, freq, which, adjacent)
    check_rotary(got[1], k, pos, freq, which, adjacent)
    # queries alone, 32-bit positions, axes in a wider tensor
    wide = torch.full((axes, N + 5), 77, dtype=torch.int32, device=DEV)
    wide[:, :N] = up(pos.astype(np.int32))
    alone = pkg.rotary(q, wide[:, :N], up(freq), **kw)
    assert same(alone[0], got[0]) and alone[1] is None
    if axes == 1:
        assert same(pkg.rotary(q, up(pos[0]), up(freq), adjacent=adjacent)[0], got[0])
    # in place
    q2, k2 = q.clone(), k.clone()
    assert pkg.rotary(q2, up(pos), up(freq), k=k2, out=(q2, k2), **kw)[0] is q2
    assert same(q2, got[0]) and same(k2, got[1])


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("N,Hq,Hk,D,rot,pad", [(5, 16, 4, 128, 128, 0), (20, 6, 2, 64, 32, 8), (4, 3, 1, 96, 40, 3), (1, 4, 2, 128, 64, 0)])
def test_rotary_in_a_projections_output(N, Hq, Hk, D, rot, pad, adjacent):
    q, k, pos, freq, which = rotary_case(N, Hq, Hk, D, rot, 2)
    ref = pkg.rotary(q, up(pos), up(freq), k=k, axes=up(which), adjacent=adjacent)
    qkv = torch.randn(N, (Hq + 2 * Hk) * D + pad, device=DEV).bfloat16()

    def part(t, first, heads):
        return t[:, first * D:(first + heads) * D].unflatten(1, (heads, D))
    part(qkv, 0, Hq).copy_(q)
    part(qkv, Hq, Hk).copy_(k)
    before = qkv.clone()
    mine = part(qkv, 0, Hq), part(qkv, Hq, Hk)
    # elsewhere first, then in place: what is not turned stays
    other = torch.zeros_like(qkv)
    got = pkg.rotary(mine[0], up(pos), up(freq), k=mine[1], axes=up(which), adjacent=adjacent, out=(part(other, 0, Hq), part(other, Hq, Hk)))
    assert same(got[0], ref[0]) and same(got[1], ref[1]) and same(qkv, before)
    assert (other[:, (Hq + Hk) * D:] == 0).all()
    pkg.rotary(mine[0], up(pos), up(freq), k=mine[1], axes=up(which), adjacent=adjacent, out=mine)
    assert same(mine[0], ref[0]) and same(mine[1], ref[1])
    assert same(qkv[:, (Hq + Hk) * D:], before[:, (Hq + Hk) * D:])


def test_rotary_far_positions_and_other_frequencies():
    N, D = 64, 64
    q, k, _, freq, _ = rotary_case(N, 2, 1, D, D, 1)
    for lo, hi in ((0, 4), (1 << 23, (1 << 23) + 100), ((1 << 31) - 200, (1 << 31) - 1), (-(1 << 31), -(1 << 31) + 99)):
        pos = np.random.default_rng(abs(hi)).integers(lo, hi, (1, N))
        for f in (freq, freq * 7.5, freq / 64, np.zeros_like(freq), -freq):
            got = pkg.rotary(q, up(pos), up(f), k=k)
            check_rotary(got[0], q, pos, f, None, False)
            check_rotary(got[1], k, pos, f, None, False)


def test_rotary_backwards_undoes_it():
    q, k, pos, freq, which = rotary_case(50, 8, 2, 128, 128, 3)
    kw = dict(axes=up(which))
    there = pkg.rotary(q, up(pos), up(freq), k=k, **kw)
    back = pkg.rotary(there[0], up(-pos), up(freq), k=there[1], **kw)
    for a, b in ((q, back[0]), (k, back[1])):  # two roundings, each 2^-8 of a value no larger than |a| + |b| of its pair
        size = a.float().abs()[..., :64] + a.float().abs()[..., 64:]
        assert ((a.float() - b.float()).abs() <= torch.cat((size, size), -1) * (3 * 2.0 ** -8)).all()


def test_rotary_axis_that_is_none():
    q, k, pos, freq, which = rotary_case(9, 4, 2, 64, 64, 2)
    which[:] = np.arange(32) % 2
    ref = pkg.rotary(q, up(pos), up(freq), axes=up(which))[0]
    which[5], which[6] = 2, 255
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = pkg.rotary(q, up(pos), up(freq), axes=up(which), dev_status=status)[0]
    assert int(status) == pkg.MOE_DEV_BAD_INDEX
    assert same(pkg.rotary(q, up(pos), up(freq), axes=up(which))[0], got)  # no status word: the same result
    off = [5, 6, 37, 38]
    on = [i for i in range(64) if i not in off]
    assert same(got[..., off], q[..., off]) and same(got[..., on], ref[..., on])


def test_rotary_nothing_else_and_no_tokens():
    for N, Hq, Hk, D, rot in ((5, 3, 2, 128, 64), (3, 2, 1, 30, 30)):
        q, k, pos, freq, _ = rotary_case(N, Hq, Hk, D, rot, 1)
        ref = pkg.rotary(q, up(pos), up(freq), k=k)
        g = Guarded(16)
        out = g((N, Hq, D), torch.bfloat16), g((N, Hk, D), torch.bfloat16)
        pkg.rotary(q, up(pos), up(freq), k=k, out=out)
        assert g.intact() and same(out[0], ref[0]) and same(out[1], ref[1])
    assert pkg.rotary(q[:0], up(pos)[:, :0], up(freq))[0].shape == (0, 2, 30)
    q[1, 0, 3] = float("nan")
    got = pkg.rotary(q, up(pos), up(freq))[0]
    bad = torch.isnan(got).nonzero().tolist()
    assert bad == [[1, 0, 3], [1, 0, 18]]


# --------------------------------------------------------------------------- sampling
def sample(rows, u, dtype=torch.float32, **settings):
    t = torch.stack([torch.as_tensor(r, dtype=torch.float32) for r in rows]).to(DEV).to(dtype)
    kw = {n: torch.as_tensor(np.broadcast_to(np.asarray(v), (len(rows),)).copy(), device=DEV).to(torch.int32 if n == "top_k" else torch.float32)
          for n, v in settings.items()}
    return pkg.sample_tokens(t, torch.as_tensor(np.asarray(u, np.float32), device=DEV), **kw).tolist()


def settings_of(r, B):
    pick = lambda v: r.choice(np.asarray(v), B)  # noqa: E731
    return dict(temperature=pick([0.0, 0.3, 0.7, 1.0, 1.0, 2.5]).astype(np.float32), top_k=pick([0, 1, 2, 5, 40, 1000, -3]).astype(np.int32),
                top_p=pick([0.0, 0.1, 0.5, 0.9, 0.99, 1.0, 1.0]).astype(np.float32), min_p=pick([0.0, 0.0, 0.01, 0.2, 1.0]).astype(np.float32))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,V", [(1, 1), (3, 2), (40, 7), (25, 100), (64, 1001), (9, 4099), (5, 32000), (3, 129021), (1, 129021),
                                 (2, 262144), (160, 5000), (300, 17)])
def test_sample(B, V, dtype):
    r = np.random.default_rng(B * 31 + V)
    x = (r.normal(size=(B, V)) * r.choice([0.1, 1.0, 3.0, 10.0], (B, 1))).astype(np.float32)
    x[r.random((B, V)) < 0.1] = -np.inf
    t = torch.from_numpy(x).to(DEV).to(dtype)
    u = r.random(B).astype(np.float32)
    for use in ((), ("temperature",), ("top_k",), ("top_p",), ("min_p",), ("temperature", "top_k", "top_p", "min_p")):
        s = {n: v for n, v in settings_of(r, B).items() if n in use}
        got = pkg.sample_tokens(t, up(u), **{n: up(v) for n, v in s.items()})
        rows = range(B) if B * V < 400000 else range(min(B, 3))
        host = t.float().cpu().numpy()
        want = [S.sample(host[b], u[b], **{n: v[b] for n, v in s.items()}) for b in rows]
        assert got[:len(want)].tolist() == want, use


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sample_ties_go_by_index(dtype):
    """Rows of a few values only: the cut of each filter falls within equal logits."""
    r = np.random.default_rng(4)
    for V in (10, 300, 9000, 60000):
        for values in ([0.0], [1.0, 0.0], [2.0, 1.0, -np.inf], [-0.0, 0.0]):
            rows = [r.choice(np.array(values, np.float32), V) for _ in range(12)]
            u = r.random(12).astype(np.float32)
            s = dict(temperature=0.8, top_k=r.integers(1, V, 12), top_p=r.choice([0.3, 0.5, 0.77], 12), min_p=0.0)
            for use in (("top_k",), ("top_p",), ("temperature", "top_k", "top_p")):
                kw = {n: s[n] for n in use}
                want = [S.sample(rows[b], u[b], **{n: np.broadcast_to(v, 12)[b] for n, v in
                                                   {n: np.asarray(v, np.float32 if n != "top_k" else int) for n, v in kw.items()}.items()})
                        for b in range(12)]
                assert sample(rows, u, dtype, **kw) == want, (V, values, use)


def test_sample_equal_logits_are_split_exactly():
    """Equal weights: token i is taken for uniform in [i / V, (i + 1) / V), borders included."""
    V, n = 1 << 12, 64
    at = np.random.default_rng(0).integers(1, V, n)
    rows = [np.zeros(V)] * n
    assert sample(rows, at / V) == at.tolist()
    below = np.nextafter((at / V).astype(np.float32), np.float32(0))
    assert sample(rows, below) == (at - 1).tolist()
    assert sample(rows, np.full(n, 0.0)) == [0] * n and sample(rows, np.full(n, np.nextafter(np.float32(1), np.float32(0)))) == [V - 1] * n
    # half of them by top_p
    assert sample(rows, np.full(n, 0.9999999), top_p=0.5) == [V // 2 - 1] * n
    assert sample(rows, np.full(n, 0.9999999), top_p=0.5, top_k=V // 2) == [V // 4 - 1] * n


def test_sample_masked_and_infinite_logits():
    low, inf, nan = -3.3895e38, np.inf, np.nan
    V = 20
    full = lambda *pairs: np.array([dict(pairs).get(i, -inf) for i in range(V)], np.float32)  # noqa: E731
    rows = [full(), np.full(V, nan), full((3, nan), (4, -5.0)), np.full(V, low), full((7, low), (9, low)), full((2, inf), (5, 1.0), (6, inf)),
            full((0, low), (1, 0.0)), full((19, -1e30))]
    for dtype in (torch.float32, torch.bfloat16):
        for kw in ({}, dict(top_k=3), dict(top_p=0.9), dict(min_p=0.5), dict(temperature=0.5, top_k=2, top_p=0.99, min_p=0.1), dict(temperature=0.0),
                   dict(temperature=inf), dict(temperature=1e-30), dict(temperature=1e30), dict(temperature=nan), dict(temperature=-1.0)):
            host = [torch.as_tensor(x).to(dtype).float().numpy() for x in rows]
            for u in (0.0, 0.37, 0.9999999):
                want = [S.sample(x, np.float32(u), **{n: (np.float32(v) if n != "top_k" else v) for n, v in kw.items()}) for x in host]
                assert sample(rows, [u] * len(rows), dtype, **kw) == want, (kw, u)


@pytest.mark.parametrize("V", [900, 30000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sample_logits_of_any_size(V, dtype):
    """Logits so near to zero, so large or so far apart that none of a fast way's assumptions holds, and mixtures."""
    r = np.random.default_rng(V)
    base = r.normal(size=(8, V))
    tiny, some = base * 1e-3, r.random((8, V)) < 0.02
    kinds = [tiny, base * 1e-6, base * 60, base * 1e4, base * 1e30, np.where(some, base, tiny), np.where(some, tiny, base), np.where(some, base * 200, base),
             np.where(some, -1e4, base), np.where(some, -np.inf, tiny), base - 100, base + 127.5, -np.abs(base) * 1e-3, np.where(some, 0.0, tiny),
             np.where(some, 0.0, base * 1e-40)]
    u = r.random(8).astype(np.float32)
    for x in kinds:
        x = torch.from_numpy(x.astype(np.float32)).to(dtype)
        for kw in ({}, dict(top_k=V // 20), dict(top_p=0.7), dict(top_k=V // 3, top_p=0.9, min_p=0.05), dict(temperature=0.01, top_k=30, top_p=0.8),
                   dict(temperature=50.0, top_p=0.5)):
            kw = {n: np.full(8, v, np.int32 if n == "top_k" else np.float32) for n, v in kw.items()}
            got = pkg.sample_tokens(x.to(DEV), up(u), **{n: up(v) for n, v in kw.items()}).tolist()
            some_rows = range(8) if V < 1000 else (0, 5)
            host = x.float().numpy()
            assert [got[b] for b in some_rows] == [S.sample(host[b], u[b], **{n: v[b] for n, v in kw.items()}) for b in some_rows], kw


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sample_one_row_as_in_a_batch(dtype):
    """A row's token does not depend on how many blocks share it: 1, 4, 20, 80 and 320 rows at a time."""
    V, B = 70001, 320
    r = np.random.default_rng(5)
    x = r.normal(size=(8, V)).astype(np.float32) * np.array([[2.5], [1e-3], [60.0], [0.3], [2.5], [2.5], [0.0], [8.0]], np.float32)
    x[4, r.random(V) < 0.9] = -np.inf
    x[5, r.random(V) < 0.001] = np.nan
    x = torch.from_numpy(x).to(dtype).to(DEV).repeat(B // 8, 1)
    u = up(r.random(B).astype(np.float32))
    kw = dict(temperature=r.choice([0.0, 0.7, 1.0, 3.0], B).astype(np.float32), top_k=r.choice([0, 1, 40, 5000, 69999], B).astype(np.int32),
              top_p=r.choice([1.0, 0.9, 0.3], B).astype(np.float32), min_p=r.choice([0.0, 0.02], B).astype(np.float32))
    kw = {n: up(v) for n, v in kw.items()}
    want = pkg.sample_tokens(x, u, **kw)
    for n in (1, 4, 20, 80):
        got = [pkg.sample_tokens(x[i:i + n], u[i:i + n], **{k: v[i:i + n] for k, v in kw.items()}) for i in range(0, B, n)]
        assert torch.equal(torch.cat(got), want), n


def test_sample_settings_outside_their_range():
    r = np.random.default_rng(8)
    rows = [r.normal(size=50).astype(np.float32)] * 6
    base = sample(rows, [0.6] * 6)
    assert sample(rows, [0.6] * 6, top_k=[0, -1, 50, 51, 1 << 30, -(1 << 30)]) == base
    assert sample(rows, [0.6] * 6, top_p=[1.0, 1.5, np.inf, np.nan, 2.0, 1.0]) == base
    assert sample(rows, [0.6] * 6, min_p=[0.0, -1.0, -np.inf, np.nan, -0.0, 0.0]) == base
    best = int(np.argmax(rows[0]))
    assert sample(rows, [0.6] * 6, top_p=[0.0, -1.0, -np.inf, 1e-30, 0.0, -0.0]) == [best] * 6
    assert sample(rows, [0.6] * 6, min_p=[1.0, 1.5, np.inf, 1e30, 1.0, 2.0]) == [best] * 6
    ends = sample(rows, [-1.0, 0.0, 1.0, np.nan, np.inf, 0.99999994])
    assert ends == [0, 0, 49, 0, 49, 49]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1000, 1003, 70001])
def test_sample_strides_and_alignment(V, dtype):
    r = np.random.default_rng(V)
    B = 6
    x = torch.from_numpy(r.normal(size=(B, V)).astype(np.float32) * 2).to(DEV).to(dtype)
    u, kw = up(r.random(B).astype(np.float32)), dict(top_k=torch.full((B,), 300, dtype=torch.int32, device=DEV),
                                                     top_p=torch.full((B,), 0.97, device=DEV))
    ref = pkg.sample_tokens(x, u, **kw)
    for pad in (1, 2, 3, 5, 8):
        wide = torch.full((B, V + pad), float("inf"), device=DEV).to(dtype)  # what lies beside a row is not looked at
        for at in range(0, pad + 1, max(1, pad // 2)):
            wide.fill_(float("inf"))
            wide[:, at:at + V] = x
            assert torch.equal(pkg.sample_tokens(wide[:, at:at + V], u, **kw), ref)
    g = Guarded(16)
    out = g((B,), torch.int32)
    pkg.sample_tokens(x, u, out=out, **kw)
    assert g.intact() and torch.equal(out, ref)
    # a row's token does not depend on the batch around it
    many = pkg.sample_tokens(x.repeat(40, 1), u.repeat(40), **{n: v.repeat(40) for n, v in kw.items()})
    assert torch.equal(many, ref.repeat(40)) and torch.equal(pkg.sample_tokens(x[:1], u[:1], **{n: v[:1] for n, v in kw.items()}), ref[:1])
    assert pkg.sample_tokens(x[:0], u[:0]).shape == (0,)


def test_sample_follows_its_distribution():
    """Evenly spread random numbers take each token as often as its weight says, to one."""
    r = np.random.default_rng(11)
    V, B = 500, 4096
    x = torch.from_numpy(r.normal(size=V).astype(np.float32) * 2).to(DEV)
    u = (torch.arange(B, device=DEV, dtype=torch.float64) + 0.5) / B
    got = pkg.sample_tokens(x.expand(B, V).contiguous(), u.float(), temperature=torch.full((B,), 0.7, device=DEV))
    p = torch.softmax(x.double() / float(np.float32(0.7)), 0)
    assert (torch.bincount(got.long(), minlength=V) - p * B).abs().max() <= 1.001
