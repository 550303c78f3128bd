"""The operators around the routed experts on the GPU against the float64 oracle.

Tolerances (none depends on a run):
* a BF16 result: half a unit in the last place, at most 2^-8 of the value (BF16 has 8 significant
  bits), plus the error of the 32-bit arithmetic before it;
* an E4M3 result: half a unit of 4 significant bits, at most 2^-4 of the value or 2^-10 (half the
  smallest step), each times its scale;
* a sum of n terms in 32 bits: (n + 8) * 2^-24 of the sum of their magnitudes;
* attention weights are rounded to 11 significant bits (2^-11 of sum p |v|, twice that with the
  rounding's effect on the exponentials), scores carry the error of their sums.
"""
import numpy as np
import pytest
import torch

from gpu_harness import DEV, F, bf16_np, pkg, to_np
from oracle import decoder as D
from test_gpu_guard_bands import Guarded

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(DEV).to(torch.bfloat16)


def f32_np(t):
    return t.float().cpu().numpy()


def assert_within(got, want, tol, what=""):
    assert got.shape == want.shape, what
    over = np.abs(got - want) - tol
    assert np.isfinite(got).all() and (over <= 0).all(), f"{what}: {over.max()} over the tolerance"


# ----------------------------------------------------------------------------- norm
def norm_case(M, H, residual, fp8, seed=0, spread=1.0):
    r = np.random.default_rng(seed * 1000 + M * 7 + H)
    x = bf16(r.normal(size=(M, H)) * spread)
    res = bf16(r.normal(size=(M, H)) * 3) if residual else None
    return x, res, bf16(1 + 0.2 * r.normal(size=H))


def check_norm(got, x, res, w, fp8, eps=1e-6):
    y, ro, y8, sc = got
    H = x.shape[1]
    want = D.add_rms_norm(f32_np(x), f32_np(w), None if res is None else f32_np(res), eps, fp8)
    slack = (H + 16) * U
    if y is not None:
        assert_within(bf16_np(y), want["y"], np.abs(want["y"]) * (2.0 ** -8 + slack) + 1e-37, "y")
    if res is None:
        assert ro is None
    elif ro is not None:
        assert_within(bf16_np(ro), want["residual"], np.abs(want["residual"]) * (2.0 ** -8 + 4 * U) + 1e-37, "residual")
    if fp8:
        s = to_np(sc).astype(np.float64)
        assert_within(s, want["scale"], want["scale"] * slack, "scale")
        groups = D.fp8_groups(H, fp8)
        held = f32_np(y8).astype(np.float64)
        tol = np.maximum(np.abs(want["y8"]) * 2.0 ** -4, 2.0 ** -10) + 448 * slack
        assert_within(held, want["y8"], tol, "y8")
        assert s.shape == (x.shape[0], len(groups))


@pytest.mark.parametrize("fp8", [None, "token", "group"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,H", [(1, 1), (1, 128), (3, 127), (5, 129), (2, 2048), (16, 2050), (7, 1531), (40, 4096),
                                 (700, 1000), (1, 32768), (2, 32767), (9, 7168), (1300, 72), (4, 12288), (3, 16392)])
def test_norm(M, H, residual, fp8):
    x, res, w = norm_case(M, H, residual, fp8)
    got = pkg.add_rms_norm(x, w, res, fp8=fp8)
    torch.cuda.synchronize()
    check_norm(got, x, res, w, fp8)


def test_norm_row_strides_in_place_and_partial_outputs():
    M, H = 37, 1024
    x, res, w = norm_case(M, H, True, "group")
    wide = torch.zeros(M, H + 24, dtype=torch.bfloat16, device=DEV)
    wide[:, :H] = x
    odd = torch.zeros(M, H + 5, dtype=torch.bfloat16, device=DEV)
    odd[:, :H] = res
    ref = pkg.add_rms_norm(x, w, res, fp8="group")
    for got in (pkg.add_rms_norm(wide[:, :H], w, odd[:, :H], fp8="group"),
                pkg.add_rms_norm(wide[:, :H], w, res, fp8="group")):
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(ref, got))
    # in place, without y
    keep = res.clone()
    y8, sc = torch.empty_like(ref[2]), torch.empty_like(ref[3])
    pkg.add_rms_norm(x, w, res, fp8="group", out=(None, res, y8, sc))
    assert torch.equal(res, ref[1]) and torch.equal(y8.view(torch.uint8), ref[2].view(torch.uint8)) and torch.equal(sc, ref[3])
    # the norm of the sum without storing the sum
    y = torch.empty_like(ref[0])
    pkg.add_rms_norm(x, w, keep, out=(y, None, None, None))
    assert torch.equal(y, ref[0])
    # no rows
    assert pkg.add_rms_norm(x[:0], w, fp8="token")[0].shape == (0, H)


@pytest.mark.parametrize("H", [256, 1531])
def test_norm_zero_tiny_and_huge_rows(H):
    x = torch.zeros(5, H, dtype=torch.bfloat16, device=DEV)
    x[1] = 1e-20          # the square underflows: eps alone is left
    x[2] = 3e4
    x[2, ::3] = -1e-3
    x[3, 0] = 1e18
    x[4, -1] = -2.0
    w = bf16(np.random.default_rng(1).normal(size=H))
    for fp8 in ("token", "group"):
        check_norm(pkg.add_rms_norm(x, w, fp8=fp8), x, None, w, fp8)


@pytest.mark.parametrize("H", [512, 515])
@pytest.mark.parametrize("M", [6, 700])
def test_norm_keeps_a_bad_row_to_itself(M, H):
    x, res, w = norm_case(M, H, True, "group")
    ref = [t.clone() for t in pkg.add_rms_norm(x, w, res, fp8="group")]
    x[1, 3] = float("nan")
    x[3, H - 1] = float("inf")
    got = pkg.add_rms_norm(x, w, res, fp8="group")
    for a, b in zip(ref, got):
        rows = torch.ones(M, dtype=torch.bool, device=DEV)
        rows[[1, 3]] = False
        assert torch.equal(a.view(torch.uint8).view(M, -1)[rows], b.view(torch.uint8).view(M, -1)[rows])
        assert torch.isnan(b[1].float()).any() and (torch.isnan(b[3].float()) | torch.isinf(b[3].float())).any()
    assert torch.isnan(got[0][1].float()).all() and torch.isnan(got[3][1]).all()


@pytest.mark.parametrize("M,H,fp8", [(3, 129, "group"), (33, 4096, "group"), (5, 1000, "token"), (600, 264, "group")])
def test_norm_writes_nothing_else(M, H, fp8):
    x, res, w = norm_case(M, H, True, fp8)
    ref = pkg.add_rms_norm(x, w, res, fp8=fp8)
    g = Guarded(16)
    out = (g((M, H), torch.bfloat16), g((M, H), torch.bfloat16), g((M, H), torch.float8_e4m3fn),
           g(tuple(ref[3].shape), torch.float32))
    pkg.add_rms_norm(x, w, res, fp8=fp8, out=out)
    assert g.intact()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(ref, out))


# --------------------------------------------------------------------------- linear
def linear_case(M, N, K, mode, seed=0):
    r = np.random.default_rng(seed * 7919 + M * 31 + N * 3 + K)
    data = r.integers(0, 256, (N, K // 2), dtype=np.uint8)
    sf = r.integers(0x18, 0x58, (N, K // 16), dtype=np.uint8)
    alpha = np.float32(0.01)
    x = r.normal(size=(M, K)) * np.where(r.random((1, K)) < 0.02, 20.0, 1.0)
    if mode is None:
        return bf16(x), None, data, sf, alpha
    groups = 1 if mode == "token" else -(-K // 128)
    scale = (r.random((M, groups)) + 0.1).astype(np.float32)
    x8 = torch.from_numpy((x * 40).astype(np.float32)).to(DEV).clamp(-448, 448).to(torch.float8_e4m3fn)
    return x8, scale, data, sf, alpha


def run_linear(x, scale, data, sf, alpha, act="identity", **kw):
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    return pkg.fp4_linear(x, up(data), up(sf), torch.tensor([alpha], device=DEV), act,
                          x_scale=None if scale is None else up(scale), **kw)


def check_linear(got, x, scale, data, sf, alpha, act="identity"):
    K = x.shape[1]
    out, y, mass = D.linear(f32_np(x), data, sf, float(alpha), act, scale)
    # the product's own error; an activation passes at most 1.2 of it on, a gate product both factors'
    err = (K + 16) * U * mass
    if act in ("swiglu", "geglu"):
        g, u = np.split(y, 2, -1)
        eg, eu = np.split(err, 2, -1)
        tol = 1.2 * eg * (np.abs(u) + eu) + np.abs(D.activate(y, act) / np.where(u == 0, 1, u)) * eu + 1.2 * eg * eu
    elif act == "relu2":
        tol = 2 * np.abs(y) * err + err * err
    else:
        tol = 1.2 * err
    assert_within(bf16_np(got), out, tol + np.abs(out) * (2.0 ** -8 + 2.0 ** -18) + 1e-30, act)


@pytest.mark.parametrize("mode", [None, "token", "group"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 15, 32), (2, 16, 48), (7, 17, 128), (8, 100, 144), (9, 513, 272),
                                   (16, 64, 2000), (3, 1000, 512), (13, 70, 4096), (17, 33, 256), (33, 40, 1040),
                                   (1, 4096, 7168), (16, 2050, 1024), (4, 300, 16384), (5, 40000, 128)])
def test_linear(M, N, K, mode):
    c = linear_case(M, N, K, mode)
    check_linear(run_linear(*c), *c)


@pytest.mark.parametrize("act", ["swiglu", "geglu", "relu2", "gelu", "relu", "silu"])
@pytest.mark.parametrize("M,N,K", [(1, 2, 16), (5, 74, 208), (16, 1026, 1024), (2, 4096, 512)])
def test_linear_activations(act, M, N, K):
    c = linear_case(M, N, K, "group" if K > 128 else None)
    check_linear(run_linear(*c, act), *c, act)


@pytest.mark.parametrize("act", ["identity", "swiglu"])
@pytest.mark.parametrize("M,N,K,mode", [(15, 44008, 4672, "group"), (16, 40016, 4720, None), (8, 50010, 1040, "token"),
                                        (4, 30002, 8208, None), (12, 60000, 256, None), (1, 39000, 2048, "group"),
                                        (20, 41000, 512, None)])
def test_linear_many_rows(M, N, K, mode, act):
    """Matrices of many turns per SM: every kind of row alignment, and x from small to more than an SM holds.
    A sample of the columns, the first and last tiles among them, is compared."""
    x, scale, data, sf, alpha = linear_case(M, N, K, mode)
    got = run_linear(x, scale, data, sf, alpha, act)
    n_out = N // 2 if act == "swiglu" else N
    cols = np.unique(np.r_[0:20, n_out - 20:n_out, np.random.default_rng(1).integers(0, n_out, 400)])
    rows = np.r_[cols, cols + n_out] if act == "swiglu" else cols
    check_linear(got[:, torch.from_numpy(cols).to(DEV)], x, scale, data[rows], sf[rows], alpha, act)


@pytest.mark.parametrize("act", ["identity", "geglu"])
@pytest.mark.parametrize("M,N,K", [(16, 40006, 528), (40, 40006, 752), (16, 80010, 720)])
def test_linear_short_unaligned_rows(M, N, K, act):
    """Rows so short that a warp takes them whole, and so aligned that only one block of 16 warps fits an SM."""
    x, scale, data, sf, alpha = linear_case(M, N, K, None)
    got = run_linear(x, scale, data, sf, alpha, act)
    n_out = N // 2 if act == "geglu" else N
    cols = np.unique(np.r_[0:300, n_out - 300:n_out])
    rows = np.r_[cols, cols + n_out] if act == "geglu" else cols
    check_linear(got[:, torch.from_numpy(cols).to(DEV)], x, scale, data[rows], sf[rows], alpha, act)


# sizes that between them are cut into every kind of block, with and without a cluster, for plain and gated products
CUTS = {"identity": [(1, 1, 1808), (3, 1, 3088), (4, 1, 528), (4, 1, 1040), (4, 1, 2064), (4, 1, 2320),
                     (4, 1, 3600), (4, 9743, 272), (4, 14682, 400), (5, 1219, 3632), (6, 1, 2064),
                     (6, 963, 1824), (6, 1448, 3680), (6, 12163, 400), (7, 1, 528), (7, 1, 1552),
                     (7, 1, 2064), (8, 1, 1040), (9, 1, 8208), (10, 3555, 784), (11, 1, 528),
                     (11, 1, 1552), (12, 1, 3088), (12, 1, 8208), (12, 971, 3648), (12, 17025, 16),
                     (13, 1, 1552), (13, 1, 3088), (15, 1, 272), (15, 1, 400), (15, 1, 2320),
                     (15, 986, 7280), (15, 3458, 800), (15, 5972, 784), (16, 1690, 1808), (16, 1970, 1808),
                     (16, 2401, 1808), (16, 2900, 1808), (16, 3527, 1888), (16, 17114, 656)],
        "swiglu": [(4, 2, 528), (6, 2, 1552), (6, 2, 2064), (6, 1456, 1808), (7, 2, 2064), (8, 2, 1040),
                   (9, 3458, 1808), (10, 2, 528), (10, 2, 1552), (10, 2, 2320), (10, 2404, 1808),
                   (10, 34050, 16), (13, 2, 272), (13, 970, 3680), (14, 2, 8208), (14, 2354, 784),
                   (14, 14598, 16), (15, 5868, 784), (15, 9780, 400), (15, 14658, 656), (16, 2, 3088),
                   (16, 986, 7184), (16, 1988, 1856), (16, 2976, 1824)]}


@pytest.mark.parametrize("act,M,N,K", [(act, *size) for act, sizes in CUTS.items() for size in sizes])
def test_linear_every_cut(act, M, N, K):
    x, scale, data, sf, alpha = linear_case(M, N, K, "group" if M % 2 else None)
    got = run_linear(x, scale, data, sf, alpha, act)
    n_out = N // 2 if act == "swiglu" else N
    cols = np.unique(np.r_[0:min(n_out, 150), max(n_out - 150, 0):n_out, np.random.default_rng(1).integers(0, n_out, 100)])
    rows = np.r_[cols, cols + n_out] if act == "swiglu" else cols
    check_linear(got[:, torch.from_numpy(cols).to(DEV)], x, scale, data[rows], sf[rows], alpha, act)


@pytest.mark.parametrize("M,N,K", [(16, 300, 65536), (9, 40, 65520), (2, 33, 40000), (16, 20000, 32784)])
def test_linear_longest_k(M, N, K):
    x, scale, data, sf, alpha = linear_case(M, N, K, None)
    got = run_linear(x, scale, data, sf, alpha)
    cols = np.unique(np.r_[0:min(N, 20), max(N - 20, 0):N, np.random.default_rng(1).integers(0, N, 60)])
    check_linear(got[:, torch.from_numpy(cols).to(DEV)], x, scale, data[cols], sf[cols], alpha)


def test_linear_row_stride_and_no_rows():
    x, scale, data, sf, alpha = linear_case(5, 60, 256, None)
    wide = torch.full((5, 256 + 40), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, :256] = x
    assert torch.equal(run_linear(wide[:, :256], None, data, sf, alpha), run_linear(x, None, data, sf, alpha))
    assert run_linear(x[:0], None, data, sf, alpha).shape == (0, 60)


@pytest.mark.parametrize("K", [512, 1040])
def test_linear_wide_range_of_activations(K):
    """Values far outside FP16's range, and tokens of very different sizes side by side."""
    x, _, data, sf, alpha = linear_case(6, 50, K, None)
    x[0] *= 1e30
    x[1] *= 1e-30
    x[2, 5] = 1e9
    x[3] = 0
    x[4, : K // 2] = 3e5
    got = run_linear(x, None, data, sf, alpha)
    check_linear(got, x, None, data, sf, alpha)
    assert (got[3] == 0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("M", [3, 12])
def test_linear_keeps_a_bad_token_to_itself(M, bad):
    x, _, data, sf, alpha = linear_case(M, 90, 512, None)
    data |= 0x11                                          # no zero weights: infinity times zero is not asked for
    ref = run_linear(x, None, data, sf, alpha).clone()
    x[1, 77] = bad
    got = run_linear(x, None, data, sf, alpha)
    rows = [m for m in range(M) if m != 1]
    assert torch.equal(got[rows], ref[rows])
    assert not torch.isfinite(got[1].float()).any()


@pytest.mark.parametrize("M,N,K", [(3, 50, 144), (16, 700, 2048), (8, 1001, 512)])
def test_linear_writes_nothing_else(M, N, K):
    c = linear_case(M, N, K, None)
    ref = run_linear(*c)
    g = Guarded(16)
    out = g((M, N), torch.bfloat16)
    run_linear(*c, out=out)
    assert g.intact() and torch.equal(out, ref)


def test_linear_of_encoded_bf16_weights():
    r = np.random.default_rng(5)
    w, x = bf16(0.02 * r.normal(size=(96, 256))), bf16(r.normal(size=(4, 256)))
    lin = pkg.NVFP4Linear.from_bf16(w)
    check_linear(lin(x), x, None, to_np(lin.w), to_np(lin.w_sf), float(lin.alpha))
    dense = f32_np(x) @ f32_np(w).T                       # 4-bit weights are within ~10 % of BF16 ones
    assert np.linalg.norm(bf16_np(lin(x)) - dense) < 0.15 * np.linalg.norm(dense)


# ---------------------------------------------------------------------------- cache
class Pool:
    """A cache of `pages` pages with `gap` bytes between them and poisoned places that hold nothing."""

    def __init__(self, pages, page, Hkv, Dh, g=1.0, gap=0):
        def pool(width):
            n = Hkv * page * width
            t = torch.full((pages, n + gap), 0x7F, dtype=torch.uint8, device=DEV)   # NaN scales, codes of -6 and 6
            return t[:, :n].view(pages, Hkv, page, width) if gap == 0 else t.as_strided(
                (pages, Hkv, page, width), (n + gap, page * width, width, 1))
        self.t = [pool(Dh // 2), pool(Dh // 16), pool(Dh // 2), pool(Dh // 16)]
        self.status = torch.zeros(4, dtype=torch.int32, device=DEV)
        self.kv = pkg.NVFP4KVCache(*self.t, k_scale=g, v_scale=g, dev_status=self.status)
        self.pages, self.page, self.Hkv, self.Dh, self.g = pages, page, Hkv, Dh, g


def sequences(pool, lens, seed=0, order=None, spread=1.0):
    """Appends whole sequences through the kernel: (page_table, lens, per-sequence held k, v float64)."""
    r = np.random.default_rng(seed)
    ps = pool.page
    used = [-(-n // ps) for n in lens]
    ids = r.permutation(pool.pages) if order is None else order
    table = np.full((len(lens), max(max(used), 1)), -7, np.int32)
    ks, vs, slots, held, at = [], [], [], [], 0
    for b, n in enumerate(lens):
        table[b, :used[b]] = ids[at:at + used[b]]
        at += used[b]
        k, v = (np.float32(spread) * r.normal(size=(n, pool.Hkv, pool.Dh)).astype(np.float32) for _ in "kv")
        k, v = (torch.from_numpy(t).bfloat16().float().numpy() for t in (k, v))
        p = np.arange(n)
        slots.append(table[b, p // ps].astype(np.int64) * ps + p % ps)
        ks.append(k)
        vs.append(v)
        held.append((D.kv_encode(k, pool.g)[2], D.kv_encode(v, pool.g)[2]) if n else (k.astype(float), v.astype(float)))
    if sum(lens):
        pool.kv.append(bf16(np.concatenate(ks)), bf16(np.concatenate(vs)),
                       torch.from_numpy(np.concatenate(slots)).to(DEV))
    return torch.from_numpy(table).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), held


def check_attend(out, lse, q, held, Hkv, scale):
    B, T, Hq, Dh = q.shape
    G = Hq // Hkv
    qf, of, lf = f32_np(q).astype(np.float64), bf16_np(out), to_np(lse).astype(np.float64)
    for b in range(B):
        k, v = held[b]
        for h in range(Hkv):
            hs = slice(h * G, (h + 1) * G)
            o, l, mass = D.attend(qf[b, :, hs], k[:, h], v[:, h], scale)
            # the largest score's terms bound the error of every score's sum
            size = np.abs(qf[b, :, hs]) @ np.abs(k[:, h]).T * abs(scale) if k.shape[0] else np.zeros((T, G, 1))
            es = (Dh + 16) * U * size.max(-1, initial=0.0) + 4 * U * np.abs(np.where(np.isfinite(l), l, 0.0))
            assert_within(of[b, :, hs], o, np.abs(o) * (2.0 ** -8 + 2.0 ** -18) + mass * (2.0 ** -10 + 4 * es[..., None]) + 1e-30, "out")
            empty = np.isneginf(l)
            assert np.array_equal(np.isneginf(lf[b, :, hs]), empty)
            assert_within(np.where(empty, 0, lf[b, :, hs]), np.where(empty, 0, l), 2 * es + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(empty, 0, l)), "lse")


def queries(B, T, Hq, Dh, seed=1, size=2.0):
    return bf16(size * np.random.default_rng(seed).normal(size=(B, T, Hq, Dh)))


@pytest.mark.parametrize("g", [1.0, 2.5])
@pytest.mark.parametrize("Hkv,Dh,page,N", [(1, 64, 16, 1), (3, 128, 32, 7), (8, 128, 64, 300)])
def test_append(Hkv, Dh, page, N, g):
    r = np.random.default_rng(N)
    pages = N // page + 3
    p = Pool(pages, page, Hkv, Dh, g, gap=48)
    before = [to_np(t).copy() for t in p.t]
    slots = r.permutation(pages * page)[:N].astype(np.int64)
    slots[N // 2] = -1
    qkv = bf16(r.normal(size=(N, 4 + 2 * Hkv, Dh)) * 10.0 ** r.integers(-3, 3, size=(N, 1, 1)))
    qkv[0, 4, :16] = 0
    k, v = qkv[:, 4:4 + Hkv], qkv[:, 4 + Hkv:]
    seen = tuple(torch.empty(N, Hkv, Dh, dtype=torch.bfloat16, device=DEV) for _ in "kv")
    p.kv.append(k, v, torch.from_numpy(slots).to(DEV), seen=seen)
    for i, t in ((0, k), (2, v)):
        data, sf, held = D.kv_encode(f32_np(t), g)
        for n, s in enumerate(slots):
            if s >= 0:
                before[i][s // page, :, s % page] = data[n]
                before[i + 1][s // page, :, s % page] = sf[n]
        assert np.array_equal(to_np(p.t[i]), before[i]) and np.array_equal(to_np(p.t[i + 1]), before[i + 1])
        assert_within(bf16_np(seen[i // 2]), held, np.abs(held) * (2.0 ** -8 + 4 * U) + 1e-37, "seen")
    assert int(p.status[0]) == 0
    p.kv.append(k, v, torch.full((N,), pages * page, dtype=torch.int64, device=DEV))
    assert int(p.status[0]) == pkg.MOE_DEV_BAD_INDEX
    assert all(np.array_equal(to_np(t), b) for t, b in zip(p.t, before))
    p.kv.append(k[:0], v[:0], torch.empty(0, dtype=torch.int64, device=DEV))


@pytest.mark.parametrize("Dh", [64, 128])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("Hkv,G,T", [(1, 1, 1), (2, 8, 1), (3, 5, 2), (2, 6, 4), (1, 16, 1), (4, 2, 3), (1, 40, 1), (1, 3, 11)])
def test_attend(Hkv, G, T, page, Dh):
    lens = [0, 1, 2, 15, 16, 17, 63, 64, 65, 130, 700]
    p = Pool(sum(-(-n // page) for n in lens) + 2, page, Hkv, Dh, 1.0 if G % 2 else 2.5)
    table, ln, held = sequences(p, lens, seed=G)
    q = queries(len(lens), T, Hkv * G, Dh)
    out, lse = p.kv.attend(q, table, ln)
    check_attend(out, lse, q, held, Hkv, Dh ** -0.5)
    assert int(p.status[0]) == 0


@pytest.mark.parametrize("B,Hkv,G,T,Dh,page,n", [(1, 1, 8, 1, 128, 64, 40000), (1, 8, 4, 1, 128, 64, 9001), (3, 2, 2, 5, 64, 16, 5000),
                                               (2, 1, 16, 2, 64, 128, 20011), (40, 2, 8, 1, 128, 32, 999)])
def test_attend_long(B, Hkv, G, T, Dh, page, n):
    lens = [n] + [(n * (b + 1)) // (B + 1) for b in range(1, B)]
    p = Pool(sum(-(-m // page) for m in lens), page, Hkv, Dh)
    table, ln, held = sequences(p, lens, seed=n)
    q = queries(B, T, Hkv * G, Dh)
    out, lse = p.kv.attend(q, table, ln, softmax_scale=0.2)
    check_attend(out, lse, q, held, Hkv, 0.2)
    again, lse2 = p.kv.attend(q, table, ln, softmax_scale=0.2)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("B,Hkv,G,T,Dh,page,n", [(20, 16, 4, 1, 128, 64, 4300), (22, 14, 4, 2, 64, 16, 5000), (1, 8, 8, 1, 128, 32, 70000),
                                               (1, 24, 3, 1, 64, 128, 33333), (300, 2, 1, 1, 128, 256, 2600)])
def test_attend_long_runs(B, Hkv, G, T, Dh, page, n):
    """Blocks that walk long runs (four 16-token runs a step), over caches of random bytes whose free places
    hold no numbers; a sample of the sequences and heads is compared."""
    r = np.random.default_rng(n)
    lens = [n] + [int(v) for v in r.integers(0, n + 1, B - 1)]
    if B > 3:
        lens[1], lens[2], lens[3] = 0, 1, 17
    used = [-(-m // page) for m in lens]
    p = Pool(sum(used) + 1, page, Hkv, Dh)
    for i in (0, 2):
        p.t[i].copy_(torch.randint(0, 256, p.t[i].shape, device=DEV).to(torch.uint8))
        p.t[i + 1].copy_(torch.randint(0x20, 0x38, p.t[i + 1].shape, device=DEV).to(torch.uint8))
    order = r.permutation(p.pages)
    table, at = np.full((B, max(used)), -1, np.int32), 0
    for b, m in enumerate(used):
        table[b, :m] = order[at:at + m]
        at += m
        if lens[b] % page:
            for i in (1, 3):
                p.t[i][int(table[b, m - 1]), :, lens[b] % page:] = 0x7F
    q = queries(B, T, Hkv * G, Dh, size=1.0)
    out, lse = p.kv.attend(q, torch.from_numpy(table).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV))
    assert int(p.status[0]) == 0 and torch.isfinite(out.float()).all()
    again = p.kv.attend(q, torch.from_numpy(table).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV))
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    for b in {0, min(1, B - 1), min(2, B - 1), min(3, B - 1), *(int(v) for v in r.integers(0, B, 4))}:
        h = int(r.integers(0, Hkv))
        pages = torch.from_numpy(table[b, :used[b]]).long().to(DEV)
        k, v = (D.nvfp4_values(to_np(p.t[i][pages, h].flatten(0, 1))[:lens[b]], to_np(p.t[i + 1][pages, h].flatten(0, 1))[:lens[b]])
                for i in (0, 2))
        sl = slice(h * G, (h + 1) * G)
        check_attend(out[b:b + 1, :, sl], lse[b:b + 1, :, sl], q[b:b + 1, :, sl], [(k[:, None], v[:, None])], 1, Dh ** -0.5)


def test_attend_spikes_far_scores_and_large_queries():
    """One score far above a long tail, scores of both signs past any exponent's range, zero queries."""
    lens, page, Dh = [3000, 3000, 3000, 3000], 64, 128
    p = Pool(200, page, 1, Dh)
    table, ln, held = sequences(p, lens, seed=9)
    q = queries(4, 1, 8, Dh)
    spike = held[0][0][1234, 0]
    q[0, 0, :] = bf16(np.tile(spike * 2, (8, 1)))         # one token's score near 2 |k|^2 / sqrt(D)
    q[1] *= 300.0                                         # softmax down to one token
    q[2] = 0
    q[3, 0, ::2] *= 1e-20
    out, lse = p.kv.attend(q, table, ln)
    check_attend(out, lse, q, held, 1, Dh ** -0.5)
    big = queries(4, 1, 8, Dh, size=1e6)                  # queries outside FP16's range, scores kept small
    out, lse = p.kv.attend(big, table, ln, softmax_scale=1e-7)
    check_attend(out, lse, big, held, 1, 1e-7)
    out, lse = p.kv.attend(q, table, ln, softmax_scale=0.0)   # plain mean of the values
    check_attend(out, lse, q, held, 1, 0.0)
    out, lse = p.kv.attend(q, table, ln, softmax_scale=-0.1)
    check_attend(out, lse, q, held, 1, -0.1)


def test_attend_bad_query_row_stays_alone():
    lens = [100, 900]
    p = Pool(20, 64, 2, 128)
    table, ln, _ = sequences(p, lens)
    q = queries(2, 2, 8, 128)
    out, lse = (t.clone() for t in p.kv.attend(q, table, ln))
    q[1, 0, 5, 17] = float("nan")
    got, got_lse = p.kv.attend(q, table, ln)
    mask = torch.ones(2, 2, 8, dtype=torch.bool, device=DEV)
    mask[1, 0, 5] = False
    assert torch.equal(got[mask], out[mask]) and torch.equal(got_lse[mask], lse[mask])
    assert torch.isnan(got[1, 0, 5].float()).all() and torch.isnan(got_lse[1, 0, 5])


@pytest.mark.parametrize("B,Hkv,G,T,Dh,page,lens,wide", [(3, 8, 4, 1, 128, 64, (9000, 700, 0), 200000), (6, 2, 3, 4, 64, 16, (5000, 64, 3, 257, 1024, 2049), 60000),
                                                         (1, 4, 8, 1, 128, 32, (2500,), 1 << 20), (2, 1, 16, 1, 128, 16, (4001, 130), 100000),
                                                         (64, 8, 2, 1, 128, 64, tuple(range(1, 3201, 50)), 131072)])
def test_attend_with_a_table_far_wider_than_the_sequences(B, Hkv, G, T, Dh, page, lens, wide):
    """The work is cut by the table's width: blocks walk a sequence in several runs, or find nothing in it."""
    p = Pool(sum(-(-n // page) for n in lens), page, Hkv, Dh)
    table, ln, held = sequences(p, list(lens), seed=B)
    far = torch.full((B, wide // page), -7, dtype=torch.int32, device=DEV)
    far[:, :table.shape[1]] = table
    q = queries(B, T, Hkv * G, Dh)
    out, lse = p.kv.attend(q, far, ln, softmax_scale=0.2)
    check_attend(out, lse, q, held, Hkv, 0.2)
    assert int(p.status[0]) == 0


def test_attend_bad_pages_and_lengths():
    lens, page = [200, 70], 16
    p = Pool(30, page, 1, 64)
    table, ln, held = sequences(p, lens)
    q = queries(2, 1, 4, 64)
    bad = table.clone()
    bad[0, 3], bad[0, 7] = p.pages, -1                    # tokens 48..63 and 112..127 are skipped
    out, lse = p.kv.attend(q, bad, ln)
    keep = np.r_[0:48, 64:112, 128:200]
    check_attend(out, lse, q, [(held[0][0][keep], held[0][1][keep]), held[1]], 1, 0.125)
    assert int(p.status[0]) == pkg.MOE_DEV_BAD_INDEX
    p.status.zero_()
    cols = -(-200 // page)
    longer = torch.tensor([cols * page + 1000, -5], dtype=torch.int32, device=DEV)
    p.t[1][bad[0, cols - 1].item()] = 0                   # the last page's free places now hold numbers (zero)
    p.t[3][bad[0, cols - 1].item()] = 0
    k, v = (np.concatenate([h[:(cols - 1) * page], np.zeros((page, 1, 64))]) for h in held[0])
    out, lse = p.kv.attend(q, table, longer)
    check_attend(out, lse, q, [(k, v), (np.zeros((0, 1, 64)), np.zeros((0, 1, 64)))], 1, 0.125)
    assert int(p.status[0]) == pkg.MOE_DEV_BAD_INDEX


def test_cache_past_four_gigabytes_and_strided_queries():
    """Pages 2 MB apart, so offsets pass 32 bits; queries, keys and values inside one projection."""
    page, Hkv, Dh, pages = 32, 2, 128, 2400
    raw = torch.zeros(pages, 2 << 20, dtype=torch.uint8, device=DEV)
    nd, ns = Hkv * page * Dh // 2, Hkv * page * Dh // 16

    def part(at, width):
        return raw.as_strided((pages, Hkv, page, width), (2 << 20, page * width, width, 1), at)
    p = Pool(1, page, Hkv, Dh)
    p.pages = pages
    p.t = [part(0, Dh // 2), part(2 * nd, Dh // 16), part(nd, Dh // 2), part(2 * nd + ns, Dh // 16)]
    p.kv = pkg.NVFP4KVCache(*p.t, dev_status=p.status)
    lens = [100, 33]
    table, ln, held = sequences(p, lens, order=np.array([2399, 0, 2200, 1100, 2398, 1300]))
    qkv = bf16(np.random.default_rng(3).normal(size=(2, 12, Dh)))
    q = qkv[:, :8].unsqueeze(1)
    out, lse = p.kv.attend(q, table, ln)
    check_attend(out, lse, q, held, Hkv, Dh ** -0.5)
    assert int(raw[1].sum()) == 0 and int(p.status[0]) == 0


def test_attend_writes_nothing_else():
    lens = [0, 5, 400, 3000]
    p = Pool(80, 64, 2, 128)
    table, ln, _ = sequences(p, lens)
    q = queries(4, 3, 10, 128)
    ref = p.kv.attend(q, table, ln)
    g = Guarded(16)
    out, lse = g(tuple(q.shape), torch.bfloat16), g((4, 3, 10), torch.float32)
    n = pkg.moe_kv_attend_workspace_bytes(p.kv.c, 4, 3, 10, table.shape[1])
    ws = g((n,), torch.uint8, 0xFF) if n else None        # whatever a workspace holds before is not used
    p.kv.attend(q, table, ln, out=out, lse=lse, workspace=ws)
    assert g.intact() and torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
    again = p.kv.attend(q, table, ln, workspace=ws)
    assert torch.equal(again[0], ref[0])


def test_the_c_entry_points_by_name():
    """The ctypes calls of the C names give what the torch layer gives."""
    x, res, w = norm_case(5, 256, True, "group")
    ref = pkg.add_rms_norm(x, w, res, fp8="group")
    got = [torch.empty_like(t) for t in ref]
    pkg.moe_add_rmsnorm(x, res, w, 1e-6, pkg.MOE_FP8_PER_GROUP, *got)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(ref, got))
    x, scale, data, sf, alpha = linear_case(5, 64, 256, "group")
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    out = torch.empty(5, 64, dtype=torch.bfloat16, device=DEV)
    pkg.moe_linear_fp4(x, up(scale), pkg.MOE_FP8_PER_GROUP, up(data), up(sf), torch.tensor([alpha], device=DEV),
                       pkg.MOE_ACT_IDENTITY, out)
    assert torch.equal(out, run_linear(x, scale, data, sf, alpha))
    lens = [3, 700]
    a, b = Pool(50, 16, 2, 64), Pool(50, 16, 2, 64)
    table, ln, _ = sequences(a, lens)
    for s, d in zip(a.t, b.t):
        d.copy_(s)
    k, v = queries(2, 1, 2, 64, seed=4)[:, 0], queries(2, 1, 2, 64, seed=5)[:, 0]
    slots = torch.tensor([int(table[0, 0]) * 16 + 2, int(table[1, 43]) * 16 + 11], device=DEV)
    a.kv.append(k, v, slots)
    pkg.moe_kv_append(b.kv.c, k, v, slots, None, None, b.status)
    assert all(torch.equal(s, d) for s, d in zip(a.t, b.t))
    q = queries(2, 1, 8, 64)
    ref = a.kv.attend(q, table, ln)
    out, lse = torch.empty_like(ref[0]), torch.empty_like(ref[1])
    n = pkg.moe_kv_attend_workspace_bytes(b.kv.c, 2, 1, 8, table.shape[1])
    ws = torch.empty(n, dtype=torch.uint8, device=DEV) if n else None
    pkg.moe_kv_attend(b.kv.c, q, 8 * 64, table, ln, 0.125, out, lse, ws, b.status)
    assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])


def test_empty_batches_tables_and_caches():
    p = Pool(4, 16, 2, 64)
    q = queries(2, 1, 4, 64)
    none = torch.empty(2, 0, dtype=torch.int32, device=DEV)
    for lens, status in (([0, 0], 0), ([5, 0], pkg.MOE_DEV_BAD_INDEX)):   # no page at all for a length above 0
        out, lse = p.kv.attend(q, none, torch.tensor(lens, dtype=torch.int32, device=DEV))
        assert (out == 0).all() and torch.isneginf(lse).all() and int(p.status[0]) == status
    out, lse = p.kv.attend(q[:0], none[:0], torch.empty(0, dtype=torch.int32, device=DEV))
    assert out.shape == (0, 1, 4, 64) and lse.shape == (0, 1, 4)
    empty = pkg.NVFP4KVCache.allocate(0, 16, 2, 64, DEV)
    table = torch.zeros(2, 3, dtype=torch.int32, device=DEV)
    out, lse = empty.attend(q, table, torch.tensor([40, 1], dtype=torch.int32, device=DEV))
    assert (out == 0).all() and torch.isneginf(lse).all() and int(empty.dev_status[0]) == pkg.MOE_DEV_BAD_INDEX


def test_norm_of_subnormal_rows_stays_finite():
    x = torch.zeros(3, 256, dtype=torch.bfloat16, device=DEV)
    x[0, ::2] = 2.0 ** -130
    x[1, 5] = 2.0 ** -126
    w = torch.full((256,), 2.0 ** -4, dtype=torch.bfloat16, device=DEV)
    for fp8 in ("token", "group"):
        y, _, y8, scale = pkg.add_rms_norm(x, w, fp8=fp8)
        assert all(torch.isfinite(t.float()).all() for t in (y, y8, scale)) and (scale >= 0).all()
        want = x.double() / np.sqrt(1e-6) * 2.0 ** -4
        # scales this small are subnormal: a few bits are left of them
        assert (y8.double() * scale[:, :1].double() - want).abs().max() <= want.abs().max() * 0.25


def test_operators_run_on_the_callers_stream_and_in_a_graph():
    """One decode step (norm, projection, append, attention) captured, then replayed on new values."""
    H, Hkv, G, Dh, page = 256, 2, 2, 64, 16
    Hq = Hkv * G
    r = np.random.default_rng(8)
    lin = pkg.NVFP4Linear.from_bf16(bf16(0.05 * r.normal(size=((Hq + 2 * Hkv) * Dh, H))))
    w = bf16(1 + 0.1 * r.normal(size=H))
    x = bf16(r.normal(size=(3, H)))
    lens = [20, 1, 300]
    p = Pool(40, page, Hkv, Dh)
    table, ln, _ = sequences(p, lens)
    slots = torch.tensor([int(table[b, (n - 1) // page]) * page + (n - 1) % page for b, n in enumerate(lens)], device=DEV)

    def step():
        _, _, y8, sc = pkg.add_rms_norm(x, w, fp8="group")
        qkv = lin(y8, sc).view(3, Hq + 2 * Hkv, Dh)
        p.kv.append(qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], slots)
        return p.kv.attend(qkv[:, :Hq].unsqueeze(1), table, ln)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step()
    for seed in (1, 2):
        x.copy_(bf16(np.random.default_rng(seed).normal(size=(3, H))))
        graph.replay()
        got = out.clone(), lse.clone()
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.current_stream())
            want = step()
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
