"""Refusals of the operators around the routed experts: at the C entry points (host checks, no
GPU) and in the Python layer."""
import ctypes

import pytest
import torch

import nvfp4_routed_moe_sort_gb300 as pkg
from nvfp4_routed_moe_sort_gb300 import _lib as L
from nvfp4_routed_moe_sort_gb300.build import build

OK, INVALID, SHAPE, MISALIGNED, WORKSPACE, CUDA, OVERLAP = range(7)

# made-up device addresses that every call must reject on the host; run only where no launch could happen
host_only = pytest.mark.skipif(torch.cuda.is_available(), reason="fake device pointers: host-only check")
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    build()
    return pkg.lib()


@host_only
def test_norm_validation(lib):
    def call(x=1 * MB, ld_x=256, r=2 * MB, ld_r=256, w=3 * MB, M=4, H=256, eps=1e-6, mode=0, y=4 * MB, ro=5 * MB,
             y8=None, sc=None):
        return lib.moe_add_rmsnorm(x, ld_x, r, ld_r, w, M, H, eps, mode, y, ro, y8, sc, None)
    assert call(M=0) == OK
    assert call(M=-1) == INVALID and call(H=0) == INVALID
    assert call(H=32769, ld_x=40000, ld_r=40000) == SHAPE
    assert call(ld_x=255) == INVALID and call(ld_r=255) == INVALID
    assert call(eps=-1e-6) == INVALID and call(eps=float("nan")) == INVALID and call(eps=float("inf")) == INVALID
    assert call(mode=3) == INVALID
    assert call(x=None) == INVALID and call(w=None) == INVALID
    assert call(y=None) == INVALID                        # no output at all
    assert call(r=None) == INVALID                        # residual_out without residual
    assert call(mode=1) == INVALID                        # E4M3 output without its tensors
    assert call(mode=1, y8=6 * MB) == INVALID             # ... without its scales
    assert call(y8=6 * MB, sc=7 * MB) == INVALID          # ... without a scale mode
    assert call(x=MB + 2) == MISALIGNED and call(ro=5 * MB + 8) == MISALIGNED
    assert call(y=1 * MB) == OVERLAP                      # y over x
    assert call(ro=4 * MB + 16) == OVERLAP                # residual_out over y
    assert call(ro=2 * MB, ld_r=264) == OVERLAP           # in place needs ld_r == H
    assert call(mode=2, y8=6 * MB, sc=6 * MB + 512) == OVERLAP


@host_only
def test_linear_validation(lib):
    def call(x=1 * MB, ld=256, xs=None, mode=0, M=4, K=256, w=2 * MB, sf=3 * MB, al=4 * MB, N=32, act=6, out=5 * MB):
        return lib.moe_linear_fp4(x, ld, xs, mode, M, K, w, sf, al, N, act, out, None)
    assert call(M=0) == OK
    assert call(M=-1) == INVALID and call(N=0) == INVALID and call(K=0) == INVALID
    assert call(K=24, ld=24) == SHAPE and call(K=65552, ld=65552) == SHAPE
    assert call(ld=255) == INVALID
    assert call(mode=3) == INVALID and call(act=7) == INVALID and call(act=-1) == INVALID
    assert call(mode=1) == INVALID                        # E4M3 without scales
    assert call(xs=6 * MB) == INVALID                     # scales with BF16
    assert call(act=0, N=31) == INVALID                   # gated: even row count
    for name in ("x", "w", "sf", "al", "out"):
        assert call(**{name: None}) == INVALID
        assert call(**{name: 9 * MB + 8}) == MISALIGNED
    assert call(ld=260) == MISALIGNED
    assert call(mode=1, xs=6 * MB, ld=264) == MISALIGNED
    assert call(out=1 * MB) == OVERLAP and call(out=2 * MB + 16) == OVERLAP


def _cache(**kw):
    f = dict(k=1 * MB, k_sf=2 * MB, v=3 * MB, v_sf=4 * MB, num_pages=4, page_size=16, num_kv_heads=2, head_dim=64,
             data_page_stride=1024, sf_page_stride=128, k_scale=1.0, v_scale=1.0)
    f.update(kw)
    return L.KVCacheT(**f)


BAD_CACHES = [(dict(head_dim=96), SHAPE), (dict(page_size=24), SHAPE), (dict(page_size=8), SHAPE),
              (dict(page_size=512), SHAPE), (dict(num_kv_heads=0), INVALID), (dict(num_pages=-1), INVALID),
              (dict(k_scale=0.0), INVALID), (dict(v_scale=float("inf")), INVALID), (dict(k=None), INVALID),
              (dict(v_sf=4 * MB + 8), MISALIGNED), (dict(data_page_stride=1008), INVALID),
              (dict(sf_page_stride=136), MISALIGNED), (dict(data_page_stride=1032), MISALIGNED)]


@host_only
@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_cache_validation(lib, kw, status):
    c = _cache(**kw)
    assert lib.moe_kv_append(c, 5 * MB, 128, 6 * MB, 128, 7 * MB, 3, None, None, None, None) == status
    assert lib.moe_kv_attend(c, 5 * MB, 512, 1, 1, 4, 6 * MB, 4, 4, 7 * MB, 0.1, 8 * MB, None, 64 * MB, 1 << 40,
                             None, None) == status
    assert lib.moe_kv_attend_workspace_bytes(c, 1, 1, 4, 4) == 0


@host_only
def test_append_validation(lib):
    c = _cache()

    def call(k=5 * MB, ldk=128, v=6 * MB, ldv=128, slots=7 * MB, N=3, ks=None, vs=None, st=None, cache=c):
        return lib.moe_kv_append(cache, k, ldk, v, ldv, slots, N, ks, vs, st, None)
    assert call(cache=ctypes.POINTER(L.KVCacheT)()) == INVALID
    assert call(N=0) == OK and call(N=-1) == INVALID
    assert call(ldk=120) == INVALID and call(ldv=132) == MISALIGNED
    assert call(k=None) == INVALID and call(slots=None) == INVALID
    assert call(ks=8 * MB) == INVALID                     # both or neither
    assert call(st=8 * MB + 4) == MISALIGNED
    assert call(k=1 * MB + 512) == OVERLAP                # new keys inside the cache
    assert call(ks=8 * MB, vs=8 * MB + 512) == OVERLAP


@host_only
def test_attend_validation(lib):
    c = _cache()

    def call(q=5 * MB, ld=256, B=2, T=1, Hq=4, table=6 * MB, ldt=4, pages=4, lens=7 * MB, scale=0.1, out=8 * MB,
             lse=9 * MB, ws=64 * MB, wsb=1 << 40, st=None):
        return lib.moe_kv_attend(c, q, ld, B, T, Hq, table, ldt, pages, lens, scale, out, lse, ws, wsb, st, None)
    assert call(B=0) == OK
    assert call(B=-1) == INVALID and call(T=0) == INVALID and call(Hq=0) == INVALID
    assert call(Hq=3) == INVALID                          # not a multiple of the kv heads
    assert call(pages=5) == INVALID and call(ld=248) == INVALID and call(scale=float("nan")) == INVALID
    assert call(B=70000) == SHAPE and call(T=70000) == SHAPE and call(pages=1 << 28, ldt=1 << 28) == SHAPE
    for name in ("q", "table", "lens", "out"):
        assert call(**{name: None}) == INVALID
        assert call(**{name: 20 * MB + 4}) == MISALIGNED
    assert call(ld=260) == MISALIGNED
    assert call(out=5 * MB) == OVERLAP and call(lse=8 * MB + 64) == OVERLAP and call(out=3 * MB) == OVERLAP
    long = 1 << 16                                        # long sequences are split: their parts need room
    need = lib.moe_kv_attend_workspace_bytes(c, 2, 1, 4, long)
    if need:
        assert call(pages=long, ldt=long, wsb=need - 1) == WORKSPACE
        assert call(pages=long, ldt=long, ws=None, wsb=need) == INVALID


def _bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def test_python_layer_refuses_wrong_tensors():
    x, w = _bf(4, 256), _bf(256)
    for bad in (dict(fp8="row"), dict(x=x.float()), dict(weight=w[:128]), dict(residual=_bf(4, 128)),
                dict(x=_bf(256, 4).T), dict(x=x)):        # the last: tensors that are not on the GPU
        with pytest.raises(ValueError):
            pkg.add_rms_norm(**{"x": x, "weight": w, **bad})
    data, sf, alpha = torch.zeros(32, 128, dtype=torch.uint8), torch.zeros(32, 16, dtype=torch.uint8), torch.ones(1)
    for bad in (dict(activation="tanh"), dict(x=_bf(4, 128)), dict(w=data[:, ::2]), dict(w_sf=sf[:, :8]),
                dict(alpha=alpha.double()), dict(x_scale=torch.ones(4, 1)), dict(x=x)):
        with pytest.raises(ValueError):
            pkg.fp4_linear(**{"x": x, "w": data, "w_sf": sf, "alpha": alpha, **bad})
    kv = [torch.zeros(3, 2, 16, n, dtype=torch.uint8) for n in (32, 4, 32, 4)]
    for i, bad in ((0, kv[0][:, :, ::2]), (1, kv[1][:2]), (2, kv[2].int()), (3, kv[0]), (0, kv[0])):
        with pytest.raises(ValueError):
            pkg.NVFP4KVCache(*kv[:i], bad, *kv[i + 1:])
