"""Refusals of the E4M3 quantiser and product, the rotary positions and the sampling at the C entry points (host
checks, no GPU)."""
import pytest
import torch

import nvfp4_routed_moe_sort_gb300 as pkg
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
def test_quantize_validation(lib):
    def call(x=1 * MB, ld=256, M=4, K=256, rows=1, y=2 * MB, sc=3 * MB):
        return lib.moe_quantize_fp8(x, ld, M, K, rows, y, sc, None)
    assert call(M=0) == OK and call(M=0, x=None) == OK
    assert call(M=-1) == INVALID and call(K=0) == INVALID and call(ld=255) == INVALID
    assert call(rows=0) == INVALID and call(rows=2) == INVALID and call(rows=-128) == INVALID
    assert call(x=None) == INVALID and call(y=None) == INVALID and call(sc=None) == INVALID
    assert call(x=MB + 1) == MISALIGNED and call(sc=3 * MB + 2) == MISALIGNED
    assert call(y=MB) == OVERLAP and call(y=MB + 2047) == OVERLAP and call(sc=MB) == OVERLAP and call(sc=2 * MB + 1020) == OVERLAP
    assert call(M=(1 << 31) - 1, K=(1 << 31) - 1, ld=1 << 31) == SHAPE and call(rows=128, M=(1 << 31) - 1) == SHAPE


@host_only
def test_linear_validation(lib):
    def call(x=1 * MB, ld=256, xs=2 * MB, mode=2, M=4, K=256, w=3 * MB, ws=4 * MB, N=32, act=6, out=5 * MB):
        return lib.moe_linear_fp8(x, ld, xs, mode, M, K, w, ws, N, act, out, None, None)
    assert call(M=0) == OK
    assert call(M=-1) == INVALID and call(N=0) == INVALID and call(K=0) == INVALID and call(ld=255) == INVALID
    assert call(mode=0) == INVALID and call(mode=3) == INVALID and call(act=7) == INVALID and call(act=-1) == INVALID
    for name in ("x", "xs", "w", "ws", "out"):
        assert call(**{name: None}) == INVALID, name
    assert call(K=24, ld=32) == SHAPE and call(K=65552, ld=65552) == SHAPE and call(N=(1 << 22) + 1) == SHAPE
    assert call(M=(1 << 22) + 1) == SHAPE
    for act in (0, 2):                                    # gated: whole blocks of 128 in each half
        assert call(act=act, N=32) == SHAPE and call(act=act, N=384) == SHAPE
    assert call(x=MB + 8) == MISALIGNED and call(w=3 * MB + 8) == MISALIGNED and call(out=5 * MB + 2) == MISALIGNED
    assert call(ld=264) == MISALIGNED and call(xs=2 * MB + 2) == MISALIGNED and call(ws=4 * MB + 1) == MISALIGNED
    assert call(out=1 * MB) == OVERLAP and call(out=2 * MB) == OVERLAP and call(out=3 * MB + 16) == OVERLAP and call(out=4 * MB) == OVERLAP


@host_only
def test_rotary_validation(lib):
    def call(q=1 * MB, ldq=512, Hq=4, k=2 * MB, ldk=256, Hk=2, D=128, rot=128, adj=0, pos=3 * MB, pb=8, ldp=16, A=1, f=4 * MB, ax=None,
             N=8, qo=5 * MB, ldqo=512, ko=6 * MB, ldko=256):
        return lib.moe_rotary(q, ldq, Hq, k, ldk, Hk, D, rot, adj, pos, pb, ldp, A, f, ax, N, qo, ldqo, ko, ldko, None, None)
    assert call(N=0) == OK
    assert call(N=-1) == INVALID and call(Hq=0) == INVALID and call(Hk=-1) == INVALID and call(D=0) == INVALID
    assert call(rot=0) == INVALID and call(rot=63) == INVALID and call(rot=130) == INVALID
    assert call(pb=2) == INVALID and call(A=0) == INVALID and call(A=2, ldp=7, ax=7 * MB) == INVALID and call(A=2) == INVALID
    assert call(ldq=511) == INVALID and call(ldqo=511) == INVALID and call(ldk=255) == INVALID and call(ldko=255) == INVALID
    assert call(D=1026, ldq=8192, ldk=8192, ldqo=8192, ldko=8192) == SHAPE and call(A=5, ax=7 * MB) == SHAPE
    assert call(Hq=1025, ldq=1 << 20, ldqo=1 << 20) == SHAPE
    for name in ("q", "k", "qo", "ko", "pos", "f"):
        assert call(**{name: None}) == INVALID, name
    assert call(q=MB + 1) == MISALIGNED and call(ko=6 * MB + 1) == MISALIGNED and call(pos=3 * MB + 4) == MISALIGNED
    assert call(pos=3 * MB + 2, pb=4) == MISALIGNED and call(f=4 * MB + 4) == MISALIGNED
    assert call(qo=MB + 16) == OVERLAP and call(qo=2 * MB) == OVERLAP and call(ko=1 * MB) == OVERLAP and call(ko=5 * MB) == OVERLAP
    assert call(qo=1 * MB, ldqo=520) == OVERLAP           # in place needs the same stride
    assert call(qo=3 * MB) == OVERLAP and call(qo=4 * MB) == OVERLAP
    # slices of one row side by side are apart; one value further they are not
    assert call(q=MB, ldq=1024, k=MB + 1024 - 2, ldk=1024, qo=MB, ldqo=1024) == OVERLAP


@host_only
def test_sample_validation(lib):
    def call(x=1 * MB, dt=1, ld=1000, B=4, V=1000, u=2 * MB, t=3 * MB, k=4 * MB, p=5 * MB, m=6 * MB, out=7 * MB):
        return lib.moe_sample(x, dt, ld, B, V, u, t, k, p, m, out, None)
    assert call(B=0) == OK
    assert call(B=-1) == INVALID and call(V=0) == INVALID and call(ld=999) == INVALID and call(dt=2) == INVALID and call(dt=-1) == INVALID
    assert call(V=(1 << 18) + 1, ld=1 << 19) == SHAPE and call(B=(1 << 24) + 1) == SHAPE
    assert call(x=None) == INVALID and call(u=None) == INVALID and call(out=None) == INVALID
    assert call(x=MB + 1) == MISALIGNED and call(x=MB + 2, dt=0) == MISALIGNED and call(out=7 * MB + 2) == MISALIGNED
    assert call(u=2 * MB + 1) == MISALIGNED and call(k=4 * MB + 2) == MISALIGNED
    for other in (1 * MB + 7996, 2 * MB, 3 * MB, 4 * MB, 5 * MB + 12, 6 * MB):
        assert call(out=other) == OVERLAP


def test_python_layer_refuses_without_a_gpu():
    bf, f32 = torch.bfloat16, torch.float32
    x = torch.zeros(4, 256)
    with pytest.raises(ValueError, match="x must be bf16 rows"):
        pkg.quantize_fp8(x)
    with pytest.raises(ValueError, match="rows must be 1 or 128"):
        pkg.quantize_fp8(x.to(bf), rows=64)
    with pytest.raises(ValueError, match="x must be float8_e4m3fn rows"):
        pkg.fp8_linear(x, torch.zeros(4, 2), torch.zeros(32, 256, dtype=torch.float8_e4m3fn), torch.zeros(1, 2))
    with pytest.raises(ValueError, match="activation must be one of"):
        pkg.fp8_linear(x, x, x, x, activation="tanh")
    with pytest.raises(ValueError, match="q must be bf16"):
        pkg.rotary(torch.zeros(4, 2, 64, dtype=bf), torch.zeros(4, dtype=torch.int64), torch.zeros(32, dtype=torch.float64))
    with pytest.raises(ValueError, match="logits must be"):
        pkg.sample_tokens(x.to(f32), torch.zeros(4))
