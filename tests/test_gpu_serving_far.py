"""Tensors of more than 2^31 values and 2^32 bytes: rows at their far ends are those of a call on these rows alone."""
import numpy as np
import pytest
import torch

from gpu_harness import DEV, pkg
from test_gpu_serving import F8, same

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def room():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def ends(M):
    return torch.cat((torch.arange(3), torch.arange(M - 300, M))).to(DEV)


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("K", [65536, 65537])
def test_quantize(K, rows):
    M = 33024  # whole blocks of 128
    x = torch.empty(M, K, dtype=torch.bfloat16, device=DEV).normal_()
    y, scale = pkg.quantize_fp8(x, rows=rows)
    y2, scale2 = pkg.quantize_fp8(x[-256:], rows=rows)
    assert same(y[-256:], y2) and same(scale[-len(scale2):], scale2) and y2.float().abs().max() == 448


@pytest.mark.parametrize("M,N,K", [(140000, 16384, 128), (40, 150000, 16384), (150000, 300, 16384)])  # far in out, in w, in x
def test_linear(M, N, K):
    """Whole numbers whose sums are exact, so that the cut of a call does not show."""
    g = torch.Generator(device=DEV).manual_seed(M)
    x, w = (torch.randint(-2, 3, s, device=DEV, generator=g, dtype=torch.int8).to(torch.bfloat16).to(F8) for s in ((M, K), (N, K)))
    xs, ws = torch.ones(M, 1, device=DEV), torch.ones(-(-N // 128), -(-K // 128), device=DEV)
    xs[-1] = ws[-1] = 2.0
    out = pkg.fp8_linear(x, xs, w, ws)
    rows, first = ends(M) if M > 300 else torch.arange(M, device=DEV), (N - 300) // 128 * 128
    exact = (x[rows].float().double() * xs[rows]) @ (w[first:].float().double() * ws[first // 128:, :1].repeat_interleave(128, 0)[:N - first]).T
    assert torch.equal(out[rows][:, first:], exact.bfloat16()) and exact.any()


def test_rotary():
    N, H, D = 140000, 128, 128
    q = torch.empty(N, H, D, dtype=torch.bfloat16, device=DEV).normal_()
    pos, freq = torch.arange(N, device=DEV), torch.rand(64, device=DEV, dtype=torch.float64)
    rows = ends(N)
    want = pkg.rotary(q[rows], pos[rows], freq)[0]
    assert same(pkg.rotary(q, pos, freq)[0][rows], want)
    odd = pkg.rotary(q, pos, freq[:31])[0][rows]  # pairs by the value
    assert same(odd, pkg.rotary(q[rows], pos[rows], freq[:31])[0])
    pkg.rotary(q, pos, freq, out=(q, None))
    assert same(q[rows], want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sample(dtype):
    B, V = 8300, 262144
    x = torch.empty(B, V, dtype=dtype, device=DEV).normal_()
    u, top_p = torch.rand(B, device=DEV), torch.full((B,), 0.9, device=DEV)
    rows = ends(B)
    for kw in ({}, dict(top_p=top_p)):
        got = pkg.sample_tokens(x, u, **kw)[rows]
        assert torch.equal(got, pkg.sample_tokens(x[rows], u[rows], **{k: v[rows] for k, v in kw.items()})) and got.unique().numel() > 200
