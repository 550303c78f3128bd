"""moe_linear_fp4 in every kind of cut (tests/linear_cuts.py) against the float64 oracle, tolerances as in
test_gpu_decoder.py: BF16 tokens, BF16 tokens of a range that takes BF16 MMAs, E4M3 tokens with either scales.
"""
import numpy as np
import pytest
import torch

from gpu_harness import DEV, pkg, to_np
from linear_cuts import CUTS, SMS
from nvfp4_routed_moe_sort_gb300._lib import linear_cut
from test_gpu_decoder import bf16, check_linear

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("i", range(len(CUTS)))
def test_linear_in_every_kind_of_cut(i):
    gated, M, N, K, *cut = CUTS[i]
    if torch.cuda.get_device_properties(DEV).multi_processor_count == SMS:
        c = linear_cut(M, K, N, gated, SMS)
        assert [c["warps"], c["across"], c["slices"], c["buffers"], c["stages"]] == cut
    gen = torch.Generator(device=DEV).manual_seed(i)
    r = np.random.default_rng(i)
    data = torch.randint(0, 256, (N, K // 2), device=DEV, generator=gen, dtype=torch.uint8)
    sf = torch.randint(0x18, 0x58, (N, K // 16), device=DEV, generator=gen, dtype=torch.uint8)
    alpha, act = torch.tensor([0.01], device=DEV), "swiglu" if gated else "identity"
    kind = ("bf16", "token", "wide", "group")[i % 4]
    x, scale = r.normal(size=(M, K)), None
    if kind == "wide":                                      # an outlier in every 128 values, under zeros for half of the rows
        at = torch.arange(5, K, 128, device=DEV)
        x[:, 5::128] = 2.0 ** 40
        half = torch.arange(0, N, 2, device=DEV)[:, None]
        data[half, at // 2] &= 0x0F
    if kind in ("bf16", "wide"):
        x = bf16(x)
    else:
        scale = (r.random((M, 1 if kind == "token" else -(-K // 128))) + 0.1).astype(np.float32)
        x = torch.from_numpy((x * 40).astype(np.float32)).to(DEV).clamp(-448, 448).to(torch.float8_e4m3fn)
    got = pkg.fp4_linear(x, data, sf, alpha, act, x_scale=None if scale is None else torch.from_numpy(scale).to(DEV))
    n_out = N // 2 if gated else N
    cols = np.unique(np.r_[0:min(n_out, 100), max(n_out - 100, 0):n_out, r.integers(0, n_out, 60)])
    if K > 12000:
        cols = cols[::3]
    rows = torch.from_numpy(np.r_[cols, cols + n_out] if gated else cols).to(DEV)
    check_linear(got[:, torch.from_numpy(cols).to(DEV)], x, scale, to_np(data[rows]), to_np(sf[rows]), float(alpha), act)
