"""Infinities and NaN in the E4M3 quantiser's blocks of 128 rows: the block's scale shows them, whatever else lies in it."""
import numpy as np
import pytest
import torch

from gpu_harness import DEV, pkg
from test_gpu_serving import same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("K", [256, 131])
@pytest.mark.parametrize("place", [(0, 0), (7, -1), (127, 3), (139, -1)])
def test_an_infinity_makes_its_groups_scale_infinite(K, rows, place):
    x = torch.ones(140, K, dtype=torch.bfloat16, device=DEV)
    ref = [t.clone() for t in pkg.quantize_fp8(x, rows=rows)]
    m, c = place[0], place[1] % K
    g, b = m // rows, c // 128
    for bad in (float("inf"), -float("inf")):
        x[m, c] = bad
        y, scale = pkg.quantize_fp8(x, rows=rows)
        assert torch.isposinf(scale[g, b]) and torch.isfinite(scale).sum() == scale.numel() - 1
        # the infinity's own code is no number (times 0), finite ones become 0; other groups stay as they were
        mine = torch.zeros(140, K, dtype=torch.bool, device=DEV)
        mine[g * rows:(g + 1) * rows, 128 * b:128 * b + 128] = True
        assert torch.isnan(y[m, c].float())
        mine[m, c] = False
        assert (y.float()[mine] == 0).all()
        mine[m, c] = True
        assert same(y.view(torch.uint8)[~mine], ref[0].view(torch.uint8)[~mine])
    x[m, c] = float("nan")
    y, scale = pkg.quantize_fp8(x, rows=rows)
    assert torch.isnan(scale[g, b]) and torch.isfinite(scale).sum() == scale.numel() - 1 and torch.isnan(y[m, c].float())
