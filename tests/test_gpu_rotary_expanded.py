"""Rotary positions of several axes that one row gives to all of them: as with the row written out."""
import pytest
import torch

from gpu_harness import pkg
from test_gpu_serving import check_rotary, rotary_case, same, up

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("N,D,rot,axes", [(1, 128, 128, 3), (7, 96, 30, 4), (33, 128, 96, 3), (5000, 64, 64, 2)])
def test_expanded_positions(N, D, rot, axes, dtype):
    q, k, pos, freq, which = rotary_case(N, 4, 2, D, rot, axes)
    row = up(pos[0]).to(dtype)
    got = pkg.rotary(q, row.expand(axes, N), up(freq), k=k, axes=up(which))
    ref = pkg.rotary(q, row.repeat(axes, 1), up(freq), k=k, axes=up(which))
    one = pkg.rotary(q, row, up(freq), k=k)
    for a, b, c, x in zip(got, ref, one, (q, k)):
        assert same(a, b) and same(a, c)
        check_rotary(a, x, pos[:1].repeat(axes, 0), freq, which, False)
