"""Rotary positions of several axes in one row, at the C entry point (host checks, no GPU)."""
import pytest
import torch

import nvfp4_routed_moe_sort_gb300 as pkg
from nvfp4_routed_moe_sort_gb300.build import build

OK, INVALID, MISALIGNED, OVERLAP, MB = 0, 1, 3, 6, 1 << 20


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake device pointers: host-only check")
def test_a_stride_of_0_is_taken_and_others_below_n_are_not():
    build()

    def call(ldp=0, A=3, N=0, ax=7 * MB, qo=5 * MB):
        return pkg.lib().moe_rotary(MB, 512, 4, None, 0, 0, 128, 128, 0, 3 * MB, 8, ldp, A, 4 * MB, ax, N, qo, 512, None, 0, None, None)
    assert call() == OK and call(ldp=8) == OK
    # with tokens, up to a check that comes after the stride's
    assert call(N=8, ax=None) == INVALID and call(N=8, qo=5 * MB + 1) == MISALIGNED
    for ldp in (1, 7, -1, -8):
        assert call(ldp=ldp, N=8, qo=5 * MB + 1) == INVALID
    assert call(N=8, qo=3 * MB) == OVERLAP and call(N=8, qo=3 * MB + 48) == OVERLAP
