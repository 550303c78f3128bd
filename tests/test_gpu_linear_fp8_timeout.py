"""The E4M3 product's bounded waits running out, through the test build (libmoe_nvfp4_test.so).

The test build does not start the copies of the first tiles' first block of K and cuts the limit of every wait to
2 ms: nothing faults, the waits run out. The call must return, report the timeout and leave the context usable: the
next call is exact.
"""
import pytest
import torch

from gpu_harness import DEV, pkg
from test_gpu_serving import linear_case, same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K,act", [(5, 300, 512, "identity"),        # a tile's K in slices
                                       (128, 20000, 144, "identity"),    # single blocks, K whole
                                       (2048, 2048, 4096, "identity"),   # pairs, one tile each
                                       (4000, 4096, 528, "swiglu")])     # pairs, several tiles each
def test_withheld_copies_time_out_and_the_next_call_is_exact(M, N, K, act):
    x, xs, w, ws = linear_case(M, N, K)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    ref = pkg.fp8_linear(x, xs, w, ws, act, dev_status=status)
    assert int(status) == 0

    def call(opts=None):
        status.zero_()
        out = torch.zeros_like(ref)
        pkg.moe_linear_fp8(x, xs, pkg.MOE_FP8_PER_GROUP, w, ws, pkg.ACTIVATIONS[act], out, status, test_options=opts)
        torch.cuda.synchronize()
        return int(status), out

    st, out = call(pkg.test_options())           # the test build with default options
    assert st == 0 and same(out, ref)
    st, _ = call(pkg.test_options(withhold_release=True, wait_limit_ns=2_000_000))
    assert st == pkg.MOE_DEV_TIMEOUT, f"status {st}: the wait for copies that never started did not run out"
    st, out = call()                             # the product path, right after
    assert st == 0 and same(out, ref)
