"""The attention's bounded waits running out, through the test build (libmoe_nvfp4_test.so).

A warp's wait for its copies gives up after a limit, sets MOE_DEV_TIMEOUT in the caller's status word, waits
(again with the limit) for the copies that are in flight and lets the block finish. Normal inputs never
reach that path. The test build does, without any fault: the copies of each sequence's first tokens are
not started, so the warps that take them wait for bytes that nothing brings, and the limit is cut to 2 ms. The
call must return, report the timeout and leave the context usable: the next call is exact.
"""
import pytest
import torch

from gpu_harness import DEV, pkg
from test_gpu_decoder import Pool, queries, sequences

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("outlier", [False, True])        # queries that a block starts again for
@pytest.mark.parametrize("lens,Hkv,G,T,Dh,page", [((40, 5), 2, 4, 1, 128, 64),            # one block a sequence
                                                  ((9000, 700, 3), 1, 8, 1, 128, 16),     # split and joined
                                                  ((6000,) * 40, 8, 4, 1, 128, 64),       # four 16-token runs a step
                                                  ((3000, 64), 2, 6, 4, 64, 32)])         # three tiles of rows
def test_withheld_copies_time_out_and_the_next_call_is_exact(lens, Hkv, G, T, Dh, page, outlier):
    p = Pool(sum(-(-n // page) for n in lens), page, Hkv, Dh)
    table, ln, _ = sequences(p, list(lens))
    B, Hq = len(lens), Hkv * G
    q = queries(B, T, Hq, Dh)
    if outlier:
        q[..., 0] = 2.0 ** 40
    n = pkg.moe_kv_attend_workspace_bytes(p.kv.c, B, T, Hq, table.shape[1])
    ws = torch.empty(n, dtype=torch.uint8, device=DEV) if n else None

    def call(opts=None):
        p.status.zero_()
        out = torch.empty(B, T, Hq, Dh, dtype=torch.bfloat16, device=DEV)
        lse = torch.empty(B, T, Hq, dtype=torch.float32, device=DEV)
        pkg.moe_kv_attend(p.kv.c, q, Hq * Dh, table, ln, Dh ** -0.5, out, lse, ws, p.status, test_options=opts)
        torch.cuda.synchronize()
        return int(p.status[0]), out, lse

    ref = p.kv.attend(q, table, ln)
    st, out, lse = call(pkg.test_options())           # the test build with default options
    assert st == 0 and torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
    st, _, _ = call(pkg.test_options(withhold_release=True, wait_limit_ns=2_000_000))
    assert st == pkg.MOE_DEV_TIMEOUT, f"status {st}: the wait for copies that never started did not run out"
    st, out, lse = call()                             # the product path, right after
    assert st == 0 and torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
