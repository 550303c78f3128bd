"""The Python layer of the E4M3 quantiser and product, the rotary positions and the sampling refuses tensors of two devices
(made-up devices: no test has two GPUs)."""
import pytest
import torch

import nvfp4_routed_moe_sort_gb300 as pkg
from nvfp4_routed_moe_sort_gb300 import decoder
from nvfp4_routed_moe_sort_gb300.build import build
from test_decoder_host import _elsewhere, host_only

BF, F8, F32, U8, I32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32, torch.uint8, torch.int32


@pytest.fixture(scope="module", autouse=True)
def native():
    build()
    return decoder._load()


def _all_refused(call, make, names):
    for name, kw in _elsewhere(make, names):
        with pytest.raises(ValueError, match=f"{name} is on cuda:1"):
            call(**kw)


@host_only
def test_tensors_of_two_devices_are_refused():
    def maker(f):
        return lambda on: f(lambda name, shape, dtype: torch.empty(shape, dtype=dtype, device=on(name)))
    _all_refused(pkg.quantize_fp8, maker(lambda t: dict(x=t("x", (4, 256), BF), out=(t("y", (4, 256), F8), t("the scales", (4, 2), F32)))), ["y", "the scales"])
    _all_refused(pkg.fp8_linear, maker(lambda t: dict(x=t("x", (4, 256), F8), x_scale=t("x_scale", (4, 2), F32), w=t("w", (32, 256), F8),
                                                      w_scale=t("w_scale", (1, 2), F32), out=t("out", (4, 32), BF), dev_status=t("dev_status", (1,), I32))),
                 ["x_scale", "w", "w_scale", "out", "dev_status"])
    _all_refused(pkg.rotary, maker(lambda t: dict(q=t("q", (4, 2, 64), BF), k=t("k", (4, 1, 64), BF), positions=t("positions", (4,), torch.int64),
                                                  inv_freq=t("inv_freq", (32,), torch.float64), axes=t("axes", (32,), U8),
                                                  out=(t("q_out", (4, 2, 64), BF), t("k_out", (4, 1, 64), BF)), dev_status=t("dev_status", (1,), I32))),
                 ["k", "positions", "inv_freq", "axes", "q_out", "k_out", "dev_status"])
    _all_refused(pkg.sample_tokens, maker(lambda t: dict(logits=t("logits", (4, 64), BF), uniform=t("uniform", (4,), F32), temperature=t("temperature", (4,), F32),
                                                         top_k=t("top_k", (4,), I32), top_p=t("top_p", (4,), F32), min_p=t("min_p", (4,), F32), out=t("out", (4,), I32))),
                 ["uniform", "temperature", "top_k", "top_p", "min_p", "out"])
