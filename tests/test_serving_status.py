"""The status word of an FP8 layer reaches the call, whatever made the layer (a stand-in for the native module: no GPU)."""
import pytest
import torch

import nvfp4_routed_moe_sort_gb300 as pkg
from nvfp4_routed_moe_sort_gb300 import decoder

TIMEOUT = pkg.MOE_DEV_TIMEOUT


class Native:
    """Calls whose waits run out: they set the bit in the word that they are given, if any."""

    def fp8_linear(self, x, x_scale, w, w_scale, act, out, dev_status):
        if dev_status is not None:
            dev_status[0] |= TIMEOUT

    def quantize_fp8(self, x, rows, y, scale):
        pass


@pytest.fixture(autouse=True)
def native(monkeypatch):
    monkeypatch.setattr(decoder, "_native", Native())


def call(layer):
    return layer(torch.zeros(4, 256).to(torch.float8_e4m3fn), torch.ones(4, 2))


def matrix():
    return torch.zeros(128, 256).to(torch.float8_e4m3fn), torch.ones(1, 2)


def test_a_wait_that_ran_out_shows_in_the_layers_own_word():
    for layer in (pkg.FP8Linear(*matrix()), pkg.FP8Linear.from_bf16(torch.zeros(128, 256, dtype=torch.bfloat16), "relu")):
        assert layer.dev_status.dtype == torch.int32 and layer.dev_status.device == layer.w.device and int(layer.dev_status[0]) == 0
        call(layer)
        assert int(layer.dev_status[0]) == TIMEOUT


def test_layers_may_share_a_word():
    word = torch.zeros(4, dtype=torch.int32)
    first = pkg.FP8Linear(*matrix(), dev_status=word)
    second = pkg.FP8Linear.from_bf16(torch.zeros(128, 256, dtype=torch.bfloat16), dev_status=word)
    assert first.dev_status is word and second.dev_status is word
    call(second)
    assert word.tolist() == [TIMEOUT, 0, 0, 0]


def test_layers_of_their_own_words_do_not_share_one():
    a, b = pkg.FP8Linear(*matrix()), pkg.FP8Linear(*matrix())
    call(a)
    assert int(a.dev_status[0]) == TIMEOUT and int(b.dev_status[0]) == 0
