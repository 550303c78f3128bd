"""What the torch layer of the E4M3 quantiser and product, the rotary positions and the sampling refuses, on tensors that
lie on the GPU: every call is right with its base arguments, and each test changes one of them. All of these are refused
on the host, before anything is launched.
"""
import pytest
import torch

from gpu_harness import DEV, pkg
from test_gpu_decoder_refusals import refused, t, wide

pytestmark = pytest.mark.gpu

BF, F8, F32, F64, U8, I32, I64 = (torch.bfloat16, torch.float8_e4m3fn, torch.float32, torch.float64, torch.uint8, torch.int32, torch.int64)


def whole(*shape, dtype):
    return torch.zeros(*shape, dtype=dtype, device=DEV)


# ------------------------------------------------------------------------- quantiser
def quantize_base():
    return dict(x=t(4, 256), rows=1, out=(t(4, 256, dtype=F8), t(4, 2, dtype=F32)))


QUANTIZE = [
    (lambda: dict(x=t(4, 256, dtype=F32)), "x must be bf16 rows"), (lambda: dict(x=t(256, 4).T), "x must be bf16 rows"),
    (lambda: dict(x=t(1024)), r"x must be \[M, K\]"), (lambda: dict(x=t(4, 256).cpu()), "x must be bf16 rows"),
    (lambda: dict(x=t(1, 256).expand(4, 256)), "MOE_ERR_INVALID_ARGUMENT"), (lambda: dict(x=[1.0]), "x must be a torch tensor"),
    (lambda: dict(rows=2), "rows must be 1 or 128"), (lambda: dict(rows=128), "the scales must be"),
    (lambda: dict(out=(t(4, 256), t(4, 2, dtype=F32))), "y must be"), (lambda: dict(out=(t(4, 255, dtype=F8), t(4, 2, dtype=F32))), "y must be"),
    (lambda: dict(out=(wide(4, 256, dtype=F8), t(4, 2, dtype=F32))), "y must be"),
    (lambda: dict(out=(t(4, 256, dtype=F8), t(4, 1, dtype=F32))), "the scales must be"),
    (lambda: dict(out=(t(4, 256, dtype=F8), t(4, 2))), "the scales must be"), (lambda: dict(out=(None, t(4, 2, dtype=F32))), "y must be a torch tensor"),
]


@pytest.mark.parametrize("i", range(len(QUANTIZE)))
def test_quantize_refuses(i):
    refused(pkg.quantize_fp8, quantize_base, QUANTIZE[i][0](), QUANTIZE[i][1])


def test_quantize_refuses_an_output_over_its_input():
    raw = torch.zeros(4096, dtype=U8, device=DEV)
    x = raw[:2048].view(BF).view(4, 256)
    refused(pkg.quantize_fp8, quantize_base, dict(x=x, out=(raw[1024:2048].view(F8).view(4, 256), t(4, 2, dtype=F32))), "MOE_ERR_OVERLAP")


# ---------------------------------------------------------------------------- product
def linear_base():
    return dict(x=t(4, 256, dtype=F8), x_scale=t(4, 2, dtype=F32), w=t(512, 256, dtype=F8), w_scale=t(4, 2, dtype=F32), out=t(4, 512))


LINEAR = [
    (lambda: dict(x=t(4, 256)), "x must be float8_e4m3fn rows"), (lambda: dict(x=wide(4, 256, dtype=F8)), "x must be float8_e4m3fn rows"),
    (lambda: dict(x=t(4, 256, dtype=F8).cpu()), "x must be float8_e4m3fn rows"), (lambda: dict(x=t(1024, dtype=F8)), r"x and w must be \[M, K\]"),
    (lambda: dict(x=t(4, 272, dtype=F8)[:, 8:264]), "MOE_ERR_MISALIGNED"), (lambda: dict(x=t(4, 264, dtype=F8)[:, :256]), "MOE_ERR_MISALIGNED"),
    (lambda: dict(x=t(4, 128, dtype=F8)), "x_scale must be"), (lambda: dict(x_scale=t(4, 3, dtype=F32)), "x_scale must be"),
    (lambda: dict(x_scale=t(3, 2, dtype=F32)), "x_scale must be"), (lambda: dict(x_scale=t(4, 2)), "x_scale must be"),
    (lambda: dict(x_scale=t(4, dtype=F32)), "x_scale must be"), (lambda: dict(x_scale=None), "x_scale must be a torch tensor"),
    (lambda: dict(w=t(512, 128, dtype=F8)), "w must be"), (lambda: dict(w=t(512, 256)), "w must be"), (lambda: dict(w=t(256, 512, dtype=F8).T), "w must be"),
    (lambda: dict(w_scale=t(3, 2, dtype=F32)), "w_scale must be"), (lambda: dict(w_scale=t(4, 1, dtype=F32)), "w_scale must be"),
    (lambda: dict(w_scale=t(2, 4, dtype=F32).T), "w_scale must be"), (lambda: dict(out=t(4, 512, dtype=F32)), "out must be"),
    (lambda: dict(out=t(4, 256)), "out must be"), (lambda: dict(out=wide(4, 512)), "out must be"), (lambda: dict(activation="swiglu"), "out must be"),
    (lambda: dict(activation="tanh"), "activation must be one of"), (lambda: dict(dev_status=t(1, dtype=F32)), "dev_status must be"),
    (lambda: dict(dev_status=whole(0, dtype=I32)), "dev_status must be"),
]


@pytest.mark.parametrize("i", range(len(LINEAR)))
def test_linear_refuses(i):
    refused(pkg.fp8_linear, linear_base, LINEAR[i][0](), LINEAR[i][1])


def test_linear_refuses_odd_k_and_gated_halves_that_are_not_blocks():
    call = dict(x=t(4, 24, dtype=F8), x_scale=t(4, 1, dtype=F32), w=t(512, 24, dtype=F8), w_scale=t(4, 1, dtype=F32))
    with pytest.raises(pkg.MoEError, match="MOE_ERR_UNSUPPORTED_SHAPE"):
        pkg.fp8_linear(**call)
    call = dict(x=t(4, 32, dtype=F8), x_scale=t(4, 1, dtype=F32), w=t(384, 32, dtype=F8), w_scale=t(3, 1, dtype=F32), activation="swiglu")
    with pytest.raises(pkg.MoEError, match="MOE_ERR_UNSUPPORTED_SHAPE"):
        pkg.fp8_linear(**call)


# ---------------------------------------------------------------------------- rotary
def rotary_base():
    return dict(q=t(4, 3, 64), positions=whole(2, 4, dtype=I64), inv_freq=whole(32, dtype=F64), k=t(4, 2, 64), axes=whole(32, dtype=U8),
                out=(t(4, 3, 64), t(4, 2, 64)))


ROTARY = [
    (lambda: dict(q=t(4, 3, 64, dtype=F32)), "q must be bf16"), (lambda: dict(q=t(12, 64)), r"q and k must be \[N"),
    (lambda: dict(q=t(3, 4, 64).transpose(0, 1)), "q must be bf16"), (lambda: dict(q=wide(4, 3, 64)), "q must be bf16"),
    (lambda: dict(q=t(4, 3, 64).cpu()), "q must be bf16"), (lambda: dict(k=t(3, 2, 64)), "k must be bf16"), (lambda: dict(k=t(4, 2, 32)), "k must be bf16"),
    (lambda: dict(k=None), "k_out must be given with k"), (lambda: dict(out=(t(4, 3, 64), None)), "k_out must be given with k"),
    (lambda: dict(out=(t(4, 2, 64), t(4, 2, 64))), "q_out must be bf16"), (lambda: dict(out=(t(4, 3, 64), t(4, 3, 64))), "k_out must be bf16"),
    (lambda: dict(positions=whole(2, 5, dtype=I64)), "positions must be"), (lambda: dict(positions=whole(2, 4, dtype=F32)), "positions must be"),
    (lambda: dict(positions=whole(4, 2, dtype=I64).T), "positions must be"), (lambda: dict(positions=whole(1, 2, 4, dtype=I64)), "positions must be"),
    (lambda: dict(positions=whole(5, 4, dtype=I64)), "MOE_ERR_UNSUPPORTED_SHAPE"), (lambda: dict(inv_freq=whole(32, dtype=F32)), "inv_freq must be"),
    (lambda: dict(inv_freq=whole(33, dtype=F64), axes=whole(33, dtype=U8)), "MOE_ERR_INVALID_ARGUMENT"), (lambda: dict(inv_freq=whole(2, 16, dtype=F64)), "inv_freq must be"),
    (lambda: dict(axes=whole(31, dtype=U8)), "axes must be"), (lambda: dict(axes=whole(32, dtype=I64)), "axes must be"), (lambda: dict(axes=None), "axes must be given"),
    (lambda: dict(dev_status=t(1)), "dev_status must be"), (lambda: dict(out=(t(1, 3, 64).expand(4, 3, 64), t(4, 2, 64))), "MOE_ERR_INVALID_ARGUMENT"),
]


@pytest.mark.parametrize("i", range(len(ROTARY)))
def test_rotary_refuses(i):
    refused(pkg.rotary, rotary_base, ROTARY[i][0](), ROTARY[i][1])


def test_rotary_refuses_outputs_over_other_values():
    rows = t(4, 6 * 64)
    q, k, v = (rows[:, 64 * i:64 * j].unflatten(1, (j - i, 64)) for i, j in ((0, 3), (3, 5), (1, 4)))
    refused(pkg.rotary, rotary_base, dict(q=q, k=k, out=(v, t(4, 2, 64))), "MOE_ERR_OVERLAP")
    refused(pkg.rotary, rotary_base, dict(q=q, k=k, out=(q, q[:, :2])), "MOE_ERR_OVERLAP")
    pkg.rotary(**{**rotary_base(), "q": q, "k": k, "out": (q, k)})
    torch.cuda.synchronize()


# --------------------------------------------------------------------------- sampling
def sample_base():
    return dict(logits=t(4, 100), uniform=t(4, dtype=F32), temperature=t(4, dtype=F32), top_k=whole(4, dtype=I32), top_p=t(4, dtype=F32),
                min_p=t(4, dtype=F32), out=whole(4, dtype=I32))


SAMPLE = [
    (lambda: dict(logits=t(4, 100, dtype=torch.float16)), "logits must be"), (lambda: dict(logits=wide(4, 100)), "logits must be"),
    (lambda: dict(logits=t(400)), r"logits must be \[B, V\]"), (lambda: dict(logits=t(4, 100).cpu()), "logits must be"),
    (lambda: dict(logits=t(1, 100).expand(4, 100)), "MOE_ERR_INVALID_ARGUMENT"), (lambda: dict(logits=t(4, (1 << 18) + 1)), "MOE_ERR_UNSUPPORTED_SHAPE"),
    (lambda: dict(uniform=t(3, dtype=F32)), "uniform must be"), (lambda: dict(uniform=t(4)), "uniform must be"), (lambda: dict(uniform=wide(4, dtype=F32)), "uniform must be"),
    (lambda: dict(uniform=None), "uniform must be a torch tensor"), (lambda: dict(temperature=t(1, dtype=F32)), "temperature must be"),
    (lambda: dict(temperature=0.7), "temperature must be a torch tensor"), (lambda: dict(top_k=whole(4, dtype=I64)), "top_k must be"),
    (lambda: dict(top_p=t(4, 1, dtype=F32)), "top_p must be"), (lambda: dict(min_p=whole(4, dtype=F64)), "min_p must be"),
    (lambda: dict(out=whole(4, dtype=I64)), "out must be"), (lambda: dict(out=whole(3, dtype=I32)), "out must be"),
]


@pytest.mark.parametrize("i", range(len(SAMPLE)))
def test_sample_refuses(i):
    refused(pkg.sample_tokens, sample_base, SAMPLE[i][0](), SAMPLE[i][1])


def test_sample_refuses_an_output_over_an_input():
    u = t(4, dtype=F32)
    refused(pkg.sample_tokens, sample_base, dict(uniform=u, out=u.view(I32)), "MOE_ERR_OVERLAP")
