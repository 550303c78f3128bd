"""What the torch layer of the operators around the routed experts refuses, on tensors that lie on the GPU: every
call is right with its base arguments, and each test changes one of them. All of these are refused on the
host, before anything is launched.
"""
import pytest
import torch

from gpu_harness import DEV, pkg

pytestmark = pytest.mark.gpu

BF, F8, F32, U8 = torch.bfloat16, torch.float8_e4m3fn, torch.float32, torch.uint8


def t(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=F32, device=DEV).to(dtype)


def wide(*shape, dtype=BF):
    """The same shape with every second value of the last dimension."""
    return t(*shape[:-1], 2 * shape[-1], dtype=dtype)[..., ::2]


def refused(call, base, change, match):
    """ValueError for a wrong tensor, MoEError for what the library itself refuses."""
    call(**base())
    torch.cuda.synchronize()
    error = pkg.MoEError if match.startswith("MOE_ERR") else ValueError
    with pytest.raises(error, match=match):
        call(**{**base(), **change})


# ---------------------------------------------------------------------------- norm
def norm_base():
    return dict(x=t(4, 256), weight=t(256), residual=t(4, 256), fp8="group",
                out=(t(4, 256), t(4, 256), t(4, 256, dtype=F8), t(4, 2, dtype=F32)))


def outs(i, new):
    o = list(norm_base()["out"])
    o[i] = new
    return dict(out=tuple(o))


NORM = [
    (lambda: dict(x=t(4, 256, dtype=F32)), "x must be bf16 rows"), (lambda: dict(x=t(256, 4).T), "x must be bf16 rows"),
    (lambda: dict(x=t(1024)), r"x must be \[M, H\]"), (lambda: dict(x=t(4, 256).cpu()), "x must be bf16 rows"),
    (lambda: dict(x=t(1, 256).expand(4, 256)), "MOE_ERR_INVALID_ARGUMENT"), (lambda: dict(x=t(4, 264)[:, 1:257]), "MOE_ERR_MISALIGNED"),
    (lambda: dict(weight=t(128)), "weight must be"), (lambda: dict(weight=wide(256)), "weight must be"),
    (lambda: dict(weight=t(256, dtype=F32)), "weight must be"), (lambda: dict(weight=t(256).cpu()), "weight must be"),
    (lambda: dict(residual=t(4, 128)), "residual must be"), (lambda: dict(residual=t(3, 256)), "residual must be"),
    (lambda: dict(residual=t(4, 256, dtype=F32)), "residual must be"), (lambda: dict(residual=None), "MOE_ERR_INVALID_ARGUMENT"),
    (lambda: outs(0, t(4, 256, dtype=F32)), "the output must be"), (lambda: outs(0, wide(4, 256)), "the output must be"),
    (lambda: outs(0, t(3, 256)), "the output must be"), (lambda: outs(1, t(4, 128)), "the residual's output must be"),
    (lambda: outs(2, t(4, 256)), "the FP8 output must be"), (lambda: outs(3, t(4, 1, dtype=F32)), "the scales must be"),
    (lambda: outs(3, t(4, 2)), "the scales must be"), (lambda: outs(2, None), "must be given with fp8"),
    (lambda: outs(3, None), "must be given with fp8"), (lambda: dict(fp8=None), "the scales must be"),
    (lambda: dict(fp8="token"), "the scales must be"), (lambda: dict(fp8="row"), "fp8 must be"),
    (lambda: dict(eps=float("nan")), "MOE_ERR_INVALID_ARGUMENT"), (lambda: dict(x=[1.0]), "x must be a torch tensor"),
]


@pytest.mark.parametrize("i", range(len(NORM)))
def test_norm_refuses(i):
    refused(pkg.add_rms_norm, norm_base, NORM[i][0](), NORM[i][1])


def test_norm_refuses_an_output_over_an_input():
    x = t(4, 256)
    refused(pkg.add_rms_norm, norm_base, {"x": x, **outs(0, x)}, "MOE_ERR_OVERLAP")


# -------------------------------------------------------------------------- linear
def linear_base():
    return dict(x=t(4, 256), w=t(32, 128, dtype=U8), w_sf=t(32, 16, dtype=U8), alpha=t(1, dtype=F32), out=t(4, 32))


def linear8_base():
    return dict(linear_base(), x=t(4, 256, dtype=F8), x_scale=t(4, 2, dtype=F32))


LINEAR = [
    (lambda: dict(x=t(4, 256, dtype=torch.float16)), "x without x_scale must be"), (lambda: dict(x=t(256, 4).T), "x without x_scale must be"),
    (lambda: dict(x=t(4, 256, dtype=F8)), "x without x_scale must be"), (lambda: dict(x=t(1024)), "x and w must be"),
    (lambda: dict(x=t(4, 128)), "w must be"), (lambda: dict(x=t(4, 256).cpu()), "x without x_scale must be"),
    (lambda: dict(x_scale=t(4, 2, dtype=F32)), "x with x_scale must be"),
    (lambda: dict(w=t(32, 128, dtype=torch.int8)), "w must be"), (lambda: dict(w=wide(32, 128, dtype=U8)), "w must be"),
    (lambda: dict(w=t(32, 128, dtype=U8).cpu()), "w must be"), (lambda: dict(w=t(33, 128, dtype=U8)), "w_sf must be"),
    (lambda: dict(w_sf=t(32, 8, dtype=U8)), "w_sf must be"), (lambda: dict(w_sf=t(32, 16, dtype=F8)), "w_sf must be"),
    (lambda: dict(w_sf=wide(32, 16, dtype=U8)), "w_sf must be"),
    (lambda: dict(alpha=t(1, dtype=torch.float64)), "alpha must be"), (lambda: dict(alpha=t(2, dtype=F32)), "alpha must be"),
    (lambda: dict(alpha=t(1, dtype=F32).cpu()), "alpha must be"),
    (lambda: dict(out=t(4, 31)), "out must be"), (lambda: dict(out=t(4, 32, dtype=F32)), "out must be"),
    (lambda: dict(out=wide(4, 32)), "out must be"), (lambda: dict(activation="swiglu"), "out must be"),
    (lambda: dict(activation="tanh"), "activation must be"),
    (lambda: dict(w=t(31, 128, dtype=U8), w_sf=t(31, 16, dtype=U8), activation="geglu"), "of an even number of rows"),
    (lambda: dict(x=t(4, 24), w=t(32, 12, dtype=U8), w_sf=t(32, 1, dtype=U8)), "MOE_ERR_UNSUPPORTED_SHAPE"),
    (lambda: dict(x=t(4, 260)[:, :256]), "MOE_ERR_MISALIGNED"),
]
LINEAR8 = [
    (lambda: dict(x_scale=t(4, 3, dtype=F32)), "x_scale must be"), (lambda: dict(x_scale=t(3, 2, dtype=F32)), "x_scale must be"),
    (lambda: dict(x_scale=t(4, 2, dtype=torch.float64)), "x_scale must be"), (lambda: dict(x_scale=wide(4, 2, dtype=F32)), "x_scale must be"),
    (lambda: dict(x_scale=t(4, 2, dtype=F32).cpu()), "x_scale must be"), (lambda: dict(x=t(4, 256)), "x with x_scale must be"),
    (lambda: dict(x=t(4, 264, dtype=F8)[:, :256]), "MOE_ERR_MISALIGNED"),
]


@pytest.mark.parametrize("i", range(len(LINEAR)))
def test_linear_refuses(i):
    refused(pkg.fp4_linear, linear_base, LINEAR[i][0](), LINEAR[i][1])


@pytest.mark.parametrize("i", range(len(LINEAR8)))
def test_linear_of_e4m3_refuses(i):
    refused(pkg.fp4_linear, linear8_base, LINEAR8[i][0](), LINEAR8[i][1])


# --------------------------------------------------------------------------- cache
def cache_base():
    return dict(k=t(6, 2, 16, 32, dtype=U8), k_sf=t(6, 2, 16, 4, dtype=U8), v=t(6, 2, 16, 32, dtype=U8), v_sf=t(6, 2, 16, 4, dtype=U8),
                dev_status=t(4, dtype=torch.int32))


CACHE = [
    (lambda: dict(k=t(6, 2, 512, dtype=U8)), "k must be"), (lambda: dict(k=t(6, 2, 16, 32, dtype=torch.int8)), "k, v and k_sf, v_sf must be"),
    (lambda: dict(v=t(5, 2, 16, 32, dtype=U8)), "k, v and k_sf, v_sf must be"), (lambda: dict(k_sf=t(6, 2, 16, 2, dtype=U8)), "k, v and k_sf, v_sf must be"),
    (lambda: dict(v_sf=t(6, 2, 16, 4, dtype=U8).cpu()), "k, v and k_sf, v_sf must be"),
    (lambda: dict(v=t(12, 2, 16, 32, dtype=U8)[::2]), "k, v and k_sf, v_sf must be"),
    (lambda: dict(k=wide(6, 2, 16, 32, dtype=U8)), "k, v and k_sf, v_sf must be"),
    (lambda: dict(k=t(6, 16, 2, 32, dtype=U8).transpose(1, 2)), "k, v and k_sf, v_sf must be"),
    (lambda: dict(dev_status=t(4, dtype=F32)), "dev_status must be"), (lambda: dict(dev_status=t(4, dtype=torch.int32).cpu()), "dev_status must be"),
]


@pytest.mark.parametrize("i", range(len(CACHE)))
def test_cache_refuses(i):
    refused(pkg.NVFP4KVCache, cache_base, CACHE[i][0](), CACHE[i][1])


@pytest.mark.parametrize("kw", [dict(k_scale=0.0), dict(v_scale=float("inf")), dict(k_scale=-1.0)])
def test_cache_of_bad_scales_is_refused_by_its_calls(kw):
    kv = pkg.NVFP4KVCache(**cache_base(), **kw)
    with pytest.raises(pkg.MoEError, match="MOE_ERR_INVALID_ARGUMENT"):
        kv.append(t(3, 2, 64), t(3, 2, 64), t(3, dtype=torch.int64))


def append_base():
    return dict(k_new=t(3, 2, 64), v_new=t(3, 2, 64), slots=t(3, dtype=torch.int64) + torch.arange(3, device=DEV),
                seen=(t(3, 2, 64), t(3, 2, 64)))


APPEND = [
    (lambda: dict(k_new=t(3, 2, 32)), "k_new must be"), (lambda: dict(k_new=t(3, 1, 64)), "k_new must be"),
    (lambda: dict(k_new=t(3, 128)), "k_new must be"), (lambda: dict(k_new=t(3, 2, 64, dtype=F32)), "k_new must be"),
    (lambda: dict(k_new=t(2, 3, 64).transpose(0, 1)), "k_new must be"), (lambda: dict(k_new=wide(3, 2, 64)), "k_new must be"),
    (lambda: dict(v_new=t(2, 2, 64)), "v_new must be"), (lambda: dict(v_new=t(3, 2, 64).cpu()), "v_new must be"),
    (lambda: dict(k_new=t(3, 132)[:, :128].unflatten(1, (2, 64))), "MOE_ERR_MISALIGNED"),
    (lambda: dict(slots=t(3, dtype=torch.int32)), "slots must be"), (lambda: dict(slots=t(4, dtype=torch.int64)), "slots must be"),
    (lambda: dict(slots=wide(3, dtype=torch.int64)), "slots must be"), (lambda: dict(slots=t(3, dtype=torch.int64).cpu()), "slots must be"),
    (lambda: dict(seen=(t(3, 2, 64, dtype=F32), t(3, 2, 64))), r"seen\[0\] must be"), (lambda: dict(seen=(t(3, 2, 64), t(2, 2, 64))), r"seen\[1\] must be"),
    (lambda: dict(seen=(t(3, 2, 64), None)), "MOE_ERR_INVALID_ARGUMENT"), (lambda: dict(seen=(wide(3, 2, 64), t(3, 2, 64))), r"seen\[0\] must be"),
]


@pytest.mark.parametrize("i", range(len(APPEND)))
def test_append_refuses(i):
    kv = pkg.NVFP4KVCache(**cache_base())
    refused(kv.append, append_base, APPEND[i][0](), APPEND[i][1])


def attend_base():
    return dict(q=t(2, 3, 4, 64), page_table=t(2, 3, dtype=torch.int32), seq_lens=t(2, dtype=torch.int32) + 20,
                out=t(2, 3, 4, 64), lse=t(2, 3, 4, dtype=F32))


ATTEND = [
    (lambda: dict(q=t(2, 12, 64)), "q must be"), (lambda: dict(q=t(2, 3, 4, 64, dtype=torch.float16)), "q must be"),
    (lambda: dict(q=t(2, 3, 4, 128)), "q must be"), (lambda: dict(q=t(2, 3, 4, 64).cpu()), "q must be"),
    (lambda: dict(q=t(2, 4, 3, 64).transpose(1, 2)), "q must be of contiguous rows"), (lambda: dict(q=t(2, 5, 4, 64)[:, :3]), "q must be of contiguous rows"),
    (lambda: dict(q=wide(2, 3, 4, 64)), "q must be of contiguous rows"), (lambda: dict(q=t(2, 3, 3, 64), out=t(2, 3, 3, 64), lse=t(2, 3, 3, dtype=F32)), "MOE_ERR_INVALID_ARGUMENT"),
    (lambda: dict(page_table=t(2, 3, dtype=torch.int64)), "page_table must be"), (lambda: dict(page_table=t(3, 3, dtype=torch.int32)), "page_table must be"),
    (lambda: dict(page_table=wide(2, 3, dtype=torch.int32)), "page_table must be"), (lambda: dict(page_table=t(6, dtype=torch.int32)), "page_table must be"),
    (lambda: dict(page_table=t(1, 3, dtype=torch.int32).expand(2, 3)), "MOE_ERR_INVALID_ARGUMENT"),
    (lambda: dict(page_table=t(2, 3, dtype=torch.int32).cpu()), "page_table must be"),
    (lambda: dict(seq_lens=t(2, dtype=torch.int64)), "seq_lens must be"), (lambda: dict(seq_lens=t(3, dtype=torch.int32)), "seq_lens must be"),
    (lambda: dict(seq_lens=wide(2, dtype=torch.int32)), "seq_lens must be"), (lambda: dict(seq_lens=t(2, dtype=torch.int32).cpu()), "seq_lens must be"),
    (lambda: dict(out=t(2, 3, 4, 32)), "out must be"), (lambda: dict(out=t(2, 3, 4, 64, dtype=F32)), "out must be"),
    (lambda: dict(out=wide(2, 3, 4, 64)), "out must be"), (lambda: dict(lse=t(2, 4, 3, dtype=F32)), "lse must be"),
    (lambda: dict(lse=t(2, 3, 4)), "lse must be"), (lambda: dict(workspace=torch.zeros(64, dtype=U8)), "workspace must be"),
    (lambda: dict(softmax_scale=float("nan")), "MOE_ERR_INVALID_ARGUMENT"), (lambda: dict(softmax_scale=float("inf")), "MOE_ERR_INVALID_ARGUMENT"),
]


@pytest.mark.parametrize("i", range(len(ATTEND)))
def test_attend_refuses(i):
    kv = pkg.NVFP4KVCache(**cache_base())
    refused(kv.attend, attend_base, ATTEND[i][0](), ATTEND[i][1])


def test_attend_refuses_too_small_a_workspace_and_an_output_in_the_cache():
    kv = pkg.NVFP4KVCache(**cache_base())

    def base():
        return dict(attend_base(), page_table=t(2, 4000, dtype=torch.int32))
    need = pkg.moe_kv_attend_workspace_bytes(kv.c, 2, 3, 4, 4000)
    assert need > 0
    refused(kv.attend, base, dict(workspace=t(need - 1, dtype=U8)), "MOE_ERR_WORKSPACE_TOO_SMALL")
    refused(kv.attend, attend_base, dict(out=kv.k.view(-1)[:2 * 3 * 4 * 64 * 2].view(BF).view(2, 3, 4, 64)), "MOE_ERR_OVERLAP")
