"""The Python layer of the operators around the routed experts: what it checks and keeps on the host."""
import math
import random
import threading
import weakref

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import nvfp4_routed_moe_sort_gb300 as pkg  # noqa: F401  (the package must be importable without a GPU)
from linear_cuts import CUTS, SMS, kinds
from nvfp4_routed_moe_sort_gb300 import decoder
from nvfp4_routed_moe_sort_gb300._lib import linear_cut
from nvfp4_routed_moe_sort_gb300.build import build


@pytest.fixture(scope="module")
def native():
    build()
    return decoder._load()


def test_a_tensor_of_another_device_is_refused(native):
    native.refuse_device("w", 0, 0)
    native.refuse_device("w", 3, 3)
    for device, current in ((1, 0), (0, 1), (7, 2)):
        with pytest.raises(ValueError, match=f"w is on cuda:{device}, the call would run on cuda:{current}"):
            native.refuse_device("w", device, current)


# tensors that say they are on a GPU and have no memory: what is refused never touches them
host_only = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up devices")


def _elsewhere(make, names):
    """(name, arguments of which that one alone is on cuda:1) for each of `names`; `make(device_of)` makes them."""
    for name in names:
        with FakeTensorMode():
            yield name, make(lambda n, name=name: "cuda:1" if n == name else "cuda:0")


@host_only
def test_tensors_of_two_devices_are_refused(native):
    bf, f8, f32, u8 = torch.bfloat16, torch.float8_e4m3fn, torch.float32, torch.uint8

    def norm(on):
        t = lambda name, shape, dtype: torch.empty(shape, dtype=dtype, device=on(name))  # noqa: E731
        return dict(x=t("x", (4, 256), bf), weight=t("weight", (256,), bf), residual=t("residual", (4, 256), bf), fp8="group",
                    out=(t("the output", (4, 256), bf), t("the residual's output", (4, 256), bf),
                         t("the FP8 output", (4, 256), f8), t("the scales", (4, 2), f32)))
    for name, kw in _elsewhere(norm, ["weight", "residual", "the output", "the residual's output", "the FP8 output", "the scales"]):
        with pytest.raises(ValueError, match=f"{name} is on cuda:1"):
            pkg.add_rms_norm(**kw)

    def linear(on):
        t = lambda name, shape, dtype: torch.empty(shape, dtype=dtype, device=on(name))  # noqa: E731
        return dict(x=t("x", (4, 256), f8), w=t("w", (32, 128), u8), w_sf=t("w_sf", (32, 16), u8), alpha=t("alpha", (1,), f32),
                    x_scale=t("x_scale", (4, 2), f32), out=t("out", (4, 32), bf))
    for name, kw in _elsewhere(linear, ["w", "w_sf", "alpha", "x_scale", "out"]):
        with pytest.raises(ValueError, match=f"{name} is on cuda:1"):
            pkg.fp4_linear(**kw)

    def cache(on):
        t = lambda name, shape, dtype=u8: torch.empty(shape, dtype=dtype, device=on(name))  # noqa: E731
        return dict(k=t("k", (3, 2, 16, 32)), k_sf=t("k_sf", (3, 2, 16, 4)), v=t("v", (3, 2, 16, 32)), v_sf=t("v_sf", (3, 2, 16, 4)),
                    dev_status=t("dev_status", (4,), torch.int32))
    for name, kw in _elsewhere(cache, ["k_sf", "v", "v_sf", "dev_status"]):
        with pytest.raises(ValueError, match=f"{name} is on cuda:1"):
            pkg.NVFP4KVCache(**kw)


@pytest.mark.parametrize("name", ["k", "k_sf", "v", "v_sf", "k_scale", "v_scale", "dev_status"])
def test_a_cache_keeps_what_it_was_made_from(name):
    """The native object has the addresses and scales: exchanging the tensor here would leave it with freed memory."""
    cache = object.__new__(pkg.NVFP4KVCache)
    with pytest.raises(AttributeError):
        setattr(cache, name, torch.zeros(1))


def test_the_linears_cut_on_any_number_of_sms(native):
    """The rule holds on a part of a GPU too: every cut fits, and clusters that run at once are some."""
    sizes = [(1, 16, 1, False), (1, 512, 2048, False), (8, 7168, 4096, True), (13, 2000, 7001, False), (16, 4096, 16384, False),
             (4, 4096, 129021, False), (2, 40000, 33, False), (16, 32784, 20000, True), (40, 1040, 40006, True), (5, 208, 74, True)]
    for sms in range(1, 200):
        for M, K, N, gated in sizes:
            try:
                c = linear_cut(M, K, N, gated, sms)
            except pkg.MoEError:
                assert sms < 10 and K > 30000, (sms, M, K, N)   # so long an x needs a cluster of up to 8 SMs
                continue
            assert 1 <= c["at_once"] <= sms * 16 and c["slices"] in (1, 2, 4, 8) and 2 <= c["warps"] <= 16, (sms, M, K, N, c)
            assert c["warps"] % c["across"] == 0 and c["slices"] * c["slice"] * 128 >= K and c["groups"] * c["tokens"] >= M
            assert c["slices"] <= sms * (16 // c["warps"])     # a cluster finds room
            tiles = c["warps"] // c["across"]
            assert tiles % (2 if gated else 1) == 0 and (c["slices"] > 1 or tiles // (2 if gated else 1) <= 15)


class _Streams:
    """Stands in for the native module: the current stream's id, while its handle never changes."""
    id = 1

    def stream_id(self):
        return self.id


@pytest.fixture
def streams(monkeypatch):
    s = _Streams()
    monkeypatch.setattr(decoder, "_native", s)
    monkeypatch.setattr(decoder.L, "current_stream", lambda: 0x5000)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return s


CPU = torch.device("cpu")


def test_scratch_is_kept_for_one_stream(streams):
    assert decoder._workspace(0, CPU) is None
    a = decoder._workspace(100, CPU)
    assert a.numel() >= 100 and decoder._workspace(60, CPU) is a
    assert decoder._workspace(200, CPU).numel() >= 200
    a = decoder._workspace(200, CPU)
    streams.id = 2                                          # another stream that got the same handle
    assert decoder._workspace(200, CPU).data_ptr() != a.data_ptr()
    streams.id = 1
    assert decoder._workspace(200, CPU) is a


def test_scratch_does_not_grow_with_streams(streams):
    alive = []
    for streams.id in range(100, 200):
        alive.append(weakref.ref(decoder._workspace(64, CPU)))
    assert sum(r() is not None for r in alive) <= 8


def test_scratch_goes_with_its_thread(streams):
    def work(out):
        out.append(weakref.ref(decoder._workspace(64, CPU)))
        out.append(decoder._workspace(64, CPU).data_ptr())
    mine, others = decoder._workspace(64, CPU), []
    for _ in range(5):
        out = []
        t = threading.Thread(target=work, args=(out,))
        t.start()
        t.join()
        others.append(out)
    assert all(ref() is None and at != mine.data_ptr() for ref, at in others)


def test_the_listed_sizes_take_the_cuts_they_are_listed_for_and_every_kind(native):
    """What tests/test_gpu_linear_cuts.py runs: the table says what the rule chooses, and no kind that ordinary sizes
    take is missing from it."""
    listed = set()
    for gated, M, N, K, warps, across, slices, buffers, stages in CUTS:
        c = linear_cut(M, K, N, gated, SMS)
        assert (c["warps"], c["across"], c["slices"], c["buffers"], c["stages"]) == (warps, across, slices, buffers, stages), (M, N, K)
        listed.update(kinds(gated, M, N, K, c))
    r = random.Random(5)
    for _ in range(20000):
        gated, M, K = r.random() < 0.5, r.randint(1, 16), max(16, int(2 ** r.uniform(4, 14)) // 16 * 16)
        if r.random() < 0.4:
            K = max(256, K // 256 * 256)
        N = max(2, int(2 ** r.uniform(1, min(17.0, 30 - math.log2(K)))) // 2 * 2)
        missing = set(kinds(gated, M, N, K, linear_cut(M, K, N, gated, SMS))) - listed
        assert not missing, (gated, M, N, K, missing)
