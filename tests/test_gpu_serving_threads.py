"""Host threads: a thread's first call of CUDA may be any of this library's, before or after other threads' calls have looked up
what is looked up once."""
import os
import subprocess
import sys
import threading

import pytest
import torch

from gpu_harness import DEV, Problem, mi, pkg
from test_gpu_serving import linear_case, rotary_case, same, up

pytestmark = pytest.mark.gpu


def in_a_new_thread(f):
    """f() as all that a new host thread does; what it raised is raised here."""
    result = []

    def work():
        try:
            result.append((f(), None))
        except BaseException as e:
            result.append((None, e))
    t = threading.Thread(target=work)
    t.start()
    t.join()
    if result[0][1] is not None:
        raise result[0][1]
    return result[0][0]


@pytest.mark.parametrize("M,N,K", [(5, 300, 1024), (130, 140, 512), (5000, 2048, 512)])  # slices, whole tiles, pairs
@pytest.mark.parametrize("way", ["c", "torch", "torch out"])
def test_linear_as_a_threads_first_call(M, N, K, way):
    x, xs, w, ws = linear_case(M, N, K)
    ref = pkg.fp8_linear(x, xs, w, ws)
    out = torch.zeros_like(ref)
    torch.cuda.synchronize()

    def call():
        if way == "c":
            pkg.moe_linear_fp8(x, xs, pkg.MOE_FP8_PER_GROUP, w, ws, pkg.MOE_ACT_IDENTITY, out, stream=0)
            return out
        return pkg.fp8_linear(x, xs, w, ws, out=out if way == "torch out" else None)
    got = in_a_new_thread(call)
    torch.cuda.synchronize()
    assert same(got, ref)


def test_the_other_operators_as_a_threads_first_call():
    x = torch.randn(40, 1024, device=DEV).bfloat16()
    q, k, pos, freq, _ = rotary_case(9, 4, 2, 64, 64, 1)
    pos, freq = up(pos), up(freq)
    logits, u = torch.randn(4, 20000, device=DEV), torch.rand(4, device=DEV)
    one = torch.randn(1, 129021, device=DEV)
    for call in (lambda: pkg.quantize_fp8(x), lambda: pkg.rotary(q, pos, freq, k=k), lambda: (pkg.sample_tokens(logits, u),),
                 lambda: (pkg.sample_tokens(one, u[:1], top_p=u[1:2]),), lambda: (pkg.add_rms_norm(x, x[0])[0],)):
        ref = call()
        torch.cuda.synchronize()
        got = in_a_new_thread(call)
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(got, ref))


@pytest.mark.parametrize("name", ["tiny", "large"])
def test_the_experts_as_a_threads_first_call(name, monkeypatch):
    cfg = mi.CONFIGS["tiny"] if name == "tiny" else mi.MoEConfig("threads", M=300, H=256, I=256, E=8, top_k=2, seed=3, weight_seed=3)
    p = Problem(cfg)
    ref = p.run_routed().clone()
    steps = p.run().clone()
    got = in_a_new_thread(p.run_routed)
    assert same(got, ref)
    # the products alone, as a thread's only call
    products = pkg._lib.moe_grouped_fp4_forward
    monkeypatch.setattr(pkg._lib, "moe_grouped_fp4_forward", lambda *a, **kw: in_a_new_thread(lambda: products(*a, **kw)))
    assert same(p.run(), steps)


CHILD = """
import sys, threading
sys.path[:0] = [{root!r}, {tests!r}]
import torch
import nvfp4_routed_moe_sort_gb300 as pkg
dev, F8 = "cuda", torch.float8_e4m3fn
g = torch.Generator(device=dev).manual_seed(1)
n = lambda *s: torch.randn(*s, device=dev, generator=g)
cases = []
for M, N, K in ((5, 300, 1024), (130, 140, 512), (5000, 2048, 512), (40, 4096, 256)) * 2:  # slices, whole tiles, pairs
    xs, ws = torch.rand(M, -(-K // 128), device=dev, generator=g), torch.rand(-(-N // 128), -(-K // 128), device=dev, generator=g)
    cases.append((n(M, K).to(F8), xs, n(N, K).to(F8), ws, torch.zeros(M, N, dtype=torch.bfloat16, device=dev)))
logits, uniform = n(2, 129021).bfloat16(), torch.rand(2, device=dev, generator=g)
top_p = torch.full((2,), 0.9, device=dev)
tokens = [torch.zeros(2, dtype=torch.int32, device=dev) for _ in cases]
streams = [torch.cuda.Stream() for _ in cases]
torch.cuda.synchronize()
pkg.lib()
go, bad = threading.Barrier(len(cases)), []

def work(i):
    try:
        x, xs, w, ws, out = cases[i]
        go.wait()
        # the C entry points, which run without the interpreter's lock
        pkg.moe_linear_fp8(x, xs, pkg.MOE_FP8_PER_GROUP, w, ws, pkg.MOE_ACT_IDENTITY, out, stream=streams[i].cuda_stream)
        pkg.moe_sample(logits, uniform, None, None, top_p, None, tokens[i], stream=streams[i].cuda_stream)
    except BaseException as e:
        bad.append(repr(e))

threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
assert not bad, bad
for x, xs, w, ws, out in cases:
    again = pkg.fp8_linear(x, xs, w, ws)
    assert again.abs().sum() > 0 and torch.equal(out, again)
again = pkg.sample_tokens(logits, uniform, top_p=top_p)
assert all(torch.equal(t, again) for t in tokens)
print("equal")
"""


def test_first_calls_of_several_threads_at_once():
    tests = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", CHILD.format(root=os.path.dirname(tests), tests=tests)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.split() == ["equal"], r.stdout[-2000:] + r.stderr[-2000:]
