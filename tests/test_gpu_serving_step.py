"""The operators of a model's step as they are used together: a prompt through E4M3 projections and rotary positions into
the cache, then steps of single tokens up to the sampled one; eagerly, on another stream, two at once, and captured."""
import numpy as np
import pytest
import torch

from gpu_harness import DEV, bf16_np, pkg, to_np
from oracle import serving as S
from test_gpu_decoder import assert_within, f32_np
from test_gpu_serving import check_linear, check_quantize, check_rotary, linear_case, rotary_case, same, up

pytestmark = pytest.mark.gpu


class Model:
    """One attention layer and a head over it; three position axes, the first half of each head turned."""

    H, heads, kv_heads, D, V, page = 512, 4, 2, 64, 5003, 16

    def __init__(self, seed=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        n = lambda *s: torch.randn(*s, device=DEV, generator=g)  # noqa: E731
        rows = self.heads + 2 * self.kv_heads
        self.norm = (1 + 0.1 * n(self.H)).bfloat16()
        self.qkv = pkg.FP8Linear.from_bf16((n(rows * self.D, self.H) / self.H ** 0.5).bfloat16())
        self.out = pkg.FP8Linear.from_bf16((n(self.H, self.heads * self.D) / 16).bfloat16())
        self.head = pkg.FP8Linear.from_bf16((n(self.V, self.H) / 8).bfloat16())
        self.freq = torch.exp2(-torch.arange(16, device=DEV, dtype=torch.float64) / 2)
        self.axes = (torch.arange(16, device=DEV) % 3).to(torch.uint8)
        self.cache = pkg.NVFP4KVCache.allocate(64, self.page, self.kv_heads, self.D)

    def keys(self, x, pos, slots):
        """Queries of tokens x [N, H], their keys and values stored: in place in the projection's output."""
        _, _, x8, scale = pkg.add_rms_norm(x, self.norm, fp8="group")
        qkv = self.qkv(x8, scale).view(x.shape[0], -1, self.D)
        q, k, v = qkv.split((self.heads, self.kv_heads, self.kv_heads), 1)
        pkg.rotary(q, pos, self.freq, k=k, axes=self.axes, out=(q, k))
        self.cache.append(k, v, slots)
        return q

    def step(self, x, pos, slots, table, lens, u, settings):
        q = self.keys(x, pos, slots)
        o, _ = self.cache.attend(q.unsqueeze(1), table, lens)
        h = x + self.out(*pkg.quantize_fp8(o.view(x.shape[0], -1)))
        _, _, x8, scale = pkg.add_rms_norm(h, self.norm, fp8="group")
        logits = self.head(x8, scale)
        return logits, pkg.sample_tokens(logits, u, **settings)


def inputs(m, B, n, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    pages = -(-(n + 4) // m.page)
    table = torch.randperm(64, device=DEV, generator=g)[:B * pages].view(B, pages).int()
    place = torch.arange(n, device=DEV)
    slots = (table[:, place // m.page].long() * m.page + place % m.page)
    x = torch.randn(B, n, m.H, device=DEV, generator=g).bfloat16()
    pos = torch.stack((place + 1000, place % 7, place // 7))[:, None].expand(3, B, n).reshape(3, -1).contiguous()
    settings = dict(temperature=torch.full((B,), 0.8, device=DEV), top_k=torch.full((B,), 40, dtype=torch.int32, device=DEV),
                    top_p=torch.full((B,), 0.95, device=DEV), min_p=torch.full((B,), 0.01, device=DEV))
    return dict(x=x, pos=pos, slots=slots, table=table, u=torch.rand(B, device=DEV, generator=g), settings=settings)


def single(c, B, n):
    """The step of the sequences' n-th token."""
    return (c["x"][:, n - 1].contiguous(), c["pos"].view(3, B, -1)[:, :, n - 1].contiguous(), c["slots"][:, n - 1].contiguous(), c["table"],
            torch.full((B,), n, dtype=torch.int32, device=DEV), c["u"], c["settings"])


def test_a_prompt_and_a_step_against_float64():
    m, B, n = Model(), 3, 37
    c = inputs(m, B, n, 1)
    # the prompt's parts, each against its definition on what it was given
    flat = c["x"].view(-1, m.H)
    _, _, x8, scale = pkg.add_rms_norm(flat, m.norm, fp8="group")
    qkv = m.qkv(x8, scale)
    check_linear(qkv, x8, scale, m.qkv.w, m.qkv.w_scale)
    q, k, _ = qkv.view(B * n, -1, m.D).split((m.heads, m.kv_heads, m.kv_heads), 1)
    q2, k2 = pkg.rotary(q, c["pos"], m.freq, k=k, axes=m.axes)
    for got, x in ((q2, q), (k2, k)):
        check_rotary(got, x, to_np(c["pos"]), to_np(m.freq), to_np(m.axes), False)
    assert same(m.keys(flat, c["pos"], c["slots"].view(-1)), q2)  # in place: the same
    # the last token again as a step: its keys are stored where they were
    args = single(c, B, n)
    logits, tokens = m.step(*args)
    o, _ = m.cache.attend(q2.view(B, n, m.heads, m.D)[:, -1:].contiguous(), c["table"], args[4])
    o8, o_scale = pkg.quantize_fp8(o.view(B, -1))
    check_quantize((o8, o_scale), o.view(B, -1), 1)
    proj = m.out(o8, o_scale)
    check_linear(proj, o8, o_scale, m.out.w, m.out.w_scale)
    _, _, x8, scale = pkg.add_rms_norm(args[0] + proj, m.norm, fp8="group")
    check_linear(logits, x8, scale, m.head.w, m.head.w_scale)
    host, s = f32_np(logits), {k: to_np(v) for k, v in c["settings"].items()}
    assert tokens.tolist() == [S.sample(host[b], float(c["u"][b]), **{k: v[b] for k, v in s.items()}) for b in range(B)]
    # attention over the turned, cached keys: against float64 of what the cache holds
    want = np.zeros((B, m.heads, m.D))
    rows = to_np(q2.view(B, n, m.heads, m.D)[:, -1].float()).astype(np.float64)
    seen = [torch.empty(B * n, m.kv_heads, m.D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    v = qkv.view(B * n, -1, m.D)[:, m.heads + m.kv_heads:]
    m.cache.append(k2, v, c["slots"].view(-1), seen=tuple(seen))
    ks, vs = (bf16_np(t).reshape(B, n, m.kv_heads, m.D) for t in seen)
    mass = np.zeros(want.shape)
    for b in range(B):
        for h in range(m.heads):
            z = ks[b, :, h // 2] @ rows[b, h] / 8
            p = np.exp(z - z.max())
            want[b, h], mass[b, h] = p @ vs[b, :, h // 2] / p.sum(), p @ np.abs(vs[b, :, h // 2]) / p.sum()
    # weights to 11 bits, values exact in BF16 (6 bits), one rounding to BF16
    assert_within(bf16_np(o)[:, 0], want, mass * 2.0 ** -9 + np.abs(want) * 2.0 ** -8)


def test_a_captured_step_follows_its_inputs():
    m, B, n = Model(), 4, 30
    c, d = inputs(m, B, n, 2), inputs(m, B, n, 3)
    m.keys(c["x"].view(-1, m.H), c["pos"], c["slots"].view(-1))
    args = [t.clone() if torch.is_tensor(t) else {k: v.clone() for k, v in t.items()} for t in single(c, B, n)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # on another stream than the tensors were made on
        eager = [t.clone() for t in m.step(*args)]
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        result = m.step(*args)
    for _ in range(3):
        graph.replay()
        assert all(same(a, b) for a, b in zip(result, eager))
    # other tokens, positions and settings in the same tensors
    e = single(d, B, n)
    args[0].copy_(e[0]), args[1].copy_(e[1]), args[5].copy_(e[5])
    args[6]["top_k"].copy_(torch.tensor([0, 1, 3, 5000], dtype=torch.int32))
    args[6]["top_p"].copy_(torch.tensor([1.0, 0.5, 0.9, 0.0]))
    args[6]["temperature"].copy_(torch.tensor([0.0, 1.0, 2.0, 0.5]))
    graph.replay()
    logits, tokens = (t.clone() for t in result)
    again = m.step(*args)
    assert same(logits, again[0]) and same(tokens, again[1])
    host, s = f32_np(logits), {k: to_np(v) for k, v in args[6].items()}
    assert tokens.tolist() == [S.sample(host[b], float(args[5][b]), **{k: v[b] for k, v in s.items()}) for b in range(B)]


def test_two_at_once_on_two_streams():
    """Calls that overlap on the GPU share nothing."""
    cases = [linear_case(40, 2048, 2048), linear_case(1500, 2048, 1024, seed=1)]
    q, k, pos, freq, which = rotary_case(2000, 16, 4, 128, 128, 3)
    x = torch.randn(32, 60000, device=DEV).bfloat16()
    u, top_p = torch.rand(32, device=DEV), torch.full((32,), 0.9, device=DEV)

    def work(i):
        return (pkg.fp8_linear(*cases[i]), *pkg.rotary(q, up(pos), up(freq), k=k, axes=up(which)), pkg.sample_tokens(x, u, top_p=top_p),
                *pkg.quantize_fp8(x[:, :4096]))
    ref = [work(i) for i in (0, 1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(work(i))
    torch.cuda.synchronize()
    for i in (0, 1):
        for g in got[i]:
            assert all(same(a, b) for a, b in zip(g, ref[i]))
