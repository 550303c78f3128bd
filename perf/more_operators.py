"""Cases and plain forms of the dense FP8 path, the rotary positions and the sampling of a model's step.

* ``quantize``: BF16 rows to E4M3 with one FP32 scale per 128 columns of a row (activations) or per
  128 x 128 block (weights).
* ``linear``: activations in E4M3 times a matrix in E4M3 with one FP32 scale per 128 x 128 block, any
  number of tokens, an optional SwiGLU over the [gate; up] rows.
* ``rotary``: queries and keys turned by their tokens' positions, one or several axes, in place in a
  projection's output.
* ``sample``: one token per row of logits: temperature, top-k, top-p and min-p, drawn by a given
  random number.

``run`` computes them in elementary torch operations in 32 bits (in 64 where angles and cumulated
weights need them), or, with ``own`` set, through the framework's entry points.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # eight tokens before a small layer's output projection: a decode step's latency
        dict(name="quantize_decode", op="quantize", M=8, K=2048, rows=1),
        # a prompt's hidden states before a 7168-wide layer's projections, the last scale group short
        dict(name="quantize_prompt", op="quantize", M=16384, K=7160, rows=1),
        # four tokens through the down projection of a small shared expert (2048 <- 512)
        dict(name="linear_small", op="linear", M=4, N=2048, K=512, act="identity", x="group"),
        # a decode batch through the gate and up rows of a shared expert of a 7168-wide layer
        dict(name="linear_decode_swiglu", op="linear", M=48, N=4096, K=7168, act="swiglu", x="group"),
        # a ragged chunk: rows, columns and K that no tile divides, one scale per token
        dict(name="linear_ragged", op="linear", M=333, N=7001, K=2000, act="identity", x="token"),
        # a long prompt through the square projection of a 7168-wide layer
        dict(name="linear_prompt", op="linear", M=8192, N=7168, K=7168, act="identity", x="group"),
        # one new token of eight sequences of a small layer, its own positions on one axis
        dict(name="rotary_decode", op="rotary", N=8, Hq=16, Hk=4, D=128, rot=128, axes=1, adjacent=False),
        # a prompt with images: time, height and width, an odd number of tokens, part of each head turned
        dict(name="rotary_images", op="rotary", N=4099, Hq=28, Hk=4, D=128, rot=96, axes=3, adjacent=False),
        # a long prompt of a layer with many heads, neighbouring values paired
        dict(name="rotary_prompt", op="rotary", N=16384, Hq=64, Hk=8, D=128, rot=128, axes=1, adjacent=True),
        # one conversation's next token out of a large vocabulary of odd size, by its nucleus alone
        dict(name="sample_one", op="sample", B=1, V=129021, dtype="bf16", kind="nucleus"),
        # seven rows of a small vocabulary in 32 bits
        dict(name="sample_small", op="sample", B=7, V=1001, dtype="f32", kind="mixed"),
        # a full serving batch, every user with settings of their own
        dict(name="sample_batch", op="sample", B=128, V=129021, dtype="bf16", kind="mixed"),
    ]


def _spread(rng, lo, hi):
    """A whole number spread evenly over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "rotary", "sample"])
    if op == "quantize":
        K = _spread(rng, 64, 8192)
        return dict(op=op, M=min(_spread(rng, 1, 16384), 16384 * 7160 // K), K=K, rows=rng.choice([1, 1, 128]))
    if op == "linear":
        K = max(64, _spread(rng, 64, 8192) // 16 * 16)
        act = rng.choice(["identity", "identity", "swiglu"])
        N = _spread(rng, 64, 16384)
        if act == "swiglu":
            N = max(1, N // 256) * 256
        M = min(_spread(rng, 1, 16384), 8192 * 7168 * 7168 // (N * K))
        return dict(op=op, M=max(1, M), N=N, K=K, act=act, x=rng.choice(["group", "group", "token"]))
    if op == "rotary":
        D = rng.choice([64, 80, 96, 128, 128, 192, 256])
        Hk = rng.choice([1, 2, 3, 4, 8])
        Hq = Hk * rng.choice([1, 2, 4, 5, 7, 8])
        rot = rng.choice([D, D, D // 2, D // 4 * 2 - 2])
        most = 16384 * 72 * 128 // ((Hq + Hk) * D)
        return dict(op=op, N=min(_spread(rng, 1, 65536), most), Hq=Hq, Hk=Hk, D=D, rot=rot, axes=rng.choice([1, 1, 2, 3, 4]),
                    adjacent=rng.random() < 0.4)
    V = _spread(rng, 17, 262144)
    return dict(op=op, B=min(_spread(rng, 1, 256), max(1, 128 * 129021 // V)), V=V, dtype=rng.choice(["bf16", "bf16", "f32"]),
                kind=rng.choice(["mixed", "mixed", "nucleus", "all"]))


def work(case):
    c = case
    if c["op"] == "quantize":
        n = c["M"] * c["K"]
        return {"bytes": 3 * n + 4 * -(-c["M"] // c["rows"]) * -(-c["K"] // 128), "flops": 3 * n}
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        g = -(-K // 128)
        out = N // 2 if c["act"] == "swiglu" else N
        return {"bytes": N * K + M * K + 4 * (-(-N // 128) * g + M * (1 if c["x"] == "token" else g)) + 2 * M * out,
                "flops": 2 * M * N * K}
    if c["op"] == "rotary":
        n = c["N"] * (c["Hq"] + c["Hk"]) * c["rot"]
        return {"bytes": 4 * n + 8 * c["axes"] * c["N"] + 9 * (c["rot"] // 2), "flops": 3 * n}
    n = c["B"] * c["V"]
    return {"bytes": n * (2 if c["dtype"] == "bf16" else 4) + 24 * c["B"], "flops": 4 * n}


# ------------------------------------------------------------------------- inputs
def _e4m3(x, rows):
    """FP32 [M, K] -> E4M3 [M, K] and FP32 scales amax / 448 (1 where amax is 0) per `rows` x 128 values."""
    M, K = x.shape
    m, n = -(-M // rows), -(-K // 128)
    b = torch.nn.functional.pad(x, (0, n * 128 - K, 0, m * rows - M)).view(m, rows, n, 128)
    amax = b.abs().amax((1, 3))
    one = torch.ones_like(amax)
    scale = torch.where(amax == 0, one, amax / 448.0)
    inv = torch.where(amax == 0, one, 448.0 / amax)
    y = (b * inv[:, None, :, None]).view(m * rows, n * 128)[:M, :K]
    return y.contiguous().to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV).manual_seed(1009 * int(seed) + 29)

    def normal(*shape):
        return torch.randn(*shape, device=DEV, generator=gen)

    def uniform(*shape):
        return torch.rand(*shape, device=DEV, generator=gen)

    if c["op"] == "quantize":
        M, K = c["M"], c["K"]
        # some channels are far larger than the others, as a model's are
        c["x_t"] = (normal(M, K) * (1.0 + 20.0 * (normal(1, K) > 2.5))).bfloat16()
        c["out"] = (torch.empty(M, K, dtype=torch.float8_e4m3fn, device=DEV),
                    torch.empty(-(-M // c["rows"]), -(-K // 128), dtype=torch.float32, device=DEV))
    elif c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        x = normal(M, K) * (0.5 + normal(M, 1).abs()) * (1.0 + 4.0 * (normal(1, K) > 2.5))
        if c["x"] == "token":
            scale = x.abs().amax(1, keepdim=True) / 448.0
            c["x_t"], c["x_scale"] = (x / scale).to(torch.float8_e4m3fn), scale
        else:
            c["x_t"], c["x_scale"] = _e4m3(x, 1)
        c["w_t"], c["w_scale"] = _e4m3(normal(N, K) / math.sqrt(K) * (0.5 + normal(N, 1).abs()), 128)
        c["out"] = torch.empty(M, N // 2 if c["act"] == "swiglu" else N, dtype=torch.bfloat16, device=DEV)
    elif c["op"] == "rotary":
        N, Hq, Hk, D, A, half = c["N"], c["Hq"], c["Hk"], c["D"], c["axes"], c["rot"] // 2
        # one projection's output holds queries, keys and values side by side
        qkv = normal(N, Hq + 2 * Hk, D).bfloat16()
        c["q_t"], c["k_t"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
        c["out"] = (torch.empty(N, Hq, D, dtype=torch.bfloat16, device=DEV), torch.empty(N, Hk, D, dtype=torch.bfloat16, device=DEV))
        c["inv_freq"] = torch.exp2(torch.arange(half, device=DEV, dtype=torch.float64) * (-math.log2(500000.0) / half))
        # far positions on the first axis (a long context), places within an image on the others
        pos = torch.randint(0, 1 << 20, (A, N), device=DEV, generator=gen)
        pos[0] = torch.randint(0, 1 << 20, (1,), device=DEV, generator=gen) + torch.arange(N, device=DEV)
        pos[1:] = pos[1:] % 1024
        c["pos"] = pos
        # neighbouring frequencies go to one axis, all axes get about as many
        c["freq_axis"] = (torch.arange(half, device=DEV) * A // half).to(torch.uint8)
    else:
        B, V = c["B"], c["V"]
        x = normal(B, V) * (1.0 + 3.0 * uniform(B, 1))
        x[:, V - V // 50:] = float("-inf")  # a padded vocabulary's tail
        # some rows may take few tokens only
        few = (torch.arange(B, device=DEV) % 5 == 3)[:, None] & (uniform(B, V) < 0.97)
        x = x.masked_fill(few, float("-inf"))
        c["x_t"] = x.bfloat16() if c["dtype"] == "bf16" else x
        c["u"] = uniform(B)

        def settings(values, dtype):
            return torch.tensor(values, dtype=dtype, device=DEV)[torch.randint(0, len(values), (B,), device=DEV, generator=gen)]

        mixed = c["kind"] == "mixed"
        c["t"] = settings([0.0, 0.6, 0.7, 0.8, 1.0, 1.3] if mixed else [0.7, 1.0], torch.float32)
        c["top_k"] = settings([0, 1, 20, 50, 200, 1000], torch.int32) if mixed else None
        c["top_p"] = None if c["kind"] == "all" else settings([0.5, 0.8, 0.9, 0.95, 1.0] if mixed else [0.8, 0.9, 0.95], torch.float32)
        c["min_p"] = settings([0.0, 0.0, 0.02, 0.1], torch.float32) if mixed else None
        c["out"] = torch.empty(B, dtype=torch.int32, device=DEV)
    return c


# ----------------------------------------------------------------------- one pass
def run(state):
    return {"quantize": _quantize, "linear": _linear, "rotary": _rotary, "sample": _sample}[state["op"]](state)


def _quantize(s):
    if own:
        import nvfp4_routed_moe_sort_gb300 as moe
        y, scale = moe.quantize_fp8(s["x_t"], rows=s["rows"], out=s["out"])
    else:
        y, scale = _e4m3(s["x_t"].float(), s["rows"])
    return {"y": y, "scale": scale}


def _linear(s):
    if own:
        import nvfp4_routed_moe_sort_gb300 as moe
        return moe.fp8_linear(s["x_t"], s["x_scale"], s["w_t"], s["w_scale"], activation=s["act"], out=s["out"])
    N, K = s["w_t"].shape
    x = s["x_t"].float() * s["x_scale"].repeat_interleave(K if s["x"] == "token" else 128, 1)[:, :K]
    w = s["w_t"].float() * s["w_scale"].repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    y = x @ w.T
    if s["act"] == "swiglu":
        gate, up = y.chunk(2, 1)
        y = gate / (1.0 + torch.exp(-gate)) * up
    return y.bfloat16()


def _rotary(s):
    if own:
        import nvfp4_routed_moe_sort_gb300 as moe
        q, k = moe.rotary(s["q_t"], s["pos"], s["inv_freq"], k=s["k_t"], axes=s["freq_axis"], adjacent=s["adjacent"], out=s["out"])
        return {"q": q, "k": k}
    rot, half = s["rot"], s["rot"] // 2
    angle = s["pos"].double()[s["freq_axis"].long()].T * s["inv_freq"]  # [N, rot / 2]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def turn(x):
        x = x.float()
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if s["adjacent"] else (x[..., :half], x[..., half:rot])
        a, b = a * cos - b * sin, a * sin + b * cos
        t = torch.stack((a, b), -1).flatten(-2) if s["adjacent"] else torch.cat((a, b), -1)
        return torch.cat((t, x[..., rot:]), -1).bfloat16()

    return {"q": turn(s["q_t"]), "k": turn(s["k_t"])}


def _sample(s):
    if own:
        import nvfp4_routed_moe_sort_gb300 as moe
        return moe.sample_tokens(s["x_t"], s["u"], temperature=s["t"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"],
                                 out=s["out"])
    V = s["V"]
    x = s["x_t"].double()
    t = s["t"].double()[:, None]
    x, order = torch.sort(x, dim=1, descending=True, stable=True)  # ties: the lowest index first
    greedy = t <= 0
    w = torch.exp((x - x[:, :1]) / torch.where(greedy, torch.ones_like(t), t))
    w = torch.where(torch.isnan(w), torch.zeros_like(w), w)  # a row that is masked everywhere
    place = torch.arange(V, device=x.device)
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        w = torch.where((place < k) | (k <= 0), w, 0.0)
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        before = torch.cumsum(w, 1) - w
        w = torch.where((before < p * w.sum(1, keepdim=True)) | (p >= 1), w, 0.0)
    if s["min_p"] is not None:
        w = torch.where(w >= s["min_p"].double()[:, None], w, 0.0)
    w = torch.where(greedy & (place > 0), 0.0, w)
    w = torch.zeros_like(w).scatter(1, order, w)  # the kept tokens in the order of their index
    cum = torch.cumsum(w, 1)
    # the first token at which the cumulated weight passes u times the total; none passed: the last one kept
    taken = ((cum > s["u"].double()[:, None] * cum[:, -1:]) & (w > 0)).to(torch.uint8).argmax(1)
    return torch.where(cum[:, -1] > 0, taken, -1).int()


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"quantize": _quantize64, "linear": _linear64, "rotary": _rotary64, "sample": _sample64}[s["op"]](s)


def _quantize64(s):
    scales, ys = [], []
    R = s["rows"]
    step = 2048
    for i in range(0, s["M"], step):
        strip = s["x_t"][i:i + step].double()
        cols, parts = [], []
        for p in strip.split(128, 1):
            top = p.abs().max(1).values
            if R > 1:
                top = torch.stack([t.max() for t in top.split(R)])
            sc = top / 448.0
            sc[sc == 0] = 1.0
            cols.append(sc)
            parts.append(p / sc.repeat_interleave(R)[:len(p), None])
        scales.append(torch.stack(cols, 1))
        ys.append(torch.cat(parts, 1))
    return {"y": torch.cat(ys), "scale": torch.cat(scales)}


def _linear64(s):
    K, half = s["K"], s["N"] // 2
    ws = s["w_scale"].double()
    w = torch.cat([strip.double() * ws[j].repeat_interleave(128)[:K] for j, strip in enumerate(s["w_t"].split(128))])
    out = []
    for i in range(0, s["M"], 2048):
        x, xs = s["x_t"][i:i + 2048].double(), s["x_scale"][i:i + 2048].double()
        x = x * xs if s["x"] == "token" else torch.cat([p * xs[:, j:j + 1] for j, p in enumerate(x.split(128, 1))], 1)
        y = x.matmul(w.t())
        if s["act"] == "swiglu":
            y = y[:, :half] * torch.sigmoid(y[:, :half]) * y[:, half:]
        out.append(y)
    return torch.cat(out)


def _rotary64(s):
    pos = s["pos"].double()
    angle = torch.stack([pos[a] * f for a, f in zip(s["freq_axis"].tolist(), s["inv_freq"].tolist())], 1)
    phase = torch.polar(torch.ones_like(angle), angle)[:, None, :]
    half, rot = s["rot"] // 2, s["rot"]

    def turn(x):
        z = x.double().clone()
        first = slice(0, rot, 2) if s["adjacent"] else slice(0, half)
        second = slice(1, rot, 2) if s["adjacent"] else slice(half, rot)
        turned = torch.complex(z[..., first], z[..., second]) * phase
        z[..., first], z[..., second] = turned.real, turned.imag
        return z

    return {"q": turn(s["q_t"]), "k": turn(s["k_t"])}


def _sample64(s):
    """Row by row on the host: the tokens in the order of their logits, ties by their index."""
    rows = s["x_t"].float().cpu().numpy().astype(np.float64)
    u = s["u"].cpu().numpy().astype(np.float64)

    def setting(name, off):
        return np.full(len(u), off) if s[name] is None else s[name].cpu().numpy().astype(np.float64)

    t, top_k, top_p, min_p = setting("t", 1.0), setting("top_k", 0), setting("top_p", 1.0), setting("min_p", 0.0)
    taken = np.full(len(u), -1, dtype=np.int32)
    for b, x in enumerate(rows):
        alive = np.flatnonzero(x > -np.inf)
        if not len(alive):
            continue
        if t[b] <= 0:
            taken[b] = np.argmax(x)
            continue
        kept = alive[np.argsort(-x[alive], kind="stable")]
        if top_k[b] > 0:
            kept = kept[:int(top_k[b])]
        z = (x[kept] - x[kept[0]]) / t[b]
        w = np.exp(z)
        if top_p[b] < 1:
            sums = np.cumsum(w)
            n = int(np.searchsorted(sums, top_p[b] * sums[-1])) + 1
            kept, w = kept[:n], w[:n]
        kept, w = kept[w >= min_p[b]], w[w >= min_p[b]]
        back = np.argsort(kept)
        sums = np.cumsum(w[back])
        taken[b] = kept[back][min(int(np.searchsorted(sums, u[b] * sums[-1], side="right")), len(kept) - 1)]
    return torch.from_numpy(taken).to(DEV)
