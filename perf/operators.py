"""Cases and plain forms of the operators around the routed experts in one decoder layer.

* ``norm``: root-mean-square norm with the residual's addition; BF16 output, and the same
  output in E4M3 with one FP32 scale per token or per 128 channels.
* ``linear``: products of one to sixteen tokens with an NVFP4 weight matrix (packed E2M1 codes,
  one E4M3 scale per 16 values, one FP32 scalar), BF16 or scaled E4M3 activations, an optional
  SwiGLU over the [gate; up] rows.
* ``attend``: a decode step over a paged NVFP4 key/value cache: the new tokens are encoded and
  stored, then every query row attends to its sequence, grouped heads, causal among the new tokens.

``run`` computes them in elementary torch operations in 32 bits, or, with ``own`` set, through
the framework's entry points.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # one token of a small layer (hidden 2048): the latency of one decode step's norm
        dict(name="norm_one_token", op="norm", M=1, H=2048, residual=True, fp8="token"),
        # a ragged chunk of a prompt with an odd hidden size: rows that start at odd addresses
        dict(name="norm_odd", op="norm", M=777, H=1531, residual=True, fp8="group"),
        # a long prompt of the 4096-wide layer, scales per 128 channels
        dict(name="norm_prompt", op="norm", M=16384, H=4096, residual=True, fp8="group"),
        # one token through the down projection of a small shared expert (2048 <- 512)
        dict(name="linear_small", op="linear", M=1, N=2048, K=512, act="identity", x="bf16"),
        # eight tokens through the gate and up rows of a 7168-wide shared expert, FP8 tokens
        dict(name="linear_swiglu_fp8", op="linear", M=8, N=4096, K=7168, act="swiglu", x="group"),
        # thirteen tokens, a row count that no tile divides and a K that is only a multiple of 16
        dict(name="linear_ragged", op="linear", M=13, N=7001, K=2000, act="identity", x="token"),
        # the output head: four tokens against a large vocabulary of odd size
        dict(name="linear_head", op="linear", M=4, N=129021, K=4096, act="identity", x="bf16"),
        # a single short conversation
        dict(name="attend_short", op="attend", B=1, q_len=1, Hkv=4, G=4, D=128, page=64, lo=37, hi=37, g=1.0, ls=1),
        # a serving batch of mixed lengths, one of its sequences empty
        dict(name="attend_ragged", op="attend", B=16, q_len=1, Hkv=4, G=8, D=128, page=64, lo=0, hi=4097, g=1.0, ls=2),
        # four drafted tokens checked at once, six query heads to a key head, small pages
        dict(name="attend_draft", op="attend", B=8, q_len=4, Hkv=2, G=6, D=64, page=16, lo=3, hi=16001, g=2.5, ls=3),
        # one long document
        dict(name="attend_long", op="attend", B=1, q_len=1, Hkv=8, G=8, D=128, page=64, lo=131071, hi=131071, g=1.0, ls=4),
        # a full batch at depth
        dict(name="attend_batch", op="attend", B=64, q_len=1, Hkv=8, G=4, D=128, page=64, lo=4000, hi=8191, g=1.0, ls=5),
    ]


def _spread(rng, lo, hi):
    """A whole number spread evenly over the logarithm of [lo, hi]; 3072 is left out."""
    n = min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return n + 1 if n == 3072 else n


def draw(rng):
    op = rng.choice(["norm", "linear", "attend"])
    if op == "norm":
        H = _spread(rng, 64, 8192)
        if rng.random() < 0.6:
            H = max(8, H // 8 * 8)
        H = 3080 if H == 3072 else H
        M = min(_spread(rng, 1, 16384), 16384 * 4096 // H)
        return dict(op=op, M=M, H=H, residual=rng.random() < 0.75, fp8=rng.choice(["none", "token", "group"]))
    if op == "linear":
        K = max(128, _spread(rng, 128, 8192) // 16 * 16)
        K = 3088 if K == 3072 else K
        N = min(_spread(rng, 64, 131072), 129021 * 4096 // K)
        act = rng.choice(["identity", "swiglu"])
        if act == "swiglu":
            N = N // 2 * 2
        N = 3070 if N == 3072 else N
        return dict(op=op, M=rng.randint(1, 16), N=N, K=K, act=act, x=rng.choice(["bf16", "token", "group"]))
    B = _spread(rng, 1, 64)
    Hkv = rng.choice([1, 2, 3, 4, 8])
    most = min(131071, max(64, 64 * 8 * 6000 // (B * Hkv)))
    hi = _spread(rng, 16, most)
    lo = rng.choice([0, hi // 2, hi])
    return dict(op=op, B=B, q_len=rng.choice([1, 1, 1, 2, 4]), Hkv=Hkv, G=rng.choice([1, 2, 4, 5, 6, 8, 16]),
                D=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]), lo=lo, hi=hi,
                g=rng.choice([1.0, 2.5]), ls=rng.randrange(1 << 20))


def _lens(c):
    """The sequences' lengths, the new tokens included: spread over [lo, hi], both ends among them."""
    r = random.Random(c["ls"])
    return [c["hi"] if i == 0 else c["lo"] if i == 1 else r.randint(c["lo"], c["hi"]) for i in range(c["B"])]


def _group(c):
    return c["H"] if c["fp8"] == "token" else 128


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["M"] * c["H"]
        b = n * (2 + 2) + 2 * c["H"] + (4 * n if c["residual"] else 0)
        if c["fp8"] != "none":
            b += n + 4 * c["M"] * -(-c["H"] // _group(c))
        return {"bytes": b, "flops": 8 * n}
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        out = N // 2 if c["act"] == "swiglu" else N
        x = M * K * 2 if c["x"] == "bf16" else M * K + 4 * M * (1 if c["x"] == "token" else -(-K // 128))
        return {"bytes": N * K * 9 // 16 + x + 2 * M * out, "flops": 2 * M * N * K}
    n, rows = sum(_lens(c)), c["B"] * c["q_len"]
    Hq = c["Hkv"] * c["G"]
    per = 2 * (c["D"] // 2 + c["D"] // 16) * c["Hkv"]  # keys and values of one token
    b = n * per + 2 * rows * Hq * c["D"] * 2 + 4 * rows * Hq + rows * (per + 8 * c["Hkv"] * c["D"])
    return {"bytes": b, "flops": 4 * n * Hq * c["D"] * c["q_len"]}


# ------------------------------------------------------------------------- inputs
def _encode(x, g):
    """FP32 values [..., n] -> packed E2M1 codes [..., n/2] and E4M3 scales [..., n/16] as bytes:
    s = (max|x| / 6) * g, q = e4m3(s), code = e2m1(x * (g / q)), each step in 32 bits."""
    b = x.unflatten(-1, (-1, 16))
    q = ((b.abs().amax(-1) / 6.0) * g).clamp(max=448.0).to(torch.float8_e4m3fn)
    qf = q.float()
    inv = torch.where(qf == 0, torch.zeros_like(qf), g / qf)
    t = b * inv.unsqueeze(-1)
    a = t.abs()
    mag = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (mag + 8 * torch.signbit(t).to(torch.uint8)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), q.view(torch.uint8)


def _decode(data, sf, values):
    """Packed codes [..., n/2] and scales [..., n/16] -> FP32 [..., n] (before the global scale);
    `values`: the sixteen codes' values."""
    v = values[torch.stack((data & 15, data >> 4), -1).flatten(-2).int()]
    return (v.unflatten(-1, (-1, 16)) * sf.view(torch.float8_e4m3fn).float().unsqueeze(-1)).flatten(-2)


def _e4m3(y, group):
    """FP32 rows -> E4M3 rows and FP32 scales amax / 448 per `group` channels."""
    M, H = y.shape
    n = -(-H // group)
    b = torch.nn.functional.pad(y, (0, n * group - H)).view(M, n, group)
    amax = b.abs().amax(-1)
    one = torch.ones_like(amax)
    scale = torch.where(amax == 0, one, amax / 448.0)
    inv = torch.where(amax == 0, one, 448.0 / amax)
    y8 = (b * inv.unsqueeze(-1)).view(M, n * group)[:, :H].contiguous().to(torch.float8_e4m3fn)
    return y8, scale


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV).manual_seed(1009 * int(seed) + 17)
    c["values"] = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV)

    def normal(*shape):
        return torch.randn(*shape, device=DEV, generator=gen)

    if c["op"] == "norm":
        M, H = c["M"], c["H"]
        c["x_t"] = (normal(M, H) * (0.5 + normal(M, 1).abs())).bfloat16()
        c["r_t"] = (normal(M, H) * 3.0).bfloat16() if c["residual"] else None
        c["w_t"] = (1.0 + 0.2 * normal(H)).bfloat16()
        n = -(-H // _group(c))
        c["out"] = (torch.empty(M, H, dtype=torch.bfloat16, device=DEV),
                    torch.empty(M, H, dtype=torch.bfloat16, device=DEV) if c["residual"] else None,
                    torch.empty(M, H, dtype=torch.float8_e4m3fn, device=DEV) if c["fp8"] != "none" else None,
                    torch.empty(M, n, dtype=torch.float32, device=DEV) if c["fp8"] != "none" else None)
    elif c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        c["w_t"] = torch.empty(N, K // 2, dtype=torch.uint8, device=DEV)
        c["sf_t"] = torch.empty(N, K // 16, dtype=torch.uint8, device=DEV)
        step = max(1, (64 << 20) // K)
        amax = 0.02 * 6.0
        c["alpha"] = torch.tensor([amax / 2688.0], device=DEV)
        for i in range(0, N, step):
            w = (0.02 * normal(min(step, N - i), K)).bfloat16().float().clamp(-amax, amax)
            c["w_t"][i:i + step], c["sf_t"][i:i + step] = _encode(w, 2688.0 / amax)
        x = normal(M, K) * (1.0 + 4.0 * (normal(1, K) > 2.5))
        if c["x"] == "bf16":
            c["x_t"], c["x_scale"] = x.bfloat16(), None
        else:
            c["x_t"], c["x_scale"] = _e4m3(x, K if c["x"] == "token" else 128)
        c["out"] = torch.empty(M, N // 2 if c["act"] == "swiglu" else N, dtype=torch.bfloat16, device=DEV)
    else:
        B, D, Hkv, ps = c["B"], c["D"], c["Hkv"], c["page"]
        lens = _lens(c)
        most = max(1, -(-max(lens) // ps))
        used = [-(-n // ps) for n in lens]
        pages = sum(used) + 3
        order = torch.randperm(pages, device=DEV, generator=gen).cpu()
        table, at = torch.full((B, most), -1, dtype=torch.int32), 0
        for b, n in enumerate(used):
            table[b, :n] = order[at:at + n].int()
            at += n
        # pages hold encoded keys and values; what lies past a sequence's end is whatever was there
        for name in ("k", "v"):
            c[name + "_pool"] = torch.empty(pages, Hkv, ps, D // 2, dtype=torch.uint8, device=DEV)
            c[name + "_sf"] = torch.empty(pages, Hkv, ps, D // 16, dtype=torch.uint8, device=DEV)
            step = max(1, (64 << 20) // (Hkv * ps * D))
            for i in range(0, pages, step):
                n = min(step, pages - i)
                x = normal(n, Hkv, ps, D) * (0.5 + normal(n, Hkv, 1, D).abs())
                c[name + "_pool"][i:i + n], c[name + "_sf"][i:i + n] = _encode(x.bfloat16().float(), c["g"])
            del x
        junk = torch.randint(0, 256, (ps, D // 16), device=DEV, generator=gen).to(torch.uint8)
        junk[:, 0] = 0x7F  # no number at all
        for b, n in enumerate(lens):
            if n % ps:
                for name in ("k", "v"):
                    c[name + "_sf"][table[b, n // ps].item(), :, n % ps:] = junk[n % ps:]
        slots = []
        for b, n in enumerate(lens):
            for i in range(c["q_len"]):
                p = n - c["q_len"] + i
                slots.append(-1 if p < 0 else int(table[b, p // ps]) * ps + p % ps)
        c["spare"] = int(order[at]) * ps  # a place that no sequence holds
        c["slots"] = torch.tensor(slots, dtype=torch.int64, device=DEV)
        c["table"], c["lens"] = table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
        rows, Hq = B * c["q_len"], Hkv * c["G"]
        # one projection's output holds queries, keys and values side by side
        qkv = normal(rows, Hq + 2 * Hkv, D)
        qkv[:, :Hq] *= 2.0
        qkv = qkv.bfloat16()
        c["q_t"] = qkv[:, :Hq].unflatten(0, (B, c["q_len"]))
        c["k_t"], c["v_t"] = qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        c["scale"] = 1.0 / math.sqrt(D)
        c["status"] = torch.zeros(4, dtype=torch.int32, device=DEV)
        c["seen"] = tuple(torch.empty(rows, Hkv, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        c["out"] = torch.empty(B, c["q_len"], Hq, D, dtype=torch.bfloat16, device=DEV)
        c["lse"] = torch.empty(B, c["q_len"], Hq, dtype=torch.float32, device=DEV)
    return c


# ----------------------------------------------------------------------- one pass
def run(state):
    return {"norm": _norm, "linear": _linear, "attend": _attend}[state["op"]](state)


def _norm(s):
    fp8 = None if s["fp8"] == "none" else s["fp8"]
    if own:
        import nvfp4_routed_moe_sort_gb300 as moe
        y, r, y8, scale = moe.add_rms_norm(s["x_t"], s["w_t"], residual=s["r_t"], eps=1e-6, fp8=fp8, out=s["out"])
    else:
        h = s["x_t"].float()
        r = None
        if s["r_t"] is not None:
            h = h + s["r_t"].float()
            r = h.bfloat16()
        f = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + 1e-6) * s["w_t"].float()
        y = f.bfloat16()
        y8, scale = _e4m3(f, _group(s)) if fp8 else (None, None)
    return {k: v for k, v in (("y", y), ("residual", r), ("y8", y8), ("scale", scale)) if v is not None}


def _linear(s):
    if own:
        import nvfp4_routed_moe_sort_gb300 as moe
        return moe.fp4_linear(s["x_t"], s["w_t"], s["sf_t"], s["alpha"], activation=s["act"], x_scale=s["x_scale"],
                              out=s["out"])
    x = s["x_t"].float()
    if s["x_scale"] is not None:
        x = x * s["x_scale"].repeat_interleave(s["K"] if s["x"] == "token" else 128, 1)[:, :s["K"]]
    y = (x @ _decode(s["w_t"], s["sf_t"], s["values"]).T) * s["alpha"]
    if s["act"] == "swiglu":
        gate, up = y.chunk(2, 1)
        y = gate / (1.0 + torch.exp(-gate)) * up
    return y.bfloat16()


def _attend(s):
    if own:
        import nvfp4_routed_moe_sort_gb300 as moe
        kv = moe.NVFP4KVCache(s["k_pool"], s["k_sf"], s["v_pool"], s["v_sf"], k_scale=s["g"], v_scale=s["g"],
                              dev_status=s["status"])
        kv.append(s["k_t"], s["v_t"], s["slots"], seen=s["seen"])
        out, lse = kv.attend(s["q_t"], s["table"], s["lens"], softmax_scale=s["scale"], out=s["out"], lse=s["lse"])
        return {"out": out, "lse": lse, "k_seen": s["seen"][0], "v_seen": s["seen"][1]}
    B, T, Hkv, G, D, ps = s["B"], s["q_len"], s["Hkv"], s["G"], s["D"], s["page"]
    held = s["slots"] >= 0
    to = torch.where(held, s["slots"], s["spare"])
    page, at, held = to // ps, to % ps, held[:, None, None]
    seen, full = [], []
    cut = s["table"].clamp(min=0).long()
    for new, data, sf in ((s["k_t"], s["k_pool"], s["k_sf"]), (s["v_t"], s["v_pool"], s["v_sf"])):  # keys, values
        code, q = _encode(new.float(), s["g"])
        # a row without a slot rewrites the spare place with what it holds
        data[page, :, at] = torch.where(held, code, data[page, :, at])
        sf[page, :, at] = torch.where(held, q, sf[page, :, at])
        seen.append((_decode(code, q, s["values"]) / s["g"]).bfloat16())
        full.append(_decode(data[cut].transpose(1, 2).flatten(2, 3), sf[cut].transpose(1, 2).flatten(2, 3), s["values"]) / s["g"])
    k, v = full
    q = s["q_t"].float().unflatten(2, (Hkv, G)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [B, Hkv, T * G, D]
    score = (q @ k.transpose(-1, -2)) * s["scale"]
    step = torch.arange(T, device=DEV).repeat_interleave(G)
    limit = s["lens"][:, None] - (T - 1) + step  # the positions that a row may see
    place = torch.arange(k.shape[2], device=DEV)
    score = torch.where(place < limit[:, None, :, None], score, float("-inf"))
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    v = torch.where(place[:, None] < s["lens"][:, None, None, None], v, 0.0)
    o = (p @ v) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + torch.log(total)).squeeze(-1)

    def heads(t):  # [B, Hkv, T * G, ...] -> [B, T, Hkv * G, ...]
        return t.unflatten(2, (T, G)).transpose(1, 2).flatten(2, 3)

    return {"out": heads(o).bfloat16(), "lse": heads(lse).contiguous(), "k_seen": seen[0], "v_seen": seen[1]}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _norm64, "linear": _linear64, "attend": _attend64}[s["op"]](s)


def _values64(data, sf):
    """Encoded bytes -> float64, from the formats' bit fields: a code is sign, two exponent bits and
    one mantissa bit; a scale is sign, four exponent bits (bias 7) and three mantissa bits."""
    lo, hi = (data & 15).double(), (data >> 4).double()
    n = torch.stack((lo, hi), -1).reshape(*data.shape[:-1], -1)
    sign = 1.0 - 2.0 * (n >= 8)
    n = n % 8
    e, m = torch.div(n, 2, rounding_mode="floor"), n % 2
    v = sign * torch.where(e == 0, m * 0.5, (1.0 + m / 2.0) * torch.exp2(e - 1.0))
    b = sf.double()
    se, sm = torch.div(b % 128, 8, rounding_mode="floor"), b % 8
    scale = torch.where(se == 0, sm / 8.0 * 2.0 ** -6, (1.0 + sm / 8.0) * torch.exp2(se - 7.0))
    scale = torch.where(b % 128 == 127, torch.full_like(scale, float("nan")), scale * (1.0 - 2.0 * (b >= 128)))
    return v * scale.repeat_interleave(16, -1)


def _norm64(s):
    out = {"y": [], "residual": [], "y8": [], "scale": []}
    for i in range(0, s["M"], 2048):
        h = s["x_t"][i:i + 2048].double()
        if s["r_t"] is not None:
            h = h + s["r_t"][i:i + 2048].double()
            out["residual"].append(h)
        y = h / torch.sqrt(h.square().sum(-1, keepdim=True) / s["H"] + 1e-6) * s["w_t"].double()
        out["y"].append(y)
        if s["fp8"] != "none":
            parts = y.split(_group(s), 1)
            scale = torch.stack([p.abs().amax(1) for p in parts], 1) / 448.0
            scale[scale == 0] = 1.0
            out["scale"].append(scale)
            out["y8"].append(torch.cat([p / scale[:, j:j + 1] for j, p in enumerate(parts)], 1))
    return {k: torch.cat(v) for k, v in out.items() if v}


def _linear64(s):
    x = s["x_t"].double()
    if s["x_scale"] is not None:
        group = s["K"] if s["x"] == "token" else 128
        x = torch.cat([p * s["x_scale"][:, j:j + 1].double() for j, p in enumerate(x.split(group, 1))], 1)
    step = max(1, (32 << 20) // s["K"])
    y = torch.cat([x @ _values64(s["w_t"][i:i + step], s["sf_t"][i:i + step]).T for i in range(0, s["N"], step)], 1)
    y = y * s["alpha"].double()
    if s["act"] == "swiglu":
        half = s["N"] // 2
        y = y[:, :half] * torch.sigmoid(y[:, :half]) * y[:, half:]
    return y


def _store64(x, g):
    """The format's rule for one block of 16 (32-bit steps by definition), in numpy: the stored
    bytes of BF16 values [..., n]."""
    scales = np.array([(1 + m / 8) * 2.0 ** (e - 7) if e else m / 8 * 2.0 ** -6 for e in range(16) for m in range(8)][:127])
    grid = np.array(E2M1)

    def nearest(a, grid):
        j = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
        lo, hi = a - grid[j - 1], grid[j] - a
        return np.where((hi < lo) | ((hi == lo) & (j % 2 == 0)), j, j - 1)

    b = x.float().cpu().numpy().reshape(*x.shape[:-1], -1, 16)
    s = (np.abs(b).max(-1) / np.float32(6)) * np.float32(g)
    code = nearest(s.astype(np.float64), scales)
    q = scales[code].astype(np.float32)
    with np.errstate(divide="ignore"):
        inv = np.where(q == 0, np.float32(0), np.float32(g) / q).astype(np.float32)
    t = b * inv[..., None]
    n = (nearest(np.abs(t).astype(np.float64), grid) + 8 * np.signbit(t)).astype(np.uint8).reshape(*x.shape[:-1], -1)
    data = torch.from_numpy(n[..., 0::2] | (n[..., 1::2] << 4)).to(DEV)
    return data, torch.from_numpy(code.astype(np.uint8)).to(DEV)


def _attend64(s):
    T, Hkv, G, D, ps, g = s["q_len"], s["Hkv"], s["G"], s["D"], s["page"], s["g"]
    lens, slots, table = s["lens"].tolist(), s["slots"].tolist(), s["table"].long()
    seen = []
    for new, data, sf in ((s["k_t"], s["k_pool"], s["k_sf"]), (s["v_t"], s["v_pool"], s["v_sf"])):
        d, q = _store64(new, g)
        for i, at in enumerate(slots):
            if at >= 0:
                data[at // ps, :, at % ps], sf[at // ps, :, at % ps] = d[i], q[i]
        seen.append(_values64(d, q) / g)
    out = torch.zeros(s["B"], T, Hkv * G, D, dtype=torch.float64, device=DEV)
    lse = torch.full((s["B"], T, Hkv * G), float("-inf"), dtype=torch.float64, device=DEV)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        cut = table[b, :-(-n // ps)]
        for h in range(Hkv):
            k, v = (_values64(s[m + "_pool"][cut, h].flatten(0, 1)[:n], s[m + "_sf"][cut, h].flatten(0, 1)[:n]) / g
                    for m in ("k", "v"))
            for t in range(max(0, T - n), T):
                seen_by = n - (T - 1) + t
                z = (s["q_t"][b, t, h * G:(h + 1) * G].double() @ k[:seen_by].T) * s["scale"]
                out[b, t, h * G:(h + 1) * G] = torch.softmax(z, -1) @ v[:seen_by]
                lse[b, t, h * G:(h + 1) * G] = torch.logsumexp(z, -1)
    return {"out": out, "lse": lse, "k_seen": seen[0], "v_seen": seen[1]}
