"""The sampled token right beside a border between two tokens, where an error of a weight shows.

A border follows from one ratio w = exp((l - max) / temperature) alone, here computed to 40 digits from the float32 inputs. The random
number (or the filter's setting) is the float32 value nearest to the border on either side that lies more than MARGIN
of it away. The weights' errors allow 2^-34 of a weight and one unit of 2^-44, which at w >= 2^-9 is another 2^-35: a border is
off by less than 2^-32 of itself, so that MARGIN = 2^-30 is never within reach. float32 values lie 2^-24 apart: a weight that is off
by 2^-20 gives a wrong token in most of the cases.
"""
import decimal
import math
from decimal import Decimal

import numpy as np
import pytest
import torch

from gpu_harness import DEV, pkg

pytestmark = pytest.mark.gpu

MARGIN = Decimal(2) ** -30
CONTEXT = decimal.Context(prec=40)


def ratio(l, top, t):
    """exp((l - top) / t) of float32 values, to 40 digits."""
    with decimal.localcontext(CONTEXT):
        return ((Decimal(float(l)) - Decimal(float(top))) / Decimal(float(t))).exp()


def beside(border):
    """The nearest float32 values below and above a border that are MARGIN of it away."""
    with decimal.localcontext(CONTEXT):
        low = high = np.float32(float(border))
        while Decimal(float(low)) >= border * (1 - MARGIN):
            low = np.nextafter(low, np.float32(-1))
        while Decimal(float(high)) <= border * (1 + MARGIN):
            high = np.nextafter(high, np.float32(2))
    return low, high


def pairs(n, least, dtype, seed):
    """Logits (smaller, larger) and temperatures whose weights' ratio lies in [least, 0.98]."""
    r = np.random.default_rng(seed)
    out = []
    while len(out) < n:
        top = np.float32(r.normal() * r.choice([0.01, 1.0, 20.0]))
        t = np.float32(r.choice([0.3, 0.6, 0.7, 1.0, 1.3, 2.5]))
        l = np.float32(top + t * math.log(r.uniform(least, 0.98)))
        if dtype == torch.bfloat16:
            l, top = (np.float32(torch.tensor(float(v)).bfloat16().float()) for v in (l, top))
        if least < math.exp((float(l) - float(top)) / float(t)) < 0.98:
            out.append((l, top, t))
    return out


def column(values, dtype=torch.float32):
    return torch.tensor(np.array(values), dtype=dtype, device=DEV)


def place(V):
    """Where a row of V tokens has its two or three: its front, middle and end, in the blocks of a long row."""
    return 0, V // 2 if V > 3 else 1, V - 1


def rows(values, V, dtype):
    """Rows of V logits of which all but those at their places are masked."""
    x = torch.full((len(values), V), -math.inf)
    for b, row in enumerate(values):
        for at, v in row.items():
            x[b, at] = float(v)
    return x.to(dtype).to(DEV)


SIZES = [(2, 512), (1003, 128), (9001, 24), (70001, 12)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,n", SIZES)
def test_the_drawn_token_beside_a_border(V, n, dtype):
    """Token 0 of weight w, a later one of weight 1: 0 for u < w / (1 + w)."""
    values, u, t, want = [], [], [], []
    for l, top, temp in pairs(n, 2.0 ** -9, dtype, V):
        w = ratio(l, top, temp)
        with decimal.localcontext(CONTEXT):
            low, high = beside(w / (1 + w))
        for number, taken in ((low, 0), (high, V - 1)):
            values.append({0: l, V - 1: top}), u.append(number), t.append(temp), want.append(taken)
    got = pkg.sample_tokens(rows(values, V, dtype), column(u), temperature=column(t)).tolist()
    assert got == want


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,n", SIZES)
def test_top_p_beside_a_border(V, n, dtype):
    """Weights 1 and w: the first alone is kept for top_p <= 1 / (1 + w). The border is resolved to 2^-24 of 1, so w is large."""
    values, p, t, want = [], [], [], []
    for l, top, temp in pairs(n, 0.5, dtype, 2 * V):
        w = ratio(l, top, temp)
        with decimal.localcontext(CONTEXT):
            low, high = beside(1 / (1 + w))
        for setting, taken in ((low, 0), (high, V - 1)):
            values.append({0: top, V - 1: l}), p.append(setting), t.append(temp), want.append(taken)
    u = column([1.0 - 2.0 ** -24] * len(p))  # the last token that is kept
    assert pkg.sample_tokens(rows(values, V, dtype), u, temperature=column(t), top_p=column(p)).tolist() == want


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,n", SIZES)
def test_top_p_of_what_top_k_keeps_beside_a_border(V, n, dtype):
    """The same with a third token of less weight, which top_k takes out of the sum."""
    a, b, c = place(max(V, 3))
    values, p, t, want = [], [], [], []
    for l, top, temp in pairs(n, 0.5, dtype, 3 * V):
        w = ratio(l, top, temp)
        with decimal.localcontext(CONTEXT):
            low, high = beside(1 / (1 + w))
        for setting, taken in ((low, b), (high, c)):
            values.append({a: l - 4 * temp, b: top, c: l}), p.append(setting), t.append(temp), want.append(taken)
    u, k = column([1.0 - 2.0 ** -24] * len(p)), column([2] * len(p), torch.int32)
    assert pkg.sample_tokens(rows(values, max(V, 3), dtype), u, temperature=column(t), top_k=k, top_p=column(p)).tolist() == want


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,n", SIZES)
def test_min_p_beside_a_border(V, n, dtype):
    """Weights w and 1: both are kept for min_p <= w."""
    values, m, t, want = [], [], [], []
    for l, top, temp in pairs(n, 2.0 ** -9, dtype, 5 * V):
        low, high = beside(ratio(l, top, temp))
        for setting, taken in ((low, 0), (high, V - 1)):
            values.append({0: l, V - 1: top}), m.append(setting), t.append(temp), want.append(taken)
    assert pkg.sample_tokens(rows(values, V, dtype), column([0.0] * len(m)), temperature=column(t), min_p=column(m)).tolist() == want


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [3, 9001])
def test_min_p_of_every_size(V, dtype):
    """From 2^-43 of the largest weight up: a third of min_p's weight is not kept, three times it is. (Such settings are no whole
    numbers of 2^-44, and are rounded up.)"""
    values, m, u, want = [], [], [], []
    for e in range(1, 44):
        for f in (1.0, 1.0 + 2.0 ** -23, 1.5, 2.0 - 2.0 ** -23):
            setting = np.float32(f * 2.0 ** -e)
            for part, taken in ((1 / 3, 0), (3.0, V - 1)):
                if setting * part < 0.9:  # tokens 1 and 0 of weight 1, the last of min_p's weight times `part`
                    values.append({0: 0.0, V - 1: math.log(float(setting) * part)})
                    m.append(setting), u.append(1.0 - 2.0 ** -24), want.append(taken)
    u = column(u)
    got = pkg.sample_tokens(rows(values, V, dtype), u, min_p=column(m)).tolist()
    # the last token's own weight is drawn only where it is at least 2^-24 of the sum
    seen = [i for i, v in enumerate(values) if v[V - 1] > -16.0 or want[i] == 0]
    assert [got[i] for i in seen] == [want[i] for i in seen]
    # reversed, it comes first and is drawn by u = 0
    back = [{0: v[V - 1], V - 1: v[0]} for v in values]
    got = pkg.sample_tokens(rows(back, V, dtype), torch.zeros_like(u), min_p=column(m)).tolist()
    assert got == [V - 1 if w == 0 else 0 for w in want]


@pytest.mark.parametrize("units", [1.02, 1.5, 1.99, 3.99, 100.9])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [3000, 1 << 18])
def test_a_long_tail_of_weights_of_a_few_units(V, dtype, units):
    """Many tokens of `units` times 2^-44, then one of 2^-12, then one of weight 1. Each may lose a unit: the borders lie within
    V units and 2^-33 of the exact ones, and beyond that the token is the exact one's; nothing is drawn that has no weight."""
    logits = torch.full((V,), math.log(units * 2.0 ** -44))
    logits[-2], logits[-1] = math.log(2.0 ** -12), 0.0
    logits = logits.to(dtype)
    w = np.exp(logits.double().numpy())
    ends = np.cumsum(w) / w.sum()
    before, middle = ends[-3], ends[-2]
    bound = V * 2.0 ** -44 + 2.0 ** -33 + units * 2.0 ** -43  # and the one that top_k takes out
    u = [middle + bound, middle - bound, before + bound, 0.999]
    want = [V - 1, V - 2, V - 2, V - 1]
    if before > bound:
        u.append(before - bound)
    u = np.float32(u)
    u[0], u[1], u[2] = np.nextafter(u[0], np.float32(1)), np.nextafter(u[1], np.float32(0)), np.nextafter(u[2], np.float32(1))
    x = logits.to(DEV).expand(len(u), V).contiguous()
    for kw in ({}, dict(top_k=column([V - 1] * len(u), torch.int32))):
        got = pkg.sample_tokens(x, column(u), **kw).tolist()
        assert got[:4] == want
        assert all(0 <= t < V - 2 for t in got[4:])
