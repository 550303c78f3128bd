"""The example's decoder layer, several tokens deep, against the same layer in float64.

The reference applies the layer's formulas to the BF16 weights and keeps its own cache in float64. What
separates the two is the 4-bit weights (each product's relative error near 0.1), the 4-bit cache and the
E4M3 and NVFP4 activations: the layer's update of the residual stream stays within 0.35 of the
reference's, and a wrong head, expert, page or residual moves it by about its own size."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from gpu_harness import DEV
from oracle import decoder as D

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("decode_layer", os.path.join(ROOT, "examples", "decode_layer.py"))
example = importlib.util.module_from_spec(spec)
spec.loader.exec_module(example)


def test_decode_layer_steps_match_float64():
    B, H, Hq, Hkv, Dh, page, steps = 3, 256, 4, 2, 64, 16, 20
    layer = example.DecodeLayer(B, H, Hq, Hkv, Dh, experts=8, top_k=2, inter=128, shared_inter=128, pages=12, page_size=page,
                                max_pages=4, seed=3)
    w = {k: v.double().cpu().numpy() for k, v in layer.w.items()}
    table = np.random.default_rng(2).permutation(12).reshape(B, 4)
    layer.page_table.copy_(torch.from_numpy(table).int())
    graph = layer.capture()          # the warm-up step stores nothing: every slot is -1
    keys = [np.zeros((0, Hkv, Dh)) for _ in range(B)]
    values = [np.zeros((0, Hkv, Dh)) for _ in range(B)]
    for t in range(steps):
        lens = [t + 1, max(t - 2, 0), t + 1]          # the second sequence starts three steps later
        x = torch.from_numpy(np.random.default_rng(t).normal(size=(B, H)).astype(np.float32)).to(DEV).bfloat16()
        layer.x.copy_(x)
        layer.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        layer.slots.copy_(torch.tensor([table[b, (n - 1) // page] * page + (n - 1) % page if n else -1 for b, n in enumerate(lens)]))
        graph.replay()
        got = layer.result.double().cpu().numpy()

        x = x.double().cpu().numpy()
        n1 = D.add_rms_norm(x, w["norm1"])["y"]
        qkv = (n1 @ w["qkv"].T).reshape(B, -1, Dh)
        o = np.zeros((B, Hq, Dh))
        for b, n in enumerate(lens):
            if n:
                keys[b] = np.concatenate([keys[b], qkv[b:b + 1, Hq:Hq + Hkv]])
                values[b] = np.concatenate([values[b], qkv[b:b + 1, Hq + Hkv:]])
            for h in range(Hkv):
                hs = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
                o[b, hs] = D.attend(qkv[b:b + 1, hs], keys[b][:, h], values[b][:, h], Dh ** -0.5)[0][0]
        h2 = o.reshape(B, -1) @ w["out"].T
        norm2 = D.add_rms_norm(h2, w["norm2"], x)
        y = norm2["y"]
        ffn = D.activate(y @ w["shared_in"].T, "swiglu") @ w["shared_out"].T
        # the routing is the layer's own: near ties may fall either way in BF16
        p = torch.softmax(torch.from_numpy(y @ w["router"].T), -1)
        for b in range(B):
            best, ids = p[b].topk(2)
            best = best / best.sum()
            for e, s in zip(ids.tolist(), best.tolist()):
                ffn[b] += s * (D.activate(y[b:b + 1] @ w["w1"][e].T, "swiglu") @ w["w2"][e].T)[0]
        want = norm2["residual"] + ffn
        for b in range(B):
            third = p[b].topk(3)[0]
            if third[1] - third[2] < 0.05:
                continue
            err = np.linalg.norm(got[b] - want[b]) / np.linalg.norm(want[b] - x[b])
            assert err < 0.35, (t, b, err)
    assert int(layer.cache.dev_status[0]) == 0
