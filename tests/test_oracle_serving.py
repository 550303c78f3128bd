"""The float64 reference of the quantiser, the E4M3 product, the rotary positions and the sampling: hand-made
values, identities and an independent library's conversions."""
import numpy as np
import pytest
import torch

from oracle import formats as F
from oracle import serving as S


def test_quantizer_against_torch_and_by_hand():
    x = np.zeros((3, 130), np.float32)
    x[0, 0], x[0, 1], x[0, 129] = 448.0, -1.0, 7.0
    x[2, 5] = -2.0 ** -10
    codes, scale = S.quantize_fp8(x)
    assert scale.tolist() == [[1.0, 7.0 / 448.0], [1.0, 1.0], [np.float32(2.0 ** -10) / np.float32(448), 1.0]]
    held = F.e4m3_decode(codes)
    assert held[0, 0] == 448 and held[0, 1] == -1 and held[0, 129] == 448 and held[2, 5] == -448
    codes, scale = S.quantize_fp8(x, 128)
    assert scale.tolist() == [[1.0, 7.0 / 448.0]] and F.e4m3_decode(codes)[2, 5] == 0  # half the smallest step: to even
    r = np.random.default_rng(0)
    x = F.bf16_round(r.normal(size=(40, 300)).astype(np.float32) * 30)
    for rows in (1, 128):
        codes, scale = S.quantize_fp8(x, rows)
        inv = np.float32(448) / (np.abs(x[:rows, :128]).max() if rows == 128 else np.abs(x[0, :128]).max())
        want = torch.from_numpy(x[:1, :128] * inv).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        assert np.array_equal(codes[:1, :128], want)


def test_linear_of_blocks_is_the_sum_of_its_blocks():
    r = np.random.default_rng(1)
    x, w = r.normal(size=(3, 300)), r.normal(size=(130, 300))
    xs, ws = r.random((3, 3)) + 0.5, r.random((2, 3)) + 0.5
    _, y, mass = S.fp8_linear(x, xs, w, ws)
    for m, n in ((0, 0), (2, 127), (1, 128), (2, 129)):
        parts = [xs[m, b] * ws[n // 128, b] * sum(x[m, k] * w[n, k] for k in range(128 * b, min(300, 128 * b + 128))) for b in range(3)]
        assert abs(y[m, n] - sum(parts)) < 1e-9 and mass[m, n] >= abs(y[m, n])
    _, one, _ = S.fp8_linear(x, xs[:, :1], w, np.ones((2, 3)))
    assert np.allclose(one, xs[:, :1] * (x @ w.T))


@pytest.mark.parametrize("adjacent", [False, True])
def test_rotary_turns(adjacent):
    x = np.zeros((2, 1, 6))
    x[:, 0, 0] = 1.0
    x[:, 0, 4:] = 5.0  # not turned
    y, size, _ = S.rotary(x, [[0, 1]], [np.pi / 2, 1.0], adjacent=adjacent)
    assert np.allclose(y[0], x[0]) and np.allclose(y[1, 0], [0, 1, 0, 0, 5, 5] if adjacent else [0, 0, 1, 0, 5, 5])
    assert (size[..., 4:] == 0).all()
    # a product of two turned vectors depends on the distance of their positions alone; a turn keeps the length
    r = np.random.default_rng(2)
    q, k, f = r.normal(size=(1, 1, 6)), r.normal(size=(1, 1, 6)), [1.0, 0.1, 0.01]

    def dot(a, b):
        return (S.rotary(q, [[a], [3 * a]], f, [0, 1, 0], adjacent)[0] * S.rotary(k, [[b], [3 * b]], f, [0, 1, 0], adjacent)[0]).sum()
    assert np.isclose(dot(5, 2), dot(105, 102)) and not np.isclose(dot(5, 2), dot(5, 3))
    assert np.isclose(np.linalg.norm(S.rotary(q, [[7], [-9]], f, [1, 1, 0], adjacent)[0]), np.linalg.norm(q))


def test_sampling_by_hand():
    l = [1.0, 3.0, 2.0, 3.0, -np.inf, np.nan]
    w = np.exp(np.array([1.0, 3, 2, 3]) - 3)
    edges = np.cumsum(w) / w.sum()
    for i in range(4):
        assert S.sample(l, edges[i] - 1e-9) == i
        if i < 3:
            assert S.sample(l, edges[i] + 1e-9) == i + 1
    assert S.sample(l, 0.9, temperature=0) == 1 and S.sample(l, 0.9, top_k=1) == 1  # ties: the lower index
    assert S.sample(l, 0.49, top_k=2) == 1 and S.sample(l, 0.51, top_k=2) == 3
    assert S.sample(l, 0.999, top_p=0.1) == 1 and S.sample(l, 0.999, top_p=0.5) == 3
    assert S.sample(l, 0.999, top_p=0.0) == 1
    # of the front three, 2 / (2 + 1 / e) = 0.8446 of the weight lies on the first two
    assert S.sample(l, 0.45, top_k=3, top_p=0.84) == 1 and S.sample(l, 0.45, top_k=3, top_p=0.85) == 2
    # two equal weights are half of the sum each only if nothing else has any
    assert S.sample([5.0, 5.0, -np.inf], 0.9, top_p=0.5) == 0 and S.sample([5.0, 5.0, -60.0], 0.9, top_p=0.5) == 1
    assert S.sample([5.0, 5.0, -2000.0], 0.9, top_p=0.5) == 1
    assert S.sample(l, 0.0, min_p=0.3) == 1 and S.sample(l, 0.0, min_p=0.1) == 0
    assert S.sample(l, 0.0, min_p=5.0) == 1 and S.sample(l, 0.999, min_p=5.0) == 3
    assert S.sample([-np.inf, np.nan], 0.5) == -1
    assert S.sample([0.0, np.inf, 1.0, np.inf], 0.6) == 3 and S.sample([0.0, np.inf, 1.0], 0.0) == 1
    assert S.sample([-0.0, 0.0], 0.0, top_k=1) == 0 and S.sample([-3.4e38] * 4, 0.6) == 2
    assert S.sample(l, 2.0) == 3 and S.sample(l, -1.0) == 0 and S.sample(l, np.nan) == 0


def test_sampling_follows_its_distribution():
    r = np.random.default_rng(3)
    l = r.normal(size=12) * 2
    p = np.exp(l / 0.7) / np.exp(l / 0.7).sum()
    n = 4000
    taken = np.bincount([S.sample(l, (i + 0.5) / n, temperature=0.7) for i in range(n)], minlength=12) / n
    assert np.abs(taken - p).max() <= 1.0 / n + 1e-12
