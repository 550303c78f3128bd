"""The oracle of the operators around the routed experts, against torch's own float64 operations,
brute force and closed forms."""
import numpy as np
import pytest
import torch

from oracle import decoder as D
from oracle import formats as F


@pytest.mark.parametrize("H", [1, 7, 128, 200])
def test_norm_against_torch(H):
    r = np.random.default_rng(H)
    x, res, w = r.normal(size=(5, H)), r.normal(size=(5, H)), r.normal(size=H)
    got = D.add_rms_norm(x, w, res, 1e-5, "group")
    want = torch.nn.functional.rms_norm(torch.tensor(x + res), (H,), torch.tensor(w), 1e-5).numpy()
    np.testing.assert_allclose(got["y"], want, rtol=1e-12)
    np.testing.assert_array_equal(got["residual"], x + res)
    assert got["scale"].shape == (5, -(-H // 128))
    np.testing.assert_allclose(got["y8"] * np.repeat(got["scale"], 128, -1)[:, :H], want, rtol=1e-12)
    assert np.abs(got["y8"]).max() == pytest.approx(448.0)


def test_norm_of_a_zero_row_keeps_scale_one():
    got = D.add_rms_norm(np.zeros((2, 130)), np.ones(130), None, 1e-6, "token")
    assert (got["scale"] == 1).all() and (got["y8"] == 0).all()


@pytest.mark.parametrize("act", ["identity", "swiglu", "geglu", "relu2", "gelu", "relu", "silu"])
def test_linear_against_torch(act):
    r = np.random.default_rng(3)
    data = r.integers(0, 256, (24, 80), dtype=np.uint8)
    sf = r.integers(0, 127, (24, 10), dtype=np.uint8)
    x = r.normal(size=(3, 160))
    scale = r.random((3, 2)) + 0.5
    out, y, mass = D.linear(x, data, sf, 2.0 ** -9, act, scale)
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)
    w = torch.zeros(24, 160, dtype=torch.float64)
    for n in range(24):
        for k in range(160):
            s = torch.tensor([int(sf[n, k // 16])], dtype=torch.uint8).view(torch.float8_e4m3fn).double()
            w[n, k] = table[(int(data[n, k // 2]) >> (4 * (k % 2))) & 15] * s
    xs = torch.tensor(x * np.concatenate([np.repeat(scale[:, :1], 128, 1), np.repeat(scale[:, 1:], 32, 1)], 1))
    z = xs @ w.T * 2.0 ** -9
    np.testing.assert_allclose(y, z.numpy(), rtol=1e-12, atol=1e-12)
    g, u = (z[:, :12], z[:, 12:]) if act in ("swiglu", "geglu") else (z, None)
    fn = torch.nn.functional
    want = {"identity": lambda: g, "swiglu": lambda: fn.silu(g) * u, "geglu": lambda: fn.gelu(g) * u,
            "relu2": lambda: fn.relu(g) ** 2, "gelu": lambda: fn.gelu(g), "relu": lambda: fn.relu(g),
            "silu": lambda: fn.silu(g)}[act]()
    np.testing.assert_allclose(out, want.numpy(), rtol=1e-11, atol=1e-12)
    assert (np.abs(y) <= mass * (1 + 1e-12)).all()


def test_kv_encode_holds_exact_values_and_bounds_the_rest():
    grid = np.concatenate([F.E2M1_MAGNITUDES, -F.E2M1_MAGNITUDES]).astype(np.float32)
    _, _, held = D.kv_encode(np.stack([grid, 4 * grid]), 1.0)
    np.testing.assert_array_equal(held, np.stack([grid, 4 * grid]))
    x = np.random.default_rng(1).normal(size=(50, 64)).astype(np.float32)
    data, sf, held = D.kv_encode(x, 2.5)
    assert data.shape == (50, 32) and sf.shape == (50, 4)
    # the block's scale is within 1/16 of amax / 6, the step at the top of the code is 1/3 of its value
    amax = np.repeat(np.abs(x.reshape(50, 4, 16)).max(-1), 16, -1)
    assert (np.abs(held - x) <= amax * (1 / 6 + 1 / 16 + 1e-6)).all()


@pytest.mark.parametrize("T,n", [(1, 1), (1, 9), (3, 2), (4, 11), (2, 0)])
def test_attend_against_torch(T, n):
    r = np.random.default_rng(T * 100 + n)
    q, k, v = r.normal(size=(T, 3, 16)), r.normal(size=(n, 16)), r.normal(size=(n, 16))
    out, lse, mass = D.attend(q, k, v, 0.3)
    for t in range(T):
        seen = n - (T - 1) + t
        if seen <= 0:
            assert (out[t] == 0).all() and (lse[t] == -np.inf).all()
            continue
        want = torch.nn.functional.scaled_dot_product_attention(
            torch.tensor(q[t][None]), torch.tensor(k[None, :seen]), torch.tensor(v[None, :seen]), scale=0.3)[0].numpy()
        np.testing.assert_allclose(out[t], want, rtol=1e-12, atol=1e-14)
        np.testing.assert_allclose(lse[t], torch.logsumexp(torch.tensor(q[t] @ k[:seen].T * 0.3), -1).numpy(), rtol=1e-12)
        assert (np.abs(out[t]) <= mass[t] + 1e-14).all()
