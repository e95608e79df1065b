"""Pins of the int8 and group norm oracle: closed forms, brute force, torch's own group norm."""
import numpy as np
import pytest
import torch

from oracle import int8 as O


def test_codes_round_trip_and_extremes():
    # integers up to 127 with 127 present: scale 1 (127 / 127), codes the integers themselves
    x = np.array([[127, -127, 0, 5, -64, 1, 2, 3]], dtype=np.float32)
    q, s = O.quantize_rows(x)
    assert s[0] == 1.0 and np.array_equal(q[0], x[0].astype(np.int8))
    # ties go to the even code
    q, _ = O.quantize_rows(np.array([[127, 0.5, 1.5, 2.5, -0.5, -1.5]], dtype=np.float32))
    assert q[0].tolist() == [127, 0, 2, 2, 0, -2]


def test_zero_tiny_and_non_finite_rows():
    x = np.array([[0, 0], [2.0 ** -101, 0], [2.0 ** -100, 0], [np.inf, 1], [np.nan, 1]], dtype=np.float32)
    q, s = O.quantize_rows(x)
    assert s[0] == 0 and s[1] == 0 and s[2] > 0 and np.isnan(s[3]) and np.isnan(s[4])
    assert q[2, 0] == 127 and not q[[0, 1, 3, 4]].any()


def test_quantization_error_is_at_most_half_a_step():
    x = np.random.default_rng(1).normal(size=(50, 64)).astype(np.float32)
    q, s = O.quantize_rows(x)
    # half a step, and the roundings of 127 / a, of the product and of the scale (127 steps of 2^-22)
    assert np.all(np.abs(q * s[:, None].astype(np.float64) - x) <= s[:, None] * (0.5 + 127 * 2.0 ** -22))


def test_linear_is_the_brute_force_sum():
    r = np.random.default_rng(2)
    xq, wq = r.integers(-127, 128, (3, 16)).astype(np.int8), r.integers(-127, 128, (5, 16)).astype(np.int8)
    sx, sw, b = r.random(3).astype(np.float32), r.random(5).astype(np.float32), r.normal(size=5)
    y = O.linear(xq, sx, wq, sw, b)
    for m in range(3):
        for n in range(5):
            acc = sum(int(xq[m, k]) * int(wq[n, k]) for k in range(16))
            assert y[m, n] == acc * float(sx[m]) * float(sw[n]) + b[n]


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_group_norm_against_torch_float64(act):
    r = np.random.default_rng(3)
    x, g, b = r.normal(size=(2, 7, 12)), r.normal(size=12), r.normal(size=12)
    t = torch.nn.functional.group_norm(torch.from_numpy(x).permute(0, 2, 1), 3, torch.from_numpy(g),
                                       torch.from_numpy(b), 1e-5).permute(0, 2, 1)
    t = torch.nn.functional.silu(t) if act == "silu" else \
        torch.nn.functional.gelu(t, approximate="tanh") if act == "gelu" else t
    assert np.allclose(O.group_norm(x, 3, g, b, 1e-5, act), t.numpy(), rtol=1e-12, atol=1e-12)


def test_smoothing_leaves_the_product_unchanged_and_helps_outliers():
    r = np.random.default_rng(4)
    X, W = r.normal(size=(64, 128)), r.normal(size=(128, 32))
    X[:, 5] *= 50
    s = np.sqrt(np.abs(X).max(0) / np.abs(W).max(1))
    assert np.allclose((X / s) @ (s[:, None] * W), X @ W)

    def err(scale):
        xq, sx = O.quantize_rows(O.smooth(X, 1.0 / scale))
        wq, sw = O.quantize_rows(np.ascontiguousarray((scale[:, None] * W).T).astype(np.float32))
        return np.linalg.norm(O.linear(xq, sx, wq, sw) - X @ W)

    assert err(s) < 0.7 * err(np.ones(128))
