"""Pins of the float64 oracle of the 8-bit frame cache (CPU)."""
import math

import numpy as np
import pytest
import torch

from oracle import cache as C


def test_e4m3_rounding_is_torchs_on_a_dense_sweep():
    x = np.concatenate([np.linspace(-448, 448, 40001), np.ldexp(np.linspace(-2, 2, 4001), -6), [0.0, -0.0]])
    ref = torch.from_numpy(x).float().to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(C.e4m3_round(x.astype(np.float32)), ref)


def test_e4m3_values_are_fixed_points_and_midpoints_go_to_even():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    codes = codes[np.isfinite(codes)]
    np.testing.assert_array_equal(C.e4m3_round(codes), codes)
    pos = np.unique(codes[codes >= 0])
    mid = C.e4m3_round((pos[:-1] + pos[1:]) / 2)
    even = np.where(np.arange(len(pos) - 1) % 2 == 0, pos[:-1], pos[1:])  # codes are ordered: even code = even index
    np.testing.assert_array_equal(mid, even)


@pytest.mark.parametrize("top,e", [(448.0, 0), (449.0, 1), (1.75, -8), (1.7578125, -7), (0.0, -124),
                                   (math.ldexp(1.0, -133), -124), (math.ldexp(255.0, 120), 119), (896.0, 1), (897.0, 2)])
def test_block_exponent_by_hand(top, e):
    assert int(C.block_exponent(np.array(top))) == e


def test_quantise_error_is_half_a_step():
    g = np.random.default_rng(0)
    x = (g.standard_normal((50, 128)) * np.exp(3 * g.standard_normal((50, 1))))
    codes, e = C.quantise(x)
    back = C.dequantise(codes, e)
    step = np.ldexp(1.0, np.repeat(e, 32, -1))
    # half a step of 4 significant bits, or half of 2^-9 in the subnormal range
    assert (np.abs(back - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * step)).all()
    assert np.abs(codes).max() <= 448
    tops = np.abs(codes.reshape(50, 4, 32)).max(-1)
    assert ((tops > 224 * (1 - 2.0 ** -4))).all()  # no smaller power of two would do


def test_norm_rope_invariants():
    g = np.random.default_rng(1)
    x = g.standard_normal((2, 3, 5, 64))
    pos = g.integers(-50, 1000, (2, 5, 2))
    f = 10000.0 ** (-np.arange(24) / 24)
    for layout in ("interleaved", "half"):
        y, _ = C.norm_rope(x, positions=pos, inv_freq=f, axis_pairs=(8, 16), layout=layout)
        np.testing.assert_allclose((y ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-12)  # a rotation
        np.testing.assert_array_equal(y[..., 48:], x[..., 48:])
        back, _ = C.norm_rope(y, positions=-pos, inv_freq=f, axis_pairs=(8, 16), layout=layout)
        np.testing.assert_allclose(back, x, atol=1e-12)
    # dot products depend on the difference of positions alone
    q, k = x[:1, :1], x[1:, :1]
    dots = []
    for shift in (0, 31):
        a, _ = C.norm_rope(q, positions=pos[:1] + shift, inv_freq=f, axis_pairs=(8, 16))
        b, _ = C.norm_rope(k, positions=pos[1:] + shift, inv_freq=f, axis_pairs=(8, 16))
        dots.append((a * b).sum(-1))
    np.testing.assert_allclose(dots[0], dots[1], atol=1e-11)
    y, _ = C.norm_rope(x, eps=0.0)
    np.testing.assert_allclose((y ** 2).mean(-1), 1.0, rtol=1e-12)
    # a complex product, pair by pair
    z = x[0, 0, 0, 0:48:2] + 1j * x[0, 0, 0, 1:48:2]
    axis = np.repeat([0, 1], [8, 16])
    z = z * np.exp(1j * pos[0, 0][axis] * f)
    y, _ = C.norm_rope(x, positions=pos, inv_freq=f, axis_pairs=(8, 16))
    np.testing.assert_allclose(y[0, 0, 0, 0:48:2] + 1j * y[0, 0, 0, 1:48:2], z, atol=1e-12)


@pytest.mark.parametrize("L,n,causal", [(3, 7, False), (3, 7, True), (5, 2, True), (4, 0, False), (1, 1, True)])
def test_attention_against_library(L, n, causal):
    g = np.random.default_rng(2)
    q, k, v = g.standard_normal((L, 64)), g.standard_normal((n, 64)), g.standard_normal((n, 64))
    o, lse, _ = C.attention(q, k, v, 0.125, causal)
    for i in range(L):
        m = max(0, n - L + i + 1) if causal else n
        if m == 0:
            assert (o[i] == 0).all() and lse[i] == -np.inf
            continue
        t = torch.from_numpy(0.125 * (k[:m] @ q[i]))
        np.testing.assert_allclose(lse[i], torch.logsumexp(t, 0).item(), atol=1e-12)
        np.testing.assert_allclose(o[i], (torch.softmax(t, 0) @ torch.from_numpy(v[:m])).numpy(), atol=1e-12)
