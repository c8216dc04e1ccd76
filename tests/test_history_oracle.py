"""Pins of the cached-history oracle (CPU): the rotation against complex multiplication and its dependence on
position differences alone, gradients against central differences, the e4m3 rounding against the list of all
e4m3 numbers, and the attention's masks and head groups against closed forms."""
import numpy as np
import pytest
import torch

from oracle import history_oracle as H
from oracle import whale_oracle as O


@pytest.mark.parametrize("layout", [H.HALVES, H.ADJACENT])
@pytest.mark.parametrize("rot", [0, 4, 8])
def test_rotation_is_complex_multiplication(layout, rot):
    rng = np.random.default_rng(rot)
    x, g, pos = rng.standard_normal((5, 2, 8)), rng.uniform(0.5, 1.5, 8), np.array([0, 1, 7, -3, 100000])
    y = H.norm_rotate(x, g, pos, rot, 100.0, layout, 1e-6)
    n = O.rms_norm(x, g, 1e-6)
    assert np.array_equal(y[..., rot:], n[..., rot:])
    u, v = H.pair_columns(rot, layout)
    for i in range(rot // 2):
        z = (n[..., u[i]] + 1j * n[..., v[i]]) * np.exp(1j * pos * 100.0 ** (-2 * i / rot))[:, None]
        assert np.allclose(y[..., u[i]], z.real, atol=1e-12) and np.allclose(y[..., v[i]], z.imag, atol=1e-12)


def test_scores_depend_on_position_differences():
    rng = np.random.default_rng(1)
    q, k, g = rng.standard_normal((1, 1, 16)), rng.standard_normal((1, 1, 16)), np.ones(16)
    s = [float(np.sum(H.norm_rotate(q, g, [p + 5], 16, 1e4, H.HALVES, 0.0) *
                      H.norm_rotate(k, g, [p], 16, 1e4, H.HALVES, 0.0))) for p in (0, 3, 900)]
    assert np.ptp(s) < 1e-10


@pytest.mark.parametrize("layout", [H.HALVES, H.ADJACENT])
def test_gradients_against_differences(layout):
    rng = np.random.default_rng(2)
    x, g, pos = rng.standard_normal((3, 2, 8)), rng.uniform(0.5, 1.5, 8), np.array([0, 9, 1234])
    dy = rng.standard_normal(x.shape)
    f = lambda x, g: float(np.sum(dy * H.norm_rotate(x, g, pos, 4, 50.0, layout, 1e-3)))  # noqa: E731
    dx, dg = H.norm_rotate_backward(x, g, pos, 4, 50.0, layout, 1e-3, dy)
    h = 1e-6
    for arr, grad, call in ((x, dx, lambda a: f(a, g)), (g, dg, lambda a: f(x, a))):
        for i in np.ndindex(arr.shape):
            e = np.zeros_like(arr)
            e[i] = h
            assert abs((call(arr + e) - call(arr - e)) / (2 * h) - grad[i]) < 1e-7


def test_e4m3_rounding_against_every_number():
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
    every = np.unique(every[np.isfinite(every)])
    assert np.array_equal(H.e4m3_round(every), every)
    mid = (every[1:] + every[:-1]) / 2
    got = H.e4m3_round(np.concatenate([mid, mid * (1 + 1e-12), mid * (1 - 1e-12)]))
    assert np.isin(got, every).all()
    x = np.concatenate([mid, np.random.default_rng(0).uniform(-448, 448, 4000)])
    near = np.abs(x[:, None] - every[None]).min(1)
    assert np.allclose(np.abs(H.e4m3_round(x) - x), near, rtol=0, atol=1e-15)
    t = torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(H.e4m3_round(x.astype(np.float32)), t)


def test_quantise_takes_the_least_exponent():
    for amax, e in ((448.0, 0), (448.5, 1), (224.0, -1), (224.1, 0), (1.75, -8), (1.7501, -7), (0.0, 0), (1e-38, -100),
                    (3e38, 119)):
        x = np.zeros((1, 32))
        x[0, 3] = -amax
        x[0, 5] = amax / 3
        v, got = H.quantise(x)
        assert got[0] == e, (amax, got[0])
        assert np.abs(v).max() <= 448.0
        if E_fine := (-100 < e < 119):
            # half a step of a 4-bit number, and half the least step
            assert E_fine and np.all(np.abs(v * 2.0 ** e - x) <= 2.0 ** -4 * np.abs(x) + 2.0 ** (e - 10))


def test_attention_masks_and_groups():
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((3, 4, 8)), rng.standard_normal((5, 2, 8)), rng.standard_normal((5, 2, 8))
    a, _ = H.attention(q, k, v, False, 0)
    for h in range(4):
        assert np.allclose(a[:, h], O.cross_attention(q[:, h], k[:, h // 2], v[:, h // 2], 1))
    c, _ = H.attention(q, k, v, True, 2)                      # rows at positions 2, 3, 4
    assert np.allclose(c[2], a[2]) and np.allclose(c[0], H.attention(q[:1], k[:3], v[:3], False, 0)[0][0])
    n, _ = H.attention(q, k, v, True, -2)                     # positions -2, -1, 0: two empty rows, one of one key
    assert not n[:2].any() and np.allclose(n[2], np.repeat(v[0], 2, axis=0))
    assert not H.attention(q, k[:0], v[:0], False, 0)[0].any()
