"""The 8-bit cache's oracle: codes and rounding against torch's own e4m3 casts,
the exponent against its definition, the commit against a plain copy."""
import numpy as np
import pytest
import torch

import oracle as O


def test_code_values_are_e4m3():
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    got = O.kv8_values(codes.numpy()[None], np.array([127], np.uint8))[0]
    assert np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("sigma", [1e-30, 1e-3, 1.0, 3e4, 1e30])
def test_rounding_is_nearest_even(sigma):
    g = torch.Generator().manual_seed(1)
    x = torch.randn((64, 48), generator=g).mul(sigma)
    codes, scale = O.kv8_quantise(x.double().numpy())
    y = x.double().numpy() * 2.0 ** (127.0 - scale)[:, None]
    want = torch.from_numpy(y).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(codes, want)
    top = np.abs(x.double().numpy()).max(1)
    power = 2.0 ** (scale - 127.0)
    assert (top <= 448 * power).all() and (top > 224 * power).all()


def test_rounding_of_every_halfway_point():
    v = O.E4M3[:127]
    mid = (v[1:] + v[:-1]) / 2
    row = np.concatenate([mid, -mid, [448.0, -448.0]])
    codes, scale = O.kv8_quantise(row[None])
    assert scale[0] == 127
    want = torch.from_numpy(row).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(codes[0], want)


def test_exponents_at_their_borders():
    for k in (-100, -3, 0, 7, 100):
        for top, s in ((448.0, k + 127), (448.0 + 2.0 ** -40, k + 128), (224.0, k + 126), (224.0 + 2.0 ** -40, k + 127)):
            assert O.kv8_quantise(np.array([[top * 2.0 ** k, 0.0]]))[1][0] == s
    for row, s in (([0.0, 0.0], 1), ([2.0 ** -140, 0.0], 1), ([np.inf, 1.0], 255), ([1.0, np.nan], 255)):
        codes, scale = O.kv8_quantise(np.array([row]))
        assert scale[0] == s and not codes.any()
    assert np.isnan(O.kv8_values(np.zeros((1, 2)), np.array([255]))).all()


def test_commit_of_a_path():
    rng = np.random.default_rng(0)
    codes = rng.integers(0, 127, (2, 2, 9, 4, 3, 16)).astype(np.uint8)
    scale = rng.integers(1, 255, (2, 2, 9, 3, 4)).astype(np.uint8)
    table, before, sbefore = np.array([8, 1, 5, 2]), codes.copy(), scale.copy()
    assert O.kv8_commit(codes, scale, table, 4, 6, [0, 2, 3, 7], 8) == 10
    at = lambda c: (table[c // 4], c % 4)  # noqa: E731
    for i, s in enumerate([0, 2, 3, 7]):
        (a, x), (b, y) = at(6 + i), at(6 + s)
        assert np.array_equal(codes[:, :, a, x], before[:, :, b, y])
        assert np.array_equal(scale[:, :, a, :, x], sbefore[:, :, b, :, y])
    rest = [c for c in range(16) if not 6 <= c < 10]
    assert all(np.array_equal(codes[:, :, at(c)[0], at(c)[1]], before[:, :, at(c)[0], at(c)[1]]) for c in rest)
    for bad in ([0, 0], [1, 0], [0, 8], [-1, 2]):
        assert O.kv8_commit(codes, scale, table, 4, 6, bad, 8) is None
    assert O.kv8_commit(codes, scale, table, 4, 14, [0, 1, 2], 8) is None
    assert O.kv8_commit(codes, scale, table, 4, 12, [0, 5], 8) is None
    assert O.kv8_commit(codes, scale, np.array([8, 9, 5, 2]), 4, 5, [0, 2], 8) is None
    assert O.kv8_commit(codes, scale, table, 4, 6, [], 8) == 6
