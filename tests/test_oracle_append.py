"""Pins of the append oracle (CPU): its e4m3 rounding against torch's over
every code and midpoint, its scale rule, and its paging against a plain copy."""

import numpy as np
import torch

from oracle import append as oa


def test_e4m3_values_are_torchs():
    want = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(oa.e4m3_values(), want)


def test_rounding_to_e4m3_is_nearest_even():
    v = oa.e4m3_values()
    x = np.concatenate([v, (v[1:] + v[:-1]) / 2, np.nextafter((v[1:] + v[:-1]) / 2, 0), v * 1.01])
    x = x[x <= 448]
    want = torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).double().numpy()
    exact = x == x.astype(np.float32)
    np.testing.assert_array_equal(oa.to_e4m3(x)[exact], want[exact])
    assert oa.to_e4m3(np.array([1e9, -1e9])).tolist() == [448.0, -448.0]


def test_block_scale_is_the_smallest_power_of_two():
    for a in (448.0, 448.0001, 447.9, 1.0, 1.75, 1.7500001, 3e-5, 0.0):
        s = oa.block_scale(a, 120)
        assert a <= 448 * s and (s == 2.0 ** -24 or a > 448 * s / 2)
    assert oa.block_scale(1e9, 7) == 128.0


def test_appending_in_pieces_equals_appending_at_once_without_scales():
    rng = np.random.default_rng(1)
    k, v = rng.standard_normal((2, 50, 2, 8))
    tab = np.stack([np.cos(np.arange(64)[:, None] * [1, .1, .01, .001]),
                    np.sin(np.arange(64)[:, None] * [1, .1, .01, .001])], -1)
    pages = [3, 0, 2, 1]
    one, many = [rng.standard_normal((4, 2, 16, 8)) for _ in range(2)], None
    many = [x.copy() for x in one]
    oa.append(one[0], one[1], None, None, [(pages, 0, 50, 7)], k, v, tab)
    at = 0
    for n in (1, 15, 1, 16, 17):
        oa.append(many[0], many[1], None, None, [(pages, at, n, 7)], k[at:at + n], v[at:at + n], tab)
        at += n
    np.testing.assert_array_equal(one[0], many[0])
    np.testing.assert_array_equal(one[1], many[1])
    flat = one[1][pages].transpose(0, 2, 1, 3).reshape(64, 2, 8)
    np.testing.assert_array_equal(flat[:50], v)
    assert not flat[50:].any()
