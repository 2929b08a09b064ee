"""The oracle of the rotated append against closed forms."""
import numpy as np
import pytest

from oracle import rope

import rope_helpers as rh


@pytest.mark.parametrize("pairs", ["halves", "adjacent"])
def test_a_rotation_is_the_complex_product(pairs):
    r = np.random.default_rng(3)
    x = r.standard_normal((5, 2, 48)).astype(np.float32).astype(np.float64)
    angle = r.uniform(-3, 3, (9, 16))
    table = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
    pos = r.integers(0, 9, (1, 5))
    y = rope.turned(x, 8, table, pos, [0] * 16, pairs)
    a, b = (slice(8, 24), slice(24, 40)) if pairs == "halves" else (slice(8, 40, 2), slice(9, 40, 2))
    z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * angle[pos[0]])[:, None]
    # three roundings to binary32 and those of cos and sin, values up to |z|
    assert np.abs(y[..., a] + 1j * y[..., b] - z).max() <= 8 * 2.0 ** -24 * np.abs(z).max()
    rest = np.r_[0:8, 40:48]
    assert (y[..., rest] == x[..., rest]).all()


def test_position_zero_leaves_rows_as_they_are_and_axes_are_taken_by_pair():
    p = rh.make(seed=1, seq_lens=[3], seq_lens_kv=[0], axes=3)
    x = np.random.default_rng(0).standard_normal((3, 1, 128)).astype(np.float32).astype(np.float64)
    same = rope.turned(x, 0, p.table, np.zeros((3, 3), int), p.pair_axis, "halves")
    assert (same == x).all()
    only = np.zeros((3, 3), int)
    only[1] = 4                                     # axis 1 alone moves: pairs 1, 4, 7, ...
    y = rope.turned(x, 0, p.table, only, p.pair_axis, "halves")
    moved = np.array([i % 3 == 1 for i in range(64)] * 2)
    assert (y[..., ~moved] == x[..., ~moved]).all() and (y[..., moved] != x[..., moved]).all()
