"""Pins of the cache oracle: values worked by hand and properties the definitions fix."""
import numpy as np
import pytest

from oracle import cache_oracle as co
from oracle import specdec_oracle as so


def test_e4m3_table_and_rounding():
    v = co.e4m3_values()
    assert v[0] == 0 and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6 and v[126] == 448 and (np.diff(v) > 0).all()
    assert co.to_e4m3(1.0) == 0x38 and co.to_e4m3(1e9) == 126
    assert co.to_e4m3(1.0625) == 0x38 and co.to_e4m3(1.1875) == 0x3a  # ties: between bytes 38|39 and 39|3a
    assert co.to_e4m3(2.0 ** -10) == 0 and co.to_e4m3(2.0 ** -10 * 1.01) == 1


def test_group_ties_go_to_the_even_code():
    x = np.array([6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25] + [-v for v in (6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25)], np.float32)
    codes, byte = co.quantise_group(x, 1.0)
    assert byte == 0x38
    assert codes.tolist() == [7, 6, 6, 4, 4, 2, 2, 0, 15, 14, 14, 12, 12, 10, 10, 8]


def test_group_extremes():
    z = np.zeros(16, np.float32)
    assert co.quantise_group(z, 1.0)[1] == 0
    for bad in (np.inf, -np.inf, np.nan):
        z[3] = bad
        codes, byte = co.quantise_group(z, 1.0)
        assert byte == 127 and not codes.any()
    codes, byte = co.quantise_group(np.full(16, 1e30, np.float32), 1.0)
    assert byte == 126 and (codes == 7).all()
    packed = codes[0::2] | (codes[1::2] << 4)
    assert (co.dequantise(packed, [byte], 0.5) == 2688 * 0.5).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_length_and_relative_angle(interleaved):
    rng = np.random.default_rng(3)
    q, k = rng.standard_normal(64), rng.standard_normal(64)
    f = 1e4 ** (-np.arange(16) / 16.0)
    a = co.rotate(q, 1000, f, interleaved=interleaved) @ co.rotate(k, 990, f, interleaved=interleaved)
    b = co.rotate(q, 110, f, interleaved=interleaved) @ co.rotate(k, 100, f, interleaved=interleaved)
    assert abs(a - b) < 1e-11
    assert np.array_equal(co.rotate(q, 77, f, interleaved=interleaved)[32:], q[32:])
    y = co.rotate(q, 5, f, weight=np.ones(64), eps=0.0)
    assert abs((y * y).mean() - 1) < 1e-12


def test_visible_matches_the_tree_mask_builder_and_the_window():
    parents = [-1, 0, 0, 1, -1, 3]
    mask, pos, _ = so.build_tree_mask(parents, 4)
    inner, depth, _ = so.build_tree_mask(parents, 0)
    sees = co.visible(6, 6, 10, 0, 0, inner, depth)
    assert np.array_equal(sees, np.asarray(mask).astype(bool))
    w = co.visible(3, 2, 9, 3, 2)  # queries at positions 7 and 8; a third does not exist
    assert np.flatnonzero(w[0]).tolist() == [0, 1, 5, 6, 7]
    assert np.flatnonzero(w[1]).tolist() == [0, 1, 6, 7, 8]
    assert not w[2].any()


def test_attention_of_equal_scores_is_the_mean():
    v = np.arange(12.0).reshape(4, 1, 3)
    out, lse, *_ = co.attend(np.zeros((1, 2, 3)), np.ones((4, 1, 3)), v, np.array([[1, 0, 1, 1]], bool), 1.0)
    assert np.allclose(out[0, 0], v[[0, 2, 3], 0].mean(0)) and np.allclose(lse, np.log(3))
