"""The comparison that smoke() makes of processed logits notices a value that should be finite and is not."""
import warnings

import numpy as np
import pytest

import __graft_entry__ as entry

WANT = np.array([[1.0, -np.inf, 2.0], [np.nan, np.inf, -3.0]])


def test_equal_and_near_values_agree():
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        assert entry.agree(WANT, WANT, 1e-5) and entry.agree(WANT + 1e-6, WANT, 1e-5)


@pytest.mark.parametrize("at,value", [((0, 0), np.nan), ((0, 0), np.inf), ((0, 0), -np.inf), ((0, 1), np.nan), ((0, 1), np.inf), ((0, 1), 0.0),
                                      ((1, 0), 0.0), ((1, 1), -np.inf), ((1, 2), -3.1)])
def test_other_values_do_not(at, value):
    got = WANT.copy()
    got[at] = value
    assert not entry.agree(got, WANT, 1e-5)
