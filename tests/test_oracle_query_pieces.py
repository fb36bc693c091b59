"""How far queries are held where attention over 8-bit pages takes them as sums of E4M3 codes (CPU): every significand of
every binade through the pieces, against what include/specdec.h says."""
import re
from pathlib import Path

import numpy as np
import pytest

from oracle import cache_oracle as co

TOP = 128.0  # a row's largest value is scaled into [TOP, 2 TOP)


def _left(x, pieces):
    for _ in range(pieces):
        x = x - co.decode8(co.encode8(x, 0), 0)
    return x


@pytest.mark.parametrize("name,bits,pieces", [("bf16", 8, 2), ("fp16", 11, 3)])
def test_values_that_are_exact(name, bits, pieces):
    header = (Path(__file__).resolve().parents[1] / "include" / "specdec.h").read_text()
    (bound,) = re.search(r"held to 2\^(-\d+) of a\s[ *]*row's largest value", header).groups()
    said = re.search(r"values from 2\^(-\d+) of it up in bf16, and from 2\^(-\d+) up in fp16, are exact", re.sub(r"\s\*\s", " ", header)).groups()[name == "fp16"]
    significands = 1 + np.arange(2 ** (bits - 1)) / 2.0 ** (bits - 1)
    exact = []
    for e in range(0, -30, -1):
        left = np.abs(_left(significands * TOP * 2.0 ** e, pieces))
        assert left.max() <= TOP * 2.0 ** int(bound)
        exact.append(not left.any())
    first = exact.index(False)  # the largest binade with a value that is not exact
    assert all(exact[:first]) and -(first - 1) == int(said)
