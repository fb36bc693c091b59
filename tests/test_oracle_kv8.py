"""The oracle of the 8-bit pages and of the logits' processing against independent statements of the same (CPU)."""
import numpy as np
import torch

from oracle import cache_oracle as co
from oracle import logits_oracle as lo


def test_codes_are_those_of_the_type():
    bytes_ = torch.arange(256, dtype=torch.uint8)
    want = bytes_.view(torch.float8_e4m3fn).double().numpy()
    got = co.decode8(bytes_.numpy(), 0)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])
    rng = np.random.default_rng(0)
    x = np.concatenate((rng.normal(0, 100, 5000), rng.normal(0, 0.02, 5000), np.arange(0, 448, 0.5), np.arange(0, 0.1, 2.0 ** -11))).astype(np.float32)
    x = np.clip(np.concatenate((x, -x)), -448, 448)
    want = torch.tensor(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(co.encode8(x.astype(np.float64), 0), want)
    assert np.array_equal(co.encode8(x.astype(np.float64) * 8, 3), want)


def test_exponents():
    assert [co.block_exponent(a) for a in (0.0, 448 * 2.0 ** -15, 448 * 2.0 ** -15 * 1.0001, 448.0, 448.1, 1.0, 57344.0, 1e9)] == [-15, -15, -14, 0, 1, -8, 7, 7]


def test_a_growing_block_keeps_its_values():
    rng = np.random.default_rng(1)
    codes, exps = np.full((32, 8), 55, np.uint8), np.full(2, 3)
    x = rng.normal(0, 1, (20, 8)).astype(np.float32)
    codes, exps = co.append8(codes, exps, x[:5], 0, 16, 1.0)
    before = co.decode8(codes[:5], exps[0])
    codes, exps = co.append8(codes, exps, x[5:] * 64, 5, 16, 1.0)
    after = co.decode8(codes[:5], exps[0])
    assert exps[0] > co.block_exponent(np.abs(x[:5]).max())
    assert (np.abs(after - before) <= np.maximum(0, 2.0 ** (exps[0] - 10))).all() and (codes[20:] == 55).all()


def test_rows_follow_their_path():
    assert lo.paths(3) == [[], [0], [0, 1], [0, 1, 2]]
    assert lo.paths(4, [-1, 0, 0, 2]) == [[], [0], [0, 1], [0, 2], [0, 2, 3]]


def test_penalties_by_hand():
    out, _ = lo.process(np.array([[2.0, -2.0, 4.0, 1.0], [2.0, -2.0, 4.0, 1.0]]), tokens=[3], counts=np.array([1, -2 ** 31, 0, 0]), repetition=2.0, presence=0.5,
                        frequency=0.25, bias=[(2, 10.0)])
    assert out.tolist() == [[1.0 - 0.75, -4.0, 14.0, 1.0], [1.0 - 0.75, -4.0, 14.0, 0.5 - 0.75]]
