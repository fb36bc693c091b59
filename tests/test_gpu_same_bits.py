"""What a row's result may depend on: its own inputs, and nothing that a kernel finds where no row is.

Tiles of the attention kernels have room for more rows than a call has.  What lies there (an earlier call's queries, the queries of
tokens that a sequence does not have) must not reach a row that counts, not even in its last bit.
"""
import pytest
import torch

import test_gpu_cache as base
import test_gpu_kv8 as kv8

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def sd(built_library):
    import speculative_decoding_token_temperature_gb300 as m
    m.load_library()
    return m


@pytest.fixture(params=["warp", "tensor_memory"])
def kernel(request, hooks):
    hooks(attend_kernel=("rule", "warp", "tensor_memory").index(request.param))
    return request.param


def _cache(bits, B, L, hkv, D, dtype):
    if bits == 8:
        return kv8.Cache(B, L, 64, 32, hkv, D, seed=L, std=100.0, exps=(-6, -6))
    return base.Cache(B, L, 64, hkv, D, dtype, bits == 4, seed=L)


def _attend(sd, c, q, lens, nq=None):
    r = sd.attend(q, c.k, c.v, c.table, base._i32(lens), query_len=None if nq is None else base._i32(nq), scale=0.05, with_lse=True, **c.kw)
    torch.cuda.synchronize()
    assert not r["status"].any()
    return r


# query rows to a key head: a part of 8, 16, 32, 128 and 256 rows, the last warp of 32 in part
ROWS = [(3, 1), (5, 2), (5, 5), (10, 4), (31, 5)]


@pytest.mark.parametrize("bits,dtype", [(16, BF16), (16, F16), (8, BF16), (8, F16), (4, F16)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,G", ROWS)
def test_an_earlier_calls_queries_do_not_count(sd, kernel, bits, dtype, D, n, G):
    """The same call behind one of a whole tile of large queries, and behind one of zeros."""
    B, hkv, L = 40, 4, 1500
    c = _cache(bits, B, L, hkv, D, dtype)
    q, full = base._q(B, n, hkv * G, D, dtype), -(-n * G // 32) * 32
    lens = [L - 7 * b for b in range(B)]
    got = []
    for std in (0.0, 300.0, 3000.0):
        _attend(sd, c, base._q(B, full, hkv, D, dtype, seed=9, std=std), lens)  # rows past n * G among them
        got.append(_attend(sd, c, q, lens))
    for r in got[1:]:
        assert torch.equal(r["out"], got[0]["out"]) and torch.equal(r["lse"], got[0]["lse"])


@pytest.mark.parametrize("bits,dtype", [(16, BF16), (16, F16), (8, BF16), (8, F16), (4, F16)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,G", ROWS)
def test_queries_of_tokens_that_do_not_exist_do_not_count(sd, kernel, bits, dtype, D, n, G):
    """A batch padded to n tokens: what the padding's queries hold does not reach the others."""
    B, hkv, L = 20, 4, 1500
    c = _cache(bits, B, L, hkv, D, dtype)
    q = base._q(B, n, hkv * G, D, dtype)
    lens, nq = [L - 7 * b for b in range(B)], [n - 1 - b % (n - 1) for b in range(B)]
    got = []
    for std in (0.0, 300.0, 3000.0, float("nan")):
        x = q.clone()
        for b in range(B):
            x[b, nq[b]:] = base._q(1, n - nq[b], hkv * G, D, dtype, seed=b, std=std)[0]
        got.append(_attend(sd, c, x, lens, nq))
    for r in got[1:]:
        assert torch.equal(r["out"], got[0]["out"]) and torch.equal(r["lse"], got[0]["lse"])
