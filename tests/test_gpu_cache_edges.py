"""The cache calls at the edges of their contracts: values that are not finite, scales and weights
next to 0, the widest windows, arguments without a truth value, workspaces.

Tolerances are those of test_gpu_cache.py unless a test derives its own.
"""
import numpy as np
import pytest
import torch

import test_gpu_cache as base
from oracle import cache_oracle as co

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def sd(built_library):
    import speculative_decoding_token_temperature_gb300 as m
    m.load_library()
    return m


@pytest.fixture(params=["rule", "warp", "tensor_memory"])
def kernel(request, hooks):
    """Each case through the kernel that the rule picks, and through each kernel."""
    hooks(attend_kernel=("rule", "warp", "tensor_memory").index(request.param))
    return request.param


def _same_places(r, c, q, lens, dtype, D, **mask):
    """Finite outputs as the oracle's, and the others at the oracle's places (an infinity may come out as NaN:
    0 times it is)."""
    for b, L in enumerate(lens):
        n = q.shape[1]
        k, v = c.rows(b, L)
        out, lse, pv, av, qk = co.attend(base._np(q[b]), k, v, co.visible(n, n, L, mask.get("window", 0), mask.get("sinks", 0)), D ** -0.5)
        odd = ~np.isfinite(out)
        got = r["out"][b].clone()
        assert np.array_equal(~np.isfinite(base._np(got)), odd), (b, np.argwhere(~np.isfinite(base._np(got)) != odd)[:4])
        got[torch.tensor(odd, device=DEV)] = 0
        out[odd] = pv[odd] = av[odd] = 0
        base._check(got, r["lse"][b], (out, lse, pv, av, qk), dtype, c.four, D, f"b={b}")


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("D,dtype", [(64, F16), (128, BF16)])
@pytest.mark.parametrize("n", [33, 64, 300])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 0), (70, 3), (600, 20)])
def test_odd_values_under_two_row_tiles(sd, four, D, dtype, n, window, sinks):
    """More than 128 query rows to a key head: two row tiles share the staged values, and a tile of slots may
    be whole for one and partial for the other.  Every request holds one such value: seen by all rows, by the
    later ones, by the earlier ones (a window's low edge), or as one of the first slots."""
    first = [100, 100, 127, 250, 5, 640, 400, 700]
    slots = [5, 104, 127 + n // 2, 130, 0, 640 + n - 2, 400 + n // 2 - 140, 2]
    lens = [p + n for p in first]
    c = base.Cache(len(lens), max(lens), 16, 1, D, dtype, four)
    for b, s in enumerate(slots):
        if four:
            c.vs[int(c.host_table[b, s // 16]), s % 16, :, b % (D // 16)] = 0x7f
        else:
            c.put("v", b, s, float("inf") if b % 3 == 1 else float("nan"))
    q = base._q(len(lens), n, 4, D, dtype)
    for _ in range(3):
        r = sd.attend(q, c.k, c.v, c.table, base._i32(lens), window=window, sinks=sinks, with_lse=True, **c.kw)
        torch.cuda.synchronize()
        assert not r["status"].any()
        _same_places(r, c, q, lens, dtype, D, window=window, sinks=sinks)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [2, 7, 20, 40])
@pytest.mark.parametrize("scale", [0.0, 1e-44, -1e-44, 1e-38])
def test_scales_next_to_zero_over_four_bit_pages(sd, kernel, D, n, scale):
    """bf16 queries below 1, whose rows carry a power of two below 1 of their own: its product with the scale
    may vanish, and masked slots stay masked."""
    c = base.Cache(2, 300, 16, 1, D, BF16, True)
    base._run(sd, c, base._q(2, n, 4, D, BF16, std=0.1), [n, 299], BF16, D, scale=scale)
