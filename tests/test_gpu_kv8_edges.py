"""More of attention over 8-bit pages against the fp64 oracle: codes of NaN where a stage of copies is filled again, and how far
queries are held."""
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


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F16, 64)])
@pytest.mark.parametrize("n", [3, 8, 16])
def test_codes_of_nan_in_stages_that_are_filled_again(sd, kernel, dtype, D, n):
    """At a window's border and among the first slots some rows see a value of NaN and others do not, so that its code is looked for
    lane by lane; the window's later slots are copied to the same places of shared memory many times over.  Every row as the formula
    has it, and every time the same bits."""
    window, sinks, B = 9000, 5, 4
    lens = [n + 16 * b + 10000 + 777 * b for b in range(B)]
    c = kv8.Cache(B, max(lens), 64, 32, 1, D, seed=n)
    for b, L in enumerate(lens):
        border = L - n - window + 1  # row i sees slots from border + i on
        for i in range(0, n, 2):
            c.v.view(torch.uint8)[int(c.host_table[b, (border + i) // 64]), (border + i) % 64, :, (11 * i) % D] = 0x7f
        c.put("v", b, sinks, 0xff)      # the first slot that nobody sees
        c.put("v", b, L - 1 - n // 2, 0x7f)
    q = base._q(B, n, 1, D, dtype)
    want = base._run(sd, c, q, lens, dtype, D, window=window, sinks=sinks, scale=0.05)
    for _ in range(10):
        r = sd.attend(q, c.k, c.v, c.table, base._i32(lens), window=window, sinks=sinks, scale=0.05, with_lse=True, **c.kw)
        torch.cuda.synchronize()
        assert torch.equal(r["out"].view(torch.int16), want["out"].view(torch.int16)) and torch.equal(r["lse"].view(torch.int32), want["lse"].view(torch.int32))


@pytest.mark.parametrize("dtype,small", [(BF16, 2.0 ** -10 * (1 + 2.0 ** -7)), (F16, 2.0 ** -7 * (1 + 2.0 ** -10))])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,n", [(1, 3), (2, 8), (4, 8), (3, 20), (5, 31)])
def test_which_kernels_hold_queries_whole(sd, kernel, dtype, small, D, G, n):
    """Queries of one large value, which meets keys of zero, and of values whose last bit E4M3 pieces cannot hold, which meet keys of
    ones: what is lost of each adds up.  With 17 to 32 rows to a key head in tensor memory a value may be off by 2^-17 of the row's largest,
    so a score by D 2^-17 scale max|q| |k|, and lse with it; everywhere else lse is as exact as fp32 sums of the whole values
    (the values are exact in fp16 relative to the row's largest).  No weight depends on it: all scores of a row are the same."""
    B, hkv, L, most = 2, 2, 300, 64.0
    c = kv8.Cache(B, L, 64, 32, hkv, D, seed=n, exps=(0, 0))
    c.k.view(torch.uint8).fill_(0x38)  # 1
    c.k.view(torch.uint8)[..., 0] = 0
    q = torch.full((B, n, hkv * G, D), most * small, device=base.DEV).to(dtype)
    q[..., 0] = most
    assert float(q[0, 0, 0, 1]) == most * small  # exact in the type
    lens, scale, k = [L, L - 7], 0.5, c.kw["k_scale"]
    r = sd.attend(q, c.k, c.v, c.table, base._i32(lens), scale=scale, with_lse=True, **c.kw)
    torch.cuda.synchronize()
    assert not r["status"].any()
    score = scale * (D - 1) * most * small * k
    pieces = kernel == "tensor_memory" and n * G <= 32
    for b, length in enumerate(lens):
        want = score + torch.log(torch.arange(length - n + 1, length + 1, dtype=torch.float64))[:, None]
        off = (r["lse"][b].double().cpu() - want).abs().max().item()
        exact = D * 2.0 ** -24 * score + 2.0 ** -13 + 2.0 ** -22 * float(want.max())
        assert off <= exact + (scale * D * 2.0 ** -17 * most * k if pieces else 0.0), (off, exact)
