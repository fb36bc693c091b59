"""The repetition penalty alone: the quotient (or product) itself, in fp32.

With no presence, frequency or bias a repeated token's logit is x / r rounded to fp32 once (x * r where x is not positive), bit for
bit, whatever r: torch's division and multiplication of fp32 numbers round to nearest, and so do the kernel's.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def sd(built_library):
    import speculative_decoding_token_temperature_gb300 as m
    m.load_library()
    return m


@pytest.mark.parametrize("r", [1.0, 1.3, 1.1, 0.7, 3.0, 2.0 ** -99, 2.0 ** 99, 1.7 * 2.0 ** 100, 1.3 * 2.0 ** 120, 1.1 * 2.0 ** -126, 1e-40, 3e38])
@pytest.mark.parametrize("V", [4096, 4099])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quotients_are_rounded_once(sd, r, V, dtype):
    B, rows = 2, 5
    g = torch.Generator().manual_seed(V)
    x = ((torch.rand(B, rows, V, generator=g) - 0.4) * 30).to(dtype).to(DEV)
    x[:, :, ::7] *= 2.0 ** -60
    x[:, :, 1::7] *= 2.0 ** 60
    x[:, :, 2::70], x[:, :, 3::70], x[:, :, 4::70] = float("inf"), float("-inf"), 0.0
    counts = (torch.rand(B, V, generator=g) < 0.5).int().to(DEV)
    counts[:, ::5] = -2 ** 31  # in the prompt
    tokens = torch.randint(0, V, (B, rows - 1), generator=g, dtype=torch.int32).to(DEV)
    counts.scatter_(1, tokens[:, :2].long(), 0)  # drafts that were not there before
    rep = torch.full((B,), r, device=DEV)
    got = sd.process_logits(x, tokens=tokens, counts=counts, repetition=rep)
    torch.cuda.synchronize()
    assert not got["status"].any()
    seen = (counts != 0)[:, None].expand(B, rows, V).clone()
    for i in range(rows):
        for j in range(i):
            seen[torch.arange(B), i, tokens[:, j].long()] = True
    f = x.float()
    want = torch.where(seen, torch.where(f > 0, f / rep[0], f * rep[0]), f).to(dtype)
    assert torch.equal(got["logits"], want)
