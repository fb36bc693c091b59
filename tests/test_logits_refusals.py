"""The logits calls refuse what they cannot run, on the host and before any launch (no GPU)."""
import pytest

from test_cache_refusals import _fake


@pytest.fixture(scope="module")
def sd(built_library):
    import speculative_decoding_token_temperature_gb300 as m
    m.load_library()
    return m


ORDER = ("logits", "dt", "tokens", "parents", "gammas", "counts", "rep", "pres", "freq", "bt", "bv", "K", "mask", "B", "rows", "V", "out",
         "status")


def _process(sd, a, **kw):
    d = dict(logits=a, dt=sd.BF16, tokens=a, parents=None, gammas=None, counts=a, rep=a, pres=a, freq=a, bt=a, bv=a, K=2, mask=a, B=1, rows=3,
             V=100, out=a, status=None)
    d.update(kw)
    return sd.load_library().specdec_process_logits(*(d[k] for k in ORDER), None)


@pytest.mark.parametrize("change,code", [
    (dict(logits=None), 1), (dict(out=None), 1), (dict(dt=2), 1), (dict(dt=9), 1), (dict(B=0), 1), (dict(rows=0), 1), (dict(V=0), 1), (dict(V=-3), 1),
    (dict(K=-1), 1), (dict(bt=None), 1), (dict(bv=None), 1), (dict(B=70000), 2), (dict(rows=8193), 2), (dict(K=1 << 24), 2), (dict(V=2 ** 31 - 65536), 2),
])
def test_process_refuses_bad_arguments(sd, change, code):
    a, keep = _fake()
    assert _process(sd, a, **change) == code


def test_process_refuses_mixed_and_misaligned(sd):
    a, keep = _fake()
    assert _process(sd, a, parents=a, tokens=None) == 1
    assert _process(sd, a, parents=a, gammas=a) == 1
    assert _process(sd, a, logits=a + 1) == 2
    assert _process(sd, a, out=a + 2, dt=sd.F32) == 2
    assert _process(sd, a, mask=a + 2) == 2


@pytest.mark.parametrize("shift", [-600, -4, 4, 300, 596])
def test_process_refuses_outputs_that_overlap_the_logits(sd, shift):
    a, keep = _fake()  # 3 rows of 100 bfloat16: 600 bytes
    assert _process(sd, a, out=a + shift, B=0) == 1
    if abs(shift) < 600:
        assert _process(sd, a, out=a + shift) == 1
        assert "lie apart" in sd.load_library().specdec_last_error().decode()


@pytest.mark.parametrize("change,code", [(dict(counts=None), 1), (dict(tokens=None), 1), (dict(B=0), 1), (dict(n=-1), 1), (dict(V=0), 1), (dict(stride=-1), 1),
                                         (dict(B=70000), 2), (dict(V=2 ** 31 - 65536), 2), (dict(n=2 ** 31 - 65536), 2)])
def test_count_refuses_bad_arguments(sd, change, code):
    a, keep = _fake()
    d = dict(counts=a, tokens=a, stride=4, num=None, B=1, n=4, V=10, prompt=0, reset=0, status=None)
    d.update(change)
    assert sd.load_library().specdec_count_tokens(*(d[k] for k in ("counts", "tokens", "stride", "num", "B", "n", "V", "prompt", "reset", "status")),
                                                  None) == code


def test_binding_refuses_host_tensors_and_wrong_shapes(sd):
    import torch
    x = torch.zeros(2, 3, 50)
    for call in (lambda: sd.process_logits(x), lambda: sd.process_logits(x.half()), lambda: sd.process_logits(x[0]),
                 lambda: sd.process_logits(x.transpose(1, 2)),
                 lambda: sd.count_tokens(torch.zeros(2, 50, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int32)),
                 lambda: sd.count_tokens(torch.zeros(50, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int32))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        sd.process_logits([1.0])
