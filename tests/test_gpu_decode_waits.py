"""GPU test of the 16-bit decode's bounded waits at limits about as long as a copy takes, where some
of a call's waits run out and others do not: what ran out is reported, a call without a report is
whole, and so is the next call under the usual limit."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv,D,B", [(32, 8, 128, 16), (4, 4, 64, 32), (16, 1, 128, 32)])
def test_limits_about_a_copy_long(pa, cuda_device, Hq, Hkv, D, B):
    g = torch.Generator(device="cuda").manual_seed(D)
    n, S = 5000, 24
    NB = S * -(-n // B)
    k, v = (torch.randn(NB, Hkv, B, D, generator=g, device="cuda").half() for _ in range(2))
    tables = torch.randperm(NB, generator=g, device="cuda").int().view(S, -1)
    lens = torch.tensor([n - 200 * i for i in range(S)], dtype=torch.int32, device="cuda")
    q = torch.randn(S, Hq, D, generator=g, device="cuda").half()
    want, out = torch.empty(S, Hq, D, device="cuda"), torch.empty(S, Hq, D, device="cuda")
    call = (k, v, tables, lens, D ** -0.5, Hkv)
    pa.pa_paged_decode_attention(want, q, *call)
    assert pa.pa_device_error(clear=True) == 0
    ran_out = 0
    try:
        for limit in (1, 30, 100, 200, 400, 600, 800, 1000, 1500, 2000, 3000, 5000, 100000, 1000000):
            pa.pa_set_wait_limit(limit)
            for _ in range(4):
                pa.pa_paged_decode_attention(out, q, *call)
                flags = pa.pa_device_error(clear=True)
                assert flags in (0, pa.DEVERR["timeout"])
                ran_out += flags != 0
                assert flags or torch.equal(out, want)
    finally:
        pa.pa_set_wait_limit(0)
    assert ran_out > 0
    pa.pa_paged_decode_attention(out, q, *call)
    assert pa.pa_device_error(clear=True) == 0 and torch.equal(out, want)
