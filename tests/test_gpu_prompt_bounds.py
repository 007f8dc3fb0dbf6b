"""GPU test of prompt attention with a bound of no queries: sequences that have some are reported and
not computed; where there are none, nothing is written or reported."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("starts,flagged", [([0, 3, 20], True), ([0, 0, 20], True), ([0, 0, 0], False),
                                            ([7, 7, 7], False)])
@pytest.mark.parametrize("max_key", [0, 20, 5000])
def test_no_queries_expected(pa, cuda_device, starts, flagged, max_key):
    q = torch.randn(20, 8, 128, device="cuda").bfloat16()
    k = torch.randn(20, 2, 128, device="cuda").bfloat16()
    out = torch.full_like(q, 7.0)
    qs = torch.tensor(starts, dtype=torch.int32, device="cuda")
    ks = torch.zeros(3, dtype=torch.int32, device="cuda") if max_key == 0 else qs
    assert pa.lib().pa_prompt_attention_workspace_bytes(2, 20, 8, 2, 128, 0, max_key) == 0
    pa.pa_prompt_attention(out, q, k, k, qs, ks, 0.1, 2, 0, max_key)
    assert pa.pa_device_error(clear=True) == (pa.DEVERR["context_len"] if flagged else 0)
    assert (out == 7).all()
