"""GPU tests of prompt attention over thousands of sequences: every sequence's rows are those that a
call of a few sequences gives, whatever mix of lengths stands around it, and the time of a call grows
with the number of sequences, not with its square."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def starts(lens):
    return torch.tensor(np.cumsum([0] + list(lens)), dtype=torch.int32, device="cuda")


def attend(pa, out, q, k, v, C, L, Hkv):
    return pa.pa_prompt_attention(out, q, k, v, starts(C), starts(L), 0.1, Hkv, max(C), max(L))


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 8, 64), (16, 4, 128)])
@pytest.mark.parametrize("kind", ["short", "mixed", "prefixes"])
def test_thousands_of_sequences(pa, cuda_device, Hq, Hkv, D, kind):
    r, S = np.random.default_rng(len(kind) + Hq), 2500
    C = r.integers(0, 40, S) if kind == "short" else np.exp(r.uniform(0, 6, S)).astype(int) - 1
    L = C + (r.integers(0, 3, S) * r.integers(0, 1500, S) if kind == "prefixes" else 0)
    L = np.maximum(L - (r.integers(0, 20, S) == 0) * r.integers(0, 30, S), 0)     # queries before the first key
    C, L = C.tolist(), L.tolist()
    g = torch.Generator(device="cuda").manual_seed(S)
    q, k, v = (torch.randn(n, h, D, generator=g, device="cuda").bfloat16()
               for n, h in ((sum(C), Hq), (sum(L), Hkv), (sum(L), Hkv)))
    out = attend(pa, torch.full_like(q, 7.0), q, k, v, C, L, Hkv)
    a, b = np.cumsum([0] + C), np.cumsum([0] + L)
    step = 125       # enough for whole units: a call whose keys are split sums them in another order
    for i in range(0, S, step):
        c, l = C[i:i + step], L[i:i + step]
        rows, keys = slice(a[i], a[i + step]), slice(b[i], b[i + step])
        need = pa.lib().pa_prompt_attention_workspace_bytes(step, sum(c), Hq, Hkv, D, max(c), max(l))
        assert need == 0
        want = attend(pa, torch.empty_like(q[rows]), q[rows], k[keys], v[keys], c, l, Hkv)
        assert torch.equal(out[rows], want), i
    assert pa.pa_device_error() == 0


def test_time_grows_with_the_number_of_sequences(pa, cuda_device):
    """4000 prompts of 70 tokens against 250: 16 times the work; 333 times the time before the
    scheduler's search went on from the last unit's."""
    took = {}
    for S in (250, 4000):
        C = [70] * S
        q, k, v = (torch.randn(70 * S, h, 64, device="cuda").bfloat16() for h in (8, 2, 2))
        out, st = torch.empty_like(q), starts(C)
        best = float("inf")
        for _ in range(4):
            begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            begin.record()
            pa.pa_prompt_attention(out, q, k, v, st, st, 0.1, 2, 70, 70)
            end.record()
            torch.cuda.synchronize()
            best = min(best, begin.elapsed_time(end))
        took[S] = best
    assert took[4000] < 4 * 16 * took[250], took
