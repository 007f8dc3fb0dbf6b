"""GPU test: every operator called from a host thread that has made no other CUDA call, as a serving
engine's worker does with tensors that were made elsewhere, gives what the main thread's call gave."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

HQ, HKV, D, B, NB, T = 8, 2, 128, 16, 8, 100


@pytest.fixture
def calls(pa, cuda_device):
    g = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").half()

    q, k, v = normal(T, HQ, D), normal(T, HKV, D), normal(T, HKV, D)
    kc, vc = normal(NB, HKV, B, D), normal(NB, HKV, B, D)
    k8, v8 = kc.to(torch.float8_e4m3fn), vc.to(torch.float8_e4m3fn)
    sc = torch.rand(NB, HKV, 2, B, generator=g, device="cuda")
    slots, pos = torch.arange(T, device="cuda"), torch.arange(T, device="cuda")
    cs = torch.rand(T, D, generator=g, device="cuda")
    table, lens = torch.arange(NB, device="cuda").int()[None], torch.full((1,), T, dtype=torch.int32, device="cuda")
    start = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    pairs = torch.tensor([[0, NB - 1]], device="cuda")
    one, out1, out = q[:1].contiguous(), torch.empty(1, HQ, D, device="cuda"), torch.empty(T, HQ, D, device="cuda")
    out16, qo = torch.empty_like(q), torch.empty_like(q)
    key, value = torch.empty_like(k), torch.empty_like(v)
    ws = pa.alloc_workspace(1, HQ, HKV, D, B, NB * B)
    return {   # each with the tensors it writes
        "rope": (lambda: pa.pa_rope_and_cache(qo, q, k, v, kc, vc, slots, pos, cs), [qo, kc, vc]),
        "rope_fp8": (lambda: pa.pa_rope_and_cache_fp8(qo, q, k, v, k8, v8, sc, slots, pos, cs), [qo, k8, v8, sc]),
        "decode_fp8": (lambda: pa.pa_paged_decode_attention_fp8(out1, one, k8, v8, sc, table, lens, 0.09, HKV,
                                                                workspace=ws), [out1]),
        "gather": (lambda: pa.pa_gather_cache_fp8(key, value, k8, v8, sc, table, start), [key, value]),
        "copy_fp8": (lambda: pa.pa_copy_blocks_fp8(k8, v8, sc, pairs), [k8, v8, sc]),
        "prompt": (lambda: pa.pa_prompt_attention(out16, q, k, v, start, start, 0.09, HKV, T, T), [out16]),
        "decode": (lambda: pa.pa_paged_decode_attention(out1, one, kc, vc, table, lens, 0.09, HKV, workspace=ws),
                   [out1]),
        "decode_step": (lambda: pa.pa_decode_step(out1, one, k[:1], v[:1], kc, vc, table, lens, 0.09, HKV,
                                                  workspace=ws), [out1, kc, vc]),
        "prefill": (lambda: pa.pa_paged_prefill_attention(out, q, kc, vc, table, lens, start, 0.09, HKV, T), [out]),
        "cache": (lambda: pa.pa_reshape_and_cache(k, v, kc, vc, slots), [kc, vc]),
    }


def bits(tensors):
    return [x.clone().view(torch.uint8) for x in tensors]


@pytest.mark.parametrize("name", ["rope", "rope_fp8", "decode_fp8", "gather", "copy_fp8", "prompt", "decode",
                                  "decode_step", "prefill", "cache"])
def test_a_thread_without_a_context(pa, calls, name):
    call, written = calls[name]
    call()
    want = bits(written)
    torch.cuda.synchronize()
    said = []

    def worker():
        try:
            call()
        except Exception as e:
            said.append(e)

    thread = threading.Thread(target=worker)
    thread.start()
    thread.join()
    assert not said, said
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(bits(written), want))
    assert pa.pa_device_error() == 0
