"""Calls given a stream and no workspace: the scratch that the binding makes for them is that
stream's.  Memory that the current stream has freed but still uses is not written, and what the
current stream allocates after the call is not the scratch of a call that has yet to run."""
import types

import pytest
import torch

pytestmark = pytest.mark.gpu

S, HQ, HKV, D, B, N = 4, 32, 8, 128, 16, 4000
CYCLES = 100_000_000       # some 50 ms


def make(name, pa):
    """A call of one operator that needs scratch, as f(out, stream), its output's make, the scratch's bytes."""
    g = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").half()

    nb = -(-N // B)
    tables = torch.randperm(S * nb, generator=g, device="cuda").int().view(S, nb)
    lens = torch.full((S,), N, dtype=torch.int32, device="cuda")
    q = normal(S, HQ, D)
    if name == "prompt":
        k, v = normal(S * N, HKV, D), normal(S * N, HKV, D)
        qs, ks = (torch.arange(S + 1, dtype=torch.int32, device="cuda") * n for n in (1, N))
        need = pa.lib().pa_prompt_attention_workspace_bytes(S, S, HQ, HKV, D, 1, N)
        return (lambda out, st: pa.pa_prompt_attention(out, q, k, v, qs, ks, 0.09, HKV, 1, N, stream=st),
                lambda: torch.zeros_like(q), need)
    need = pa.pa_paged_decode_workspace_bytes(S, HQ, HKV, D, B, nb * B)
    made = lambda: torch.zeros(S, HQ, D, device="cuda")      # noqa: E731
    kc, vc = normal(S * nb, HKV, B, D), normal(S * nb, HKV, B, D)
    if name == "decode_fp8":
        kc, vc = (x.to(torch.float8_e4m3fn) for x in (kc, vc))
        sc = torch.rand(S * nb, HKV, 2, B, generator=g, device="cuda")
        return (lambda out, st: pa.pa_paged_decode_attention_fp8(out, q, kc, vc, sc, tables, lens, 0.09, HKV,
                                                                 stream=st), made, need)
    if name == "decode":
        return (lambda out, st: pa.pa_paged_decode_attention(out, q, kc, vc, tables, lens, 0.09, HKV, stream=st),
                made, need)
    kn, vn = normal(S, HKV, D), normal(S, HKV, D)
    return (lambda out, st: pa.pa_decode_step(out, q, kn, vn, kc, vc, tables, lens, 0.09, HKV, stream=st),
            made, need)


@pytest.mark.parametrize("name", ["decode_fp8", "prompt", "decode", "decode_step"])
def test_scratch_is_the_calls_stream_s(pa, cuda_device, name):
    call, made, need = make(name, pa)
    assert need > 0
    want, got, later = made(), made(), made()
    call(want, None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    # freed by the host, read by the current stream's later work
    x = torch.full((need,), 7, dtype=torch.uint8, device="cuda")
    y = torch.empty_like(x)
    torch.cuda.synchronize()
    torch.cuda._sleep(CYCLES)
    y.copy_(x)
    del x
    call(got, side)
    torch.cuda.synchronize()
    assert (y == 7).all() and torch.equal(got, want)
    # the call waits on its stream; what the current stream allocates meanwhile stays as it is
    del y
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(CYCLES)
    call(later, side)
    z = torch.full((need,), 7, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert (z == 7).all() and torch.equal(later, want)
    assert pa.pa_device_error() == 0


@pytest.mark.parametrize("name", ["decode_fp8", "prompt", "decode", "decode_step"])
def test_a_stream_known_by_its_handle(pa, cuda_device, name):
    """Any object with a cuda_stream names the stream, the default stream among them."""
    call, made, _ = make(name, pa)
    want = made()
    call(want, None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, torch.cuda.default_stream(), torch.cuda.ExternalStream(side.cuda_stream)):
        for given in (stream, types.SimpleNamespace(cuda_stream=stream.cuda_stream)):
            got = made()
            torch.cuda.synchronize()
            call(got, given)
            torch.cuda.synchronize()
            assert torch.equal(got, want)
