"""GPU tests of attention over packed prompts (pa_prompt_attention) against a
plain 64-bit form, one sequence and head at a time.

Tolerance of an output row, from the arithmetic: with A = sum_t p_t |v_t|,
  eps/2 A         the weights' rounding to the type (eps/2 of each), and
  2^-25 sum |v|   the smallest fp16 step, for weights near zero (their sum is at least 1)
  2^-23 L A       the product's fp32 sums, 2^-24 2 (D + 8) z A the scores' (z: the largest sum
                  of |q k| scale of the row), 2^-20 A exp2 and the joins
  eps/2 |out|     the output's rounding."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(autouse=True)
def clean_error_word(pa, cuda_device):
    pa.pa_device_error(clear=True)
    yield
    assert pa.pa_device_error(clear=True) == 0     # tests that expect a flag clear it themselves


def starts(lens):
    return torch.tensor(np.cumsum([0] + list(lens)), dtype=torch.int32, device="cuda")


def inputs(C, L, Hq, Hkv, D, dtype, seed, extra=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, Tk = sum(C) + extra, sum(L) + extra
    q, k, v = (torch.randn(n, h, D, generator=g, device="cuda").to(dtype)
               for n, h in ((T, Hq), (Tk, Hkv), (Tk, Hkv)))
    return q, k, v


def check_sequence(out, q, k, v, scale):
    """One sequence's rows: out, q [C, Hq, D], k, v [L, Hkv, D]."""
    (C, Hq, D), L, Hkv = q.shape, len(k), k.shape[1]
    eps = torch.finfo(q.dtype).eps
    row, key = (torch.arange(n, device="cuda") for n in (C, L))
    seen = key <= L - C + row[:, None]
    for h in range(Hq):
        K, V, Q = k[:, h // (Hq // Hkv)].double(), v[:, h // (Hq // Hkv)].double(), q[:, h].double()
        got = out[:, h].double()
        z = (Q @ K.T * scale).masked_fill(~seen, -float("inf"))
        p = torch.softmax(z, -1).masked_fill(~seen.any(-1, keepdim=True), 0.0)
        want, A = p @ V, p @ V.abs()
        most = ((Q.abs() @ K.abs().T) * abs(scale) * seen).amax(-1, True) if L else torch.zeros(C, 1, device="cuda")
        tol = ((eps / 2 + 2.0 ** -20 + 2.0 ** -23 * L + 2.0 ** -23 * (D + 8) * most) * A
               + 2.0 ** -25 * (seen.double() @ V.abs()))
        tol = tol * (1 + eps) + eps / 2 * want.abs() + 2.0 ** -25
        bad = (got - want).abs() / tol.clamp(min=1e-30)
        assert torch.isfinite(got).all() and (bad <= 1).all(), (h, bad.max().item(), bad.argmax().item())
        if not seen.any(-1).all():
            assert (got[~seen.any(-1)] == 0).all()


def run(pa, C, L, q, k, v, scale, max_query=None, max_key=None, out=None, **kw):
    if out is None:
        out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    return pa.pa_prompt_attention(out, q, k, v, starts(C), starts(L), scale, k.shape[1],
                                  max(C) if max_query is None else max_query,
                                  max(L) if max_key is None else max_key, **kw)


def check(out, C, L, q, k, v, scale, which=None):
    a, b = np.cumsum([0] + list(C)), np.cumsum([0] + list(L))
    for i in range(len(C)) if which is None else which:
        if C[i]:
            check_sequence(out[a[i]:a[i + 1]], q[a[i]:a[i + 1]], k[b[i]:b[i + 1]], v[b[i]:b[i + 1]], scale)
    assert (out[a[-1]:] == 7).all()


SHAPES = [("bf16", 8, 2, 128), ("f16", 4, 4, 64), ("bf16", 16, 1, 64), ("f16", 5, 1, 128),
          ("bf16", 3, 3, 128), ("f16", 12, 4, 128), ("bf16", 9, 1, 64)]


@pytest.mark.parametrize("dtype,Hq,Hkv,D", SHAPES)
@pytest.mark.parametrize("C,L", [
    ([1], [1]),
    ([5], [5]),
    ([1, 0, 130, 17], [1, 9, 130, 17]),
    ([127, 128, 129, 255, 256, 257], [127, 128, 129, 255, 256, 257]),
    ([1, 5, 64, 300, 0, 33], [128, 129, 700, 301, 0, 2000]),
    ([64, 300, 10, 200], [0, 290, 3, 7]),             # queries before the first key
    ([900], [1000]),
])
def test_ragged(pa, dtype, Hq, Hkv, D, C, L):
    q, k, v = inputs(C, L, Hq, Hkv, D, DT[dtype], seed=sum(C) + Hq, extra=9)
    k[sum(L):], v[sum(L):], q[sum(C):] = float("nan"), float("nan"), float("nan")
    out = run(pa, C, L, q, k, v, D ** -0.5)
    check(out, C, L, q, k, v, D ** -0.5)
    assert torch.equal(out, run(pa, C, L, q, k, v, D ** -0.5))


@pytest.mark.parametrize("dtype,Hq,Hkv,D", [("bf16", 64, 8, 128), ("f16", 4, 4, 64), ("bf16", 10, 2, 128)])
def test_few_queries_many_keys(pa, dtype, Hq, Hkv, D):
    """The keys are split over CTAs and joined."""
    C, L = [5, 40, 1, 17, 3], [4000, 9001, 1, 130, 2]
    need = pa.lib().pa_prompt_attention_workspace_bytes(5, sum(C), Hq, Hkv, D, 40, 9001)
    assert need > 0
    q, k, v = inputs(C, L, Hq, Hkv, D, DT[dtype], seed=3)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")      # NaN everywhere
    out = run(pa, C, L, q, k, v, D ** -0.5, workspace=ws)
    check(out, C, L, q, k, v, D ** -0.5)


@pytest.mark.parametrize("L", [1792, 1793, 2049, 2176, 2177, 4000])
def test_one_query_tile_and_odd_tiles(pa, L):
    """One query tile takes the K/V tiles in turn with itself; the last piece may hold one tile,
    and another sequence's queries may stand before its first key."""
    C, L = [3, 8], [L, 5]
    q, k, v = inputs(C, L, 4, 1, 128, torch.bfloat16, seed=31)
    assert pa.lib().pa_prompt_attention_workspace_bytes(2, 11, 4, 1, 128, 8, L[0]) > 0
    check(run(pa, C, L, q, k, v, 0.09), C, L, q, k, v, 0.09)


def test_output_on_any_16_bytes(pa):
    """An output that begins in the middle of a 32-byte sector."""
    C = [200, 70]
    q, k, v = inputs(C, C, 4, 2, 64, torch.float16, seed=32)
    out = torch.full((q.numel() + 8,), 7.0, dtype=q.dtype, device="cuda")[8:].view(q.shape)
    assert out.data_ptr() % 32 == 16
    check(run(pa, C, C, q, k, v, 0.125, out=out), C, C, q, k, v, 0.125)


def test_large_values(pa):
    """bf16 values far outside fp16's range."""
    C = [150]
    q, k, v = inputs(C, C, 4, 2, 64, torch.bfloat16, seed=33)
    v *= 1e30
    q, k = q * 1e8, k * 1e-8
    out = run(pa, C, C, q, k, v, 0.125)
    check_sequence(out, q, k, v, 0.125)


def test_two_streams(pa):
    """Split calls on two streams at once, workspaces from the binding."""
    C, L = [5, 9], [6000, 3000]
    a, b = (inputs(C, L, 16, 2, 128, torch.bfloat16, seed=i) for i in (41, 42))
    want = [run(pa, C, L, *x, 0.09) for x in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for r in range(5):
        for i, x in enumerate((a, b)):
            out = torch.full_like(x[0], 7.0)
            streams[i].wait_stream(torch.cuda.current_stream())
            got[i].append(run(pa, C, L, *x, 0.09, out=out, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])


def test_larger_bounds_than_lengths(pa):
    """max_query_len and max_key_len may be anything that covers the lengths."""
    C, L = [100, 37], [300, 37]
    q, k, v = inputs(C, L, 8, 2, 128, torch.bfloat16, seed=4)
    for mq, mk in ((100, 300), (5000, 300), (100, 20000), (4096, 4096)):
        check(run(pa, C, L, q, k, v, 0.1, mq, mk), C, L, q, k, v, 0.1)


def test_many_sequences(pa):
    C = [(7 * i) % 41 for i in range(700)]
    L = [c + (i % 3) * 100 for i, c in enumerate(C)]
    q, k, v = inputs(C, L, 4, 2, 64, torch.float16, seed=5)
    check(run(pa, C, L, q, k, v, 0.125), C, L, q, k, v, 0.125, which=list(range(0, 700, 23)) + [699])


@pytest.mark.parametrize("scale", [0.0, -0.1, 1.5])
def test_scales(pa, scale):
    """Zero (the mean of what is seen), negative, steep (maxima that move by more than 2^8)."""
    C, L = [300, 70], [300, 400]
    q, k, v = inputs(C, L, 4, 1, 128, torch.bfloat16, seed=6)
    check(run(pa, C, L, q, k, v, scale), C, L, q, k, v, scale)


def test_growing_scores(pa):
    """Scores that grow along the keys: the running maximum moves in every tile."""
    C, L = [600], [600]
    q, k, v = inputs(C, L, 4, 2, 64, torch.float16, seed=7)
    q[:], k[:] = q.abs(), k.abs() * torch.linspace(0.1, 4, 600, device="cuda")[:, None, None]
    check(run(pa, C, L, q, k, v, 0.5), C, L, q, k, v, 0.5)


def test_columns_of_a_projection(pa):
    C = [40, 333, 128]
    qkv = torch.randn(sum(C), 8 + 2 + 2, 128, device="cuda").bfloat16()
    q, k, v = qkv[:, :8], qkv[:, 8:10], qkv[:, 10:]
    out = run(pa, C, C, q, k, v, 0.09)
    check(out, C, C, q, k, v, 0.09)
    assert torch.equal(out, run(pa, C, C, q.contiguous(), k.contiguous(), v.contiguous(), 0.09))


def test_another_sequences_nan_stays_there(pa):
    C, L = [70, 50, 300], [70, 500, 300]
    q, k, v = inputs(C, L, 4, 2, 128, torch.bfloat16, seed=8)
    q[70:120] = float("nan")
    k[70:570], v[70:570] = float("nan"), float("inf")
    out = run(pa, C, L, q, k, v, 0.09)
    assert out[70:120].isnan().all()
    out[70:120] = 0
    check_sequence(out[:70], q[:70], k[:70], v[:70], 0.09)
    check_sequence(out[120:], q[120:], k[570:], v[570:], 0.09)


def test_nan_reaches_the_rows_that_see_it(pa):
    q, k, v = inputs([400], [400], 4, 4, 64, torch.float16, seed=9)
    k[201, 1, 3], q[20, 2, 5], v[300, 3, 7] = float("nan"), float("nan"), float("nan")
    out = run(pa, [400], [400], q, k, v, 0.125)
    assert out[201:, 1].isnan().all() and out[:201, 1].isfinite().all()
    assert out[20, 2].isnan().all() and out[21:, 2].isfinite().all() and out[:20, 2].isfinite().all()
    assert out[300:, 3, 7].isnan().all() and out[:45, 3].isfinite().all()
    assert out[:, 3, :7].isfinite().all() and out[:, 0].isfinite().all()


def test_bad_starts_are_flagged(pa):
    C, L = [30, 40, 50], [30, 40, 50]
    q, k, v = inputs(C, L, 4, 2, 64, torch.bfloat16, seed=10)
    for mq, mk in ((49, 50), (50, 49)):          # the third is longer than was said
        out = run(pa, C, L, q, k, v, 0.1, mq, mk)
        assert pa.pa_device_error(clear=True) == pa.DEVERR["context_len"]
        assert (out[70:] == 7).all()
        check_sequence(out[:30], q[:30], k[:30], v[:30], 0.1)
        check_sequence(out[30:70], q[30:70], k[30:70], v[30:70], 0.1)
    out = torch.full_like(q, 7.0)
    bad = torch.tensor([0, 30, 70, 121], dtype=torch.int32, device="cuda")     # one past the end
    pa.pa_prompt_attention(out, q, k, v, bad, starts(L), 0.1, 2, 60, 60)
    assert pa.pa_device_error(clear=True) == pa.DEVERR["context_len"]
    assert (out[70:] == 7).all() and not (out[:70] == 7).any()
    back = torch.tensor([0, 30, 20, 120], dtype=torch.int32, device="cuda")    # decreasing
    pa.pa_prompt_attention(out, q, k, v, starts(C), back, 0.1, 2, 100, 100)
    assert pa.pa_device_error(clear=True) == pa.DEVERR["context_len"]


def test_no_keys_at_all(pa):
    q = torch.randn(20, 4, 64, device="cuda").half()
    k = torch.empty(0, 2, 64, dtype=torch.float16, device="cuda")
    out = torch.full_like(q, 7.0)
    z = torch.zeros(2, dtype=torch.int32, device="cuda")
    pa.pa_prompt_attention(out, q, k, k, starts([20]), z, 0.1, 2, 20, 0)
    assert (out == 0).all()


def test_wait_limit(pa):
    """Waits that run out are reported and the next call is whole."""
    C = [700, 300]
    q, k, v = inputs(C, C, 8, 8, 128, torch.bfloat16, seed=11)
    try:
        pa.pa_set_wait_limit(1)
        run(pa, C, C, q, k, v, 0.09)
        assert pa.pa_device_error(clear=True) & pa.DEVERR["timeout"]
    finally:
        pa.pa_set_wait_limit(0)
    check(run(pa, C, C, q, k, v, 0.09), C, C, q, k, v, 0.09)


def test_captured_and_replayed_with_other_lengths(pa):
    """One captured call, replayed with other starts and inputs on another stream."""
    T = 700
    q, k, v = inputs([T], [T], 8, 2, 128, torch.bfloat16, seed=12)
    out = torch.full_like(q, 7.0)
    qs = starts([350, 350])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pa.pa_prompt_attention(out, q, k, v, qs, qs, 0.09, 2, T, T)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pa.pa_prompt_attention(out, q, k, v, qs, qs, 0.09, 2, T, T)
    for C in ([1, 699], [350, 300], [0, 5], [700, 0]):
        out.fill_(7.0)
        qs.copy_(starts(C))
        q.copy_(torch.randn(q.shape, device="cuda"))
        graph.replay()
        check(out, C, C, q, k, v, 0.09)


def test_rows_behind_2_31_elements(pa):
    """280000 tokens of 64 heads in sequences of 70: the last ones lie 2.3e9 elements in."""
    S, n, H, D = 4000, 70, 64, 128
    C = [n] * S
    q = torch.empty(S * n, H, D, dtype=torch.bfloat16, device="cuda").normal_()
    k = torch.empty_like(q).normal_()
    v = torch.empty_like(q).normal_()
    out = run(pa, C, C, q, k, v, 0.09)
    check(out, C, C, q, k, v, 0.09, which=[0, S - 1])
