"""What the binding of the rotary write, the 8-bit pool's calls and prompt attention refuses:
tensors of another place, type, shape or layout, before anything is launched."""
import pytest
import torch

pytestmark = pytest.mark.gpu

T, HQ, HKV, D, B, NB, S = 5, 8, 2, 64, 16, 6, 2


def f16(*shape):
    return torch.zeros(*shape, dtype=torch.float16, device="cuda")


def i32(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


@pytest.fixture
def pool():
    codes = torch.zeros(NB, HKV, B, D, device="cuda").to(torch.float8_e4m3fn)
    return {"k_cache": codes, "v_cache": codes.clone(),
            "kv_scale": torch.zeros(NB, HKV, 2, B, device="cuda")}


def refused(call, good, cases):
    call(**good)
    torch.cuda.synchronize()
    for error, change in cases:
        with pytest.raises(error):
            call(**{**good, **change})
            pytest.fail(f"taken: {list(change)}")
    call(**good)
    torch.cuda.synchronize()


def test_rope(pa, pool):
    good = dict(q_out=f16(T, HQ, D), q=f16(T, HQ, D), key=f16(T, HKV, D), value=f16(T, HKV, D),
                **pool, slot_mapping=torch.arange(T, device="cuda"),
                positions=torch.arange(T, device="cuda"),
                cos_sin=torch.ones(32, D, device="cuda"), sections=(D // 2,), interleaved=False)
    two = torch.zeros(2, T, dtype=torch.int64, device="cuda")
    refused(pa.pa_rope_and_cache_fp8, good, [
        (ValueError, dict(key=torch.zeros(T, HKV, D, dtype=torch.float16))),        # on the host
        (ValueError, dict(slot_mapping=torch.arange(T))),
        (TypeError, dict(key=f16(T, HKV, D).float())),
        (TypeError, dict(q=f16(T, HQ, D).bfloat16())),
        (TypeError, dict(slot_mapping=i32(0, 1, 2, 3, 4))),
        (TypeError, dict(k_cache=pool["k_cache"].view(torch.uint8))),
        (TypeError, dict(kv_scale=None)),
        (TypeError, dict(value=3)),
        (ValueError, dict(value=f16(T, HKV + 1, D))),
        (ValueError, dict(q_out=f16(T + 1, HQ, D))),
        (ValueError, dict(q=f16(T, D, HQ).transpose(1, 2))),                        # heads not dense
        (ValueError, dict(key=f16(T, HKV * D + 4)[:, :HKV * D].view(T, HKV, D))),   # odd stride
        (ValueError, dict(key=f16(1, HKV, D).expand(T, HKV, D))),
        (ValueError, dict(kv_scale=torch.zeros(NB, HKV, B, 2, device="cuda"))),
        (ValueError, dict(v_cache=pool["k_cache"][:, :, ::2])),
        (ValueError, dict(positions=two, sections=None)),                           # unnamed axes
        (ValueError, dict(positions=two, sections=(D // 2,))),
        (ValueError, dict(cos_sin=torch.ones(32, D, 1, device="cuda"))),
        (TypeError, dict(sections=5)),
        (TypeError, dict(interleaved=torch.ones(2))),                               # neither true nor false
        (pa.PAError, dict(sections=(D // 2 - 1,))),
        (pa.PAError, dict(cos_sin=torch.ones(32, D - 8, device="cuda"), sections=None)),
    ])
    for sixteen in (False, True):     # the 16-bit pool has its own type
        kv = [f16(NB, HKV, B, D).to(torch.bfloat16 if sixteen else torch.float16) for _ in "kv"]
        rest = {n: x for n, x in good.items() if n not in pool}
        if sixteen:
            with pytest.raises(TypeError):
                pa.pa_rope_and_cache(**rest, k_cache=kv[0], v_cache=kv[1])
        else:
            pa.pa_rope_and_cache(**rest, k_cache=kv[0], v_cache=kv[1])
    torch.cuda.synchronize()


def test_decode(pa, pool):
    good = dict(out=torch.zeros(S, HQ, D, device="cuda"), q=f16(S, HQ, D), **pool,
                block_tables=i32(0, 1, 2, 3).view(S, 2), context_lens=i32(20, 1), scale=0.125,
                num_kv_heads=HKV)
    refused(pa.pa_paged_decode_attention_fp8, good, [
        (TypeError, dict(out=f16(S, HQ, D))),
        (TypeError, dict(q=f16(S, HQ, D).float())),
        (TypeError, dict(scale="x")),
        (TypeError, dict(max_context_len=1.5)),
        (ValueError, dict(q=f16(S, D, HQ).transpose(1, 2))),
        (ValueError, dict(num_kv_heads=HKV + 1)),
        (ValueError, dict(context_lens=i32(20))),
        (ValueError, dict(block_tables=i32(0, 1, 2, 3))),
        (ValueError, dict(out=torch.zeros(S, HQ, D))),
        (ValueError, dict(max_context_len=1 << 40)),
        (ValueError, dict(workspace=torch.zeros(1 << 20, dtype=torch.uint8))),
        (pa.PAError, dict(workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))),
        (pa.PAError, dict(max_context_len=33)),              # more than the table holds
        (pa.PAError, dict(max_context_len=-1)),
    ])


def test_copy_and_gather(pa, pool):
    pairs = torch.tensor([[0, 5]], device="cuda")
    refused(pa.pa_copy_blocks_fp8, dict(**pool, block_mapping=pairs), [
        (TypeError, dict(block_mapping=pairs.int())),
        (ValueError, dict(block_mapping=pairs.cpu())),
        (ValueError, dict(block_mapping=pairs.view(2))),
        (ValueError, dict(k_cache=pool["k_cache"][0])),
    ])
    good = dict(key=f16(T, HKV, D), value=f16(T, HKV, D), **pool,
                block_tables=i32(0, 1, 2, 3).view(S, 2), key_start=i32(0, 2, 5))
    refused(pa.pa_gather_cache_fp8, good, [
        (TypeError, dict(value=f16(T, HKV, D).bfloat16())),
        (TypeError, dict(key_start=torch.tensor([0, 2, 5], device="cuda"))),
        (ValueError, dict(key=f16(T, HKV + 1, D))),
        (ValueError, dict(key=f16(T, 2 * HKV, D)[:, ::2])),
        (ValueError, dict(key_start=i32(0, 2))),
        (ValueError, dict(key_start=torch.tensor(3, dtype=torch.int32, device="cuda"))),
    ])


def test_prompt(pa):
    good = dict(out=f16(T, HQ, D), q=f16(T, HQ, D), key=f16(T, HKV, D), value=f16(T, HKV, D),
                query_start=i32(0, 2, T), key_start=i32(0, 2, T), scale=0.125, num_kv_heads=HKV,
                max_query_len=3, max_key_len=3)
    refused(pa.pa_prompt_attention, good, [
        (TypeError, dict(out=f16(T, HQ, D).float())),
        (TypeError, dict(key=f16(T, HKV, D).bfloat16())),
        (TypeError, dict(query_start=torch.tensor([0, 2, T], device="cuda"))),
        (TypeError, dict(max_query_len=None)),
        (ValueError, dict(num_kv_heads=HQ)),
        (ValueError, dict(value=f16(T + 1, HKV, D))),
        (ValueError, dict(key_start=i32(0, T))),
        (ValueError, dict(q=f16(T, HQ * 2, D)[:, ::2])),
        (ValueError, dict(key=f16(1, HKV, D).expand(T, HKV, D))),
        (ValueError, dict(out=f16(T, HQ, D).cpu())),
        (ValueError, dict(max_key_len=1 << 40)),
        (pa.PAError, dict(max_key_len=-1)),
        (pa.PAError, dict(q=f16(T, HQ - 1, D), out=f16(T, HQ - 1, D))),
    ])
