"""The rotary write, the 8-bit pool's calls and prompt attention refuse bad
arguments on the host, before any CUDA call; empty calls do nothing."""
import ctypes

import pytest
import torch

NUL = None
ARG, UNSUPPORTED, WORKSPACE = -1, -2, -7
P = 1 << 20      # an aligned address that is never read: a check refuses the call first


def sections(*n):
    return (ctypes.c_int * len(n))(*n)


def rope(pa, fp8=False, ptr=NUL, sect=(64,), axes=1, rot=128, most=100, qs=4096, ks=1024, vs=1024,
         toks=4, qh=32, kv=8, hd=128, bs=16, nblk=10, dt=1, cos=None, pos=None, q=None):
    L = pa.lib()
    fn = L.pa_rope_and_cache_fp8 if fp8 else L.pa_rope_and_cache
    q = ptr if q is None else q
    pool = [ptr] * (3 if fp8 else 2)
    return fn(q, q, ptr, ptr, *pool, ptr, ptr if pos is None else pos, ptr if cos is None else cos,
              sections(*sect) if sect else NUL, axes, rot, most, 0, qs, qs, ks, vs, toks, qh, kv, hd,
              bs, nblk, dt, NUL)


@pytest.mark.parametrize("fp8", [False, True])
def test_rope(pa, fp8):
    assert rope(pa, fp8, toks=0) == 0
    assert rope(pa, fp8) == ARG                              # null pointers
    assert rope(pa, fp8, toks=-1) == ARG
    assert rope(pa, fp8, dt=2) == ARG
    assert rope(pa, fp8, kv=0) == ARG
    assert rope(pa, fp8, rot=130) == ARG                     # wider than a head
    assert rope(pa, fp8, hd=96, rot=96) == UNSUPPORTED
    assert rope(pa, fp8, bs=8) == UNSUPPORTED
    assert rope(pa, fp8, rot=24, sect=(12,)) == UNSUPPORTED  # not a multiple of 16
    assert rope(pa, fp8, axes=5, sect=(16, 16, 16, 8, 8)) == UNSUPPORTED
    assert rope(pa, fp8, axes=2, sect=(32, 31)) == ARG       # do not add up
    assert rope(pa, fp8, axes=2, sect=(65, -1)) == ARG
    assert rope(pa, fp8, most=0) == ARG
    assert rope(pa, fp8, sect=None) == ARG
    assert rope(pa, fp8, ptr=P + 8) == ARG                   # alignment
    assert rope(pa, fp8, ptr=P, ks=1023) == ARG              # shorter than a row
    assert rope(pa, fp8, ptr=P, vs=1028) == ARG              # not a multiple of 8
    assert rope(pa, fp8, ptr=P, qs=4000) == ARG
    assert rope(pa, fp8, ptr=P, qh=0) == ARG                 # queries, but no heads


def test_decode_fp8(pa):
    def call(ptr=NUL, kv=8, seqs=4, qh=32, hd=128, bs=16, maxb=4, most=64, nblk=10, dt=1, ws=NUL, n=0):
        return pa.lib().pa_paged_decode_attention_fp8(ptr, ptr, ptr, ptr, ptr, ptr, ptr, 1.0, kv, seqs,
                                                      qh, hd, bs, maxb, most, nblk, dt, ws, n, NUL)
    assert call(seqs=0) == 0
    assert call() == ARG
    assert call(qh=30) == ARG and call(dt=3) == ARG and call(seqs=-1) == ARG
    assert call(kv=1) == UNSUPPORTED and call(bs=24) == UNSUPPORTED and call(hd=256) == UNSUPPORTED
    assert call(most=65) == ARG and call(nblk=0) == ARG and call(maxb=0) == ARG
    assert call(nblk=1 << 24) == UNSUPPORTED                 # rows beyond 2^31
    assert call(ptr=P + 4) == ARG
    assert call(ptr=P) == WORKSPACE and call(ptr=P, ws=P + 16, n=1 << 30) == WORKSPACE


def test_gather_and_copies(pa):
    def gather(ptr=NUL, seqs=2, toks=5, kv=8, hd=128, bs=16, maxb=4, nblk=10, dt=1):
        return pa.lib().pa_gather_cache_fp8(ptr, ptr, ptr, ptr, ptr, ptr, ptr, seqs, toks, kv, hd, bs,
                                            maxb, nblk, dt, NUL)
    assert gather(seqs=0) == 0 and gather(toks=0) == 0
    assert gather() == ARG and gather(ptr=P + 8) == ARG and gather(maxb=0) == ARG
    assert gather(toks=-1) == ARG and gather(dt=5) == ARG
    assert gather(hd=80) == UNSUPPORTED and gather(toks=(1 << 31) - 1) == UNSUPPORTED

    def copy(ptr=NUL, n=3, kv=8, hd=128, bs=16, nblk=10):
        return pa.lib().pa_copy_blocks_fp8(ptr, ptr, ptr, ptr, n, kv, hd, bs, nblk, NUL)
    assert copy(n=0) == 0
    assert copy() == ARG and copy(ptr=P + 8) == ARG and copy(n=-1) == ARG and copy(kv=0) == ARG
    assert copy(hd=100) == UNSUPPORTED and copy(ptr=P, n=1 << 30) == UNSUPPORTED


def test_prompt(pa):
    def call(ptr=NUL, kv=8, seqs=2, toks=64, keys=64, qh=32, hd=128, mq=32, mk=32, qs=4096, ks=1024,
             vs=1024, dt=1):
        return pa.lib().pa_prompt_attention(ptr, ptr, ptr, ptr, ptr, ptr, 1.0, kv, seqs, toks, keys,
                                            qh, hd, mq, mk, qs, ks, vs, dt, NUL, 0, NUL)
    assert call(seqs=0) == 0 and call(toks=0) == 0 and call(mq=0) == 0
    assert call() == ARG and call(ptr=P + 8) == ARG
    assert call(qh=30) == ARG and call(dt=2) == ARG and call(mk=-1) == ARG and call(keys=-1) == ARG
    assert call(kv=1) == UNSUPPORTED and call(hd=96) == UNSUPPORTED and call(mq=1 << 30) == UNSUPPORTED
    assert call(ptr=P, qs=4095) == ARG and call(ptr=P, ks=1020) == ARG and call(ptr=P, vs=8) == ARG
    size = pa.lib().pa_prompt_attention_workspace_bytes
    assert size(2, 64, 30, 8, 128, 32, 32) == 0 and size(-1, 64, 32, 8, 128, 32, 32) == 0


def test_binding_refuses(pa):
    """Tensors of the wrong place, type, shape or layout raise."""
    h = torch.float16
    q, k = torch.zeros(3, 4, 64, dtype=h), torch.zeros(3, 2, 64, dtype=h)
    pool = torch.zeros(4, 2, 16, 64, dtype=h)
    codes, scale = pool.to(torch.float8_e4m3fn), torch.zeros(4, 2, 2, 16)
    slots, cs = torch.zeros(3, dtype=torch.int64), torch.zeros(8, 64)
    start = torch.tensor([0, 3], dtype=torch.int32)
    table, lens = torch.zeros(3, 1, dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    calls = [
        lambda: pa.pa_rope_and_cache(q, q, k, k, pool, pool, slots, slots, cs),
        lambda: pa.pa_rope_and_cache_fp8(q, q, k, k, codes, codes, scale, slots, slots, cs),
        lambda: pa.pa_paged_decode_attention_fp8(q.float(), q, codes, codes, scale, table, lens, 1.0, 2),
        lambda: pa.pa_copy_blocks_fp8(codes, codes, scale, torch.zeros(1, 2, dtype=torch.int64)),
        lambda: pa.pa_gather_cache_fp8(k, k, codes, codes, scale, table, start),
        lambda: pa.pa_prompt_attention(q, q, k, k, start, start, 1.0, 2, 3, 3),
    ]
    for call in calls:
        with pytest.raises(ValueError):
            call()


@pytest.mark.gpu
def test_binding_refuses_on_the_gpu(pa, cuda_device):
    def cuda(x):
        return x.to(cuda_device)
    h = torch.float16
    q, k = cuda(torch.zeros(3, 4, 64, dtype=h)), cuda(torch.zeros(3, 2, 64, dtype=h))
    codes, scale = cuda(torch.zeros(4, 2, 16, 64)).to(torch.float8_e4m3fn), cuda(torch.zeros(4, 2, 2, 16))
    pool = codes.to(h)
    slots, cs = cuda(torch.zeros(3, dtype=torch.int64)), cuda(torch.zeros(8, 64))
    start = cuda(torch.tensor([0, 3], dtype=torch.int32))
    table, lens = cuda(torch.zeros(3, 1, dtype=torch.int32)), cuda(torch.ones(3, dtype=torch.int32))
    wide = cuda(torch.zeros(3, 2, 128, dtype=h))[..., ::2]
    out = q.float()
    rope, rope8 = pa.pa_rope_and_cache, pa.pa_rope_and_cache_fp8
    bad = [
        lambda: rope(q, q, k, k, pool.bfloat16(), pool, slots, slots, cs),
        lambda: rope(q, q, k, k.float(), pool, pool, slots, slots, cs),
        lambda: rope(q, q, k, k, pool, pool, slots.int(), slots, cs),
        lambda: rope(q, q, k, k, pool, pool, slots, slots[:2], cs),
        lambda: rope(q, q, k, wide, pool, pool, slots, slots, cs),
        lambda: rope(q[:2], q, k, k, pool, pool, slots, slots, cs),
        lambda: rope(q, q, k, k, pool, pool, slots, slots, cs, (8, 24)),
        lambda: rope(q, q, k.float(), k.float(), pool, pool, slots, slots, cs),
        lambda: rope8(q, q, k, k, pool, codes, scale, slots, slots, cs),
        lambda: rope8(q, q, k, k, codes, codes, scale[:3], slots, slots, cs),
        lambda: pa.pa_paged_decode_attention_fp8(q, q, codes, codes, scale, table, lens, 1.0, 2),
        lambda: pa.pa_paged_decode_attention_fp8(out, q, codes, codes, scale, table, lens, 1.0, 4),
        lambda: pa.pa_paged_decode_attention_fp8(out, q, codes, codes, scale, table[:2], lens, 1.0, 2),
        lambda: pa.pa_paged_decode_attention_fp8(out, q, codes, codes, scale, table, lens, 1.0, 2, 17),
        lambda: pa.pa_copy_blocks_fp8(codes, codes, scale, torch.zeros(1, 3, dtype=torch.int64, device=cuda_device)),
        lambda: pa.pa_gather_cache_fp8(k, k.bfloat16(), codes, codes, scale, table[:1], start),
        lambda: pa.pa_gather_cache_fp8(k, k, codes, codes, scale, table, start),
        lambda: pa.pa_prompt_attention(q, q, k, k, start, start[:1], 1.0, 2, 3, 3),
        lambda: pa.pa_prompt_attention(q, q, k, k, start, start, 1.0, 4, 3, 3),
        lambda: pa.pa_prompt_attention(out, q, k, k, start, start, 1.0, 2, 3, 3),
        lambda: pa.pa_prompt_attention(q, q, wide, k, start, start, 1.0, 2, 3, 3),
        lambda: pa.pa_prompt_attention(q, q, k, k, start, start, 1.0, 2, -1, 3),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((TypeError, ValueError, pa.PAError)):
            call()
            pytest.fail(f"call {i} was taken")
