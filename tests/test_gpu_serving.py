"""The operators together, as a serving engine uses them: prompts of mixed
lengths through rotary write and prompt attention, decode steps over the 8-bit
pool, a fork with copy-on-write, and a second request that finds its prefix in
the cache and gathers it -- each step against a 64-bit model of the same
tokens."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

HQ, HKV, D, B = 8, 2, 64, 16


def turn(x, pos, table):
    h = D // 2
    c, s = table[pos, :h].double()[:, None], table[pos, h:].double()[:, None]
    a, b = x[..., :h].double(), x[..., h:].double()
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def attend(q, k, v):
    """64-bit causal attention: the queries are the last of the keys' positions."""
    C, L = len(q), len(k)
    seen = torch.arange(L, device="cuda") <= L - C + torch.arange(C, device="cuda")[:, None]
    k, v = (x.repeat_interleave(HQ // HKV, 1) for x in (k, v))
    z = torch.einsum("chd,lhd->hcl", q, k) / math.sqrt(D)
    return torch.einsum("hcl,lhd->chd", torch.softmax(z.masked_fill(~seen, -math.inf), -1), v)


def test_prompts_decode_fork_and_prefix(pa, cuda_device):
    g = torch.Generator(device="cuda").manual_seed(0)
    NB, table = 64, torch.cat([f(torch.arange(512, device="cuda")[:, None]
                                 * 10000.0 ** (-torch.arange(0, D, 2, device="cuda") / D))
                               for f in (torch.cos, torch.sin)], 1).float().contiguous()
    bm = pa.BlockManager(NB, B)
    kc, vc = (torch.full((NB, HKV, B, D), float("nan"), device="cuda").to(torch.float8_e4m3fn)
              for _ in range(2))
    sc = torch.full((NB, HKV, 2, B), float("nan"), device="cuda")
    scale = 1 / math.sqrt(D)
    model = {}          # sequence -> 64-bit turned keys and values of its tokens

    def write(seqs, counts, slots):
        """New tokens of each sequence: turned queries, and K/V into the pool and the model."""
        T = sum(counts)
        qkv = torch.randn(T, HQ + 2 * HKV, D, generator=g, device="cuda").bfloat16()
        q, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:]
        at = [len(model[s][0]) if s in model else 0 for s in seqs]
        pos = torch.cat([torch.arange(a, a + n, device="cuda") for a, n in zip(at, counts)])
        qo = torch.empty(T, HQ, D, dtype=torch.bfloat16, device="cuda")
        pa.pa_rope_and_cache_fp8(qo, q, k, v, kc, vc, sc, torch.as_tensor(slots, device="cuda"), pos, table)
        tk = turn(k, pos, table)
        i = 0
        for s, n in zip(seqs, counts):
            old = model.get(s, (tk[:0], v.double()[:0]))
            model[s] = (torch.cat([old[0], tk[i:i + n]]), torch.cat([old[1], v[i:i + n].double()]))
            i += n
        return qo, tk.bfloat16(), v.contiguous(), turn(q, pos, table)

    def slots_of(seq, first, n):
        blocks = torch.as_tensor(bm.block_tables([seq], NB)[0][0])
        at = torch.arange(first, first + n)
        return blocks.long()[at // B] * B + at % B

    # e4m3 keys and values: an element is off by 2^-4 of itself, a score by the sum of D such
    # errors (independent: 2^-4 |q| |k| / sqrt(D) ~ 2^-4 sqrt(D) scale, some 0.06 each) and the output
    # by a fraction of |v|; bf16 ones by 2^-8.  Bars on the root mean square, against 1 for v.
    def close(got, want, bar):
        err = (got.double() - want).pow(2).mean().sqrt().item()
        assert err <= bar, err

    # 1. three fresh prompts: rotary write, then attention from the projections
    counts = [37, 5, 130]
    for s, n in enumerate(counts):
        bm.allocate(s, n)
    qo, k16, v16, tq = write([0, 1, 2], counts, torch.cat([slots_of(s, 0, n) for s, n in enumerate(counts)]))
    start = torch.tensor(np.cumsum([0] + counts), dtype=torch.int32, device="cuda")
    out = torch.empty_like(qo)
    pa.pa_prompt_attention(out, qo, k16, v16, start, start, scale, HKV, 130, 130)
    a = np.cumsum([0] + counts)
    close(out, torch.cat([attend(tq[a[i]:a[i + 1]], *model[i]) for i in range(3)]), 2.0 ** -6)

    # 2. a fork, then decode steps; the first write into a shared block copies it
    bm.fork(2, 3)
    model[3] = model[2]
    seqs = [0, 1, 2, 3]
    for step in range(20):
        slots, pairs = bm.append_slots(seqs)
        if len(pairs):
            pa.pa_copy_blocks_fp8(kc, vc, sc, torch.as_tensor(np.asarray(pairs), device="cuda"))
        qo, _, _, tq = write(seqs, [1] * 4, np.asarray(slots))
        tables, lens = bm.block_tables(seqs, 12)
        dout = torch.empty(4, HQ, D, device="cuda")
        pa.pa_paged_decode_attention_fp8(dout, qo, kc, vc, sc, torch.as_tensor(tables, device="cuda"),
                                         torch.as_tensor(lens, device="cuda"), scale, HKV)
        close(dout, torch.cat([attend(tq[i:i + 1], *model[s]) for i, s in enumerate(seqs)]), 2.0 ** -4)
    assert len(pairs) == 0 and torch.equal(model[2][0][:130], model[3][0][:130])

    # 3. a chunk behind a cached context: gather it, append the new rows, attend
    n, L = 29, len(model[3][0])
    slots, _ = bm.append_slots([3] * n)
    qo, k16, v16, tq = write([3], [n], np.asarray(slots))
    tables, _ = bm.block_tables([3], 12)
    key, value = (torch.empty(L + n, HKV, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pa.pa_gather_cache_fp8(key, value, kc, vc, sc, torch.as_tensor(tables, device="cuda"),
                           torch.tensor([0, L], dtype=torch.int32, device="cuda"))
    key[L:], value[L:] = k16, v16
    out = torch.empty_like(qo)
    pa.pa_prompt_attention(out, qo, key, value, torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                           torch.tensor([0, L + n], dtype=torch.int32, device="cuda"), scale, HKV, n, L + n)
    close(out, attend(tq, *model[3]), 2.0 ** -4)
    assert pa.pa_device_error() == 0
    bm.close()


def test_turned_keys_with_the_queries(pa, cuda_device):
    """One pass turns a fused projection's query and key heads for prompt attention and fills the
    16-bit pool; the next chunk decodes over that pool as the prompt attends over itself."""
    g = torch.Generator(device="cuda").manual_seed(5)
    lens = [70, 1, 33]
    T, S = sum(lens), len(lens)
    ang = torch.arange(128, device="cuda")[:, None] * 10000.0 ** (-torch.arange(0, D, 2, device="cuda") / D)
    table = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
    qkv = torch.randn(T, HQ + 2 * HKV, D, generator=g, device="cuda").bfloat16()
    k, v = qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:]
    pos = torch.cat([torch.arange(n, device="cuda") for n in lens])
    nb = [-(-n // B) for n in lens]
    blocks = torch.randperm(sum(nb), generator=torch.Generator().manual_seed(6)).int()
    tables = torch.zeros(S, max(nb), dtype=torch.int32)
    for s, own in enumerate(blocks.split(nb)):
        tables[s, :nb[s]] = own
    slots = torch.cat([tables[s].long()[torch.arange(n) // B] * B + torch.arange(n) % B
                       for s, n in enumerate(lens)]).cuda()
    kc, vc = (torch.zeros(sum(nb), HKV, B, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    turned = torch.empty(T, HQ + HKV, D, dtype=torch.bfloat16, device="cuda")
    pa.pa_rope_and_cache(turned, qkv[:, :HQ + HKV], k, v, kc, vc, slots, pos, table)
    # the pool's keys are those handed to prompt attention, and V's rows are v's
    at = slots // B, slice(None), slots % B
    assert torch.equal(kc[at], turned[:, HQ:]) and torch.equal(vc[at], v)
    start = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda")
    out = torch.empty(T, HQ, D, dtype=torch.bfloat16, device="cuda")
    scale = 1 / math.sqrt(D)
    pa.pa_prompt_attention(out, turned[:, :HQ], turned[:, HQ:], v, start, start, scale, HKV, 70, 70)
    # a prompt's last token attends over all of it, as decode's new token does.  Decode is fp32
    # from the same 16-bit inputs; the prompt rounds each weight and the output to bf16, off by at
    # most 2^-8 of themselves, together 2^-7 of the largest |v|
    last = (start[1:] - 1).long()
    dec = torch.empty(S, HQ, D, device="cuda")
    ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = pa.alloc_workspace(S, HQ, HKV, D, B, max(nb) * B)
    pa.pa_paged_decode_attention(dec, turned[last, :HQ].contiguous(), kc, vc, tables.cuda(), ctx, scale, HKV,
                                 workspace=ws)
    assert (out[last].float() - dec).abs().max().item() <= 2.0 ** -7 * v.float().abs().max().item()
    assert pa.pa_device_error() == 0
