"""The operators around the 8-bit paged cache: cases, plain forms and the library's calls.

Five operators, each a case's "op":

* ``rope``    rotary positions on q and k (one or several position axes) and the
              write of K/V into their slots, into an e4m3 pool with one scale
              per token, kv head and K or V, or into a 16-bit pool.
* ``decode``  attention of one new token per sequence over the e4m3 pool.
* ``prompt``  causal attention over packed prompts of different lengths.
* ``gather``  cached rows out of the e4m3 pool, packed, in 16 bits.
* ``copy``    copy-on-write copies of e4m3 blocks with their scales.

``run`` computes a case in plain torch operations (``own`` false) or by the
library's calls (``own`` true); ``exact`` computes it in 64 bits, one sequence
and one head at a time.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
E4M3 = torch.float8_e4m3fn
TOP = 448.0            # largest e4m3 value
LEAST = 2.0 ** -100    # smallest magnitude a row's scale is made for
MAX_POSITION = 32768


def listed():
    gqa = {"q_heads": 32, "kv_heads": 8, "dim": 128, "block": 16, "dtype": "bf16"}
    return [
        # the step of a decode batch: 256 new tokens, text positions
        {"name": "rope decode step", "op": "rope", **gqa, "tokens": 256, "rotary": 128,
         "axes": 1, "pairs": False, "fp8": True},
        # prompts with images, 16K tokens: time, height and width positions
        {"name": "rope image prompts", "op": "rope", **gqa, "tokens": 16384, "rotary": 128,
         "axes": 3, "pairs": False, "fp8": True},
        # one user, small heads: the latency of a call
        {"name": "decode one sequence", "op": "decode", "q_heads": 4, "kv_heads": 4, "dim": 64,
         "block": 16, "dtype": "f16", "seqs": 1, "low": 777, "high": 777, "mix": 1},
        # a serving batch of mixed lengths, 16 to 4096 tokens
        {"name": "decode mixed batch", "op": "decode", **gqa, "seqs": 256, "low": 16,
         "high": 4096, "mix": 2},
        # a few long documents, 16K to 32K tokens, wide groups
        {"name": "decode long contexts", "op": "decode", "q_heads": 64, "kv_heads": 8,
         "dim": 128, "block": 32, "dtype": "bf16", "seqs": 8, "low": 16384, "high": 32768,
         "mix": 3},
        # short last chunks after long cached prefixes: few rows, many keys
        {"name": "prompt chunks on prefixes", "op": "prompt", "q_heads": 64, "kv_heads": 8,
         "dim": 128, "dtype": "bf16", "seqs": 3, "low": 5, "high": 40, "before_low": 4000,
         "before_high": 16000, "mix": 4},
        # a batch of fresh prompts of mixed lengths, no grouped heads
        {"name": "prompt ragged batch", "op": "prompt", "q_heads": 40, "kv_heads": 40,
         "dim": 128, "dtype": "f16", "seqs": 16, "low": 64, "high": 2048, "before_low": 0,
         "before_high": 0, "mix": 5},
        # one long prompt
        {"name": "prompt one of 8192", "op": "prompt", "q_heads": 32, "kv_heads": 8, "dim": 128,
         "dtype": "bf16", "seqs": 1, "low": 8192, "high": 8192, "before_low": 0,
         "before_high": 0, "mix": 6},
        # a prefix hit of one request
        {"name": "gather one prefix", "op": "gather", **gqa, "seqs": 1, "low": 300, "high": 300,
         "mix": 7},
        # the cached contexts of a batch of chunks
        {"name": "gather batch of contexts", "op": "gather", **gqa, "seqs": 16, "low": 512,
         "high": 8192, "mix": 8},
        # the copies of one step of forked sequences
        {"name": "copy one step", "op": "copy", **gqa, "pairs": 37},
        # every branch of many forks writes for the first time
        {"name": "copy first writes", "op": "copy", **gqa, "pairs": 2048},
    ]


def draw(rng):
    def logint(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rope", "decode", "prompt", "gather", "copy", "decode", "prompt"])
    q_heads, kv_heads = rng.choice([(32, 8), (40, 40), (64, 8), (4, 4), (12, 4), (16, 1), (10, 2)])
    c = {"op": op, "q_heads": q_heads, "kv_heads": kv_heads, "dim": rng.choice([64, 128]),
         "dtype": rng.choice(["bf16", "f16"])}
    if op != "prompt":
        c["block"] = rng.choice([16, 32])
    if op == "rope":
        axes = rng.choice([1, 3])
        width = (q_heads + 2 * kv_heads) * c["dim"]
        most = max(2, 16384 * 48 * 128 // width)
        return {**c, "tokens": logint(1, min(most, 16384)), "axes": axes,
                "rotary": c["dim"] if axes > 1 else rng.choice([c["dim"], c["dim"] // 2]),
                "pairs": rng.random() < 0.3, "fp8": rng.random() < 0.7}
    c["mix"] = rng.randrange(1 << 20)
    if op == "copy":
        del c["mix"]
        return {**c, "pairs": logint(1, 2048 * 8 * 16 * 128
                                     // (kv_heads * c["block"] * c["dim"]) // 4 + 1)}
    if op == "prompt":
        high = logint(1, 2048)
        before = rng.choice([0, 0, logint(1, 8192)])
        pairs = high * (high + before) * q_heads
        seqs = logint(1, max(1, min(16, 8192 * 8192 * 8 // pairs)))
        return {**c, "seqs": seqs, "low": rng.randint(1, high), "high": high,
                "before_low": rng.randint(0, before), "before_high": before}
    # decode and gather: at most 128K tokens of 8 heads of 128, padded to the longest
    high = logint(1, 32768)
    most = (1 << 17) * 8 * 128 // (kv_heads * c["dim"] * high)
    if most < 1:
        high, most = 4096, max(1, (1 << 17) * 8 * 128 // (kv_heads * c["dim"] * 4096))
    return {**c, "seqs": logint(1, min(256, most)), "low": rng.randint(0, high), "high": high}


def lengths(case, low="low", high="high", salt=0):
    """The case's lengths, spread over their logarithm (from `low` to `high`)."""
    r, lo, hi = random.Random(case["mix"] + salt), case[low], case[high]
    return [min(hi, max(lo, int(round(math.exp(r.uniform(math.log(lo + 1), math.log(hi + 1)))) - 1)))
            for _ in range(case["seqs"])]


def sections_of(case):
    """Frequency pairs of each position axis: a quarter for time, the rest for height and width."""
    half = case["rotary"] // 2
    if case["axes"] == 1:
        return (half,)
    t, h = half // 4, (half - half // 4) // 2
    return (t, h, half - t - h)


def starts(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def quantised(x):
    """e4m3 codes [..., D] of x and their scales [...]."""
    top = x.float().abs().amax(-1).clamp(min=LEAST)
    return (x.float() * (TOP / top)[..., None]).to(E4M3), top / TOP


def made_pool(case, blocks, g):
    """An e4m3 pool as cached normal K and V leave it: codes, codes, scales [.., 2, B]."""
    shape = (blocks, case["kv_heads"], case["block"], case["dim"])
    k, ks = quantised(torch.randn(shape, generator=g, device="cuda"))
    v, vs = quantised(torch.randn(shape, generator=g, device="cuda"))
    return k, v, torch.stack([ks, vs], 2).contiguous()


def paged(case, lens, g):
    """A pool in which the sequences' blocks lie in random order, and their tables."""
    block = case["block"]
    need = [-(-n // block) for n in lens]
    blocks = sum(need) + 8
    order = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    wide = max(1, max(need))
    tables = torch.full((len(lens), wide), -1, dtype=torch.int32, device="cuda")
    at = torch.tensor(starts(need)[:-1], device="cuda")[:, None] + torch.arange(wide, device="cuda")
    used = torch.arange(wide, device="cuda") < torch.tensor(need, device="cuda")[:, None]
    tables[used] = order[at[used]]
    return (*made_pool(case, blocks, g), tables)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    hq, hkv, dim = case["q_heads"], case["kv_heads"], case["dim"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)

    def ints(values, kind=torch.int32):
        return torch.tensor(values, dtype=kind, device="cuda")

    if case["op"] == "rope":
        tokens, block, rot = case["tokens"], case["block"], case["rotary"]
        # q, k and v are columns of one projection's output
        qkv = normal(tokens, (hq + 2 * hkv), dim)
        blocks = -(-tokens // block) + 4
        slots = torch.randperm(blocks * block, generator=g, device="cuda")[:tokens]
        slots[torch.rand(tokens, generator=g, device="cuda") < 0.02] = -1   # already cached
        angle = (torch.arange(MAX_POSITION, dtype=torch.float64, device="cuda")[:, None]
                 * 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot))
        pool = torch.zeros(blocks, hkv, block, dim, device="cuda")
        kind = E4M3 if case["fp8"] else dtype
        return {"case": case, "q": qkv[:, :hq], "k": qkv[:, hq:hq + hkv], "v": qkv[:, hq + hkv:],
                "q_out": torch.zeros(tokens, hq, dim, dtype=dtype, device="cuda"),
                "k_cache": pool.to(kind), "v_cache": pool.to(kind),
                "kv_scale": torch.zeros(blocks, hkv, 2, block, device="cuda"),
                "slots": slots, "sections": sections_of(case),
                "positions": torch.randint(MAX_POSITION, (case["axes"], tokens), generator=g,
                                           device="cuda"),
                "cos_sin": torch.cat([angle.cos(), angle.sin()], 1).float()}
    if case["op"] == "copy":
        n = case["pairs"]
        k, v, scale = made_pool(case, 2 * n + 8, g)
        pairs = torch.randperm(2 * n + 8, generator=g, device="cuda")[:2 * n].view(n, 2)
        return {"case": case, "k_cache": k, "v_cache": v, "kv_scale": scale,
                "pairs": pairs.contiguous()}
    lens = lengths(case)
    if case["op"] == "prompt":
        before = lengths(case, "before_low", "before_high", 1)
        keys = [a + b for a, b in zip(lens, before)]
        t, tk = sum(lens), sum(keys)
        return {"case": case, "q": normal(t, hq, dim), "k": normal(tk, hkv, dim),
                "v": normal(tk, hkv, dim), "out": torch.zeros(t, hq, dim, dtype=dtype, device="cuda"),
                "query_start": ints(starts(lens)), "key_start": ints(starts(keys)),
                "max_query": max(lens), "max_key": max(keys), "scale": dim ** -0.5}
    k, v, scale, tables = paged(case, lens, g)
    state = {"case": case, "k_cache": k, "v_cache": v, "kv_scale": scale, "tables": tables,
             "lens": ints(lens), "longest": max(lens)}
    if case["op"] == "gather":
        state["key_start"] = ints(starts(lens))
        state["key"], state["value"] = (torch.zeros(sum(lens), hkv, dim, dtype=dtype, device="cuda")
                                        for _ in range(2))
    else:
        state["q"] = normal(case["seqs"], hq, dim)
        state["out"] = torch.zeros(case["seqs"], hq, dim, device="cuda")
        state["scale"] = dim ** -0.5
        # scratch, larger than any of these calls asks for
        state["workspace"] = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    return state


# ------------------------------------------------------------------ plain forms

def rotated(x, s):
    """x [T, H, D] in 32 bits with its first `rotary` columns turned by the table's angles."""
    case, half = s["case"], s["case"]["rotary"] // 2
    pair = torch.arange(half, device=x.device)
    row = torch.cat([p[:, None].expand(-1, n)                # each pair's position: [T, half]
                     for p, n in zip(s["positions"], s["sections"])], 1)
    c, n = (s["cos_sin"][row, pair + d][:, None] for d in (0, half))
    x = x.float()
    if case["pairs"]:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * c - b * n, b * c + a * n], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def plain_rope(s):
    block = s["case"]["block"]
    s["q_out"].copy_(rotated(s["q"], s))
    kept = s["slots"] >= 0
    slot = s["slots"][kept]
    at, off = slot // block, slot % block
    for n, x, cache in ((0, rotated(s["k"], s), s["k_cache"]), (1, s["v"].float(), s["v_cache"])):
        x = x[kept]
        if s["case"]["fp8"]:
            codes, scale = quantised(x)
            cache.view(torch.uint8)[at, :, off] = codes.view(torch.uint8)
            s["kv_scale"][:, :, n][at, :, off] = scale
        else:
            cache[at, :, off] = x.to(cache.dtype)
    return [s["q_out"], s["k_cache"], s["v_cache"], s["kv_scale"]]


def cached(s, n, tables):
    """Rows of K (n = 0) or V (n = 1) through the tables, in 32 bits: [S, L, Hkv, D]."""
    codes = (s["k_cache"], s["v_cache"])[n].view(torch.uint8)[tables].view(E4M3)
    x = codes.float() * s["kv_scale"][tables][:, :, :, n, :, None]      # [S, nb, Hkv, B, D]
    return x.transpose(2, 3).flatten(1, 2)


def softmax_product(scores, seen, v):
    """softmax over the keys that are seen, times v; rows that see nothing give zeros."""
    scores.masked_fill_(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    return (p @ v) / total.masked_fill(total == 0, 1.0)


def plain_decode(s):
    hkv, dim = s["case"]["kv_heads"], s["case"]["dim"]
    tables = s["tables"].clamp(min=0).long()
    k, v = (cached(s, n, tables).transpose(1, 2) for n in (0, 1))       # [S, Hkv, L, D]
    q = s["q"].float().view(len(tables), hkv, -1, dim)
    scores = (q @ k.transpose(-1, -2)) * s["scale"]
    seen = torch.arange(k.shape[2], device=q.device) < s["lens"][:, None]
    s["out"].copy_(softmax_product(scores, seen[:, None, None], v).flatten(1, 2))
    return s["out"]


def plain_gather(s):
    tables = s["tables"].clamp(min=0).long()
    seen = (torch.arange(tables.shape[1] * s["case"]["block"], device=tables.device)
            < s["lens"][:, None])
    s["key"].copy_(cached(s, 0, tables)[seen])
    s["value"].copy_(cached(s, 1, tables)[seen])
    return [s["key"], s["value"]]


def plain_copy(s):
    src, dst = s["pairs"][:, 0], s["pairs"][:, 1]
    for x in (s["k_cache"].view(torch.uint8), s["v_cache"].view(torch.uint8), s["kv_scale"]):
        x[dst] = x[src]
    return [s["k_cache"], s["v_cache"], s["kv_scale"]]


def padded(x, start, longest):
    """Packed rows [T, H, D] as [S, longest, H, D] in 32 bits, and which of them are rows."""
    at = torch.arange(longest, device=x.device)
    first, size = start[:-1, None].long(), (start[1:] - start[:-1])[:, None]
    return x[(first + at).clamp(max=x.shape[0] - 1)].float(), at < size


def plain_prompt(s):
    case = s["case"]
    hkv, group = case["kv_heads"], case["q_heads"] // case["kv_heads"]
    q, rows = padded(s["q"], s["query_start"], s["max_query"])
    k, keys = padded(s["k"], s["key_start"], s["max_key"])
    v, _ = padded(s["v"], s["key_start"], s["max_key"])
    n, c = rows.shape
    k, v = (x.transpose(1, 2).contiguous() for x in (k, v))             # [S, Hkv, L, D]
    q = q.view(n, c, hkv, group, -1).permute(0, 2, 3, 1, 4).reshape(n, hkv, group * c, -1)
    scores = ((q @ k.transpose(-1, -2)).mul_(s["scale"])).view(n, hkv, group, c, -1)
    size_q, size_k = ((x[1:] - x[:-1])[:, None, None] for x in (s["query_start"], s["key_start"]))
    last = size_k - size_q + torch.arange(c, device=q.device)[:, None]
    seen = (torch.arange(k.shape[2], device=q.device) <= last) & keys[:, None]
    o = softmax_product(scores, seen[:, None, None], v[:, :, None])     # [S, Hkv, G, C, D]
    s["out"].copy_(o.permute(0, 3, 1, 2, 4).flatten(2, 3)[rows])
    return s["out"]


# ------------------------------------------------------------------ the library's calls

def own_call(s):
    import paged_kv_cache_414_b200 as pa
    op, hkv = s["case"]["op"], s["case"]["kv_heads"]
    if op == "rope":
        if s["case"]["fp8"]:
            pa.pa_rope_and_cache_fp8(s["q_out"], s["q"], s["k"], s["v"], s["k_cache"],
                                     s["v_cache"], s["kv_scale"], s["slots"], s["positions"],
                                     s["cos_sin"], s["sections"], interleaved=s["case"]["pairs"])
        else:
            pa.pa_rope_and_cache(s["q_out"], s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"],
                                 s["slots"], s["positions"], s["cos_sin"], s["sections"],
                                 interleaved=s["case"]["pairs"])
        return [s["q_out"], s["k_cache"], s["v_cache"], s["kv_scale"]]
    if op == "decode":
        return pa.pa_paged_decode_attention_fp8(
            s["out"], s["q"], s["k_cache"], s["v_cache"], s["kv_scale"], s["tables"], s["lens"],
            s["scale"], hkv, s["longest"], s["workspace"])
    if op == "gather":
        pa.pa_gather_cache_fp8(s["key"], s["value"], s["k_cache"], s["v_cache"], s["kv_scale"],
                               s["tables"], s["key_start"])
        return [s["key"], s["value"]]
    if op == "copy":
        pa.pa_copy_blocks_fp8(s["k_cache"], s["v_cache"], s["kv_scale"], s["pairs"])
        return [s["k_cache"], s["v_cache"], s["kv_scale"]]
    return pa.pa_prompt_attention(s["out"], s["q"], s["k"], s["v"], s["query_start"],
                                  s["key_start"], s["scale"], hkv, s["max_query"], s["max_key"])


def run(state):
    if own:
        return own_call(state)
    return {"rope": plain_rope, "decode": plain_decode, "prompt": plain_prompt,
            "gather": plain_gather, "copy": plain_copy}[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    hq, hkv, dim = case["q_heads"], case["kv_heads"], case["dim"]
    cell = hkv * (2 * dim + 8)                # a cached token: codes and scales of K and V
    if case["op"] == "rope":
        t = case["tokens"]
        row = cell if case["fp8"] else 4 * hkv * dim
        table = 4 * case["rotary"] * min(t, MAX_POSITION)
        return {"bytes": t * (4 * hq * dim + 4 * hkv * dim + row + 8 + 8 * case["axes"]) + table,
                "flops": t * (hq + hkv) * case["rotary"] * 3}
    if case["op"] == "copy":
        return {"bytes": case["pairs"] * (2 * cell * case["block"] + 16), "flops": 0}
    lens = lengths(case)
    n = sum(lens)
    if case["op"] == "prompt":
        before = lengths(case, "before_low", "before_high", 1)
        seen = sum(c * b + c * (c + 1) // 2 for c, b in zip(lens, before))
        return {"bytes": 4 * n * hq * dim + 4 * (n + sum(before)) * hkv * dim,
                "flops": 4 * seen * hq * dim}
    read = n * cell + 4 * sum(-(-x // case["block"]) for x in lens)
    if case["op"] == "gather":
        return {"bytes": read + 4 * n * hkv * dim, "flops": 2 * n * hkv * dim}
    return {"bytes": read + case["seqs"] * hq * dim * 6, "flops": 4 * n * hq * dim}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    """From the definitions, in 64 bits.  Which e4m3 code a value next to the border between
    two gets is no number to compare: None there."""
    s = prepare(case, seed)
    hq, hkv, dim, block = case["q_heads"], case["kv_heads"], case["dim"], case.get("block")
    if case["op"] == "copy":
        order = torch.arange(len(s["k_cache"]), device="cuda")
        order[s["pairs"][:, 1]] = s["pairs"][:, 0]            # which block each one now equals
        return [s["k_cache"].double()[order], s["v_cache"].double()[order],
                s["kv_scale"].double()[order]]
    if case["op"] == "rope":
        half, pool = case["rotary"] // 2, s["k_cache"].double()
        turn = []
        for x in (s["q"].double(), s["k"].double()):
            y, first = x.clone(), 0
            for axis, many in enumerate(s["sections"]):
                for j in range(first, first + many):
                    a, b = (2 * j, 2 * j + 1) if case["pairs"] else (j, j + half)
                    line = s["cos_sin"][s["positions"][axis]].double()
                    c, n = line[:, j, None], line[:, half + j, None]
                    y[..., a] = x[..., a] * c - x[..., b] * n
                    y[..., b] = x[..., b] * c + x[..., a] * n
                first += many
            turn.append(y)
        slot = s["slots"]
        to, frm = slot[slot >= 0], torch.nonzero(slot >= 0)[:, 0]
        rows = [turn[1][frm], s["v"].double()[frm]]
        if case["fp8"]:
            scale = torch.zeros(s["kv_scale"].shape, dtype=torch.float64, device="cuda")
            for n, x in enumerate(rows):
                scale[to // block, :, n, to % block] = x.abs().max(-1).values.clamp(min=LEAST) / TOP
            return [turn[0], None, None, scale]
        caches = []
        for x in rows:
            c = pool.clone()
            c[to // block, :, to % block] = x
            caches.append(c)
        return [turn[0], *caches, s["kv_scale"].double()]
    if case["op"] in ("decode", "gather"):
        lens, out = lengths(case), []
        for i, n in enumerate(lens):
            at = torch.arange(n, device="cuda")
            blk, off = s["tables"][i].long()[at // block], at % block
            kv = [(c.view(torch.uint8)[blk, :, off].view(E4M3).double()
                   * s["kv_scale"][blk, :, m, off].double()[..., None])
                  for m, c in enumerate((s["k_cache"], s["v_cache"]))]   # [n, Hkv, D]
            if case["op"] == "gather":
                out.append(kv)
            elif n == 0:
                out.append(torch.zeros(hq, dim, dtype=torch.float64, device="cuda"))
            else:
                q = s["q"][i].double().view(hkv, -1, dim)
                p = torch.softmax(torch.einsum("hgd,nhd->hgn", q, kv[0]) * s["scale"], -1)
                out.append(torch.einsum("hgn,nhd->hgd", p, kv[1]).reshape(hq, dim))
        if case["op"] == "gather":
            return [torch.cat([kv[m] for kv in out]) for m in (0, 1)]
        return torch.stack(out)
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    qs, ks = s["query_start"].tolist(), s["key_start"].tolist()
    for i in range(case["seqs"]):
        c, n = qs[i + 1] - qs[i], ks[i + 1] - ks[i]
        later = torch.ones(c, n, dtype=torch.bool, device="cuda").triu(n - c + 1)
        for h in range(hq):
            kh = h // (hq // hkv)
            q = s["q"][qs[i]:qs[i + 1], h].double()
            k, v = (x[ks[i]:ks[i + 1], kh].double() for x in (s["k"], s["v"]))
            z = (q @ k.T * s["scale"]).masked_fill_(later, -math.inf)
            o[qs[i]:qs[i + 1], h] = torch.softmax(z, -1) @ v
    return o
