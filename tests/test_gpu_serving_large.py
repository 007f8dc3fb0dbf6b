"""GPU tests of the paths that only large calls take: a warp's second token and further ones in the
rotary write, cut contexts of more than a thousand sequences (with the merge of several heads at
once) and forced cuts in 8-bit decode, hundreds of sequences in the gather.  Against 64-bit forms;
the tolerances count fp32 operations (2^-24) and roundings to a type (half its eps)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
E4M3 = torch.float8_e4m3fn
U32 = 2.0 ** -24


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ------------------------------------------------------------------ rotary write

def turned(x, c, s, pairs):
    """x [T, H, D] with its first columns turned by c, s [T, half], in 64 bits, and the size of what
    was added up for each element."""
    half = c.shape[1]
    first, second = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if pairs
                     else (slice(0, half), slice(half, 2 * half)))
    y, c, s = x.double().clone(), c.double()[:, None], s.double()[:, None]
    a, b = x[..., first].double(), x[..., second].double()
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    size = x.double().abs().clone()
    size[..., first] = (a * c).abs() + (b * s).abs()
    size[..., second] = (b * c).abs() + (a * s).abs()
    return y, size


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype,Hq,Hkv,D,B,T,rot,sect,pairs", [
    ("bf16", 5, 1, 128, 16, 8001, 128, (20, 24, 20), False),
    ("f16", 3, 3, 64, 32, 11111, 32, (16,), True),
    ("bf16", 16, 8, 128, 16, 4097, 64, (5, 27), False),
])
def test_rope_of_many_tokens(pa, cuda_device, dtype, Hq, Hkv, D, B, T, rot, sect, pairs, fp8):
    """Every warp takes several tokens, some of which are skipped (bad positions) or not stored."""
    dt, g, most = DT[dtype], generator(T), 5000
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device="cuda").to(dt)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    angle = torch.rand(most, rot // 2, generator=g, device="cuda") * 6.2832
    cs = torch.cat([angle.cos(), angle.sin()], 1)
    NB = -(-T // B) + 5
    slots = torch.randperm(NB * B, generator=g, device="cuda")[:T]
    slots[torch.rand(T, generator=g, device="cuda") < 0.05] = -1
    pos = torch.randint(most, (len(sect), T), generator=g, device="cuda")
    bad = torch.rand(T, generator=g, device="cuda") < 0.02
    bad[:2], bad[-1] = True, True
    pos[0, bad], pos[-1, 1] = most, -1
    q_out = torch.full((T, Hq, D), 9.0, dtype=dt, device="cuda")
    kind = E4M3 if fp8 else dt
    caches = [torch.full((NB, Hkv, B, D), 7.0, device="cuda").to(kind) for _ in range(2)]
    sc = torch.full((NB, Hkv, 2, B), 5.0, device="cuda")
    write = pa.pa_rope_and_cache_fp8 if fp8 else pa.pa_rope_and_cache
    write(q_out, q, k, v, *caches, *([sc] if fp8 else []), slots, pos, cs, sect, pairs)
    assert pa.pa_device_error(clear=True) == pa.DEVERR["position"]
    axis = torch.cat([torch.full((n,), a) for a, n in enumerate(sect)]).cuda()
    at = pos[axis].T.clamp(0, most - 1)                              # [T, half]
    j = torch.arange(rot // 2, device="cuda")
    c, s = cs[at, j], cs[at, rot // 2 + j]
    (yq, sq), (yk, sk) = (turned(x, c, s, pairs) for x in (q, k))
    e = torch.finfo(dt).eps / 2
    off = (q_out.double() - yq).abs() <= e * yq.abs() + (1 + e) * 3 * U32 * sq + 2.0 ** -25
    assert off[~bad].all() and (q_out[bad] == 9).all()
    keep = (slots >= 0) & ~bad
    blk, row = slots[keep] // B, slots[keep] % B
    untouched = torch.ones(NB, B, dtype=torch.bool, device="cuda")
    untouched[blk, row] = False
    for n, (cache, x, size) in enumerate(((caches[0], yk, sk), (caches[1], v.double(), v.double().abs()))):
        x, size = x[keep], size[keep]
        raw = cache.view(torch.uint8) if fp8 else cache
        got = raw[blk, :, row].view(kind).double()
        if fp8:
            scale = sc[:, :, n][blk, :, row].double()
            assert ((scale - x.abs().amax(-1) / 448).abs() <= 5 * U32 * size.amax(-1) / 448).all()
            tol = x.abs() * 2.0 ** -4 + scale[..., None] * 2.0 ** -10 + 8 * U32 * size.amax(-1, True)
            assert ((got * scale[..., None] - x).abs() <= tol).all()
            assert (sc[:, :, n].transpose(1, 2)[untouched] == 5).all()
        else:
            assert ((got - x).abs() <= e * x.abs() + (1 + e) * 3 * U32 * size + 2.0 ** -25).all()
        assert (cache.transpose(1, 2)[untouched].double() == 7).all()


# ------------------------------------------------------------------ 8-bit pool

def made_pool(lens, Hkv, B, D, seed):
    """A pool, its tables, and NaN in every row that no sequence holds."""
    g, need = generator(seed), [-(-n // B) for n in lens]
    NB = sum(need) + 3
    k, v = (torch.randn(NB, Hkv, B, D, generator=g, device="cuda").mul(100).clamp(-448, 448).to(E4M3)
            for _ in range(2))
    sc = torch.rand(NB, Hkv, 2, B, generator=g, device="cuda").add(0.2) / 100
    order = torch.randperm(NB, generator=g, device="cuda").int().cpu()
    tables = torch.full((len(lens), max(need)), -7, dtype=torch.int32)
    dead = torch.ones(NB, B, dtype=torch.bool)
    first = 0
    for i, n in enumerate(need):
        tables[i, :n] = order[first:first + n]
        first += n
        dead[tables[i, :n].long()] = False
        if lens[i] % B:
            dead[tables[i, n - 1].long(), lens[i] % B:] = True
    dead = dead.cuda()[:, None].expand(-1, Hkv, -1)
    for c in (k, v):
        c.view(torch.uint8)[dead] = 0x7F
    sc.transpose(2, 3)[dead] = float("nan")
    return k, v, sc, tables.cuda()


def rows_of(codes, scale, which, table, n, B):
    at = torch.arange(n, device="cuda")
    blk, off = table.long()[at // B], at % B
    return codes.view(torch.uint8)[blk, :, off].view(E4M3).double(), scale[blk, :, which, off].double()


def check_decode(out, q, k, v, sc, tables, lens, B, scale):
    """A score: D products, scaled and shifted, which moves a weight twice; some steps for the
    weight's halves, exp2 and the joins; half of fp16's smallest step is 2^-39 of a tile's largest
    weight times V scale."""
    worst = torch.zeros((), dtype=torch.float64, device="cuda")
    for i, n in enumerate(lens):
        if n == 0:
            assert (out[i] == 0).all()
            continue
        (kc, ks), (c, vs) = (rows_of(x, sc, w, tables[i], n, B) for w, x in ((0, k), (1, v)))
        qq, K = q[i].double().view(k.shape[1], -1, q.shape[2]), kc * ks[..., None]
        y = torch.softmax(torch.einsum("hgd,nhd->hgn", qq, K) * scale, -1) * vs.T[:, None]
        terms = (torch.einsum("hgd,nhd->hgn", qq.abs(), K.abs()) * abs(scale)).amax()
        tol = (U32 * (2 * (q.shape[2] + 8) * terms + 64) * torch.einsum("hgn,nhd->hgd", y, c.abs())
               + 2.0 ** -39 * y.amax(-1, keepdim=True) * c.abs().sum(0)[:, None])
        off = (out[i].double().view(tol.shape) - torch.einsum("hgn,nhd->hgd", y, c)).abs() / tol
        worst = torch.maximum(worst, torch.nan_to_num(off, nan=torch.inf).amax())
    assert worst <= 1, worst.item()


@pytest.mark.parametrize("dtype,Hq,Hkv,D,B", [("bf16", 6, 2, 64, 16), ("f16", 12, 2, 128, 32),
                                              ("bf16", 26, 2, 64, 32), ("f16", 3, 1, 128, 16)])
def test_decode_fp8_of_many_cut_sequences(pa, cuda_device, dtype, Hq, Hkv, D, B):
    S = 1117
    lens = [0 if i % 11 == 3 else 200 + (37 * i) % 401 for i in range(S)]
    k, v, sc, tables = made_pool(lens, Hkv, B, D, seed=Hq)
    q = torch.randn(S, Hq, D, generator=generator(5), device="cuda").to(DT[dtype])
    out = torch.full((S, Hq, D), float("nan"), device="cuda")
    pa.pa_paged_decode_attention_fp8(out, q, k, v, sc, tables, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                     D ** -0.5, Hkv)
    assert pa.pa_device_error(clear=True) == 0
    check_decode(out, q, k, v, sc, tables, lens, B, D ** -0.5)


@pytest.mark.parametrize("ctas,tiles", [(1, 1), (2, 1), (0, 3), (1, 7), (4, 1000)])
@pytest.mark.parametrize("dtype,Hq,Hkv,D,B", [("bf16", 13, 1, 128, 16), ("f16", 20, 4, 64, 32),
                                              ("bf16", 9, 3, 128, 32)])
def test_decode_fp8_launch_shapes(pa, cuda_device, dtype, Hq, Hkv, D, B, ctas, tiles):
    lens = [1, 0, 33, 500, 64, 2500, 31, 32, 97, 0, 1000, 5]
    k, v, sc, tables = made_pool(lens, Hkv, B, D, seed=D)
    q = torch.randn(len(lens), Hq, D, generator=generator(6), device="cuda").to(DT[dtype])
    out = torch.full((len(lens), Hq, D), float("nan"), device="cuda")
    try:
        pa.pa_decode_tuning(ctas_per_sm=ctas, min_tiles_per_warp=tiles)
        pa.pa_paged_decode_attention_fp8(out, q, k, v, sc, tables,
                                         torch.tensor(lens, dtype=torch.int32, device="cuda"), D ** -0.5, Hkv)
    finally:
        pa.pa_decode_tuning()
    assert pa.pa_device_error(clear=True) == 0
    check_decode(out, q, k, v, sc, tables, lens, B, D ** -0.5)


def test_gather_of_many_sequences(pa, cuda_device):
    B, Hkv, D, dt = 16, 2, 64, torch.bfloat16
    lens = [(13 * i) % 41 if i % 3 else 0 for i in range(777)]
    k, v, sc, tables = made_pool(lens, Hkv, B, D, seed=8)
    start = torch.tensor(np.cumsum([5] + lens), dtype=torch.int32, device="cuda")
    T = 5 + sum(lens)
    key, value = (torch.full((T + 7, Hkv, D), 7.0, dtype=dt, device="cuda") for _ in range(2))
    pa.pa_gather_cache_fp8(key, value, k, v, sc, tables, start)
    assert pa.pa_device_error(clear=True) == 0
    for w, (got, codes) in enumerate(((key, k), (value, v))):
        parts = [rows_of(codes, sc, w, tables[i], n, B) for i, n in enumerate(lens) if n]
        want = torch.cat([c * s[..., None] for c, s in parts])
        # one fp32 product, one rounding
        assert ((got[5:T].double() - want).abs() <= (torch.finfo(dt).eps / 2 + 2 * U32) * want.abs()).all()
        assert (got[:5] == 7).all() and (got[T:] == 7).all()
