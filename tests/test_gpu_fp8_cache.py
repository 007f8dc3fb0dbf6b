"""GPU tests of the rotary cache write and of the 8-bit pool's operators
(decode attention, gather, block copies) against plain 64-bit forms.

Tolerances come from the arithmetic: a rounding to a type is off by at most
eps / 2 of the value (e4m3: 2^-4 of it, or half its smallest step, 2^-10), an
fp32 operation by 2^-24."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
E4M3 = torch.float8_e4m3fn
LEAST = 2.0 ** -100
U32 = 2.0 ** -24


def half_eps(dtype):
    return torch.finfo(dtype).eps / 2


@pytest.fixture(autouse=True)
def clean_error_word(pa, cuda_device):
    pa.pa_device_error(clear=True)
    yield
    assert pa.pa_device_error(clear=True) == 0     # tests that expect a flag clear it themselves


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def table(rotary, most=4096):
    ang = (torch.arange(most, dtype=torch.float64, device="cuda")[:, None]
           * 10000.0 ** (-torch.arange(0, max(rotary, 2), 2, dtype=torch.float64, device="cuda")
                         / max(rotary, 2)))
    return torch.cat([ang.cos(), ang.sin()], 1)[:, :2 * (rotary // 2)].float().contiguous()


def turned(x, positions, cos_sin, sections, pairs):
    """x [T, H, D] turned, in 64 bits, and for each element the size of what was added up."""
    y, size = x.double().clone(), x.double().abs().clone()
    half, first = cos_sin.shape[1] // 2, 0
    for axis, many in enumerate(sections):
        line = cos_sin[positions[axis]].double()
        for j in range(first, first + many):
            a, b = (2 * j, 2 * j + 1) if pairs else (j, j + half)
            c, s = line[:, j, None], line[:, half + j, None]
            xa, xb = x[..., a].double(), x[..., b].double()
            y[..., a], y[..., b] = xa * c - xb * s, xb * c + xa * s
            size[..., a] = xa.abs() * c.abs() + xb.abs() * s.abs()
            size[..., b] = xb.abs() * c.abs() + xa.abs() * s.abs()
        first += many
    return y, size


def dequantised(codes, scale):
    return codes.double() * scale.double()[..., None]


def make_pool(NB, Hkv, B, D, seed, spread=1.0):
    """Random codes (no NaN) and scales: k, v, kv_scale, and their values in 64 bits."""
    g = generator(seed)
    k, v = (torch.randn(NB, Hkv, B, D, generator=g, device="cuda").mul(100).clamp(-448, 448).to(E4M3)
            for _ in range(2))
    scale = torch.rand(NB, Hkv, 2, B, generator=g, device="cuda").add(0.2).mul(spread / 100)
    return k, v, scale


def make_tables(lens, B, NB, seed, width=None):
    g = generator(seed)
    need = [-(-n // B) for n in lens]
    order = torch.randperm(NB, generator=g, device="cuda").to(torch.int32)
    assert sum(need) <= NB
    wide = max(1, max(need)) if width is None else width
    t = torch.full((len(lens), wide), -7, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):
        t[i, :n] = order[at:at + n]
        at += n
    return t


def poison_unused(k, v, scale, tables, lens, B):
    """NaN codes and scales in every row that no sequence holds."""
    used = torch.zeros(k.shape[0], B, dtype=torch.bool, device="cuda")
    for i, n in enumerate(lens):
        at = torch.arange(n, device="cuda")
        used[tables[i].long()[at // B], at % B] = True
    dead = (~used)[:, None, :].expand(-1, k.shape[1], -1)
    for c in (k, v):
        c.view(torch.uint8)[dead] = 0x7F
    scale[:, :, 0][dead] = float("nan")
    scale[:, :, 1][dead] = float("inf")


def rows_of(codes, scale, which, table_row, n, B):
    """Cached rows of one sequence in 64 bits: [n, Hkv, D]."""
    at = torch.arange(n, device="cuda")
    blk, off = table_row.long()[at // B], at % B
    return (codes.view(torch.uint8)[blk, :, off].view(E4M3).double()
            * scale[blk, :, which, off].double()[..., None])


# ------------------------------------------------------------------ rotary write

ROPE = [
    # dtype, Hq, Hkv, D, B, tokens, rotary, sections, pairs
    ("bf16", 32, 8, 128, 16, 1, 128, None, False),
    ("f16", 4, 4, 64, 32, 5, 64, None, True),
    ("bf16", 3, 1, 128, 32, 333, 128, (16, 24, 24), False),
    ("f16", 16, 1, 128, 16, 77, 64, (3, 20, 9), True),
    ("bf16", 10, 2, 64, 16, 130, 16, (1, 2, 0, 5), False),
    ("f16", 12, 4, 64, 16, 1000, 32, (0, 16), False),
    ("bf16", 40, 40, 128, 16, 700, 128, (64,), True),       # four heads a thread
    ("f16", 6, 2, 128, 16, 9, 0, None, False),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype,Hq,Hkv,D,B,T,rot,sect,pairs", ROPE)
def test_rope_and_cache(pa, dtype, Hq, Hkv, D, B, T, rot, sect, pairs, fp8):
    dt, g = DT[dtype], generator(T + rot)
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device="cuda").to(dt)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]      # columns of one projection
    NB = -(-T // B) + 3
    slots = torch.randperm(NB * B, generator=g, device="cuda")[:T]
    slots[::7] = -1
    sections = (rot // 2,) if sect is None else sect
    pos = torch.randint(4096, (len(sections), T), generator=g, device="cuda")
    cs = table(rot) if rot else None
    q_out = torch.full((T, Hq, D), 9.0, dtype=dt, device="cuda")
    kind = E4M3 if fp8 else dt
    kc, vc = (torch.full((NB, Hkv, B, D), 7.0, device="cuda").to(kind) for _ in range(2))
    sc = torch.full((NB, Hkv, 2, B), 5.0, device="cuda")
    args = (slots, pos[0].contiguous() if sect is None else pos, cs, sect, pairs)
    if fp8:
        pa.pa_rope_and_cache_fp8(q_out, q, k, v, kc, vc, sc, *args)
    else:
        pa.pa_rope_and_cache(q_out, q, k, v, kc, vc, *args)
    if rot:
        (yq, sq), (yk, sk) = (turned(x, pos, cs, sections, pairs) for x in (q, k))
    else:
        yq, sq, yk, sk = q.double(), q.double().abs(), k.double(), k.double().abs()
    # two products and a sum in fp32, then one rounding
    e = half_eps(dt)
    assert ((q_out.double() - yq).abs() <= e * yq.abs() + (1 + e) * 3 * U32 * sq + 2.0 ** -25).all()
    keep = slots >= 0
    at, off = slots[keep] // B, slots[keep] % B
    for n, (cache, x, size) in enumerate(((kc, yk, sk), (vc, v.double(), v.double().abs()))):
        x, size = x[keep], size[keep]
        raw = cache.view(torch.uint8) if fp8 else cache
        got = raw[at, :, off].view(E4M3 if fp8 else dt)
        if fp8:
            scale = sc[:, :, n][at, :, off].double()
            amax = x.abs().amax(-1)
            want = amax.clamp(min=LEAST) / 448
            # the largest element's 3 fp32 operations, the division's one
            assert ((scale - want).abs() <= 5 * U32 * size.amax(-1) / 448).all()
            err = (dequantised(got, scale) - x).abs()
            # e4m3 rounding; the fp32 operations before it (the turn 3, x * inv and inv 2)
            tol = x.abs() * 2.0 ** -4 + scale[..., None] * 2.0 ** -10 + 8 * U32 * size.amax(-1, True)
            assert (err <= tol).all()
            # the row's largest element keeps the whole range
            assert (got.double().abs().amax(-1) == 448).all()
        else:
            assert ((got.double() - x).abs() <= e * x.abs() + (1 + e) * 3 * U32 * size + 2.0 ** -25).all()
        # every other row as it was
        raw = raw.clone()
        fill = torch.tensor(7.0, device="cuda").to(kind)
        raw[at, :, off] = fill.view(torch.uint8) if fp8 else fill
        assert (raw.view(kind).double() == 7.0).all()
    if fp8:
        for n in (0, 1):
            sc[:, :, n][at, :, off] = 5.0
        assert (sc == 5.0).all()


def test_rope_in_place_and_keys_only(pa):
    g = generator(1)
    q, k, v = (torch.randn(50, h, 128, generator=g, device="cuda").bfloat16() for h in (8, 2, 2))
    cs, pos = table(128), torch.randint(4096, (50,), generator=g, device="cuda")
    slots = torch.arange(50, device="cuda")
    out, mine = torch.empty_like(q), q.clone()
    caches = [[torch.zeros(4, 2, 16, 128, device="cuda").bfloat16() for _ in range(2)] for _ in range(3)]
    pa.pa_rope_and_cache(out, q, k, v, *caches[0], slots, pos, cs)
    pa.pa_rope_and_cache(mine, mine, k, v, *caches[1], slots, pos, cs)
    pa.pa_rope_and_cache(None, None, k, v, *caches[2], slots, pos, cs)
    assert torch.equal(out, mine)
    for c in caches[1:]:
        assert torch.equal(c[0], caches[0][0]) and torch.equal(c[1], caches[0][1])


def test_rows_of_zeros_tiny_huge_and_nan(pa):
    """Scales of degenerate rows: zeros read back as zeros, a row below 2^-100 as zeros or its
    e4m3 steps of 2^-100 / 448, an infinite row as NaN, a NaN element as NaN, the others kept."""
    x = torch.randn(6, 1, 64, device="cuda")
    x[0] = 0
    x[1] *= 2.0 ** -130
    x[2] *= 2.0 ** 120
    x[3, 0, 5] = float("inf")
    x[4, 0, 9] = float("nan")
    k = x.bfloat16()
    kc, vc = (torch.zeros(1, 1, 16, 64, device="cuda").to(E4M3) for _ in range(2))
    sc = torch.zeros(1, 1, 2, 16, device="cuda")
    pa.pa_rope_and_cache_fp8(None, None, k, k, kc, vc, sc, torch.arange(6, device="cuda"), None, None)
    got = dequantised(kc[0, 0, :6], sc[0, 0, 0, :6])
    assert (got[0] == 0).all()
    tol = k[:, 0].double().abs() * 2.0 ** -4 + (sc[0, 0, 0, :6].double() * 2.0 ** -10)[:, None]
    for r in (1, 2, 5):
        assert ((got[r] - k[r, 0].double()).abs() <= tol[r] * (1 + 4 * U32)).all()
    assert got[3].isnan().all()
    bad = torch.arange(64, device="cuda") == 9
    assert got[4][bad].isnan().all() and ((got[4] - k[4, 0].double()).abs() <= tol[4] * (1 + 4 * U32))[~bad].all()


def test_bad_slots_and_positions_are_flagged(pa):
    g = generator(2)
    q, k, v = (torch.randn(40, h, 64, generator=g, device="cuda").half() for h in (4, 2, 2))
    cs = table(64, 100)
    slots = torch.arange(40, device="cuda")
    slots[3] = 48                                       # one past the pool
    pos = torch.randint(100, (2, 40), generator=g, device="cuda")
    pos[1, 5], pos[0, 7] = 100, -1
    out = torch.full_like(q, 9.0)
    kc, vc = (torch.full((3, 2, 16, 64), 7.0, device="cuda").half() for _ in range(2))
    pa.pa_rope_and_cache(out, q, k, v, kc, vc, slots, pos, cs, (10, 22))
    assert pa.pa_device_error(clear=True) == pa.DEVERR["slot"] | pa.DEVERR["position"]
    rows = kc.transpose(1, 2).reshape(48, 2, 64)
    for t in (5, 7):
        assert (out[t] == 9).all() and (rows[t] == 7).all()
    assert (rows[3] == 7).all() and (rows[40:] == 7).all()
    assert not (out[3] == 9).all() and not (rows[6] == 7).all()


# ------------------------------------------------------------------ decode

def decode_reference(q, k, v, scale_t, tables, lens, B, scale):
    """64-bit outputs and, for each, what 2^-24 is multiplied with in the tolerance."""
    S, Hq, D = q.shape
    Hkv = k.shape[1]
    out, tol = torch.zeros(S, Hq, D, dtype=torch.float64, device="cuda"), torch.zeros(S, 1, 1, device="cuda")
    for i, n in enumerate(lens):
        if n == 0:
            continue
        K, V = (rows_of(c, scale_t, w, tables[i], n, B) for w, c in ((0, k), (1, v)))
        qq = q[i].double().view(Hkv, -1, D)
        z = torch.einsum("hgd,nhd->hgn", qq, K) * scale
        out[i] = torch.einsum("hgn,nhd->hgd", torch.softmax(z, -1), V).reshape(Hq, D)
        # a score is a sum of D products, scaled and shifted: D + 8 operations of what its terms
        # add up to; a weight is off by that, twice (its own and the sum's), by 2^-22 from its
        # two halves and by a few steps of exp2 and of the joins; the output by that of |V|
        terms = (torch.einsum("hgd,nhd->hgn", qq.abs(), K.abs()) * abs(scale)).max()
        tol[i] = (2 * (D + 8) * terms + 64) * V.abs().max()
    return out, tol.double() * U32


DECODE = [
    # dtype, Hq, Hkv, D, B
    ("bf16", 32, 8, 128, 16), ("f16", 8, 8, 128, 32), ("bf16", 64, 8, 128, 32),
    ("f16", 16, 1, 128, 16), ("bf16", 10, 1, 64, 16), ("f16", 4, 4, 64, 32),
    ("bf16", 12, 4, 64, 16), ("f16", 9, 1, 128, 32),
]
LENS = [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 700, 0, 2049, 5]


@pytest.mark.parametrize("dtype,Hq,Hkv,D,B", DECODE)
def test_decode_fp8_ragged(pa, dtype, Hq, Hkv, D, B):
    NB = sum(-(-n // B) for n in LENS) + 5
    k, v, sc = make_pool(NB, Hkv, B, D, seed=Hq + D)
    tables = make_tables(LENS, B, NB, 3)
    poison_unused(k, v, sc, tables, LENS, B)
    q = torch.randn(len(LENS), Hq, D, generator=generator(4), device="cuda").to(DT[dtype])
    out = torch.full((len(LENS), Hq, D), float("nan"), device="cuda")
    lens = torch.tensor(LENS, dtype=torch.int32, device="cuda")
    pa.pa_paged_decode_attention_fp8(out, q, k, v, sc, tables, lens, D ** -0.5, Hkv)
    want, tol = decode_reference(q, k, v, sc, tables, LENS, B, D ** -0.5)
    assert ((out.double() - want).abs() <= tol).all(), ((out.double() - want).abs() / tol).max()
    again = torch.empty_like(out)
    pa.pa_paged_decode_attention_fp8(again, q, k, v, sc, tables, lens, D ** -0.5, Hkv)
    assert torch.equal(out, again)


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_decode_fp8_scales_and_sizes(pa, scale):
    """A scale of zero (the mean), a negative one, a steep softmax; q and V from 2^-60 to 2^60."""
    lens, B, Hkv, D = [300, 129, 40], 16, 2, 64
    k, v, sc = make_pool(40, Hkv, B, D, seed=9)
    sc[:, :, 1] *= torch.tensor([2.0 ** -60, 2.0 ** 60], device="cuda")[:, None]
    tables = make_tables(lens, B, 40, 5)
    q = torch.randn(3, 8, D, generator=generator(6), device="cuda").bfloat16()
    out = torch.empty(3, 8, D, device="cuda")
    pa.pa_paged_decode_attention_fp8(out, q, k, v, sc, tables,
                                     torch.tensor(lens, dtype=torch.int32, device="cuda"), scale, Hkv)
    for h in range(Hkv):      # one kv head at a time: its own size of V
        part = slice(4 * h, 4 * h + 4)
        want, tol = decode_reference(q[:, part], k[:, h:h + 1], v[:, h:h + 1], sc[:, h:h + 1],
                                     tables, lens, B, scale)
        assert ((out[:, part].double() - want).abs() <= tol).all()


def test_decode_fp8_long_context_and_odd_table(pa):
    """One long sequence split over every warp, and a table whose last tile is half a tile."""
    B, Hkv, D = 16, 8, 128
    lens = [16 * 2051, 16 * 3 - 1]
    k, v, sc = make_pool(2060, Hkv, B, D, seed=11)
    tables = make_tables(lens, B, 2060, 12, width=2051)
    q = torch.randn(2, 32, D, generator=generator(13), device="cuda").half()
    out = torch.empty(2, 32, D, device="cuda")
    pa.pa_paged_decode_attention_fp8(out, q, k, v, sc, tables,
                                     torch.tensor(lens, dtype=torch.int32, device="cuda"), D ** -0.5, Hkv)
    want, tol = decode_reference(q, k, v, sc, tables, lens, B, D ** -0.5)
    assert ((out.double() - want).abs() <= tol).all()


def test_decode_fp8_many_short_sequences(pa):
    B, Hkv, D, S = 16, 1, 64, 1500
    lens = [(7 * i) % 50 for i in range(S)]
    NB = sum(-(-n // B) for n in lens)
    k, v, sc = make_pool(NB, Hkv, B, D, seed=14)
    tables = make_tables(lens, B, NB, 15)
    q = torch.randn(S, 2, D, generator=generator(16), device="cuda").bfloat16()
    out = torch.empty(S, 2, D, device="cuda")
    pa.pa_paged_decode_attention_fp8(out, q, k, v, sc, tables,
                                     torch.tensor(lens, dtype=torch.int32, device="cuda"), D ** -0.5, Hkv)
    want, tol = decode_reference(q, k, v, sc, tables, lens, B, D ** -0.5)
    assert ((out.double() - want).abs() <= tol).all()


def test_decode_fp8_bad_tables_are_flagged(pa):
    """A block outside the pool is left out, a length past the table is cut, both flagged."""
    B, Hkv, D = 16, 2, 64
    k, v, sc = make_pool(12, Hkv, B, D, seed=17)
    tables = torch.tensor([[0, 12, 2], [3, 4, 5]], dtype=torch.int32, device="cuda")
    q = torch.randn(2, 4, D, generator=generator(18), device="cuda").half()
    out = torch.empty(2, 4, D, device="cuda")
    pa.pa_paged_decode_attention_fp8(out, q, k, v, sc, tables,
                                     torch.tensor([48, 60], dtype=torch.int32, device="cuda"),
                                     D ** -0.5, Hkv)
    assert pa.pa_device_error(clear=True) == pa.DEVERR["block_id"] | pa.DEVERR["context_len"]
    short = torch.tensor([[0, 2], [3, 4]], dtype=torch.int32, device="cuda")
    want, tol = decode_reference(q[:1], k, v, sc, short[:1], [32], B, D ** -0.5)
    assert ((out[:1].double() - want).abs() <= tol).all()
    want, tol = decode_reference(q[1:], k, v, sc, tables[1:], [48], B, D ** -0.5)
    assert ((out[1:].double() - want).abs() <= tol).all()


def test_decode_fp8_nan_and_infinite_rows_reach_their_outputs(pa):
    B, Hkv, D = 16, 2, 64
    k, v, sc = make_pool(8, Hkv, B, D, seed=19)
    k.view(torch.uint8)[0, 0, 3, 7] = 0x7F              # sequence 0, kv head 0
    sc[2, 1, 1, 5] = float("inf")                       # sequence 1, kv head 1
    tables = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    q = torch.randn(2, 4, D, generator=generator(20), device="cuda").half()
    out = torch.empty(2, 4, D, device="cuda")
    pa.pa_paged_decode_attention_fp8(out, q, k, v, sc, tables,
                                     torch.tensor([32, 32], dtype=torch.int32, device="cuda"),
                                     D ** -0.5, Hkv)
    assert out[0, :2].isnan().all() and out[0, 2:].isfinite().all()
    assert not out[1, 2:].isfinite().any() and out[1, :2].isfinite().all()


def test_decode_fp8_wait_limit(pa):
    """Waits that run out are reported and the next call is whole.  (270 MB of cache, more than
    the L2 holds: a tile's copy takes longer than the work on the tile before it.)"""
    B, Hkv, D, n = 16, 8, 128, 131072
    k, v, sc = make_pool(n // B, Hkv, B, D, seed=21)
    tables = make_tables([n], B, n // B, 22)
    q = torch.randn(1, 32, D, generator=generator(23), device="cuda").half()
    out = torch.empty(1, 32, D, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    try:
        pa.pa_set_wait_limit(1)
        pa.pa_paged_decode_attention_fp8(out, q, k, v, sc, tables, lens, D ** -0.5, Hkv)
        assert pa.pa_device_error(clear=True) & pa.DEVERR["timeout"]
    finally:
        pa.pa_set_wait_limit(0)
    pa.pa_paged_decode_attention_fp8(out, q, k, v, sc, tables, lens, D ** -0.5, Hkv)
    want, tol = decode_reference(q, k, v, sc, tables, [n], B, D ** -0.5)
    assert ((out.double() - want).abs() <= tol).all()


# ------------------------------------------------------------------ gather, copies

@pytest.mark.parametrize("dtype,Hkv,D,B", [("bf16", 8, 128, 16), ("f16", 1, 64, 32), ("bf16", 3, 64, 16)])
def test_gather(pa, dtype, Hkv, D, B):
    lens = [0, 1, 17, 0, 0, 300, 33, 16, 0]
    NB = sum(-(-n // B) for n in lens) + 2
    k, v, sc = make_pool(NB, Hkv, B, D, seed=31)
    tables = make_tables(lens, B, NB, 32)
    poison_unused(k, v, sc, tables, lens, B)
    T = sum(lens)
    start = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda")
    key, value = (torch.full((T + 20, Hkv, D), 7.0, dtype=DT[dtype], device="cuda") for _ in range(2))
    pa.pa_gather_cache_fp8(key, value, k, v, sc, tables, start)
    e = half_eps(DT[dtype])
    for w, (got, codes) in enumerate(((key, k), (value, v))):
        want = torch.cat([rows_of(codes, sc, w, tables[i], n, B) for i, n in enumerate(lens)])
        # one fp32 product, one rounding (2^-25: half the smallest fp16 step)
        assert ((got[:T].double() - want).abs() <= (e + 2 * U32) * want.abs() + 2.0 ** -25).all()
        assert (got[T:] == 7).all()


def test_gather_leaves_rows_of_no_sequence(pa):
    k, v, sc = make_pool(6, 2, 16, 64, seed=34)
    tables = torch.tensor([[4, 1]], dtype=torch.int32, device="cuda")
    key, value = (torch.full((60, 2, 64), 7.0, dtype=torch.float16, device="cuda") for _ in range(2))
    pa.pa_gather_cache_fp8(key, value, k, v, sc, tables, torch.tensor([9, 40], dtype=torch.int32, device="cuda"))
    want = rows_of(k, sc, 0, tables[0], 31, 16)
    assert ((key[9:40].double() - want).abs() <= (2.0 ** -11 + 2 * U32) * want.abs() + 2.0 ** -25).all()
    for got in (key, value):
        assert (got[:9] == 7).all() and (got[40:] == 7).all()


def test_gather_bad_tables_are_flagged(pa):
    k, v, sc = make_pool(6, 2, 16, 64, seed=33)
    tables = torch.tensor([[0, 6], [2, 3]], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 32, 70], dtype=torch.int32, device="cuda")   # 38 > 2 blocks of 16
    key, value = (torch.full((70, 2, 64), 7.0, dtype=torch.float16, device="cuda") for _ in range(2))
    pa.pa_gather_cache_fp8(key, value, k, v, sc, tables, start)
    assert pa.pa_device_error(clear=True) == pa.DEVERR["block_id"] | pa.DEVERR["context_len"]
    assert (key[16:32] == 7).all() and (value[64:] == 7).all()
    assert not (key[:16] == 7).any() and not (value[32:64] == 7).any()


@pytest.mark.parametrize("Hkv,D,B,n", [(8, 128, 16, 37), (1, 64, 32, 1), (3, 64, 16, 70000), (40, 128, 32, 3)])
def test_copy_blocks_fp8(pa, Hkv, D, B, n):
    g = generator(41)
    small = min(n, 300)
    k, v, sc = make_pool(2 * small + 3, Hkv, B, D, seed=42)
    order = torch.randperm(2 * small + 3, generator=g, device="cuda")
    pairs = order[:2 * small].view(small, 2).contiguous()
    many = pairs[torch.arange(n, device="cuda") % small]        # past 65535 pairs: the same ones again
    want = [x.clone() for x in (k.view(torch.uint8), v.view(torch.uint8), sc)]
    for x in want:
        x[pairs[:, 1]] = x[pairs[:, 0]]
    pa.pa_copy_blocks_fp8(k, v, sc, many.contiguous())
    for x, y in zip((k.view(torch.uint8), v.view(torch.uint8), sc), want):
        assert torch.equal(x, y)


def test_copy_blocks_fp8_bad_pairs_are_flagged(pa):
    k, v, sc = make_pool(4, 2, 16, 64, seed=43)
    want = k.view(torch.uint8).clone()
    want[2] = want[1]
    pa.pa_copy_blocks_fp8(k, v, sc, torch.tensor([[0, 4], [1, 2], [-1, 3]], device="cuda"))
    assert pa.pa_device_error(clear=True) == pa.DEVERR["copy_pair"]
    assert torch.equal(k.view(torch.uint8), want)


# ------------------------------------------------------------------ large pools, streams, graphs

def test_blocks_behind_2_31_bytes(pa):
    """Write, copy, decode and gather at the far end of a pool of 2.2 GB for K and for V."""
    B, Hkv, D = 16, 8, 128
    NB = 135000
    kc, vc = (torch.empty(NB, Hkv, B, D, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2))
    sc = torch.empty(NB, Hkv, 2, B, device="cuda")
    g = generator(51)
    k, v = (torch.randn(40, Hkv, D, generator=g, device="cuda").half() for _ in range(2))
    slots = torch.arange(40, device="cuda") + (NB - 3) * B
    pa.pa_rope_and_cache_fp8(None, None, k, v, kc, vc, sc, slots, None, None)
    pa.pa_copy_blocks_fp8(kc, vc, sc, torch.tensor([[NB - 2, 5], [NB - 3, NB - 5]], device="cuda"))
    tables = torch.tensor([[NB - 5, 5, NB - 1]], dtype=torch.int32, device="cuda")
    key, value = (torch.empty(40, Hkv, D, dtype=torch.float16, device="cuda") for _ in range(2))
    pa.pa_gather_cache_fp8(key, value, kc, vc, sc, tables, torch.tensor([0, 40], dtype=torch.int32, device="cuda"))
    for got, x in ((key, k), (value, v)):
        top = x.double().abs().amax(-1, keepdim=True)
        # e4m3 and fp16 roundings
        tol = x.double().abs() * (2.0 ** -4 + 2.0 ** -10) + top * (2.0 ** -10 / 448 + 2.0 ** -20)
        assert ((got.double() - x.double()).abs() <= tol).all()
    q = torch.randn(1, 32, D, generator=g, device="cuda").half()
    out = torch.empty(1, 32, D, device="cuda")
    pa.pa_paged_decode_attention_fp8(out, q, kc, vc, sc, tables,
                                     torch.tensor([40], dtype=torch.int32, device="cuda"), D ** -0.5, Hkv)
    want, tol = decode_reference(q, kc, vc, sc, tables, [40], B, D ** -0.5)
    assert ((out.double() - want).abs() <= tol).all()


def test_captured_and_replayed_on_another_stream(pa):
    """A decode step (rotary write, then attention) captured once and replayed with new
    positions, slots, lengths and inputs gives what eager calls give."""
    B, Hkv, D, S, Hq = 16, 4, 128, 3, 16
    cs = table(D)
    kc, vc, sc = make_pool(30, Hkv, B, D, seed=61)
    tables = make_tables([160, 160, 160], B, 30, 62)
    qkv = torch.empty(S, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device="cuda")
    qo, out = torch.empty(S, Hq, D, dtype=torch.bfloat16, device="cuda"), torch.empty(S, Hq, D, device="cuda")
    slots, pos = (torch.zeros(S, dtype=torch.int64, device="cuda") for _ in range(2))
    lens = torch.ones(S, dtype=torch.int32, device="cuda")
    ws = pa.alloc_workspace(S, Hq, Hkv, D, B, 160)

    def step(kc, vc, sc):
        pa.pa_rope_and_cache_fp8(qo, qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], kc, vc, sc,
                                 slots, pos, cs)
        pa.pa_paged_decode_attention_fp8(out, qo, kc, vc, sc, tables, lens, D ** -0.5, Hkv, workspace=ws)

    def set_inputs(n):
        qkv.copy_(torch.randn(qkv.shape, generator=generator(n), device="cuda"))
        at = torch.tensor([n, n + 33, 2 * n], device="cuda")
        pos.copy_(at)
        lens.copy_(at + 1)
        slots.copy_(torch.gather(tables.long(), 1, (at // B)[:, None])[:, 0] * B + at % B)

    set_inputs(1)
    eager = [x.clone() for x in (kc, vc, sc)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(kc, vc, sc)                       # warm-up on the stream
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(kc, vc, sc)
    for n in (1, 2, 15, 16, 40):
        set_inputs(n)
        graph.replay()
        got = out.clone()
        step(*eager)
        assert torch.equal(got, out)
    torch.cuda.synchronize()
    for x, y in zip((kc, vc), eager):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert torch.equal(sc, eager[2])


def test_two_calls_at_once_on_two_streams(pa):
    """Decode calls on two streams, each with the workspace the binding makes for it, between
    allocations that would reuse that memory too early."""
    B, Hkv, D, S = 16, 8, 128, 64
    lens = [(97 * i) % 1500 for i in range(S)]
    NB = sum(-(-n // B) for n in lens)
    k, v, sc = make_pool(NB, Hkv, B, D, seed=71)
    tables = make_tables(lens, B, NB, 72)
    ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = [torch.randn(S, 32, D, generator=generator(i), device="cuda").bfloat16() for i in (1, 2)]
    want = [torch.empty(S, 32, D, device="cuda") for _ in q]
    for a, b in zip(want, q):
        pa.pa_paged_decode_attention_fp8(a, b, k, v, sc, tables, ctx, D ** -0.5, Hkv)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in q]
    got = [[torch.zeros_like(want[0]) for _ in range(6)] for _ in q]
    torch.cuda.synchronize()
    for r in range(6):
        for i, st in enumerate(streams):
            pa.pa_paged_decode_attention_fp8(got[i][r], q[i], k, v, sc, tables, ctx, D ** -0.5, Hkv, stream=st)
            torch.full((4 << 20,), float("nan"), device="cuda")      # on the current stream
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])
