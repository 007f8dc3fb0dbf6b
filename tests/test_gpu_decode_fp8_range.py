"""GPU test of the 8-bit decode where the V rows of a sequence differ widely in
size: the tokens that count may be the small ones.

Tolerance of an output, from the arithmetic, with w the weights, c the codes and
vs the scales of V: a score is a sum of D products, scaled and shifted (D + 8
operations of 2^-24 of what its terms add up to), which moves a weight twice (its
own and the sum's), and a weight's two fp16 halves, exp2 and the joins cost some
more steps of it: 2^-24 (2 (D + 8) z + 64) sum_t w_t vs_t |c_t|.  The halves end
at fp16's smallest step: half of one is 2^-39 of the largest w vs of the tile,
for each token: 2^-39 max_t (w_t vs_t) sum_t |c_t|."""
import pytest
import torch

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def reference(q, k, ks, v, vs, scale):
    """One sequence: q [Hq, D], codes [n, Hkv, D], scales [n, Hkv], in 64 bits: outputs, tolerance."""
    Hkv, D = k.shape[1:]
    qq, K, c = q.double().view(Hkv, -1, D), k.double() * ks.double()[..., None], v.double()
    z = torch.einsum("hgd,nhd->hgn", qq, K) * scale
    y = torch.softmax(z, -1) * vs.double().T[:, None]               # w vs: [Hkv, G, n]
    out = torch.einsum("hgn,nhd->hgd", y, c)
    terms = (torch.einsum("hgd,nhd->hgn", qq.abs(), K.abs()) * abs(scale)).amax()
    tol = (2.0 ** -24 * (2 * (D + 8) * terms + 64) * torch.einsum("hgn,nhd->hgd", y, c.abs())
           + 2.0 ** -39 * y.amax(-1, keepdim=True) * c.abs().sum(0)[:, None])
    return out.reshape(q.shape), tol.reshape(q.shape)


# (tokens, steps of log2 between the sizes of V of neighbouring tokens' kinds, log2 that the large
# ones' weights stay behind by)
SIZES = [(32, 24, 70), (32, 40, 80), (20, 60, 100), (700, 30, 60), (700, 50, 45), (3000, 45, 90)]


@pytest.mark.parametrize("dtype,Hq,Hkv,D,B", [("bf16", 8, 2, 128, 16), ("f16", 3, 1, 64, 32),
                                              ("bf16", 14, 2, 128, 32), ("f16", 16, 1, 64, 16),
                                              ("f16", 13, 1, 128, 16), ("bf16", 7, 1, 64, 16)])
@pytest.mark.parametrize("every", [1, 33])
@pytest.mark.parametrize("n,size,behind", SIZES)
def test_small_rows_beside_large_ones(pa, cuda_device, dtype, Hq, Hkv, D, B, every, n, size, behind):
    """Tokens of large V and next to no weight among tokens of small V that have all of it: in
    one tile (every second token) and in tiles of their own (every second tile)."""
    g = torch.Generator(device="cuda").manual_seed(n + size + Hq)
    NB = -(-n // B)
    codes = [torch.randn(NB, Hkv, B, D, generator=g, device="cuda").mul(100).clamp(-448, 448).to(E4M3)
             for _ in range(2)]
    sc = torch.rand(NB, Hkv, 2, B, generator=g, device="cuda").add(0.5) / 100
    token = torch.arange(NB * B, device="cuda").view(NB, 1, B)
    large = (token // every) % 2 == 1
    # column 0 of K is its row's largest, q's is `behind`: the scores of the two kinds lie apart
    scale = 1 / 64
    raw = codes[0].view(torch.uint8)
    raw[..., 0] = torch.tensor(448.0).to(E4M3).view(torch.uint8).item()
    raw[..., 0] |= (large.expand(NB, Hkv, B).to(torch.uint8) << 7)              # its sign
    sc[:, :, 0] = 1 / 448
    sc[:, :, 1] *= torch.where(large, 2.0 ** (size / 2), 2.0 ** (-size / 2))
    q = torch.randn(1, Hq, D, generator=g, device="cuda") / 4
    q[..., 0] = behind * 0.6931 / 2 / scale
    q = q.to(DT[dtype])
    table = torch.randperm(NB, generator=g, device="cuda").int()
    pool = [torch.empty_like(x.view(torch.uint8)) for x in codes]
    scales = torch.empty_like(sc)
    for to, x in zip(pool, codes):
        to[table.long()] = x.view(torch.uint8)
    scales[table.long()] = sc
    out = torch.empty(1, Hq, D, device="cuda")
    pa.pa_paged_decode_attention_fp8(out, q, pool[0].view(E4M3), pool[1].view(E4M3), scales, table[None],
                                     torch.tensor([n], dtype=torch.int32, device="cuda"), scale, Hkv)
    rows = [x.transpose(1, 2).reshape(NB * B, Hkv, D)[:n] for x in (c.double() for c in codes)]
    per = [sc[:, :, i].transpose(1, 2).reshape(NB * B, Hkv)[:n] for i in (0, 1)]
    want, tol = reference(q[0], rows[0], per[0], rows[1], per[1], scale)
    off = (out[0].double() - want).abs() / tol
    assert (off <= 1).all(), off.max().item()
    assert pa.pa_device_error() == 0
