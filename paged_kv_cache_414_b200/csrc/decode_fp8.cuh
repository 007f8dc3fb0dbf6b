// Paged decode attention over an 8-bit cache, for sm_100a.
//
// For sequence s and query head h of kv head kh, with e4m3 codes K^, V^ and
// per-token scales ks, vs (layouts in fp8_cache.cuh):
//   out[s, h] = sum_t w_t vs_t V^_t,   w = softmax_t(scale ks_t <q, K^_t>).
// The scales never touch the codes: ks_t multiplies the finished score and
// vs_t the weight, so both products run on the codes as they lie in the pool.
//
// Work split, launch plan and split merge are those of the 16-bit decode
// kernel (decode_attention.cuh): the tiles of all (sequence, kv head) pairs,
// numbered in order, are cut into equal contiguous ranges, one per warp, each
// warp streams its range through its own ring of bulk copies, and cut
// segments leave partials for the merge kernel.  Here a tile is 32 tokens
// whatever the block size (two blocks of 16 or one of 32): half the bytes per
// token would otherwise leave twice the bookkeeping per byte.
//
// Arithmetic.  Codes become fp16 exactly (cvt.rn.f16x2.e4m3x2), so both
// products are fp16 warp MMAs (m16n8k16, fp32 accumulation) for fp16 and bf16
// queries alike:
//   * a query row is scaled by the power of two that puts its largest element
//     in [2^14, 2^15) before it is rounded to fp16: exact for fp16 queries and
//     for bf16 elements down to 2^-39 of the row's largest;
//   * a weight times its vs_t is scaled by the power of two that puts the
//     tile's largest vs in the same range and goes in as a hi + lo pair of
//     fp16 values (2^-22 relative), so the output keeps ~fp32 accuracy;
//   * a tile's P.V is summed in fresh accumulators and folded into the running
//     output by one FMA with the softmax correction, so long segments never
//     add small products to a large tensor-core accumulator.
// Fragments come from shared memory by plain 16-byte loads, not ldmatrix: the
// reduction order of an MMA is free as long as both operands agree, so lane
// (g, c) takes D/4 neighbouring codes of K row g, and D/8 neighbouring columns
// of V for its four tokens; bytes of two tokens are paired with one byte
// permute before the conversion.  With the copies' 128-byte (D = 128) or
// 64-byte (D = 64) swizzle the K loads and D = 128's V loads are free of bank
// conflicts.
//
// Bound: HBM, 2 D + 8 bytes per token and kv head.
#pragma once

#include <cuda_fp8.h>

#include "decode_attention.cuh"

namespace pa {

constexpr int kF8Tile = 32;   // tokens per tile

struct DecodeFp8Params {
  DecodeParams d;             // max_blocks counts tiles of 32 tokens here
  const float *kv_scale;
  int table_blocks;           // blocks per row of the block table
  int block_size;
  int q_bf16;
};

// A packed pair of e4m3 codes (low 16 bits) as a packed pair of fp16 values.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t x) {
  uint32_t y;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
      : "=r"(y)
      : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t e4m3x2_hi_to_f16x2(uint32_t x) {
  uint32_t y;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, hi;\n\t}"
      : "=r"(y)
      : "r"(x));
  return y;
}

// 2^x by the hardware approximation (2 ulp, results below 2^-126 are zero).
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ float lds_f32(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}

__device__ __forceinline__ void st_global_hint4(float *dst, float4 v, uint64_t policy) {
  asm volatile("st.global.L2::cache_hint.v4.f32 [%0], {%1, %2, %3, %4}, %5;" ::"l"(dst), "f"(v.x),
               "f"(v.y), "f"(v.z), "f"(v.w), "l"(policy)
               : "memory");
}

// Power of two with the exponent field e (1..254).
__device__ __forceinline__ float pow2_field(int e) { return __int_as_float(e << 23); }

// Exponent field e of the magnitude `bits`, clamped so that the two powers of
// two that take it to [2^14, 2^15) and back (fields 268 - e and e - 14) are
// normal numbers.
__device__ __forceinline__ int scale_field(uint32_t bits) {
  const int e = (int)((bits >> 23) & 0xffu);
  return min(max(e, 15), 254);
}

template <int D, int NT>
struct Fp8Path {
  static constexpr int W = D / 16;    // words of K per lane and row = k-steps of q.K
  static constexpr int MM = D / 16;   // m-tiles of P.V
  float o[MM][NT][4];                 // d = (D/8) g + 2 mm + (r >> 1), head 8 n + 2 c + (r & 1)
  float m[NT][2], l[NT][2];
  float qs[NT][2];                    // scale * log2(e) * 2^-shift of the accumulators' heads
  uint32_t qf[W][NT][2];

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int a = 0; a < MM; ++a)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) o[a][n][r] = 0.f;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        m[n][r] = -INFINITY;
        l[n][r] = 0.f;
      }
  }

  // Lane (g, c): columns (D/4) c .. of query row 8 n + g, as scaled fp16.
  __device__ __forceinline__ void load_q(const uint8_t *q, int G, bool bf16, float scale_log2,
                                         int lane) {
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int head = n * 8 + g;
      uint32_t raw[2 * W];
      uint32_t top = 0;
      const uint4 *row = reinterpret_cast<const uint4 *>(q + (size_t)head * (D * 2) + c * (D / 2));
#pragma unroll
      for (int i = 0; i < W / 2; ++i) {
        const uint4 v = head < G ? row[i] : make_uint4(0, 0, 0, 0);
        raw[4 * i] = v.x, raw[4 * i + 1] = v.y, raw[4 * i + 2] = v.z, raw[4 * i + 3] = v.w;
      }
#pragma unroll
      for (int i = 0; i < 2 * W; ++i) {
        const float2 f = bf16 ? Mma<__nv_bfloat16>::unpack(raw[i]) : Mma<__half>::unpack(raw[i]);
        top = max(top, max(__float_as_uint(fabsf(f.x)), __float_as_uint(fabsf(f.y))));
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = scale_field(top);
      const float up = pow2_field(268 - e);
      const float down = pow2_field(e - 14) * scale_log2;
#pragma unroll
      for (int i = 0; i < 2 * W; ++i) {
        const float2 f = bf16 ? Mma<__nv_bfloat16>::unpack(raw[i]) : Mma<__half>::unpack(raw[i]);
        qf[i >> 1][n][i & 1] = Mma<__half>::pack(f.x * up, f.y * up);
      }
      qs[n][0] = __shfl_sync(0xffffffffu, down, 8 * c);        // row 2 c is held by lanes 8 c ..
      qs[n][1] = __shfl_sync(0xffffffffu, down, 8 * c + 4);
    }
  }

  // One tile: codes at kb, vb, scales at sb ([block][K or V][B] floats), `live`
  // the tokens that count.
  __device__ __forceinline__ void tile(uint32_t kb, uint32_t vb, uint32_t sb, int B, uint32_t live,
                                       int lane) {
    const int g = lane >> 2, c = lane & 3;
    float sc[2][NT][4];
    // ---- scores: S^T[token][head]
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) sc[t][n][r] = 0.f;
      uint32_t k0[W], k1[W];   // rows 16 t + g and + 8
#pragma unroll
      for (int i = 0; i < W / 4; ++i) {
        const int row = 16 * t + g;
        uint32_t a;
        if constexpr (D == 128)
          a = kb + row * 128 + (((2 * c + i) ^ g) << 4);
        else
          a = kb + row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
        const uint4 v = lds128(a), u = lds128(a + 8 * D);   // row + 8: the same swizzle
        k0[4 * i] = v.x, k0[4 * i + 1] = v.y, k0[4 * i + 2] = v.z, k0[4 * i + 3] = v.w;
        k1[4 * i] = u.x, k1[4 * i + 1] = u.y, k1[4 * i + 2] = u.z, k1[4 * i + 3] = u.w;
      }
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const uint32_t a[4] = {e4m3x2_to_f16x2(k0[w]), e4m3x2_to_f16x2(k1[w]),
                               e4m3x2_hi_to_f16x2(k0[w]), e4m3x2_hi_to_f16x2(k1[w])};
#pragma unroll
        for (int n = 0; n < NT; ++n) Mma<__half>::run(sc[t][n], a, qf[w][n][0], qf[w][n][1]);
      }
    }
    // ---- the tokens' scales: K's for the scores, V's for the weights
    float vs[2][2];
    {
      const int sub = lane / B;
      const uint32_t mine = sb + 4 * ((2 * sub + 1) * B + lane - sub * B);   // V scale of token `lane`
      const uint32_t bits =
          (live >> lane) & 1 ? __float_as_uint(fabsf(lds_f32(mine))) : 0u;
      const int e = scale_field(__reduce_max_sync(0xffffffffu, bits));
      const float up = pow2_field(268 - e);
      vdown = pow2_field(e - 14);
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int tok = 16 * t + g + 8 * x, s = tok / B;
          const uint32_t a = sb + 4 * (2 * s * B + tok - s * B);
          const bool on = (live >> tok) & 1;
          const float ks = lds_f32(a);
          vs[t][x] = on ? lds_f32(a + 4 * B) * up : 0.f;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r)
              sc[t][n][2 * x + r] = on ? sc[t][n][2 * x + r] * (ks * qs[n][r]) : -INFINITY;
        }
    }
    // ---- running maximum and sum of each head
    float alpha[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float v = fmaxf(fmaxf(sc[0][n][r], sc[0][n][2 + r]), fmaxf(sc[1][n][r], sc[1][n][2 + r]));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
        const float mn = fmaxf(m[n][r], v);
        // all scores so far -inf (a -inf in q or K): weights of 0, not NaN
        const float ref = mn == -INFINITY ? 0.f : mn;
        alpha[n][r] = exp2_approx(m[n][r] - ref);
        m[n][r] = mn;
        float s = 0.f;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float pv = exp2_approx(sc[t][n][2 * x + r] - ref);
            sc[t][n][2 * x + r] = pv * vs[t][x];
            s += pv;
          }
        l[n][r] = l[n][r] * alpha[n][r] + s;
      }
    // ---- weights (times vs) as B operands: hi + lo
    uint32_t ph[2][NT][2], pl[2][NT][2];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float a = sc[t][n][2 * x], b = sc[t][n][2 * x + 1];
          const uint32_t h = Mma<__half>::pack(a, b);
          const float2 f = Mma<__half>::unpack(h);
          ph[t][n][x] = movmatrix_trans(h);
          pl[t][n][x] = movmatrix_trans(Mma<__half>::pack(a - f.x, b - f.y));
        }
    // ---- O^T[d][head] = alpha O^T + 2^.. V^T P^T
    constexpr int XW = D / 32;   // words of V per lane and token
    uint32_t vw[2][4][XW];       // tokens 16 t + 2 c + {0, 1, 8, 9}
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 16 * t + 2 * c + (i & 1) + 8 * (i >> 1);
        if constexpr (D == 128) {
          const uint4 v = lds128(vb + row * 128 + ((g ^ (row & 7)) << 4));
          vw[t][i][0] = v.x, vw[t][i][1] = v.y, vw[t][i][2] = v.z, vw[t][i][3] = v.w;
        } else {
          const uint2 v = lds64(vb + row * 64 + (((g >> 1) ^ ((row >> 1) & 3)) << 4) + (g & 1) * 8);
          vw[t][i][0] = v.x, vw[t][i][1] = v.y;
        }
        // a token that does not count may hold any bits, NaN codes too
        if (live != 0xffffffffu && !((live >> row) & 1))
#pragma unroll
          for (int x = 0; x < XW; ++x) vw[t][i][x] = 0u;
      }
#pragma unroll
    for (int x = 0; x < XW; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int a = 2 * x + y;                      // columns 2 a, 2 a + 1 of this lane's
        const uint32_t sel = y ? 0x7362u : 0x5140u;   // bytes 2 y, 2 y + 1 of both tokens
        float acc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[n][r] = 0.f;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const uint32_t u = __byte_perm(vw[t][0][x], vw[t][1][x], sel);
          const uint32_t v = __byte_perm(vw[t][2][x], vw[t][3][x], sel);
          const uint32_t f[4] = {e4m3x2_to_f16x2(u), e4m3x2_hi_to_f16x2(u), e4m3x2_to_f16x2(v),
                                 e4m3x2_hi_to_f16x2(v)};
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            Mma<__half>::run(acc[n], f, ph[t][n][0], ph[t][n][1]);
            Mma<__half>::run(acc[n], f, pl[t][n][0], pl[t][n][1]);
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            o[a][n][r] = fmaf(acc[n][r], vdown, o[a][n][r] * alpha[n][r & 1]);
      }
  }
  float vdown;   // 2^-shift of the current tile's weights

  // Write the segment: normalised output, or a partial for the merge.
  __device__ __forceinline__ void finish(const DecodeParams &p, int s, int h, bool complete,
                                         int slot, int lane) {
    const int g = lane >> 2, c = lane & 3;
    const int G = p.group;
    const uint64_t pol = l2_policy_evict_last();   // partials stay in L2 for the merge
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float lt = l[n][r];
        lt += __shfl_xor_sync(0xffffffffu, lt, 4);
        lt += __shfl_xor_sync(0xffffffffu, lt, 8);
        lt += __shfl_xor_sync(0xffffffffu, lt, 16);
        const int head = n * 8 + 2 * c + r;
        if (head >= G) continue;
        const float f = complete ? (lt == 0.f ? 0.f : 1.f / lt) : 1.f;
        float *dst = (complete ? p.out + ((int64_t)s * p.num_q_heads + (int64_t)h * G) * D
                               : p.part_o + (int64_t)slot * G * D) +
                     head * D + (D / 8) * g;
#pragma unroll
        for (int a = 0; a < MM; a += 2) {
          const float4 v = make_float4(o[a][n][r] * f, o[a][n][2 + r] * f, o[a + 1][n][r] * f,
                                       o[a + 1][n][2 + r] * f);
          if (complete)
            *reinterpret_cast<float4 *>(dst + 2 * a) = v;
          else
            st_global_hint4(dst + 2 * a, v, pol);
        }
        if (!complete && g == 0) {
          float *pm = p.part_ml + ((int64_t)slot * G + head) * 2;
          st_global_hint(pm, m[n][r], pol);
          st_global_hint(pm + 1, lt, pol);
        }
      }
  }
};

// Lane-parallel description of up to 32 consecutive tiles of one sequence.
struct Fp8Batch {
  int s, L, nt;             // warp-uniform: sequence, its length, its tiles
  int n;                    // tiles in the batch (0 = none)
  int my_h, my_j;           // this lane's tile
  int id0, id1;             // its blocks (block size 32: id1 unused)
};

__device__ __forceinline__ void make_fp8_batch(const DecodeFp8Params &p, Fp8Batch &tb, int s, int L,
                                               int nt, int h, int j, int64_t remaining, int lane) {
  tb.s = s;
  tb.L = L;
  tb.nt = nt;
  const int64_t left = (int64_t)p.d.num_kv_heads * nt - ((int64_t)h * nt + j);
  const int64_t n = left < remaining ? left : remaining;
  tb.n = n < 32 ? (int)n : 32;
  tb.my_h = 0;
  tb.my_j = 0;
  tb.id0 = tb.id1 = -1;
  if (lane < tb.n) {
    const int64_t at = (int64_t)h * nt + j + lane;
    tb.my_h = (int)(at / nt);
    tb.my_j = (int)(at - (int64_t)tb.my_h * nt);
    const int32_t *row = p.d.block_tables + (int64_t)s * p.table_blocks;
    const int per = kF8Tile / p.block_size, b0 = tb.my_j * per;
    const int used = min(ceil_div_i(L, p.block_size), p.table_blocks);
    if (b0 < used) tb.id0 = __ldg(row + b0);
    if (per == 2 && b0 + 1 < used) tb.id1 = __ldg(row + b0 + 1);
  }
}

// Smem of one CTA: per warp and stage a K and a V tile, 64 scales, the group's
// query rows, a tile descriptor and a barrier.
__host__ __device__ constexpr int fp8_stage_bytes(int D) { return 2 * kF8Tile * D; }
constexpr int kF8ScaleBytes = kF8Tile * 2 * 4;
struct Fp8Tile {
  int s, h, flags;
  uint32_t live;
};

template <int D, int NT, int NW>
__global__ void __launch_bounds__(NW * 32, NT == 1 ? 3 : 2)
    paged_decode_fp8_kernel(const __grid_constant__ CUtensorMap kmap,
                            const __grid_constant__ CUtensorMap vmap, const DecodeFp8Params pp) {
  constexpr int TILE = kF8Tile * D;
  constexpr int STAGE = fp8_stage_bytes(D);
  const DecodeParams &p = pp.d;
  const int G = p.group, B = pp.block_size;
  const int qbytes = G * D * 2;
  const int nstage = p.nstage;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = p.num_seqs, Hkv = p.num_kv_heads;

  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int k0 = warp * nstage, all = NW * nstage;
  uint8_t *stages = smem + (size_t)k0 * STAGE;
  uint8_t *scales = smem + (size_t)all * STAGE + (size_t)k0 * kF8ScaleBytes;
  uint8_t *qslots = smem + (size_t)all * (STAGE + kF8ScaleBytes) + (size_t)k0 * qbytes;
  uint8_t *after_q = smem + (size_t)all * (STAGE + kF8ScaleBytes + qbytes);
  Fp8Tile *info = reinterpret_cast<Fp8Tile *>(after_q) + k0;
  uint64_t *bars = reinterpret_cast<uint64_t *>(after_q + (size_t)all * sizeof(Fp8Tile)) + k0;

  __shared__ long long red[NW];
  __shared__ int loc_s[NW];
  __shared__ long long loc_base[NW];
  __shared__ int loc_L[NW];

  if (threadIdx.x == 0) {
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
  }
  if (lane == 0)
    for (int k = 0; k < nstage; ++k) mbar_init(&bars[k], 1);
  grid_dependency_wait();
  allow_dependent_launch();

  // ---- plan: total tiles, this CTA's warp ranges
  const long long w_total = (long long)gridDim.x * NW;
  const long long w = (long long)blockIdx.x * NW + warp;
  long long U = 0, w_active = 0;
  cta_plan<kF8Tile, NW>(
      p, w_total, [&](int k, long long U_, long long wa_) -> long long {
        const long long wk = (long long)blockIdx.x * NW + k;
        return wk < wa_ ? (wk * U_) / wa_ : -1;
      },
      true, red, loc_s, loc_base, loc_L, U, w_active);
  if (lane == 0) fence_barrier_init();
  __syncwarp();
  const bool active = w < w_active;
  const long long u0 = active ? (w * U) / w_active : 0;
  const long long u1 = active ? ((w + 1) * U) / w_active : 0;
  long long *meta = p.meta + w * kMetaWords;
  if (!active) {
    if (lane < kMetaWords) meta[lane] = lane == 3 ? U : (lane == 4 ? w_active : 0);
    return;
  }

  // ---- this warp's first tile
  const int s0 = loc_s[warp];
  const long long base0 = loc_base[warp];
  const int L0 = loc_L[warp];
  const int nt0 = ceil_div_i(L0, kF8Tile);
  const long long r0 = u0 - base0;
  const int h0 = (int)(r0 / nt0);
  const int j0 = (int)(r0 - (long long)h0 * nt0);
  if (lane < kMetaWords) {   // descriptor for the merge, as in the 16-bit kernel
    const long long seg_lo = base0 + (long long)h0 * nt0;
    long long v = 1;
    switch (lane) {
      case 0: v = u0; break;
      case 1: v = seg_lo; break;
      case 2: v = seg_lo + nt0; break;
      case 3: v = U; break;
      case 4: v = w_active; break;
      case 5: v = s0; break;
      case 6: v = h0; break;
      default: v = 1;
    }
    meta[lane] = v;
  }
  const long long ntiles = u1 - u0;

  // ---- issue cursor
  Fp8Batch cur, nxt;
  long long issued = 0;
  int cur_k = 0;
  make_fp8_batch(pp, cur, s0, L0, nt0, h0, j0, ntiles, lane);
  auto follow = [&](const Fp8Batch &b, long long remaining) {   // the batch after b
    Fp8Batch r = b;
    r.n = 0;
    if (remaining <= 0) return r;
    int h = __shfl_sync(0xffffffffu, b.my_h, b.n - 1);
    int j = __shfl_sync(0xffffffffu, b.my_j, b.n - 1) + 1;
    int s = b.s, L = b.L, nt = b.nt;
    if (j == nt) { j = 0; ++h; }
    while (h >= Hkv || nt == 0) {   // next sequence with tiles
      ++s;
      if (s >= S) return r;
      L = seq_len_clamped<kF8Tile>(p, s);
      nt = ceil_div_i(L, kF8Tile);
      h = 0;
      j = 0;
    }
    make_fp8_batch(pp, r, s, L, nt, h, j, remaining, lane);
    return r;
  };
  nxt = follow(cur, ntiles - cur.n);

  const uint64_t stream_policy = l2_policy_evict_first();
  const int per = kF8Tile / B;
  auto issue = [&](int stage) {
    if (cur_k == cur.n) {
      cur = nxt;
      cur_k = 0;
      nxt = follow(cur, ntiles - issued - cur.n);
    }
    const int h = __shfl_sync(0xffffffffu, cur.my_h, cur_k);
    const int j = __shfl_sync(0xffffffffu, cur.my_j, cur_k);
    const int id0 = __shfl_sync(0xffffffffu, cur.id0, cur_k);
    const int id1 = __shfl_sync(0xffffffffu, cur.id1, cur_k);
    const int len = min(kF8Tile, cur.L - j * kF8Tile);
    const bool in0 = id0 >= 0 && id0 < p.num_blocks;
    const bool in1 = per == 2 && len > B && id1 >= 0 && id1 < p.num_blocks;
    const bool first = j == 0 || issued == 0;
    uint64_t *bar = &bars[stage];
    fence_proxy_async_smem();   // this lane's reads of the stage, before copies into it
    if (lane == 0) {
      Fp8Tile ti;
      ti.s = cur.s;
      ti.h = h;
      ti.flags = (first ? TF_FIRST : 0) |
                 (j == cur.nt - 1 || issued == ntiles - 1 ? TF_LAST : 0) |
                 (j == 0 ? TF_J0 : 0) | (j == cur.nt - 1 ? TF_JEND : 0);
      const uint32_t below = len == 32 ? 0xffffffffu : (1u << len) - 1u;
      ti.live = below & ((in0 ? (per == 2 ? 0x0000ffffu : 0xffffffffu) : 0u) |
                         (in1 ? 0xffff0000u : 0u));
      if (ti.live != below) {   // a block outside the pool, or past the table's end
        const bool past = j * per + (in0 ? 1 : 0) >= pp.table_blocks;
        flag_error(past ? PA_DEVERR_CONTEXT_LEN : PA_DEVERR_BLOCK_ID);
      }
      info[stage] = ti;
      const uint32_t bytes =
          (in0 + in1) * (2 * B * D + 8 * B) + (first ? (uint32_t)qbytes : 0u);
      if (bytes)
        mbar_arrive_expect_tx(bar, bytes);
      else
        mbar_arrive(bar);
      if (first)
        bulk_load(qslots + (size_t)stage * qbytes,
                  p.q + ((int64_t)cur.s * p.num_q_heads + (int64_t)h * G) * (D * 2), qbytes, bar);
    }
    __syncwarp();
    // lanes 0 .. 3 per - 1: K codes, V codes and scales of one block each
    const int b = lane / 3, kind = lane - 3 * b;
    if (b < per && (b == 0 ? in0 : in1)) {
      const int tile = (b == 0 ? id0 : id1) * Hkv + h;
      uint8_t *dst = stages + (size_t)stage * STAGE + b * B * D;
      if (kind == 0)
        tma_load_2d_hint(dst, &kmap, 0, tile * B, bar, stream_policy);
      else if (kind == 1)
        tma_load_2d_hint(dst + TILE, &vmap, 0, tile * B, bar, stream_policy);
      else
        bulk_load(scales + (size_t)stage * kF8ScaleBytes + b * 8 * B,
                  pp.kv_scale + (int64_t)tile * 2 * B, 8 * B, bar);
    }
    ++cur_k;
    ++issued;
  };

  const int pre = ntiles < nstage ? (int)ntiles : nstage;
  for (int k = 0; k < pre; ++k) issue(k);

  // ---- consume
  Fp8Path<D, NT> st;
  st.reset();
  bool seg_from0 = false;
  int seg_index = 0, stage = 0;
  uint32_t parity = 0;
  for (long long i = 0; i < ntiles; ++i) {
    if (!mbar_wait_bounded(&bars[stage], parity, p.wait_ns)) {
      if (lane == 0) flag_error(PA_DEVERR_TIMEOUT);
      // copies still in flight, this tile's and later ones, land before the
      // warp leaves
      for (long long k = i; k < issued; ++k)
        mbar_wait_bounded(&bars[k % nstage], (uint32_t)((k / nstage) & 1), kDrainLimitNs);
      return;
    }
    const Fp8Tile ti = info[stage];
    if (ti.flags & TF_FIRST) {
      st.reset();
      st.load_q(qslots + (size_t)stage * qbytes, G, pp.q_bf16 != 0, p.scale_log2, lane);
      seg_from0 = (ti.flags & TF_J0) != 0;
    }
    if (ti.live) {
      const uint32_t kb = smem_addr(stages + (size_t)stage * STAGE);
      st.tile(kb, kb + TILE, smem_addr(scales + (size_t)stage * kF8ScaleBytes), B, ti.live, lane);
    }
    if (ti.flags & TF_LAST) {
      const bool complete = seg_from0 && (ti.flags & TF_JEND);
      st.finish(p, ti.s, ti.h, complete, (int)(2 * w + (seg_index == 0 ? 0 : 1)), lane);
      ++seg_index;
    }
    __syncwarp();
    if (i + nstage < ntiles) issue(stage);
    if (++stage == nstage) {
      stage = 0;
      parity ^= 1;
    }
  }
}

}  // namespace pa
