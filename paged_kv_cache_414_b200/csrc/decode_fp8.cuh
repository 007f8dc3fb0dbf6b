// Paged decode attention over an 8-bit cache, for sm_100a.
//
// For sequence s and query head h of kv head kh, with e4m3 codes K^, V^ and
// per-token scales ks, vs (layouts in fp8_cache.cuh):
//   out[s, h] = sum_t w_t vs_t V^_t,   w = softmax_t(scale ks_t <q, K^_t>).
// The scales never touch the codes: ks_t multiplies the finished score and
// vs_t the weight, so both products run on the codes as they lie in the pool.
//
// Work split as in the 16-bit decode kernel (decode_attention.cuh): the tiles of
// all (sequence, kv head) pairs, numbered in order, are cut into equal
// contiguous ranges, one per warp, and cut segments leave partials for the
// merge kernel.  Every warp finds its range by itself.  Where no context can be
// longer than a few tiles, ranges are cut between pairs only and there is
// nothing to merge.  Here a tile is 32 tokens
// whatever the block size (two blocks of 16 or one of 32): half the bytes per
// token would otherwise leave twice the bookkeeping per byte.  Every kv head of
// a sequence begins with a tile of no tokens that stands for what a segment
// costs besides its tiles (its query rows, its output): short sequences would
// otherwise make some warps' equal shares take a quarter longer than the mean.
//
// A warp has one buffer for K and one for V, filled by tensor copies: the next
// tile's K is asked for as soon as the scores are made, its V after P.V, so
// either is on its way during about half of a tile's work, and 8 to 16 warps
// per SM cover for each other.  One elected lane issues, from warp-uniform
// values: six lanes with a copy each took 1400 cycles per tile instead of 850,
// and so did 16-byte asynchronous copies by all lanes.
//
// Arithmetic.
//   * Codes become fp16 exactly (cvt.rn.f16x2.e4m3x2) and both products are
//     fp16 warp MMAs (m16n8k16, fp32 accumulation) for fp16 and bf16 queries
//     alike.  (With the e4m3 warp MMA on e4m3 pieces of the queries the decode
//     of 256 mixed sequences took 6 percent longer.)
//   * A query row is scaled by the power of two that puts its largest element
//     in [2^14, 2^15) before it is rounded to fp16: exact for fp16 queries and
//     for bf16 elements down to 2^-39 of the row's largest.
//   * A weight times its vs_t is scaled by the power of two that puts the
//     tile's largest vs in the same range and goes in as a hi + lo pair of
//     fp16 values (2^-22 relative), so the output keeps ~fp32 accuracy.
//   * Groups of up to four heads (HPL = 1) give each head two neighbouring of
//     the eight MMA columns: a lane then holds the scores of one head, half the
//     softmax work, and hi and lo share one P.V MMA.  Wider groups (HPL = 2)
//     need the columns for heads and take two.
//   * A tile's P.V is summed in fresh accumulators and folded into the running
//     output by one FMA with the softmax correction, so long segments never
//     add small products to a large tensor-core accumulator.
// Fragments come from shared memory by plain 16-byte loads, not ldmatrix: the
// reduction order of an MMA is free as long as both operands agree, so lane
// (g, c) takes D/4 neighbouring codes of K row g, and D/8 neighbouring columns
// of V for its four tokens; bytes of two tokens are paired with one byte
// permute before the conversion.  Chunks are swizzled within 128-byte (D = 128)
// or 64-byte (D = 64) rows, with which the K loads and D = 128's V loads are
// free of bank conflicts.
//
// Bound: HBM, 2 D + 8 bytes per token and kv head; held back by the
// instructions of a tile.  Of its 4100 cycles (D = 128, eight heads, 12 warps
// per SM) a warp waits 380 for copies, takes 900 for the scores, 2030 for
// weights and output and 820 for the copies' bookkeeping.  375 MB of 64 / 8
// heads take 71 us, 5.3 TB/s, and 79 with the merge in a loop of calls; 407 MB
// of 256 mixed sequences 79 to 80 with it.  Groups above eight pay for their
// registers (two CTAs per SM): 375 MB of 128 / 8 heads take 116 us.
#pragma once

#include <cuda_fp8.h>

#include "decode_attention.cuh"
#include "prefill_attention.cuh"   // fast_exp2

namespace pa {

constexpr int kF8Tile = 32;   // tokens per tile

// Tiles of a kv head of a sequence of L tokens: the empty first one, then its
// tokens 32 at a time.
__device__ __forceinline__ int fp8_tiles(int L) {
  return L > 0 ? (L + kF8Tile - 1) / kF8Tile + 1 : 0;
}

struct DecodeFp8Params {
  float *out;                    // [S, Hq, D]
  const uint8_t *q;              // [S, Hq, D], 16 bits
  const float *kv_scale;         // [NB, Hkv, 2, B]
  const int32_t *block_tables;   // [S, max_blocks]
  const int32_t *context_lens;   // [S]
  int4 *meta;                    // [w_total]: the segment each range begins in, for the merge
  float2 *part_ml;               // [2 w_total][G]  (max in log2 units, sum)
  float *part_o;                 // [2 w_total][G][D]
  float scale_log2;              // scale * log2(e)
  int num_seqs, num_q_heads, num_kv_heads, group;
  int max_blocks, num_blocks, block_size;
  int q_bf16;
  int min_tiles;                 // fewest tiles a warp is given; 0: whole (sequence, kv head) pairs
  uint64_t wait_ns;              // limit of a wait on a copy before giving up (2 s by default)
};

// Length of sequence s, cut to what its row of the block table can hold.
__device__ __forceinline__ int fp8_length(const DecodeFp8Params &p, int s) {
  const int L = __ldg(p.context_lens + s);
  return max(0, min(L, p.max_blocks * p.block_size));
}

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

// One lane of a fully active warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(e));
  return e != 0;
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

// D = A B (+ C), A and B fp16.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1, const float *c) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]),
        "f"(c[2]), "f"(c[3]));
}

// NT sets of 4 HPL heads; lane (g, c) works on heads (4 n + c) HPL + e of set n.
template <int D, int NT, int HPL>
struct Fp8Path {
  static constexpr int W = D / 16;           // words of K per lane and row = k-steps of q.K
  static constexpr int MM = D / 16;          // m-tiles of P.V
  float o[MM][NT][HPL][2];                   // d = (D/8) g + 2 mm + r
  float m[NT][HPL], l[NT][HPL];
  float qs[NT][HPL];                         // scale * log2(e) * 2^-shift of the head's q
  uint32_t qf[W][NT][2];
  int k_off[2], v_off[2];                    // this lane's chunks of K rows g, V rows 2 c and 2 c + 1

  __device__ __forceinline__ void init(int lane) {
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = 2 * c + i;
      if constexpr (D == 128) {
        k_off[i] = g * 128 + (((2 * c + i) ^ g) << 4);
        v_off[i] = row * 128 + ((g ^ row) << 4);
      } else {
        k_off[i] = g * 64 + ((c ^ (g >> 1)) << 4);   // one chunk a row: i = 1 is not used
        v_off[i] = row * 64 + (((g >> 1) ^ (row >> 1)) << 4) + (g & 1) * 8;
      }
    }
    reset();
  }

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < HPL; ++e) {
#pragma unroll
        for (int a = 0; a < MM; ++a) o[a][n][e][0] = o[a][n][e][1] = 0.f;
        m[n][e] = -INFINITY;
        l[n][e] = 0.f;
      }
  }

  // Lane (g, c): columns (D/4) c .. of the query row of MMA column g, as scaled fp16.
  __device__ __forceinline__ void load_q(const uint8_t *q, int G, bool bf16, float scale_log2,
                                         int lane) {
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int head = HPL == 1 ? n * 4 + (g >> 1) : n * 8 + g;
      uint32_t raw[2 * W];
      uint32_t top = 0;               // the largest magnitude, as 16 bits
      const uint4 *row = reinterpret_cast<const uint4 *>(q + (size_t)head * (D * 2) + c * (D / 2));
#pragma unroll
      for (int i = 0; i < W / 2; ++i) {
        const uint4 v = head < G ? row[i] : make_uint4(0, 0, 0, 0);
        raw[4 * i] = v.x, raw[4 * i + 1] = v.y, raw[4 * i + 2] = v.z, raw[4 * i + 3] = v.w;
      }
#pragma unroll
      for (int i = 0; i < 2 * W; ++i) top = __vmaxu2(top, raw[i] & 0x7fff7fffu);
      top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
      top = max(top & 0xffffu, top >> 16);
      const float big = bf16 ? __uint_as_float(top << 16) : __half2float(__ushort_as_half(top));
      const int e = scale_field(__float_as_uint(big));
      const float up = pow2_field(268 - e);
      const float down = pow2_field(e - 14) * scale_log2;
#pragma unroll
      for (int i = 0; i < 2 * W; ++i) {
        const float2 f = bf16 ? Mma<__nv_bfloat16>::unpack(raw[i]) : Mma<__half>::unpack(raw[i]);
        qf[i >> 1][n][i & 1] = Mma<__half>::pack(f.x * up, f.y * up);
      }
#pragma unroll
      for (int e2 = 0; e2 < HPL; ++e2)       // column 2 c + e2 was loaded by lanes 8 c + 4 e2 ..
        qs[n][e2] = __shfl_sync(0xffffffffu, down, 8 * c + 4 * e2);
    }
  }

  float sc[2][NT][2][HPL];     // scores of tokens 16 t + g + 8 x

  // Scores of one tile, S^T[token][head]: K codes at kb, scales at sb ([block][K
  // or V][B]).
  __device__ __forceinline__ void scores(const uint8_t *kb, const float *sb, int B, int lane) {
    const int g = lane >> 2;
    const float zero[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      uint32_t k0[W], k1[W];     // rows 16 t + g and + 8 (the same swizzle)
#pragma unroll
      for (int i = 0; i < W / 4; ++i) {
        const uint8_t *a = kb + k_off[i] + t * (16 * D);
        const uint4 v = *reinterpret_cast<const uint4 *>(a);
        const uint4 u = *reinterpret_cast<const uint4 *>(a + 8 * D);
        k0[4 * i] = v.x, k0[4 * i + 1] = v.y, k0[4 * i + 2] = v.z, k0[4 * i + 3] = v.w;
        k1[4 * i] = u.x, k1[4 * i + 1] = u.y, k1[4 * i + 2] = u.z, k1[4 * i + 3] = u.w;
      }
      float s[NT][4];
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const uint32_t a[4] = {e4m3x2_to_f16x2(k0[w]), e4m3x2_to_f16x2(k1[w]),
                               e4m3x2_hi_to_f16x2(k0[w]), e4m3x2_hi_to_f16x2(k1[w])};
#pragma unroll
        for (int n = 0; n < NT; ++n) mma_f16(s[n], a, qf[w][n][0], qf[w][n][1], w == 0 ? zero : s[n]);
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float ks = sb[t * (512 / B) + g + 8 * x];   // token 16: the next block, or this one
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < HPL; ++e) sc[t][n][x][e] = s[n][2 * x + e] * (ks * qs[n][e]);
      }
    }
  }

  // The same tile's part of the output: V codes at vb, `live` the tokens that
  // count.
  __device__ __forceinline__ void output(const uint8_t *vb, const float *sb, int B, uint32_t live,
                                         int lane) {
    const int g = lane >> 2, c = lane & 3;
    const float zero[4] = {0.f, 0.f, 0.f, 0.f};
    float vs[2][2];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int x = 0; x < 2; ++x) vs[t][x] = sb[t * (512 / B) + B + g + 8 * x];
    if (live != 0xffffffffu) {                  // tokens that do not count
      const uint32_t mask = live >> g;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if (!((mask >> (16 * t + 8 * x)) & 1)) {
            vs[t][x] = 0.f;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < HPL; ++e) sc[t][n][x][e] = -INFINITY;
          }
    }
    // ---- running maximum and sum of each head; weights (times vs) as B operands
    float alpha[NT][HPL], vdown[NT][HPL];    // vdown: 2^-shift of a head's weights
    uint32_t ph[2][NT][2], pl[2][NT][2];     // HPL = 1: hi and lo both in ph
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float hi[HPL][2][2], lo[HPL][2][2];
      uint32_t top[HPL];                     // largest weight times vs, as bits
#pragma unroll
      for (int e = 0; e < HPL; ++e) {
        float v = fmaxf(fmaxf(sc[0][n][0][e], sc[0][n][1][e]), fmaxf(sc[1][n][0][e], sc[1][n][1][e]));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
        const float mn = fmaxf(m[n][e], v);
        // all scores so far -inf (a -inf in q or K): weights of 0, not NaN
        const float ref = mn == -INFINITY ? 0.f : mn;
        alpha[n][e] = fast_exp2(m[n][e] - ref);
        m[n][e] = mn;
        float sum = 0.f;
        top[e] = 0;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float pv = fast_exp2(sc[t][n][x][e] - ref);
            sum += pv;
            lo[e][t][x] = pv * vs[t][x];
            top[e] = max(top[e], __float_as_uint(fabsf(lo[e][t][x])));
          }
        l[n][e] = l[n][e] * alpha[n][e] + sum;
      }
      // the exponents of both heads' largest go through the shuffles together
      uint32_t tops = HPL == 1 ? top[0] >> 16 : __byte_perm(top[0], top[HPL - 1], 0x7632);
#pragma unroll
      for (int d = 4; d < 32; d <<= 1)
        tops = __vmaxu2(tops, __shfl_xor_sync(0xffffffffu, tops, d));
#pragma unroll
      for (int e = 0; e < HPL; ++e) {
        const int field = scale_field(e == 0 ? tops << 16 : tops);
        const float up = pow2_field(268 - field);
        vdown[n][e] = pow2_field(field - 14);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float y = lo[e][t][x] * up;
            hi[e][t][x] = __half2float(__float2half_rn(y));
            lo[e][t][x] = y - hi[e][t][x];
          }
      }
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          ph[t][n][x] = movmatrix_trans(
              Mma<__half>::pack(hi[0][t][x], HPL == 1 ? lo[0][t][x] : hi[HPL - 1][t][x]));
          if constexpr (HPL == 2)
            pl[t][n][x] = movmatrix_trans(Mma<__half>::pack(lo[0][t][x], lo[1][t][x]));
        }
    }
    // ---- O^T[d][head] = alpha O^T + 2^.. V^T P^T
    constexpr int XW = D / 32;   // words of V per lane and token
    uint32_t vw[2][4][XW];       // tokens 16 t + 2 c + {0, 1, 8, 9}
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint8_t *a = vb + v_off[i & 1] + (16 * t + 8 * (i >> 1)) * D;
        if constexpr (D == 128) {
          const uint4 v = *reinterpret_cast<const uint4 *>(a);
          vw[t][i][0] = v.x, vw[t][i][1] = v.y, vw[t][i][2] = v.z, vw[t][i][3] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2 *>(a);
          vw[t][i][0] = v.x, vw[t][i][1] = v.y;
        }
      }
    if (live != 0xffffffffu) {   // a token that does not count may hold any bits, NaN codes too
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = 16 * t + 2 * c + (i & 1) + 8 * (i >> 1);
#pragma unroll
          for (int x = 0; x < XW; ++x) vw[t][i][x] = (live >> row) & 1 ? vw[t][i][x] : 0u;
        }
    }
#pragma unroll
    for (int x = 0; x < XW; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int a = 2 * x + y;                      // columns 2 a, 2 a + 1 of this lane's
        const uint32_t sel = y ? 0x7362u : 0x5140u;   // bytes 2 y, 2 y + 1 of both tokens
        float acc[NT][4];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const uint32_t u = __byte_perm(vw[t][0][x], vw[t][1][x], sel);
          const uint32_t v = __byte_perm(vw[t][2][x], vw[t][3][x], sel);
          const uint32_t f[4] = {e4m3x2_to_f16x2(u), e4m3x2_hi_to_f16x2(u), e4m3x2_to_f16x2(v),
                                 e4m3x2_hi_to_f16x2(v)};
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_f16(acc[n], f, ph[t][n][0], ph[t][n][1], t == 0 ? zero : acc[n]);
            if constexpr (HPL == 2) mma_f16(acc[n], f, pl[t][n][0], pl[t][n][1], acc[n]);
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < HPL; ++e)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float add = HPL == 1 ? acc[n][2 * r] + acc[n][2 * r + 1] : acc[n][2 * r + e];
              o[a][n][e][r] = fmaf(add, vdown[n][e], o[a][n][e][r] * alpha[n][e]);
            }
      }
  }

  // Write the segment: normalised output, or a partial for the merge.
  __device__ __forceinline__ void finish(const DecodeFp8Params &p, int s, int h, bool complete,
                                         int slot, int lane) {
    const int g = lane >> 2, c = lane & 3;
    const int G = p.group;
    const uint64_t pol = l2_policy_evict_last();   // partials stay in L2 for the merge
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < HPL; ++e) {
        float lt = l[n][e];
        lt += __shfl_xor_sync(0xffffffffu, lt, 4);
        lt += __shfl_xor_sync(0xffffffffu, lt, 8);
        lt += __shfl_xor_sync(0xffffffffu, lt, 16);
        const int head = (n * 4 + c) * HPL + e;
        if (head >= G) continue;
        const float f = complete ? (lt == 0.f ? 0.f : 1.f / lt) : 1.f;
        float *dst = (complete ? p.out + ((int64_t)s * p.num_q_heads + (int64_t)h * G) * D
                               : p.part_o + (int64_t)slot * G * D) +
                     head * D + (D / 8) * g;
#pragma unroll
        for (int a = 0; a < MM; a += 2) {
          const float4 v = make_float4(o[a][n][e][0] * f, o[a][n][e][1] * f, o[a + 1][n][e][0] * f,
                                       o[a + 1][n][e][1] * f);
          if (complete)
            *reinterpret_cast<float4 *>(dst + 2 * a) = v;
          else
            st_global_hint4(dst + 2 * a, v, pol);
        }
        if (!complete && g == 0) {
          p.part_ml[(int64_t)slot * G + head] = make_float2(m[n][e], lt);
        }
      }
  }
};

// A tile as its warp's ring holds it: first rows of its blocks in the code
// pools (-1: no such block), the tokens that count, TF_ flags and kv head << 8.
struct Fp8Tile {
  int row0, row1;
  uint32_t live;
  int head_flags;
};
constexpr int kF8Ring = 64;

// The walk of a warp through its tiles, described up to 32 at a time, lane by
// lane: begin() fetches the block ids of the next run of tiles of one
// sequence, end() writes the run into the ring.
struct Fp8Walk {
  int s, L, nt, h, j;        // next tile to describe (warp-uniform)
  int described;             // tiles described so far
  int n;                     // tiles between begin() and end()
  int id0, id1, my_h, my_j;  // this lane's tile of them

  __device__ __forceinline__ void begin(const DecodeFp8Params &p, int ntiles, int lane) {
    while (h >= p.num_kv_heads || nt == 0) {   // next sequence with tiles
      h = 0;
      j = 0;
      if (s + 1 >= p.num_seqs) {   // only if lengths changed under the kernel: empty tiles
        L = 0;
        nt = 1;
        break;
      }
      ++s;
      L = fp8_length(p, s);
      nt = fp8_tiles(L);
    }
    const int64_t left = (int64_t)(p.num_kv_heads - h) * nt - j;
    n = min((int)min(left, (int64_t)32), ntiles - described);
    my_h = h;
    my_j = j + lane;                 // a few steps, one when nt >= 32
    while (my_j >= nt) my_j -= nt, ++my_h;
    id0 = id1 = -1;
    if (lane < n) {
      const int per = kF8Tile / p.block_size, b0 = (my_j - 1) * per;
      const int32_t *table = p.block_tables + (int64_t)s * p.max_blocks + b0;
      const bool two = per == 2 && L - (my_j - 1) * kF8Tile > p.block_size;
      if (my_j > 0 && b0 < p.max_blocks) id0 = __ldg(table);
      if (my_j > 0 && two && b0 + 1 < p.max_blocks) id1 = __ldg(table + 1);
    }
  }

  __device__ __forceinline__ void end(const DecodeFp8Params &p, Fp8Tile *ring, int *ring_s,
                                      int ntiles, int lane) {
    if (lane < n) {
      const int B = p.block_size, per = kF8Tile / B;
      const int len = my_j == 0 ? 0 : min(kF8Tile, L - (my_j - 1) * kF8Tile);
      const uint32_t below = len == 32 ? 0xffffffffu : (1u << len) - 1u;
      const bool in0 = id0 >= 0 && id0 < p.num_blocks, in1 = id1 >= 0 && id1 < p.num_blocks;
      const bool first = my_j == 0, last = my_j == nt - 1;
      const int at = described + lane;
      Fp8Tile t;
      t.row0 = in0 ? (id0 * p.num_kv_heads + my_h) * B : -1;
      t.row1 = in1 ? (id1 * p.num_kv_heads + my_h) * B : -1;
      t.live = below & ((in0 ? (per == 2 ? 0x0000ffffu : 0xffffffffu) : 0u) |
                        (in1 ? 0xffff0000u : 0u));
      t.head_flags = (my_h << 8) | (first || at == 0 ? TF_FIRST : 0) | (first ? TF_J0 : 0) |
                     (last || at == ntiles - 1 ? TF_LAST : 0) | (last ? TF_JEND : 0);
      if (t.live != below)           // a block outside the pool, or past the table's end
        flag_error((my_j - 1) * per + (in0 ? 1 : 0) >= p.max_blocks ? PA_DEVERR_CONTEXT_LEN
                                                                : PA_DEVERR_BLOCK_ID);
      ring[at & (kF8Ring - 1)] = t;
      ring_s[at & (kF8Ring - 1)] = s;
    }
    const int last_h = __shfl_sync(0xffffffffu, my_h, n - 1);
    const int last_j = __shfl_sync(0xffffffffu, my_j, n - 1);
    described += n;
    n = 0;
    h = last_h + (last_j == nt - 1 ? 1 : 0);
    j = last_j == nt - 1 ? 0 : last_j + 1;
    __syncwarp();
  }
};

// Smem of one warp: a K and a V tile, two tiles' scales, the group's query
// rows, a ring of tile descriptions, two barriers; in whole swizzle atoms.
constexpr int kF8ScaleFloats = 2 * kF8Tile;
__host__ __device__ constexpr int fp8_warp_bytes(int D, int G) {
  return (2 * kF8Tile * D + 2 * kF8ScaleFloats * 4 + G * D * 2 +
          kF8Ring * (int)(sizeof(Fp8Tile) + 4) + 16 + 1023) /
         1024 * 1024;
}

// CTAs per SM that registers allow.
__host__ __device__ constexpr int fp8_ctas(int NT, int HPL) {
  return NT * HPL == 1 ? 4 : (NT * HPL == 2 ? 3 : 2);
}

// Sum over the lanes before this one, and over all of them.
__device__ __forceinline__ int warp_scan(int v, int lane, int *total) {
  int incl = v;
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, x);
    if (lane >= x) incl += y;
  }
  *total = __shfl_sync(0xffffffffu, incl, 31);
  return incl - v;
}

template <int D, int NT, int HPL, int NW>
__global__ void __launch_bounds__(NW * 32, fp8_ctas(NT, HPL))
    paged_decode_fp8_kernel(const __grid_constant__ CUtensorMap kmap,
                            const __grid_constant__ CUtensorMap vmap, const DecodeFp8Params p) {
  constexpr int TILE = kF8Tile * D;
  const int G = p.group, B = p.block_size, S = p.num_seqs;
  const int qbytes = G * D * 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *kbuf = smem + (size_t)warp * fp8_warp_bytes(D, G), *vbuf = kbuf + TILE;
  float *scales = reinterpret_cast<float *>(vbuf + TILE);
  uint8_t *qbuf = reinterpret_cast<uint8_t *>(scales + 2 * kF8ScaleFloats);
  Fp8Tile *ring = reinterpret_cast<Fp8Tile *>(qbuf + qbytes);
  int *ring_s = reinterpret_cast<int *>(ring + kF8Ring);
  uint64_t *kbar = reinterpret_cast<uint64_t *>(ring_s + kF8Ring), *vbar = kbar + 1;

  if (lane == 0) {
    mbar_init(kbar, 1);
    mbar_init(vbar, 1);
    fence_barrier_init();
  }
  if (threadIdx.x == 0) {
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
  }
  grid_dependency_wait();
  allow_dependent_launch();

  const int w_total = gridDim.x * NW, w = blockIdx.x * NW + warp;
  // empty sequences' rows, and lengths that the table cannot hold
  for (int s = w; s < S; s += w_total) {
    const int L = __ldg(p.context_lens + s);
    if (lane == 0 && (L < 0 || L > p.max_blocks * B)) flag_error(PA_DEVERR_CONTEXT_LEN);
    if (L <= 0) {
      float4 *row = reinterpret_cast<float4 *>(p.out + (int64_t)s * p.num_q_heads * D);
      for (int k = lane; k < p.num_q_heads * D / 4; k += 32) row[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  // ---- this warp's range: ntiles tiles from tile j0 of kv head h0 of sequence s0 on
  int s0, h0, j0, L0, nt0, ntiles, w_active = 0;
  long long u0 = 0, U = 0;
  if (p.min_tiles == 0) {
    const long long pairs = (long long)S * p.num_kv_heads;
    const long long a = pairs * w / w_total, e = pairs * (w + 1) / w_total;
    int sum = 0;
    for (long long i = a + lane; i < e; i += 32)
      sum += fp8_tiles(fp8_length(p, (int)(i / p.num_kv_heads)));
    ntiles = __reduce_add_sync(0xffffffffu, sum);
    if (ntiles == 0) return;
    s0 = (int)(a / p.num_kv_heads);
    h0 = (int)(a - (long long)s0 * p.num_kv_heads);
    j0 = 0;
    L0 = fp8_length(p, s0);
    nt0 = fp8_tiles(L0);
  } else {
    // lane l counts the tiles (of one kv head) of sequences per * l ..
    const int per = (S + 31) / 32;
    int mine = 0;
#pragma unroll 8
    for (int k = 0; k < per; ++k) {
      const int s = lane * per + k;
      mine += s < S ? fp8_tiles(fp8_length(p, s)) : 0;
    }
    int total;
    const int before = warp_scan(mine, lane, &total);
    U = (long long)total * p.num_kv_heads;
    w_active = (int)min((long long)w_total, (U + p.min_tiles - 1) / p.min_tiles);
    if (w >= w_active) {
      if (lane == 0) p.meta[w] = make_int4(0, 0, 0, 0);
      return;
    }
    const long long u01 = (long long)(w + (lane & 1)) * U / w_active;
    u0 = __shfl_sync(0xffffffffu, u01, 0);
    ntiles = (int)(__shfl_sync(0xffffffffu, u01, 1) - u0);
    // the sequence that tile u0 belongs to: first the lane that counted it, then
    // that lane's sequences 32 at a time
    const int t0 = (int)(u0 / p.num_kv_heads);
    const int owner =
        31 - __clz(__ballot_sync(0xffffffffu, before <= t0));   // the last one that begins before
    int base = __shfl_sync(0xffffffffu, before, owner);
    s0 = owner * per;
    L0 = 0;
    for (int k0 = 0; k0 < per; k0 += 32) {
      const int s = owner * per + k0 + lane;
      const int L = k0 + lane < per && s < S ? fp8_length(p, s) : 0;
      int sum;
      const int at = base + warp_scan(fp8_tiles(L), lane, &sum);
      if (base + sum <= t0) {
        base += sum;
        continue;
      }
      const int hit = 31 - __clz(__ballot_sync(0xffffffffu, at <= t0));
      s0 = owner * per + k0 + hit;
      base = __shfl_sync(0xffffffffu, at, hit);
      L0 = __shfl_sync(0xffffffffu, L, hit);
      break;
    }
    nt0 = fp8_tiles(L0);
    const long long r0 = u0 - (long long)base * p.num_kv_heads;
    h0 = (int)(r0 / nt0);
    j0 = (int)(r0 - (long long)h0 * nt0);
  }

  // ---- the walk, and the copies of a tile
  Fp8Walk walk;
  walk.s = s0, walk.L = L0, walk.nt = nt0, walk.h = h0, walk.j = j0;
  walk.described = 0;
  walk.begin(p, ntiles, lane);
  walk.end(p, ring, ring_s, ntiles, lane);
  // the next run, if the ring has room for it: its block ids travel meanwhile
  auto look_ahead = [&](int consumed) {
    if (walk.n == 0 && walk.described < ntiles && walk.described - consumed <= kF8Ring - 32)
      walk.begin(p, ntiles, lane);
  };
  look_ahead(0);

  const uint64_t stream_policy = l2_policy_evict_first();
  // K, scales and, where a segment begins, query rows of tile i
  auto copy_k = [&](int i, const Fp8Tile &t) {
    const int row0 = __shfl_sync(0xffffffffu, t.row0, 0);
    const int row1 = __shfl_sync(0xffffffffu, t.row1, 0);
    const bool first = __shfl_sync(0xffffffffu, t.head_flags, 0) & TF_FIRST;
    float *sc = scales + (i & 1) * kF8ScaleFloats;
    fence_proxy_async_smem();      // this lane's reads of the buffers, before copies into them
    __syncwarp();
    if (elect_one()) {
      mbar_arrive_expect_tx(kbar, ((row0 >= 0) + (row1 >= 0)) * (B * D + 8 * B) +
                                      (first ? (uint32_t)qbytes : 0u));
      if (row0 >= 0) {
        tma_load_2d_hint(kbuf, &kmap, 0, row0, kbar, stream_policy);
        bulk_load(sc, p.kv_scale + (int64_t)row0 * 2, 8 * B, kbar);
      }
      if (row1 >= 0) {
        tma_load_2d_hint(kbuf + B * D, &kmap, 0, row1, kbar, stream_policy);
        bulk_load(sc + 2 * B, p.kv_scale + (int64_t)row1 * 2, 8 * B, kbar);
      }
      if (first) {
        const int64_t row = (int64_t)ring_s[i & (kF8Ring - 1)] * p.num_q_heads +
                            (int64_t)(t.head_flags >> 8) * G;
        bulk_load(qbuf, p.q + row * (D * 2), qbytes, kbar);
      }
    }
  };
  auto copy_v = [&](const Fp8Tile &t) {
    const int row0 = __shfl_sync(0xffffffffu, t.row0, 0);
    const int row1 = __shfl_sync(0xffffffffu, t.row1, 0);
    fence_proxy_async_smem();
    __syncwarp();
    if (elect_one()) {
      mbar_arrive_expect_tx(vbar, ((row0 >= 0) + (row1 >= 0)) * B * D);
      if (row0 >= 0) tma_load_2d_hint(vbuf, &vmap, 0, row0, vbar, stream_policy);
      if (row1 >= 0) tma_load_2d_hint(vbuf + B * D, &vmap, 0, row1, vbar, stream_policy);
    }
  };
  // The description of tile i.
  auto next_tile = [&](int i) {
    const int used = max(i - 1, 0);    // the tile before is still being worked on
    if (i == walk.described) {
      look_ahead(used);
      walk.end(p, ring, ring_s, ntiles, lane);
      look_ahead(used);
    }
    return ring[i & (kF8Ring - 1)];
  };
  Fp8Tile ti = next_tile(0);
  copy_k(0, ti);
  copy_v(ti);

  // ---- for the merge, while the first copies travel: if this range begins
  // inside a segment and no earlier one does, the segment's (sequence, kv
  // head), its first partial and the number of them; the others are the first
  // partials of the ranges behind the first
  if (p.min_tiles > 0) {
    const long long lo = u0 - j0, hi = lo + nt0;
    // the range that holds tile u: the largest c with c U / w_active <= u
    const long long c01 = (((lane & 1) ? hi : lo + 1) * w_active - 1) / U;
    const int c_lo = (int)__shfl_sync(0xffffffffu, c01, 0);
    const int c_hi = (int)__shfl_sync(0xffffffffu, c01, 1);
    const bool starts = (long long)c_lo * U / w_active == lo;   // range c_lo begins with the segment
    const bool merge = j0 > 0 && c_lo == w - 1;
    if (lane == 0)
      p.meta[w] = make_int4(merge ? s0 * p.num_kv_heads + h0 : 0, 2 * c_lo + (starts ? 0 : 1),
                            c_lo, merge ? c_hi - c_lo + 1 : 0);
  }

  // every lane waits; the warp goes on only if all of them saw the phase (lanes
  // whose limits ran out alone would leave the others' shuffles without a source)
  auto wait_all = [&](uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, p.wait_ns));
  };
  Fp8Path<D, NT, HPL> st;
  st.init(lane);
  bool seg_from0 = false;
  int seg_index = 0;
  for (int i = 0; i < ntiles; ++i) {
    const Fp8Tile tn = i + 1 < ntiles ? next_tile(i + 1) : ti;
    const float *sc = scales + (i & 1) * kF8ScaleFloats;
    if (!wait_all(kbar, i & 1)) {
      if (lane == 0) flag_error(PA_DEVERR_TIMEOUT);
      // copies still in flight land before the warp leaves
      mbar_wait_bounded(kbar, i & 1, kDrainLimitNs);
      mbar_wait_bounded(vbar, i & 1, kDrainLimitNs);
      return;
    }
    if (ti.head_flags & TF_FIRST) {
      st.reset();
      st.load_q(qbuf, G, p.q_bf16 != 0, p.scale_log2, lane);
      seg_from0 = (ti.head_flags & TF_J0) != 0;
    }
    if (ti.live) st.scores(kbuf, sc, B, lane);
    if (i + 1 < ntiles) copy_k(i + 1, tn);
    if (!wait_all(vbar, i & 1)) {
      if (lane == 0) flag_error(PA_DEVERR_TIMEOUT);
      mbar_wait_bounded(vbar, i & 1, kDrainLimitNs);
      if (i + 1 < ntiles) mbar_wait_bounded(kbar, (i + 1) & 1, kDrainLimitNs);
      return;
    }
    if (ti.live) st.output(vbuf, sc, B, ti.live, lane);
    if (i + 1 < ntiles) copy_v(tn);
    if (ti.head_flags & TF_LAST) {
      const bool complete = seg_from0 && (ti.head_flags & TF_JEND);
      st.finish(p, ring_s[i & (kF8Ring - 1)], ti.head_flags >> 8, complete,
                2 * w + (seg_index == 0 ? 0 : 1), lane);
      ++seg_index;
    }
    ti = tn;
  }
}

// ============================================================================
// Merge of split segments.  A warp looks at `span` ranges (one per lane) and
// merges the segments that are first cut at one of them, GMW heads at a time:
// with many segments about every range begins inside one.  With few long ones
// (GMW = 1) a segment has many partials: each head goes to a CTA, whose four
// warps share the partials.
// ============================================================================
template <int D, int GMW>
__global__ void __launch_bounds__(128)
    paged_decode_fp8_merge_kernel(const DecodeFp8Params p, int w_total, int span, int groups) {
  constexpr int VPL = D / 32;
  constexpr int UNR = 16 / GMW;   // partials per batch of loads
  using VecT = typename std::conditional<VPL == 4, float4, float2>::type;
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  constexpr bool kShare = GMW == 1;
  __shared__ float joined[kShare ? 4 : 1][D + 2];   // each warp's sums, their maximum and weight
  const int warp = threadIdx.x >> 5;
  const int t = kShare ? blockIdx.x : blockIdx.x * 4 + warp;
  const int G = p.group, g0 = t % groups * GMW, b = t / groups * span + lane;
  const int4 mine = lane < span && b < w_total ? __ldcg(p.meta + b) : make_int4(0, 0, 0, 0);
  unsigned todo = __ballot_sync(0xffffffffu, mine.w > 0);
  while (todo) {
    const int src = __ffs(todo) - 1;
    todo &= todo - 1;
    const int sh = __shfl_sync(0xffffffffu, mine.x, src);
    const int first = __shfl_sync(0xffffffffu, mine.y, src);
    const int c_lo = __shfl_sync(0xffffffffu, mine.z, src);
    const int n = __shfl_sync(0xffffffffu, mine.w, src);
    float M[GMW], den[GMW], num[GMW][VPL];
#pragma unroll
    for (int g = 0; g < GMW; ++g) {
      M[g] = -INFINITY;
      den[g] = 0.f;
#pragma unroll
      for (int v = 0; v < VPL; ++v) num[g][v] = 0.f;
    }
    for (int k0 = kShare ? warp * 32 : 0; k0 < n; k0 += kShare ? 128 : 32) {
      const int k = k0 + lane, cnt = min(n - k0, 32);
      const bool ok = k < n;
      const long long row = (long long)(k == 0 ? first : 2 * (c_lo + k)) * G + g0;
      VecT buf[UNR][GMW];
      auto fetch = [&](int j0) {
#pragma unroll
        for (int u = 0; u < UNR; ++u) {
          const long long rj = __shfl_sync(0xffffffffu, row, min(j0 + u, cnt - 1));
#pragma unroll
          for (int g = 0; g < GMW; ++g)
            buf[u][g] = __ldcg(reinterpret_cast<const VecT *>(
                p.part_o + (rj + min(g, G - 1 - g0)) * D + lane * VPL));
        }
      };
      float2 ml[GMW];
#pragma unroll
      for (int g = 0; g < GMW; ++g)
        ml[g] = ok ? __ldcg(p.part_ml + row + min(g, G - 1 - g0)) : make_float2(-INFINITY, 0.f);
      fetch(0);
      float wk[GMW];
#pragma unroll
      for (int g = 0; g < GMW; ++g) {
        float cm = ml[g].x;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) cm = fmaxf(cm, __shfl_xor_sync(0xffffffffu, cm, x));
        const float Mn = fmaxf(M[g], cm);
        const float so = M[g] == -INFINITY ? 0.f : exp2f(M[g] - Mn);
        wk[g] = ml[g].x == -INFINITY ? 0.f : exp2f(ml[g].x - Mn);
        float dl = wk[g] * ml[g].y;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) dl += __shfl_xor_sync(0xffffffffu, dl, x);
        den[g] = den[g] * so + dl;
#pragma unroll
        for (int v = 0; v < VPL; ++v) num[g][v] *= so;
        M[g] = Mn;
      }
      for (int j0 = 0; j0 < cnt; j0 += UNR) {
        if (j0 > 0) fetch(j0);
#pragma unroll
        for (int u = 0; u < UNR; ++u) {
          if (j0 + u >= cnt) break;
#pragma unroll
          for (int g = 0; g < GMW; ++g) {
            const float wj = __shfl_sync(0xffffffffu, wk[g], j0 + u);
            num[g][0] = fmaf(wj, buf[u][g].x, num[g][0]);
            num[g][1] = fmaf(wj, buf[u][g].y, num[g][1]);
            if constexpr (VPL == 4) {
              num[g][2] = fmaf(wj, buf[u][g].z, num[g][2]);
              num[g][3] = fmaf(wj, buf[u][g].w, num[g][3]);
            }
          }
        }
      }
    }
    if constexpr (kShare) {
#pragma unroll
      for (int v = 0; v < VPL; ++v) joined[warp][lane * VPL + v] = num[0][v];
      if (lane == 0) joined[warp][D] = M[0], joined[warp][D + 1] = den[0];
      __syncthreads();
      float top = -INFINITY;
#pragma unroll
      for (int k = 0; k < 4; ++k) top = fmaxf(top, joined[k][D]);
      den[0] = 0.f;
#pragma unroll
      for (int v = 0; v < VPL; ++v) num[0][v] = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {   // (a warp without partials: a maximum of -inf)
        const float wk = joined[k][D] == -INFINITY ? 0.f : exp2f(joined[k][D] - top);
        den[0] = fmaf(wk, joined[k][D + 1], den[0]);
#pragma unroll
        for (int v = 0; v < VPL; ++v) num[0][v] = fmaf(wk, joined[k][lane * VPL + v], num[0][v]);
      }
      __syncthreads();
      if (warp > 0) continue;
    }
    float *dst = p.out + ((int64_t)sh * G + g0) * D + lane * VPL;
#pragma unroll
    for (int g = 0; g < GMW; ++g) {
      if (g0 + g >= G) break;
      const float inv = den[g] == 0.f ? 0.f : 1.f / den[g];
      if constexpr (VPL == 4)
        *reinterpret_cast<float4 *>(dst + g * D) =
            make_float4(num[g][0] * inv, num[g][1] * inv, num[g][2] * inv, num[g][3] * inv);
      else
        *reinterpret_cast<float2 *>(dst + g * D) = make_float2(num[g][0] * inv, num[g][1] * inv);
    }
  }
}

}  // namespace pa
