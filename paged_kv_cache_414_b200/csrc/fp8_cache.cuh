// The 8-bit cache's own operators and the rotary cache write, for sm_100a.
//
// An 8-bit pool holds e4m3 codes, K and V each [NB, Hkv, B, D] bytes, and one
// fp32 scale per (block, kv head, K or V, token): kv_scale [NB, Hkv, 2, B].
// A cached element is code * scale; a row's scale is max(amax, 2^-100) / 448
// with amax the row's largest magnitude and 448 e4m3's largest value, so a
// row's largest element keeps e4m3's full 4 significant bits whatever the
// row's size, and a row of zeros needs no special case.  (One scale per token
// rather than per block or per pool: writing a token never re-scales another.)
//
// All three kernels move bytes: their bound is HBM, or the launch for small
// calls.
#pragma once

#include <cuda_fp8.h>
#include <stdint.h>

#include "pa_device.cuh"

namespace pa {

constexpr float kE4m3Max = 448.f;
constexpr float kLeastAmax = 7.888609052210118e-31f;   // 2^-100

struct RopeParams {
  void *q_out;                 // [T, Hq, D], row stride q_out_stride elements
  const void *q, *k, *v;       // [T, H, D], row strides below
  void *k_cache, *v_cache;
  float *kv_scale;             // e4m3 pool only
  const int64_t *slots;        // [T]
  const int64_t *positions;    // [axes, T]
  const float *cos_sin;        // [max_position, rotary]: cosines, then sines
  long long q_out_stride, q_stride, k_stride, v_stride;
  long long num_slots;
  int num_tokens, num_q_heads, num_kv_heads, block_size;
  int rotary, axes, max_position;
  int sect[3];                 // frequency pairs before axis 1, 2, 3
  int splits, passes;          // warps to a token, and passes of each
};

// Rotary positions and the cache write.  Frequency pair j of a head's first
// `rotary` columns is turned by the angle of the position its axis gives:
//   a' = a cos - b sin,  b' = b cos + a sin,
// (a, b) = columns (j, j + rotary/2), or (2j, 2j + 1) with PAIRS.  D/16 lanes
// share a head row, 16 columns each, chosen so that lane l owns the pairs
// 8l .. 8l+7 in either order and both its loads and its 16-bit stores are
// 16-byte vectors; a row's amax is a shuffle among its lanes.
//
// A warp takes a token's heads 512 / D at a time -- the query heads, then K's
// and V's -- so that the cosines and sines of its lanes are fetched once per
// token; a pass's rows are loaded two passes ahead, the next token's positions
// and slot a token ahead.  With few tokens `splits` warps share one.
//
// Bound: HBM.  16384 tokens of 32 q and 8 kv heads of 128 (378 MB in and out)
// take 78 us, 4.9 TB/s; with four heads to a thread and no loop they took 119
// (15 warps per SM, all waiting for the same things at the same time).  256
// tokens take 3.5 us, a launch.
template <typename T, int D, bool FP8, bool PAIRS>
__global__ void __launch_bounds__(256, 3) rope_and_cache_kernel(const RopeParams p) {
  constexpr int LPR = D / 16, HPP = 32 / LPR;   // lanes of a head row, heads of a pass
  grid_dependency_wait();
  allow_dependent_launch();
  const int lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR;
  const int nq = p.num_q_heads, nkv = p.num_kv_heads;
  const int pq = (nq + HPP - 1) / HPP, all = pq + (2 * nkv + HPP - 1) / HPP;   // passes of a token
  const int units = p.num_tokens * p.splits, step = gridDim.x * 8;
  int unit = blockIdx.x * 8 + (threadIdx.x >> 5);

  const bool turns = 16 * l < p.rotary;
  const int e0 = PAIRS || !turns ? 16 * l : 8 * l;
  const int e1 = PAIRS || !turns ? 16 * l + 8 : p.rotary / 2 + 8 * l;
  const int j0 = 8 * l;
  auto axis_of = [&](int j) {
    return (j >= p.sect[0] ? 1 : 0) + (j >= p.sect[1] ? 1 : 0) + (j >= p.sect[2] ? 1 : 0);
  };
  const int axis0 = axis_of(j0);
  const bool one_axis = axis0 == axis_of(j0 + 7);
  const bool mixed = __any_sync(0xffffffffu, turns && !one_axis);

  // lane a < axes: the token's position on that axis; lane 4: its slot
  auto fetch = [&](int u) -> long long {
    if (u >= units) return 0;
    const int t = u / p.splits;
    if (lane < p.axes) return p.positions[(long long)lane * p.num_tokens + t];
    return lane == 4 ? p.slots[t] : 0;
  };
  long long next = fetch(unit);
  for (; unit < units; unit += step) {
    const long long now = next;
    next = fetch(unit + step);
    const int t = unit / p.splits, part = unit - t * p.splits;
    const bool bad = lane < p.axes && (now < 0 || now >= p.max_position);
    const long long slot = __shfl_sync(0xffffffffu, now, 4);
    if (__any_sync(0xffffffffu, bad)) {   // the token is skipped altogether
      if (bad && part == 0) flag_error(PA_DEVERR_POSITION);
      continue;
    }
    bool keep = slot >= 0;
    if (slot >= p.num_slots) {
      if (part == 0 && lane == 0) flag_error(PA_DEVERR_SLOT);
      keep = false;
    }
    const long long blk = keep ? slot / p.block_size : 0;
    const int off = keep ? (int)(slot - blk * p.block_size) : 0;
    const int p0 = part * p.passes, p1 = min(p0 + p.passes, all);

    const T *qrow = static_cast<const T *>(p.q) + t * p.q_stride + sub * D;
    const T *krow = static_cast<const T *>(p.k) + t * p.k_stride;
    const T *vrow = static_cast<const T *>(p.v) + t * p.v_stride;
    uint4 x0[2], x1[2];                                     // the next two passes' rows
    auto load = [&](int ps, uint4 (&y)[2]) {
      const T *row = nullptr;
      if (ps < min(pq, p1)) {
        if (ps * HPP + sub < nq) row = qrow + ps * (HPP * D);
      } else if (ps < p1) {
        const int h = (ps - pq) * HPP + sub;
        if (h < 2 * nkv) row = h < nkv ? krow + h * D : vrow + (h - nkv) * D;
      }
      y[0] = row ? *reinterpret_cast<const uint4 *>(row + e0) : make_uint4(0, 0, 0, 0);
      y[1] = row ? *reinterpret_cast<const uint4 *>(row + e1) : make_uint4(0, 0, 0, 0);
    };
    load(p0, x0);
    load(p0 + 1, x1);

    float c[8], s[8];
    const long long pos = __shfl_sync(0xffffffffu, now, axis0);
    if (turns && one_axis) {
      const float *f = p.cos_sin + pos * p.rotary + j0;
#pragma unroll
      for (int m = 0; m < 8; m += 4) {
        const float4 fc = __ldg(reinterpret_cast<const float4 *>(f + m));
        const float4 fs = __ldg(reinterpret_cast<const float4 *>(f + p.rotary / 2 + m));
        c[m] = fc.x, c[m + 1] = fc.y, c[m + 2] = fc.z, c[m + 3] = fc.w;
        s[m] = fs.x, s[m + 1] = fs.y, s[m + 2] = fs.z, s[m + 3] = fs.w;
      }
    }
    if (mixed) {                          // a section ends among some lane's pairs
#pragma unroll
      for (int m = 0; m < 8; ++m) {
        const long long at = __shfl_sync(0xffffffffu, now, axis_of(j0 + m));
        if (turns && !one_axis) {
          const float *f = p.cos_sin + at * p.rotary + j0 + m;
          c[m] = __ldg(f);
          s[m] = __ldg(f + p.rotary / 2);
        }
      }
    }

    // columns e0 .. e0+7, then e1 .. e1+7, turned if `turn`
    auto unpack = [&](const uint4 (&y)[2], bool turn, float (&f)[16]) {
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint32_t g[4] = {y[w].x, y[w].y, y[w].z, y[w].w};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const float2 v2 = Mma<T>::unpack(g[m]);
          f[8 * w + 2 * m] = v2.x;
          f[8 * w + 2 * m + 1] = v2.y;
        }
      }
      if (turn) {
#pragma unroll
        for (int m = 0; m < 8; ++m) {
          const int ia = PAIRS ? 2 * m : m, ib = PAIRS ? 2 * m + 1 : m + 8;
          const float a = f[ia], b = f[ib];
          f[ia] = a * c[m] - b * s[m];
          f[ib] = b * c[m] + a * s[m];
        }
      }
    };
    auto store16 = [&](T *row, const float (&f)[16]) {
#pragma unroll
      for (int w = 0; w < 2; ++w)
        *reinterpret_cast<uint4 *>(row + (w ? e1 : e0)) =
            make_uint4(Mma<T>::pack(f[8 * w], f[8 * w + 1]),
                       Mma<T>::pack(f[8 * w + 2], f[8 * w + 3]),
                       Mma<T>::pack(f[8 * w + 4], f[8 * w + 5]),
                       Mma<T>::pack(f[8 * w + 6], f[8 * w + 7]));
    };
    int ps = p0;
    T *qout = static_cast<T *>(p.q_out) + t * p.q_out_stride + sub * D;
#pragma unroll 1
    for (; ps < min(pq, p1); ++ps) {
      const uint4 y[2] = {x0[0], x0[1]};
      x0[0] = x1[0], x0[1] = x1[1];
      load(ps + 2, x1);
      float f[16];
      unpack(y, turns, f);
      if (ps * HPP + sub < nq) store16(qout + ps * (HPP * D), f);
    }
    // rows of the pool: K or V head h of this token
    const long long tile0 = blk * nkv;
#pragma unroll 1
    for (; ps < p1; ++ps) {
      const uint4 y[2] = {x0[0], x0[1]};
      x0[0] = x1[0], x0[1] = x1[1];
      load(ps + 2, x1);
      const int h = (ps - pq) * HPP + sub;
      const bool is_k = h < nkv;
      const long long tile = tile0 + (is_k ? h : h - nkv);
      const long long row = tile * p.block_size + off;
      const bool put = keep && h < 2 * nkv;
      float f[16];
      unpack(y, turns && is_k, f);
      if constexpr (!FP8) {
        if (put) store16(static_cast<T *>(is_k ? p.k_cache : p.v_cache) + row * D, f);
      } else {
        float amax = 0.f;
#pragma unroll
        for (int m = 0; m < 16; ++m) amax = fmaxf(amax, fabsf(f[m]));
#pragma unroll
        for (int d = 1; d < LPR; d <<= 1)
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
        if (put) {
          const float top = fmaxf(amax, kLeastAmax);
          const float inv = kE4m3Max / top;
          uint32_t w4[4];
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(
                make_float2(f[4 * m] * inv, f[4 * m + 1] * inv), __NV_SATFINITE, __NV_E4M3);
            const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(
                make_float2(f[4 * m + 2] * inv, f[4 * m + 3] * inv), __NV_SATFINITE, __NV_E4M3);
            w4[m] = (uint32_t)lo | ((uint32_t)hi << 16);
          }
          uint8_t *dst = static_cast<uint8_t *>(is_k ? p.k_cache : p.v_cache) + row * D;
          *reinterpret_cast<uint2 *>(dst + e0) = make_uint2(w4[0], w4[1]);
          *reinterpret_cast<uint2 *>(dst + e1) = make_uint2(w4[2], w4[3]);
          if (l == 0) p.kv_scale[(tile * 2 + (is_k ? 0 : 1)) * p.block_size + off] = top / kE4m3Max;
        }
      }
    }
  }
}

// Copy-on-write copies of 8-bit blocks: a pair's K codes, V codes and scales
// are three runs of 16-byte vectors, walked as one; each thread loads all its
// vectors before it stores any (no destination is also a source).  Bound: HBM;
// 2048 pairs of 16 tokens x 8 heads of 128 (138 MB in and out) take 24 us, 5.8
// TB/s, and 37 pairs 2.9 us, a launch.
constexpr int kCopy8Unroll = 8;
__global__ void __launch_bounds__(256)
    copy_blocks_fp8_kernel(uint4 *k_cache, uint4 *v_cache, uint4 *kv_scale,
                           const int64_t *__restrict__ block_mapping, int code_vec, int scale_vec,
                           int chunks, int num_blocks) {
  grid_dependency_wait();
  allow_dependent_launch();
  const long long pair = blockIdx.x / chunks;
  const int chunk = (int)(blockIdx.x - pair * chunks);
  const int64_t src = __ldg(block_mapping + 2 * pair);
  const int64_t dst = __ldg(block_mapping + 2 * pair + 1);
  if (src < 0 || src >= num_blocks || dst < 0 || dst >= num_blocks) {
    if (chunk == 0 && threadIdx.x == 0) flag_error(PA_DEVERR_COPY_PAIR);
    return;
  }
  const int total = 2 * code_vec + scale_vec;
  const int beg = chunk * (256 * kCopy8Unroll) + threadIdx.x;
  auto at = [&](int i, int64_t b) -> uint4 * {
    if (i < code_vec) return k_cache + b * code_vec + i;
    if (i < 2 * code_vec) return v_cache + b * code_vec + (i - code_vec);
    return kv_scale + b * scale_vec + (i - 2 * code_vec);
  };
  uint4 r[kCopy8Unroll];
#pragma unroll
  for (int k = 0; k < kCopy8Unroll; ++k)
    if (beg + k * 256 < total) r[k] = *at(beg + k * 256, src);
#pragma unroll
  for (int k = 0; k < kCopy8Unroll; ++k)
    if (beg + k * 256 < total) *at(beg + k * 256, dst) = r[k];
}

struct GatherParams {
  void *key, *value;            // [T, Hkv, D]
  const uint8_t *k_cache, *v_cache;
  const float *kv_scale;
  const int32_t *block_tables;  // [S, max_blocks]
  const int32_t *key_start;     // [S + 1]
  int num_seqs, num_tokens, num_kv_heads, block_size, max_blocks, num_blocks;
};

// Cached rows out of the 8-bit pool, packed and in 16 bits (each code * scale
// is rounded once, to nearest).  A CTA takes kGatherRows output rows: its
// first row's sequence is the number of sequences that end at or before it,
// counted by all threads at once (one load deep, no search), the others
// follow from it; then K and V of every head, in an order that reads a
// block's tokens of one head one after the other.  gridDim.y splits the
// heads.  Rows before the first sequence and behind the last are left as they are.
// Bound: HBM; 247 MB in and out take 48 us, 5.1 TB/s (more rows to a CTA, deeper
// or shallower loads: the same or slower), 300 tokens 3.0 us, a launch.
constexpr int kGatherRows = 16;
template <typename T, int D>
__global__ void __launch_bounds__(256) gather_cache_fp8_kernel(const GatherParams p) {
  constexpr int LPR = D / 16;   // lanes of a row, 16 codes each
  constexpr int UNR = 4;
  __shared__ long long cell[kGatherRows];   // (block * Hkv * B + offset), or -1
  grid_dependency_wait();
  allow_dependent_launch();
  const int r0 = blockIdx.x * kGatherRows;
  int s0 = 0;
  for (int i0 = 0; i0 < p.num_seqs; i0 += 256) {
    const int i = i0 + threadIdx.x;
    s0 += __syncthreads_count(i < p.num_seqs && __ldg(p.key_start + i + 1) <= r0);
  }
  if (threadIdx.x < kGatherRows) {
    const int r = r0 + threadIdx.x;
    int s = s0;
    while (s < p.num_seqs && __ldg(p.key_start + s + 1) <= r) ++s;
    long long c = -1;
    if (r < p.num_tokens && s < p.num_seqs) {
      const long long pos = (long long)r - __ldg(p.key_start + s);
      if (pos >= (long long)p.max_blocks * p.block_size) {
        flag_error(PA_DEVERR_CONTEXT_LEN);
      } else if (pos >= 0) {   // (rows before the first sequence are no one's)
        const int blk = __ldg(p.block_tables + (long long)s * p.max_blocks + pos / p.block_size);
        if (blk < 0 || blk >= p.num_blocks)
          flag_error(PA_DEVERR_BLOCK_ID);
        else
          c = (long long)blk * p.num_kv_heads * p.block_size + pos % p.block_size;
      }
    }
    cell[threadIdx.x] = c;
  }
  __syncthreads();
  const int B = p.block_size;
  const int rows = 2 * p.num_kv_heads * kGatherRows;        // K rows of every head, then V rows
  const int step = gridDim.y * (256 / LPR);
  const int l = threadIdx.x % LPR;
  for (int base = blockIdx.y * (256 / LPR) + threadIdx.x / LPR; base < rows; base += UNR * step) {
    uint4 w[UNR];
    float sc[UNR];
#pragma unroll
    for (int k = 0; k < UNR; ++k) {
      const int i = base + k * step;
      const int row = i % kGatherRows, hv = i / kGatherRows;   // hv: (K or V, head)
      const long long c = i < rows ? cell[row] : -1;
      if (c >= 0) {
        const int isv = hv >= p.num_kv_heads, h = isv ? hv - p.num_kv_heads : hv;
        const long long tok = c + (long long)h * B;            // row of the code pool
        w[k] = __ldg(reinterpret_cast<const uint4 *>((isv ? p.v_cache : p.k_cache) + tok * D) + l);
        // scale [blk, h, isv, off]: tile = (tok / B), off = tok % B
        const long long tile = tok / B;
        sc[k] = __ldg(p.kv_scale + (tile * 2 + isv) * B + (tok - tile * B));
      }
    }
#pragma unroll
    for (int k = 0; k < UNR; ++k) {
      const int i = base + k * step;
      const int row = i % kGatherRows, hv = i / kGatherRows;
      if (i >= rows || cell[row] < 0) continue;
      const int isv = hv >= p.num_kv_heads, h = isv ? hv - p.num_kv_heads : hv;
      const uint32_t g[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
      uint32_t y[8];
#pragma unroll
      for (int m = 0; m < 8; ++m) {
        const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(
            (__nv_fp8x2_storage_t)(g[m >> 1] >> (16 * (m & 1))), __NV_E4M3);
        const float2 f = __half22float2(__half2(hr));
        y[m] = Mma<T>::pack(f.x * sc[k], f.y * sc[k]);
      }
      T *dst = static_cast<T *>(isv ? p.value : p.key) +
               ((long long)(r0 + row) * p.num_kv_heads + h) * D + 16 * l;
      reinterpret_cast<uint4 *>(dst)[0] = make_uint4(y[0], y[1], y[2], y[3]);
      reinterpret_cast<uint4 *>(dst)[1] = make_uint4(y[4], y[5], y[6], y[7]);
    }
  }
}

}  // namespace pa
