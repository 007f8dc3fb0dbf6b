// Causal attention over packed prompts, on the fifth-generation tensor cores
// (tcgen05, accumulators in tensor memory).  K and V come straight from the
// projections, packed like the queries; no pool and no block tables.
//
// Sequence s has C queries (rows query_start[s] ..) and L keys (rows
// key_start[s] ..); query i stands at position p = L - C + i and
//   out = softmax_{t <= p}(scale <q, k_t>) v,   zeros where p < 0.
//
// Work unit: (sequence, pair of query tiles, kv head, piece of the keys).  A
// query tile is 128 rows = tq = 128 / G tokens x the G heads of one kv head;
// tiles A and B (2 tq consecutive tokens) share every K/V tile of 128 keys.
// Units are numbered longest first over all sequences -- found in the kernel by
// a search over the lengths that goes on from a CTA's last unit -- and CTAs, one
// per SM, take them in that order: the first by blockIdx, the next by cancelling
// CTAs that have not been launched yet (clusterlaunchcontrol), so that loads, the
// tensor-memory allocation and the barriers of one unit run on into the next.
//
//   warps 0-3   softmax and output of tile A, one thread per row
//   warps 4-7   the same for tile B
//   warp 8      TMA producer
//   warp 9      MMA issue: per K/V tile j, O_A += P_A V_j, S_A(j+1) = Q_A K^T,
//               then the same for B, so one tile's softmax runs under the
//               other's MMAs
//   warp 10     scheduler: finds the next unit one unit ahead
//   warp 11     zeroes V rows behind the last visible key (they may hold
//               another sequence's NaN, and 0 x NaN would reach every row)
//
// P replaces S in tensor memory, in the inputs' 16-bit type: rounding the
// weights (at most 2^-8 or 2^-11 each, independent) costs about as much as rounding
// the output does.  Maximum, sum and O are fp32.  O is rescaled only when a
// row's maximum grows by more than 2^8 (weights then stay below 2^8).
//
// Bound: the chain of a tile's softmax between its two products, at half of the
// tensor cores' rate (the exponentials' unit is busy for as long).  One prompt
// of 8192 tokens, 32 / 8 heads of 128: 459 us, 1.2 PFLOP/s of visible pairs;
// 16 prompts of 64 to 2048 tokens, 40 heads: 209 us, 0.69 (their units have few
// tiles, and the diagonal ones count half); 256 prompts of 70 tokens, 32 / 8
// heads of 128: 124 us, 4000 of them 1.91 ms (the units' fixed costs).  Measured
// and left: a polynomial on the FMA units for a quarter of the exponentials (498
// us), scores in halves of 64 keys with two in flight (590), two threads to a row
// (783), the next unit's first scores before this one's last P.V (465), heads in
// groups whose K/V fit the L2 cache (as before or slower), masks as selects in
// registers instead of a pass over the tile (457, with spills).
#pragma once

#include <limits.h>

#include "prefill_attention.cuh"
#include "prompt_umma.cuh"

namespace pa {

struct PromptParams {
  void *out;                   // [T, Hq, D]
  const int32_t *query_start;  // [S + 1]
  const int32_t *key_start;    // [S + 1]
  float *part_o;               // [units][pieces][256][D], keys split only
  float2 *part_ml;             // [units][pieces][256]  (max in log2 units, sum)
  int4 *part_of;               // [units]  first token, tokens, parts of tiles A and B (tokens
                               // negative: of one query tile, see PromptUnit::alternate)
  float scale_log2;            // scale * log2(e)
  int num_seqs, num_tokens, num_key_tokens, num_q_heads, num_kv_heads, group;
  int tq;                      // tokens per query tile
  int max_query, max_key;
  int pieces;                  // pieces of the keys in the grid
  int piece_tiles;             // K/V tiles per piece
  long long wait_cycles;       // limit of a wait before giving up
  uint32_t wait_hint;          // and of one try, in ns
};

constexpr int kPrRows = 128;
constexpr int kPrKeys = 128;
constexpr int kPrThreads = 384;
constexpr int kPrSeqCache = 256;   // sequences whose (first key, units) a CTA keeps
constexpr int kPrConsumers = 11;   // warps that read a unit's description

// A unit as the scheduler describes it.
struct PromptUnit {
  int n[2];        // K/V tiles of query tiles A and B in this piece; n[0] < 0: no more units
  int tiles;       // K/V tiles in all
  int alternate;   // there is only tile A, and B stands for it too: A takes the even K/V tiles,
                   // B the odd ones, each with a partial of its own
  int first_key;   // global row of the piece's first key
  int token0;      // global row of tile A's first token
  int tokens;      // of tiles A and B
  int pos0;        // position of tile A's first token, less that of the piece's first key
  int kv_head;
  int slot;        // index of its partials
};

template <int D>
struct PromptSmem {
  static constexpr int NCH = D / 64;
  static constexpr int STAGES = D == 128 ? 2 : 4;
  static constexpr int REGION = kPrRows * 128;
  static constexpr int Q_TILE = NCH * REGION;
  static constexpr int KV_BYTES = NCH * kPrKeys * 128;
  static constexpr int OFF_K = 2 * Q_TILE;
  static constexpr int OFF_V = OFF_K + STAGES * KV_BYTES;
  static constexpr int BYTES = OFF_V + STAGES * KV_BYTES + 1024;   // the slack aligns the base
};

// Bounded wait that also gives up when another role has: a dozen instructions,
// so that the kernel's loops stay within the instruction caches.  (With pf_wait
// at every wait the kernel had 111 KB of code.)  The limit is in SM clock
// cycles, two to a nanosecond; it is also the hint for how long one try may
// sleep.  Who gives up sets `abort`, which the kernel reports at its end.
__device__ __forceinline__ bool prompt_wait(uint64_t *bar, uint32_t parity, volatile int *abort,
                                            long long limit_cycles, uint32_t hint_ns) {
  if (mbar_test_wait(bar, parity)) return true;
  const long long c0 = clock64();
  uint32_t ok;
  do {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity), "r"(hint_ns)
        : "memory");
    if (ok) return true;
  } while (!*abort && clock64() - c0 <= limit_cycles);
  *abort = 1;
  return false;
}

// ---------------------------------------------------------------- units

// A sequence: its first query and key rows and how many; no queries if it is not
// one that can be computed.
struct PromptSeq {
  int q0, C, k0, L;
};
__device__ __forceinline__ PromptSeq prompt_seq(const PromptParams &p, int s, bool report) {
  const int q0 = __ldg(p.query_start + s), q1 = __ldg(p.query_start + s + 1);
  const int k0 = __ldg(p.key_start + s), k1 = __ldg(p.key_start + s + 1);
  if (q0 < 0 || q1 < q0 || q1 > p.num_tokens || k0 < 0 || k1 < k0 || k1 > p.num_key_tokens ||
      q1 - q0 > p.max_query || k1 - k0 > p.max_key) {
    if (report) flag_error(PA_DEVERR_CONTEXT_LEN);
    return PromptSeq{0, 0, 0, 0};
  }
  return PromptSeq{q0, q1 - q0, k0, k1 - k0};
}

// What the numbering needs of it: units are its pairs of query tiles (y of
// them), pair i has order x + i, which grows with the keys it sees.
__device__ __forceinline__ int2 prompt_order(const PromptParams &p, const PromptSeq &q) {
  const int w = 2 * p.tq;
  return make_int2(max(0, q.L - q.C) / w, (q.C + w - 1) / w);
}

// Where the last search ended: the units of order `level` begin with number
// `above`, and `seen` of them are of sequences before i0.  A CTA's unit numbers
// grow, so the next search goes on from there: with every search from the
// start, the cost of a call grew with the square of the number of sequences
// (4000 prompts of 70 tokens took 43 ms).  All sequences are still gone over
// where a CTA passes from one order to the next.
struct PromptCursor {
  int level = -1, above = 0, i0 = 0, seen = 0;
  int total = INT_MAX;   // units in all, once a search has gone past the last one
};

// Unit number v in order of decreasing length (ties by sequence): its pair and
// sequence, or false past the last one.  A whole warp; lane i holds sequence i
// and its order, the further ones' orders are in `cache` as far as that goes.
__device__ __forceinline__ bool prompt_find(const PromptParams &p, const int2 *cache,
                                            const PromptSeq &mine, int2 order, int v,
                                            PromptCursor &at, PromptSeq *found, int *pair) {
  const int lane = threadIdx.x & 31;
  if (v >= at.total) return false;
  auto further = [&](int i) {
    return i < kPrSeqCache ? cache[i] : prompt_order(p, prompt_seq(p, i, false));
  };
  auto at_least = [&](int e) {   // units of order e or more
    int n = min(max(order.x + order.y - e, 0), order.y);
#pragma unroll 1
    for (int i = lane + 32; i < p.num_seqs; i += 32) {
      const int2 q = further(i);
      n += min(max(q.x + q.y - e, 0), q.y);
    }
    return __reduce_add_sync(0xffffffffu, n);
  };
  // at_least(lo) > v >= at_least(hi) = above, once lo is known not to be -1
  int hi = (p.max_query + p.max_key) / (2 * p.tq) + 2, above = 0;
  if (p.num_seqs <= 32) hi = __reduce_max_sync(0xffffffffu, order.x + order.y);
  bool known = at.level >= 0 && v >= at.above + at.seen, next = false;
#pragma unroll 1
  while (true) {
    if (!known) {
      int lo = -1;
#pragma unroll 1
      while (hi - lo > 1) {
        const int mid = next ? hi - 1 : (lo + hi) >> 1, n = at_least(mid);
        next = false;
        if (n > v) {
          lo = mid;
        } else {
          hi = mid;
          above = n;
        }
      }
      if (lo < 0) {
        at.total = above;
        return false;
      }
      at.level = lo, at.above = above, at.i0 = 0, at.seen = 0;
    }
    const int lo = at.level;
    int left = v - at.above - at.seen;
#pragma unroll 1
    for (; at.i0 < p.num_seqs; at.i0 += 32) {
      const int i0 = at.i0, i = i0 + lane;
      const int2 q = i0 == 0 ? order : (i < p.num_seqs ? further(i) : make_int2(0, 0));
      const bool has = q.x <= lo && lo < q.x + q.y;
      const unsigned who = __ballot_sync(0xffffffffu, has);
      const int many = __popc(who);
      if (left < many) {
        const unsigned which = __ballot_sync(
            0xffffffffu, has && __popc(who & ((1u << lane) - 1u)) == left);
        const int src = __ffs(which) - 1;
        *pair = lo - __shfl_sync(0xffffffffu, q.x, src);
        if (i0 == 0) {
          found->q0 = __shfl_sync(0xffffffffu, mine.q0, src);
          found->C = __shfl_sync(0xffffffffu, mine.C, src);
          found->k0 = __shfl_sync(0xffffffffu, mine.k0, src);
          found->L = __shfl_sync(0xffffffffu, mine.L, src);
        } else {
          *found = prompt_seq(p, i0 + src, false);
        }
        return true;
      }
      left -= many;
      at.seen += many;
    }
    // the order is through: v is in one below, mostly the next
    hi = lo, above = at.above + at.seen;
    known = false, next = true;
  }
}

// Tiles of 128 keys that the tokens up to position `last` see.
__device__ __forceinline__ int prompt_tiles(int last) { return last < 0 ? 0 : last / kPrKeys + 1; }

// Tokens and positions of a pair of query tiles.
struct PromptPair {
  int token0, tokens, pos0, key0;
  int tiles[2];   // of A and B over the whole length
};
__device__ __forceinline__ PromptPair prompt_pair(const PromptParams &p, const PromptSeq &q,
                                                  int pair) {
  PromptPair u;
  const int t0 = pair * 2 * p.tq;
  u.token0 = q.q0 + t0;
  u.tokens = min(2 * p.tq, q.C - t0);
  u.pos0 = q.L - q.C + t0;
  u.key0 = q.k0;
  u.tiles[0] = prompt_tiles(u.pos0 + min(p.tq, u.tokens) - 1);
  u.tiles[1] = u.tokens > p.tq ? prompt_tiles(u.pos0 + u.tokens - 1) : 0;
  return u;
}

// ---------------------------------------------------------------- launch control

// Ask for a CTA that has not been launched yet; the answer (16 bytes) lands in
// `dst` and completes them on `bar`.
__device__ __forceinline__ void try_cancel(void *dst, uint64_t *bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], "
      "[%1];" ::"r"(smem_addr(dst)),
      "r"(smem_addr(bar))
      : "memory");
}
// blockIdx.x of the CTA that was cancelled in this one's favour, or -1.
__device__ __forceinline__ int cancelled_block(const void *answer) {
  uint32_t ok, x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 h;\n\t"
      "ld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
      : "=r"(ok), "=r"(x)
      : "r"(smem_addr(answer))
      : "memory");
  return ok ? (int)x : -1;
}

// 32 bytes in one store (32-byte aligned).
__device__ __forceinline__ void st_global_v8(void *dst, const uint32_t *v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                   reinterpret_cast<uint64_t>(dst)),
               "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// max(a, b, c), NaN if any is.
__device__ __forceinline__ float fmax3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// ---------------------------------------------------------------- the kernel

template <typename T, int D>
__global__ void __launch_bounds__(kPrThreads, 1)
    prompt_attention_kernel(const __grid_constant__ CUtensorMap qmap,
                            const __grid_constant__ CUtensorMap kmap,
                            const __grid_constant__ CUtensorMap vmap, const PromptParams p) {
  using L = PromptSmem<D>;
  constexpr int NCH = L::NCH, NST = L::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t *sQ = smem, *sK = smem + L::OFF_K, *sV = smem + L::OFF_V;

  __shared__ uint64_t full_k[NST], full_v[NST], empty_k[NST], empty_v[NST];
  __shared__ uint64_t q_full, q_empty;      // both query tiles: landed, read by their last S
  __shared__ uint64_t s_full[2], p_half[2], p_full[2], o_done[2];
  __shared__ uint64_t v_tail, v_clean;      // the last V tile: landed; its tail is zeros
  __shared__ uint64_t unit_full[2], unit_empty[2];
  __shared__ uint64_t answer_bar, drain;
  __shared__ __align__(16) uint4 answer;
  __shared__ PromptUnit units[2];
  __shared__ int2 seqs[kPrSeqCache];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  volatile int *abort = &abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.group;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&full_k[i], 1);
      mbar_init(&full_v[i], 1);
      mbar_init(&empty_k[i], 1);
      mbar_init(&empty_v[i], 1);
    }
    mbar_init(&q_full, 1);
    mbar_init(&q_empty, 1);
    mbar_init(&v_tail, 1);
    mbar_init(&v_clean, 32);
    mbar_init(&answer_bar, 1);
    mbar_init(&drain, 1);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&s_full[x], 1);
      mbar_init(&p_half[x], 4);
      mbar_init(&p_full[x], 4);
      mbar_init(&o_done[x], 1);
      mbar_init(&unit_full[x], 1);
      mbar_init(&unit_empty[x], kPrConsumers);
    }
    abort_flag = 0;
    fence_barrier_init();
  }
  if (threadIdx.x == 32) {
    prefetch_tensormap(&qmap);
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
  }
  if (warp == 9) {
    tmem_alloc(&tmem_slot, kPfTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  grid_dependency_wait();
  allow_dependent_launch();

  // every lane waits; the warp goes on only if all of them saw the phase
  auto wait_all = [&](uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, prompt_wait(bar, parity, abort, p.wait_cycles, p.wait_hint));
  };
  // the next unit, by its number in this CTA
  int taken = 0;
  auto next_unit = [&](PromptUnit &u) {
    const int b = taken & 1;
    if (!wait_all(&unit_full[b], (taken >> 1) & 1)) return false;
    u = units[b];
    __syncwarp();
    if (lane == 0) mbar_arrive(&unit_empty[b]);
    ++taken;
    return u.n[0] >= 0;
  };

  // The softmax keeps a row's 128 scores in registers: 208 each for its 256
  // threads, 80 for the others, of the 384 x 168 that the block starts with.
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == 10) {
      // ------------------------------------------------------------ scheduler
      const PromptSeq mine =
          lane < p.num_seqs ? prompt_seq(p, lane, blockIdx.x == 0) : PromptSeq{0, 0, 0, 0};
      const int2 order = prompt_order(p, mine);
#pragma unroll 1
      for (int i = lane + 32; i < p.num_seqs; i += 32) {
        if (i >= kPrSeqCache && blockIdx.x != 0) break;   // (one CTA reports)
        const int2 q = prompt_order(p, prompt_seq(p, i, blockIdx.x == 0));
        if (i < kPrSeqCache) seqs[i] = q;
      }
      __syncwarp();
      int block = blockIdx.x, made = 0, asked = 0;
      PromptCursor cursor;
      while (true) {
        PromptUnit u;
        u.n[0] = -1;
        bool give = block < 0;
        if (block >= 0) {
          const int piece = block % p.pieces, rest = block / p.pieces;
          const int kh = rest % p.num_kv_heads, v = rest / p.num_kv_heads;
          PromptSeq q;
          int pair;
          if (prompt_find(p, seqs, mine, order, v, cursor, &q, &pair)) {
            const PromptPair w = prompt_pair(p, q, pair);
            const int j0 = piece * p.piece_tiles;
            u.n[0] = min(max(w.tiles[0] - j0, 0), p.piece_tiles);
            u.n[1] = min(max(w.tiles[1] - j0, 0), p.piece_tiles);
            u.tiles = max(u.n[0], u.n[1]);
            u.alternate = p.pieces > 1 && w.tokens <= p.tq;
            if (u.alternate) {
              u.n[1] = u.n[0] / 2;
              u.n[0] -= u.n[1];
            }
            u.first_key = w.key0 + j0 * kPrKeys;
            u.token0 = w.token0;
            u.tokens = w.tokens;
            u.pos0 = w.pos0 - j0 * kPrKeys;
            u.kv_head = kh;
            u.slot = block;
            give = u.tiles > 0 || p.pieces == 1;   // no keys: rows of zeros
            if (p.pieces > 1 && piece == 0 && lane == 0) {
              // what the join needs: parts with keys (of the last one's two, B's
              // has none if it is one tile long)
              const int parts[2] = {(w.tiles[0] + p.piece_tiles - 1) / p.piece_tiles,
                                    (w.tiles[1] + p.piece_tiles - 1) / p.piece_tiles};
              p.part_of[rest] =
                  u.alternate ? make_int4(w.token0, -w.tokens, parts[0],
                                          parts[0] - (w.tiles[0] % p.piece_tiles == 1))
                              : make_int4(w.token0, w.tokens, parts[0], parts[1]);
            }
          } else if (p.pieces > 1 && piece == 0 && lane == 0) {
            p.part_of[rest] = make_int4(0, 0, 0, 0);
          }
        }
        if (give) {
          const int b = made & 1;
          if (made >= 2 && !wait_all(&unit_empty[b], ((made >> 1) - 1) & 1)) break;
          if (lane == 0) {
            units[b] = u;
            mbar_arrive(&unit_full[b]);
          }
          ++made;
        }
        if (block < 0 || *abort) break;
        if (lane == 0) {
          fence_proxy_async_smem();   // the last answer was read before the next is written
          mbar_arrive_expect_tx(&answer_bar, 16);
          try_cancel(&answer, &answer_bar);
        }
        __syncwarp();
        if (!wait_all(&answer_bar, asked & 1)) {
          // it lands before the CTA exits
          mbar_wait_bounded(&answer_bar, asked & 1, kPfDrainLimitNs);
          break;
        }
        ++asked;
        block = cancelled_block(&answer);
        __syncwarp();
      }
    } else if (warp == 8) {
      // ------------------------------------------------------------ producer
      PromptUnit u;
      int it = 0, loads = 0, vloads = 0, nq = 0;   // K/V tiles, units with a Q
      bool ok = true;
      while (ok && next_unit(u)) {
        for (int j = 0; ok && j < u.tiles; ++j, ++it) {
          const int st = it % NST;
          const uint32_t free_phase = (it / NST - 1) & 1;
          if (it >= NST && !(ok = wait_all(&empty_k[st], free_phase))) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(&full_k[st], L::KV_BYTES);
            for (int c = 0; c < NCH; ++c)
              tma_load_3d(sK + st * L::KV_BYTES + c * kPrKeys * 128, &kmap, c * 64, u.kv_head,
                          u.first_key + j * kPrKeys, &full_k[st]);
          }
          loads = it + 1;
          if (j == 0) {
            if (nq > 0 && !(ok = wait_all(&q_empty, (nq - 1) & 1))) break;
            const bool two = u.tokens > p.tq;
            if (lane == 0) {
              mbar_arrive_expect_tx(&q_full, (two ? 2 : 1) * NCH * 128 * p.tq * G);
              for (int c = 0; c < NCH; ++c) {
                tma_load_3d(sQ + c * L::REGION, &qmap, c * 64, u.kv_head * G, u.token0, &q_full);
                if (two)
                  tma_load_3d(sQ + L::Q_TILE + c * L::REGION, &qmap, c * 64, u.kv_head * G,
                              u.token0 + p.tq, &q_full);
              }
            }
            ++nq;
          }
          if (it >= NST && !(ok = wait_all(&empty_v[st], free_phase))) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(&full_v[st], L::KV_BYTES);
            for (int c = 0; c < NCH; ++c)
              tma_load_3d(sV + st * L::KV_BYTES + c * kPrKeys * 128, &vmap, c * 64, u.kv_head,
                          u.first_key + j * kPrKeys, &full_v[st]);
          }
          vloads = it + 1;
        }
      }
      // copies still in flight must land before the CTA exits
      if (lane == 0) {
        for (int j = max(0, loads - NST); j < loads; ++j)
          mbar_wait_bounded(&full_k[j % NST], (j / NST) & 1, kPfDrainLimitNs);
        for (int j = max(0, vloads - NST); j < vloads; ++j)
          mbar_wait_bounded(&full_v[j % NST], (j / NST) & 1, kPfDrainLimitNs);
        if (nq > 0) mbar_wait_bounded(&q_full, (nq - 1) & 1, kPfDrainLimitNs);
      }
    } else if (warp == 9) {
      // ------------------------------------------------------------ MMA issue
      constexpr bool kBf = std::is_same<T, __nv_bfloat16>::value;
      const uint32_t idS = umma_idesc_f16(kBf, kPrRows, kPrKeys, false, false);
      const uint32_t idO = umma_idesc_f16(kBf, kPrRows, D, false, true);
      const uint64_t dQ0 = umma_desc_sw128(smem_addr(sQ), 16, 1024);
      const uint64_t dK0 = umma_desc_sw128(smem_addr(sK), 16, 1024);
      const uint64_t dV0 = umma_desc_sw128(smem_addr(sV), kPrKeys * 128, 1024);
      constexpr uint32_t kStageStep = L::KV_BYTES >> 4, kQStep = L::Q_TILE >> 4;
      bool alternate = false;
      auto issue_s = [&](int x, int st) {       // S_x = Q_x K^T
        const uint64_t dq = dQ0 + (alternate ? 0 : x) * kQStep, dk = dK0 + st * kStageStep;
        const uint32_t d = tmem + x * 256;
        constexpr uint32_t kRegion = L::REGION >> 4;
        if constexpr (D == 128)
          umma_ss_group8<0, 2, 4, 6, kRegion, kRegion + 2, kRegion + 4, kRegion + 6>(d, dq, dk, idS,
                                                                                      0u);
        else
          umma_ss_group4<0, 2, 4, 6>(d, dq, dk, idS, 0u);
        umma_commit(&s_full[x]);
      };
      // O_x (+)= P_x V, the first or last 64 keys of the tile
      auto issue_pv0 = [&](int x, int st, bool first) {
        const uint32_t pj = tmem + x * 256;
        umma_ts_group4<0, 8, 16, 24, 0, 128, 256, 384>(pj + 128, pj, dV0 + st * kStageStep, idO,
                                                       first ? 0u : 1u);
      };
      auto issue_pv1 = [&](int x, int st) {
        const uint32_t pj = tmem + x * 256;
        umma_ts_group4<32, 40, 48, 56, 512, 640, 768, 896>(pj + 128, pj, dV0 + st * kStageStep, idO,
                                                           1u);
      };
      PromptUnit u;
      unsigned it = 0, p_phase = 0;             // p_phase bit x: parity of the P awaited from tile x
      int nq = 0, nclean = 0;
      bool ok = true;
      // O_x += P_x V of one tile, as its two halves come
      auto add_pv = [&](int x, int st, bool first) {
        const uint32_t parity = (p_phase >> x) & 1;
        p_phase ^= 1u << x;
        if (!wait_all(&p_half[x], parity)) return false;
        tc_fence_after();
        issue_pv0(x, st, first);
        if (!wait_all(&p_full[x], parity)) return false;
        tc_fence_after();
        issue_pv1(x, st);
        return true;
      };
      while (ok && next_unit(u)) {
        const int nm = u.tiles;
        if (nm == 0) continue;
        const bool tail = u.pos0 + u.tokens < nm * kPrKeys;   // keys behind the last position
        alternate = u.alternate;
        ok = wait_all(&q_full, nq & 1);
        ++nq;
        // step j: P.V of K/V tile j and the scores that then have room -- tile
        // j + 1's of both query tiles, or tile j + 2's of the one whose turn it is
        const int ahead = alternate ? 2 : 1;
#pragma unroll 1
        for (int j = -ahead; ok && j < nm; ++j) {
          const unsigned tv = it + j, tk = tv + ahead;
          const int st = tv % NST, sn = tk % NST;
          const bool more = j + ahead < nm;
          if (j >= 0) {
            ok = wait_all(&full_v[st], (tv / NST) & 1);
            if (ok && tail && j + 1 == nm) {
              if (lane == 0) mbar_arrive(&v_tail);
              ok = wait_all(&v_clean, nclean++ & 1);
            }
          }
          if (ok && more) ok = wait_all(&full_k[sn], (tk / NST) & 1);
#pragma unroll 1
          for (int x = 0; ok && x < 2; ++x) {
            if (alternate ? x != (j & 1) : j >= (x ? u.n[1] : u.n[0])) continue;
            if (j >= 0) {
              ok = add_pv(x, st, j < ahead);
              if (!ok) break;
            }
            tc_fence_after();
            if (alternate ? more : j + 1 < (x ? u.n[1] : u.n[0])) issue_s(x, sn);
            else if (j >= 0) umma_commit(&o_done[x]);
          }
          if (!ok) break;
          if (j >= 0) umma_commit(&empty_v[st]);
          if (more) umma_commit(&empty_k[sn]);
          if (j + ahead + 1 == nm) umma_commit(&q_empty);
        }
        it += nm;
      }
      umma_commit(&drain);
      mbar_wait_bounded(&drain, 0, kPfDrainLimitNs);
    } else {
      // ------------------------------------------------------------ V tail
      // (asked by the MMA warp, which reaches the tile in order: a wait on the
      // tile's own barrier alone could meet an earlier phase of it)
      PromptUnit u;
      int it = 0, asked = 0;
      while (next_unit(u)) {
        const int nm = u.tiles;
        it += nm;
        // rows of the last tile that count
        const int live = u.pos0 + u.tokens - (nm - 1) * kPrKeys;
        if (nm == 0 || live >= kPrKeys) continue;
        const int st = (it - 1) % NST;
        if (!wait_all(&v_tail, asked++ & 1) || !wait_all(&full_v[st], ((it - 1) / NST) & 1)) break;
        uint8_t *v0 = sV + st * L::KV_BYTES;
        for (int i = live * 8 + lane; i < kPrKeys * 8; i += 32)
#pragma unroll
          for (int c = 0; c < NCH; ++c)
            *reinterpret_cast<uint4 *>(v0 + c * kPrKeys * 128 + i * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();   // read next by the tensor cores (async proxy)
        mbar_arrive(&v_clean);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax + output
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int x = warp >> 2;                 // query tile
    const int r = threadIdx.x & 127;         // this thread's row, and lane of tensor memory
    const int t = r / G, t_lo = (r - lane) / G;
    const uint32_t tS = tmem + x * 256 + ((uint32_t)((warp & 3) * 32) << 16), tO = tS + 128;
    const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
    const bool pos_scale = p.scale_log2 > 0.f;
    const float sl2 = pos_scale ? p.scale_log2 : 1.f;   // else the scores are scaled first
    PromptUnit u;
    int ns = 0, no = 0;
    bool ok = true;
    while (ok && next_unit(u)) {
      const int n = x ? u.n[1] : u.n[0];
      const int tx = u.alternate ? 0 : x * p.tq;               // the query tile's first token
      const bool row_ok = t < p.tq && tx + t < u.tokens;
      const int pos = row_ok ? u.pos0 + tx + t : u.pos0 + u.tokens - 1;
      const int pos_lo = u.pos0 + tx + t_lo;                   // of this warp's first row
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j, ++ns) {
        ok = wait_all(&s_full[x], ns & 1);
        if (!ok) break;
        tc_fence_after();
        // keys past a row's position, and a scale that is not positive: the
        // scores are first rewritten where they lie
        const int first = (u.alternate ? 2 * j + x : j) * kPrKeys;   // the tile's first key
        const int lim = pos - first;                           // keys 0 .. lim of the tile count
        // of its four runs of 32 keys, every row of this warp sees those before `whole`
        const int whole = max((pos_lo - first + 1) >> 5, 0);
        if (whole < 4 || !pos_scale) {
#pragma unroll 1
          for (int c = pos_scale ? whole : 0; c < 4; ++c) {
            uint32_t w[32];
            tmem_load32(tS + c * 32, w);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float z = __uint_as_float(w[i]) * (pos_scale ? 1.f : p.scale_log2);
              w[i] = c * 32 + i <= lim ? __float_as_uint(z) : 0xff800000u;   // -inf
            }
            tmem_store32_async(tS + c * 32, w);
          }
          tmem_store_wait();
        }
        uint32_t v[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_load32_async(tS + c * 32, v + c * 32);
        tmem_load_wait();
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_loaded(v + c * 32);
        float mx[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) mx[i] = __uint_as_float(v[i]);
#pragma unroll
        for (int i = 4; i < 124; i += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mx[k] = fmax3_nan(mx[k], __uint_as_float(v[i + 2 * k]), __uint_as_float(v[i + 2 * k + 1]));
        mx[0] = fmax3_nan(mx[0], __uint_as_float(v[124]), __uint_as_float(v[125]));
        mx[1] = fmax3_nan(mx[1], __uint_as_float(v[126]), __uint_as_float(v[127]));
        const float mt = fmax3_nan(fmax3_nan(mx[0], mx[1], mx[2]), mx[3], mx[3]) * sl2;
        // The reference moves only when the maximum has grown by more than 8
        // (log2 units); the negation takes a NaN along, and the row ends as NaN.
        const bool bump = !(mt <= m + 8.f);
        const float m_new = bump ? mt : m;
        const float ref = m_new == -INFINITY ? 0.f : m_new;    // nothing seen: weights of 0
        const float alpha = bump ? fast_exp2(m - ref) : 1.f;
        m = m_new;
        // O is stable: S(j) was committed after P.V(j-1)
        if (j > 0 && __any_sync(0xffffffffu, bump)) {
#pragma unroll 1
          for (int c = 0; c < D; c += 8) {
            uint32_t o[8];
            tmem_load8(tO + c, o);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_store8(tO + c, o);
          }
        }
        // weights, 32 keys at a time, and their sum
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t h[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int k = c * 32 + 2 * i, s = (i & 1) * 2;
            float x0, x1;
            ffma2(x0, x1, __uint_as_float(v[k]), __uint_as_float(v[k + 1]), sl2, sl2, -ref, -ref);
            const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
            fadd2(sum[s], sum[s + 1], sum[s], sum[s + 1], p0, p1);
            h[i] = Mma<T>::pack(p0, p1);
          }
          tmem_store16_async(tS + c * 16, h);
          if (c == 1) {              // P.V may begin on the first half
            tmem_store_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_half[x]);
          }
        }
        l = l * alpha + ((sum[0] + sum[1]) + (sum[2] + sum[3]));
        tmem_store_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[x]);
      }
      if (!ok) break;
      if (n > 0) {
        ok = wait_all(&o_done[x], no++ & 1);
        if (!ok) break;
        tc_fence_after();
      }
      if (p.pieces > 1) {
        if (n > 0) {      // fp32 partial, as it is, with its maximum and sum
          const long long row = (long long)u.slot * 256 + x * 128 + r;
          float *dst = p.part_o + row * D;
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            uint32_t o[16];
            tmem_load16(tO + c, o);
            if (row_ok) {
              st_global_v8(dst + c, o);
              st_global_v8(dst + c + 8, o + 8);
            }
          }
          if (row_ok) p.part_ml[row] = make_float2(m, l);
        }
      } else {
        const bool none = l == 0.f;          // nothing seen: zeros, whatever V holds
        const float inv = 1.f / l;
        T *dst = static_cast<T *>(p.out) +
                 ((long long)(u.token0 + tx + t) * p.num_q_heads + u.kv_head * G + r - t * G) * D;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32], h[16];
          if (n > 0) tmem_load32(tO + c, o);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            h[i] = none ? 0u
                        : Mma<T>::pack(__uint_as_float(o[2 * i]) * inv,
                                       __uint_as_float(o[2 * i + 1]) * inv);
          if (row_ok) {
            if (wide) {                      // whole 32-byte sectors
              st_global_v8(dst + c, h);
              st_global_v8(dst + c + 16, h + 8);
            } else {
#pragma unroll
              for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<uint4 *>(dst + c + 2 * i) =
                    make_uint4(h[i], h[i + 1], h[i + 2], h[i + 3]);
            }
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && abort_flag) flag_error(PA_DEVERR_TIMEOUT);
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, kPfTmemCols);
  }
}

// Join of the pieces of the keys: a warp takes one of the 256 rows of a (pair
// of query tiles, kv head), each lane D / 32 columns.
template <typename T, int D>
__global__ void __launch_bounds__(256) prompt_join_kernel(const PromptParams p) {
  constexpr int VPL = D / 32, UNR = 8;
  using VecT = typename std::conditional<VPL == 4, float4, float2>::type;
  grid_dependency_wait();
  allow_dependent_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.y * 8 + warp, x = row >> 7, r = row & 127;
  const int t = r / p.group, g = r - t * p.group;
  const int4 of = __ldcg(p.part_of + blockIdx.x);
  const bool alternate = of.y < 0;
  const int token = x * p.tq + t;
  if (t >= p.tq || token >= abs(of.y) || (alternate && x > 0) || of.x < 0 ||
      of.x + token >= p.num_tokens)
    return;
  // part i of the row's: of its own query tile, then (alternate) of B's rows
  const int own = min(x ? of.w : of.z, p.pieces), n = own + (alternate ? min(of.w, p.pieces) : 0);
  const long long first = (long long)blockIdx.x * p.pieces * 256 + row;
  float M = -INFINITY, den = 0.f, num[VPL];
#pragma unroll
  for (int v = 0; v < VPL; ++v) num[v] = 0.f;
  for (int k0 = 0; k0 < n; k0 += 32) {
    const int k = k0 + lane, cnt = min(n - k0, 32);
    const long long at = first + (k < own ? (long long)k * 256 : (long long)(k - own) * 256 + 128);
    const float2 ml = k < n ? __ldcg(p.part_ml + at) : make_float2(-INFINITY, 0.f);
    // the largest so far; a NaN goes along
    float top = ml.x;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      const float y = __shfl_xor_sync(0xffffffffu, top, d);
      top = fmax3_nan(top, y, y);
    }
    top = fmax3_nan(top, M, M);
    const float ref = top == -INFINITY ? 0.f : top;
    const float keep = exp2f(M - ref), wk = exp2f(ml.x - ref);   // no keys seen: 0
    float sum = wk * ml.y;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    den = den * keep + sum;
#pragma unroll
    for (int v = 0; v < VPL; ++v) num[v] *= keep;
    M = top;
    for (int j0 = 0; j0 < cnt; j0 += UNR) {
      VecT o[UNR];
#pragma unroll
      for (int j = 0; j < UNR; ++j) {
        const long long aj = __shfl_sync(0xffffffffu, at, min(j0 + j, cnt - 1));
        o[j] = __ldcg(reinterpret_cast<const VecT *>(p.part_o + aj * D) + lane);
      }
#pragma unroll
      for (int j = 0; j < UNR; ++j) {
        if (j0 + j >= cnt) break;
        const float wj = __shfl_sync(0xffffffffu, wk, j0 + j);
        num[0] = fmaf(wj, o[j].x, num[0]);
        num[1] = fmaf(wj, o[j].y, num[1]);
        if constexpr (VPL == 4) {
          num[2] = fmaf(wj, o[j].z, num[2]);
          num[3] = fmaf(wj, o[j].w, num[3]);
        }
      }
    }
  }
  const bool none = M == -INFINITY;   // nothing seen: zeros, whatever V holds
  const float inv = 1.f / den;
#pragma unroll
  for (int v = 0; v < VPL; ++v) num[v] = none ? 0.f : num[v] * inv;
  const int kh = blockIdx.x % p.num_kv_heads;
  T *dst = static_cast<T *>(p.out) +
           ((long long)(of.x + token) * p.num_q_heads + kh * p.group + g) * D + lane * VPL;
  if constexpr (VPL == 4)
    *reinterpret_cast<uint2 *>(dst) =
        make_uint2(Mma<T>::pack(num[0], num[1]), Mma<T>::pack(num[2], num[3]));
  else
    *reinterpret_cast<uint32_t *>(dst) = Mma<T>::pack(num[0], num[1]);
}

}  // namespace pa
