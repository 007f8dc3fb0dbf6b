// C entry points around the 8-bit paged cache: rotary positions with the cache
// write, decode attention, gather and block copies, and attention over packed
// prompts.  Included by library.cu behind pa_kernels.cu, whose helpers
// (tensor-map encoder, argument checks, wait limit) it uses.
#pragma once

namespace {

bool aligned_stride(long long elements, int head_dim, int heads) {
  return elements >= (long long)heads * head_dim && elements % 8 == 0;
}

// Launch with programmatic stream serialisation: the grid may be scheduled
// while the kernel before it on the stream finishes, and waits for it before
// its first global access.
template <typename... KArgs, typename... Args>
cudaError_t launch_dependent(void (*kern)(KArgs...), dim3 grid, int threads, size_t smem,
                             cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  if (e != cudaSuccess) cudaGetLastError();
  return e;
}

// ---------------------------------------------------------------- rotary cache write

template <typename T, int D, bool FP8, bool PAIRS>
int launch_rope(pa::RopeParams &p, int sms, cudaStream_t stream) {
  constexpr int HPP = 512 / D;   // heads of a pass
  const int all = (p.num_q_heads + HPP - 1) / HPP + (2 * p.num_kv_heads + HPP - 1) / HPP;
  // As many warps to a token as leave every SM its 24, one pass each at most.
  const long long resident = 24ll * sms;
  p.splits = (int)std::max(1ll, std::min<long long>(all, resident / p.num_tokens));
  p.passes = (all + p.splits - 1) / p.splits;
  p.splits = (all + p.passes - 1) / p.passes;
  const long long units = (long long)p.num_tokens * p.splits;
  const unsigned grid = (unsigned)std::min<long long>((units + 7) / 8, 3ll * sms);
  const cudaError_t e = launch_dependent(pa::rope_and_cache_kernel<T, D, FP8, PAIRS>, dim3(grid),
                                         256, 0, stream, p);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

template <typename T, int D>
int dispatch_rope(pa::RopeParams &p, bool fp8, bool pairs, int sms, cudaStream_t stream) {
  if (fp8)
    return pairs ? launch_rope<T, D, true, true>(p, sms, stream)
                 : launch_rope<T, D, true, false>(p, sms, stream);
  return pairs ? launch_rope<T, D, false, true>(p, sms, stream)
               : launch_rope<T, D, false, false>(p, sms, stream);
}

int rope_and_cache(bool fp8, void *q_out, const void *q, const void *key, const void *value,
                   void *k_cache, void *v_cache, float *kv_scale, const int64_t *slot_mapping,
                   const int64_t *positions, const float *cos_sin, const int *sections,
                   int num_axes, int rotary_dim, int max_position, int interleaved,
                   long long q_out_stride, long long q_stride, long long key_stride,
                   long long value_stride, int num_tokens, int num_q_heads, int num_kv_heads,
                   int head_dim, int block_size, int num_blocks, pa_dtype dtype,
                   cudaStream_t stream) {
  if (num_tokens < 0 || num_q_heads < 0 || num_kv_heads <= 0 || num_blocks < 0 || head_dim <= 0 ||
      block_size <= 0 || rotary_dim < 0 || rotary_dim > head_dim)
    return PA_ERR_ARG;
  if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_ARG;
  if (!supported_shape(head_dim, block_size)) return PA_ERR_UNSUPPORTED;
  if (rotary_dim % 16 != 0) return PA_ERR_UNSUPPORTED;
  int bound[3] = {1 << 30, 1 << 30, 1 << 30};   // pairs before axis 1, 2, 3
  if (rotary_dim > 0) {
    if (num_axes < 1 || num_axes > 4) return PA_ERR_UNSUPPORTED;
    if (max_position <= 0 || !sections) return PA_ERR_ARG;
    int sum = 0;
    for (int a = 0; a < num_axes; ++a) {
      if (sections[a] < 0 || sections[a] > rotary_dim / 2) return PA_ERR_ARG;
      if (a > 0) bound[a - 1] = sum;
      sum += sections[a];
    }
    if (sum != rotary_dim / 2) return PA_ERR_ARG;
  }
  if (num_tokens == 0) return PA_OK;
  const int q_heads = q ? num_q_heads : 0;
  if (!key || !value || !k_cache || !v_cache || !slot_mapping || (fp8 && !kv_scale) ||
      (rotary_dim > 0 && (!positions || !cos_sin)) || (q && !q_out) || (q && num_q_heads == 0))
    return PA_ERR_ARG;
  if (!aligned(key, 16) || !aligned(value, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(slot_mapping, 8) || !aligned(q, 16) || !aligned(q_out, 16) ||
      !aligned(kv_scale, 16) || !aligned(positions, 8) || !aligned(cos_sin, 16))
    return PA_ERR_ARG;
  if (!aligned_stride(key_stride, head_dim, num_kv_heads) ||
      !aligned_stride(value_stride, head_dim, num_kv_heads) ||
      (q && (!aligned_stride(q_stride, head_dim, num_q_heads) ||
             !aligned_stride(q_out_stride, head_dim, num_q_heads))))
    return PA_ERR_ARG;
  if (num_tokens >= (1 << 30) || num_kv_heads > (1 << 20) || num_q_heads > (1 << 20))
    return PA_ERR_UNSUPPORTED;
  int dev;
  if (current_device(&dev) != PA_OK) return PA_ERR_CUDA;
  const int sms = sm_count(dev);
  if (sms <= 0) return PA_ERR_CUDA;
  pa::RopeParams p;
  p.q_out = q_out;
  p.q = q;
  p.k = key;
  p.v = value;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.kv_scale = kv_scale;
  p.slots = slot_mapping;
  p.positions = positions;
  p.cos_sin = cos_sin;
  p.q_out_stride = q_out_stride;
  p.q_stride = q_stride;
  p.k_stride = key_stride;
  p.v_stride = value_stride;
  p.num_slots = (long long)num_blocks * block_size;
  p.num_tokens = num_tokens;
  p.num_q_heads = q_heads;
  p.num_kv_heads = num_kv_heads;
  p.block_size = block_size;
  p.rotary = rotary_dim;
  p.axes = rotary_dim > 0 ? num_axes : 0;
  p.max_position = max_position;
  for (int a = 0; a < 3; ++a) p.sect[a] = bound[a];
  if (dtype == PA_BF16)
    return head_dim == 128 ? dispatch_rope<__nv_bfloat16, 128>(p, fp8, interleaved != 0, sms, stream)
                           : dispatch_rope<__nv_bfloat16, 64>(p, fp8, interleaved != 0, sms, stream);
  return head_dim == 128 ? dispatch_rope<__half, 128>(p, fp8, interleaved != 0, sms, stream)
                         : dispatch_rope<__half, 64>(p, fp8, interleaved != 0, sms, stream);
}

// ---------------------------------------------------------------- 8-bit decode

// The code pool as rows of D bytes; a box is one (block, kv head) tile, with
// the swizzle as wide as a row.
bool encode_code_map(CUtensorMap *m, const void *base, long long rows, int D, int B) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)D};
  cuuint32_t box[2] = {(cuuint32_t)D, (cuuint32_t)B};
  cuuint32_t estr[2] = {1u, 1u};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int NT, int HPL>
int launch_decode_fp8(pa::DecodeFp8Params &p, const CUtensorMap &kmap, const CUtensorMap &vmap,
                      uint8_t *workspace, size_t workspace_bytes, int max_context, int dev, int sms,
                      cudaStream_t stream) {
  auto kern = pa::paged_decode_fp8_kernel<D, NT, HPL, kWarpsPerCta>;
  const int G = p.group;
  const size_t smem = 1024 + (size_t)kWarpsPerCta * pa::fp8_warp_bytes(D, G);   // 1024: alignment
  const int most = pa::fp8_ctas(NT, HPL), want = g_tune_ctas.load();
  const int ctas = want > 0 ? std::min(want, most) : most;
  static pa::SmemLimit<kMaxDevices> limit;
  if (!limit.raise(dev, smem, [&](size_t n) { return set_smem(kern, n); })) return PA_ERR_CUDA;
  const long long pairs = (long long)p.num_seqs * p.num_kv_heads;
  const long long tiles = (max_context + pa::kF8Tile - 1) / pa::kF8Tile + 1;   // of a pair, at most
  // Short contexts are not cut (a warp takes a pair's tiles in less time than a
  // cut, its partials and the merge cost): up to 64 tokens (one sequence of 40
  // tokens, 32 / 8 heads: 7.4 us whole, 8.7 cut), or 128 where the pairs alone
  // give every eighth warp work (128 sequences of 128: 13.2 and 16.8; but one
  // of 128: 10.3 and 8.7, 128 of 512: 34.2 and 34.0).  Else at least two tiles
  // to a warp, or one where that still leaves warps without work (one sequence
  // of 256: 9.3 us with one, 10.4 with two, 13.2 with four).
  const int mt = g_tune_min_tiles.load();
  const long long most_warps = (long long)sms * ctas * kWarpsPerCta;
  const bool whole = tiles <= 3 || (tiles <= 5 && pairs * 8 >= most_warps);
  p.min_tiles = mt > 0 ? mt : (whole ? 0 : (pairs * tiles * 2 <= most_warps && tiles <= 64 ? 1 : 2));
  // No more warps than can have work.
  const long long useful = p.min_tiles == 0 ? pairs : (pairs * tiles + p.min_tiles - 1) / p.min_tiles;
  const int grid = (int)std::min<long long>((useful + kWarpsPerCta - 1) / kWarpsPerCta,
                                            (long long)sms * ctas);
  const int w_total = grid * kWarpsPerCta;
  size_t off_ml, off_o;
  if (workspace_bytes < workspace_for(w_total, G, D, &off_ml, &off_o)) return PA_ERR_WORKSPACE;
  p.meta = reinterpret_cast<int4 *>(workspace);
  p.part_ml = reinterpret_cast<float2 *>(workspace + off_ml);
  p.part_o = reinterpret_cast<float *>(workspace + off_o);
  if (launch_dependent(kern, dim3(grid), kWarpsPerCta * 32, smem, stream, kmap, vmap, p) !=
      cudaSuccess)
    return PA_ERR_CUDA;
  if (p.min_tiles == 0) return PA_OK;   // nothing was cut
  // Segments are at least as many as (sequence, kv head) pairs, cuts at most as
  // many as ranges: with many pairs a warp takes one range and four heads, else
  // a CTA as many ranges as there are to a pair, and one head.
  int span = 1;
  while (span < 32 && pairs * span * 2 <= w_total) span *= 2;
  const int heads = span > 1 ? 1 : 4, groups = (G + heads - 1) / heads;
  const long long warps = (long long)((w_total + span - 1) / span) * groups;
  const dim3 mgrid((unsigned)(span > 1 ? warps : (warps + 3) / 4));
  const cudaError_t e =
      span > 1 ? launch_dependent(pa::paged_decode_fp8_merge_kernel<D, 1>, mgrid, 128, 0, stream, p,
                                  w_total, span, groups)
               : launch_dependent(pa::paged_decode_fp8_merge_kernel<D, 4>, mgrid, 128, 0, stream, p,
                                  w_total, span, groups);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

template <int D, typename... Args>
int dispatch_decode_fp8(pa::DecodeFp8Params &p, Args... args) {
  if (p.group <= 4) return launch_decode_fp8<D, 1, 1>(p, args...);
  if (p.group <= 8) return launch_decode_fp8<D, 1, 2>(p, args...);
  return launch_decode_fp8<D, 2, 2>(p, args...);
}

// ---------------------------------------------------------------- packed prompts

// K or V [Tk, Hkv, D] with any token stride as a 3-D map (D, Hkv, Tk); a box is
// 64 columns of one head x 128 tokens.  Q [T, Hq, D] the same way, a box 64
// columns x the G heads of one kv head x tq tokens.
bool encode_rows_map(CUtensorMap *m, const void *base, long long rows, int heads, int D,
                     long long stride, int box_heads, int box_rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
  cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
  cuuint32_t box[3] = {64u, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void *>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How a call is cut up: units of (pair of query tiles, kv head), at most
// `units` of them, and pieces of the keys when the units alone leave SMs idle.
struct PromptPlan {
  long long units;
  int tq, pieces, piece_tiles;
  size_t workspace;
};

// The keys are split if that takes at least so many K/V tiles off the longest
// CTA's way: partials and their join cost what about ten tiles do.
constexpr long long kSplitGain = 12;

PromptPlan plan_prompt(int num_seqs, int num_tokens, int num_q_heads, int num_kv_heads,
                       int head_dim, int max_query, int max_key, int sms) {
  PromptPlan pl;
  pl.tq = pa::kPrRows / (num_q_heads / num_kv_heads);
  if (max_query == 0) {   // one CTA, which reports sequences that have queries all the same
    pl.units = pl.pieces = pl.piece_tiles = 1;
    pl.workspace = 0;
    return pl;
  }
  const long long w = 2 * pl.tq;
  const long long pairs = std::min((long long)num_seqs * ((max_query + w - 1) / w),
                                   num_tokens / w + num_seqs);
  pl.units = pairs * num_kv_heads;
  const long long tiles = std::max(1, (max_key + pa::kPrKeys - 1) / pa::kPrKeys);
  pl.pieces = 1;
  pl.piece_tiles = (int)tiles;
  if (pl.units < sms) {
    const long long per = std::max(2ll, (pl.units * tiles + sms - 1) / sms);
    if (per + kSplitGain <= tiles) {
      pl.piece_tiles = (int)per;
      pl.pieces = (int)((tiles + per - 1) / per);
    }
  }
  pl.workspace =
      pl.pieces > 1 ? (size_t)pl.units * (pl.pieces * 256ll * (head_dim * 4 + 8) + 16) : 0;
  return pl;
}

// What plan_prompt takes; out of range for the entry points below.
int check_prompt(int num_seqs, int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                 int max_query, int max_key) {
  if (num_seqs < 0 || num_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      max_query < 0 || max_key < 0 || num_q_heads % num_kv_heads != 0)
    return PA_ERR_ARG;
  if ((head_dim != 64 && head_dim != 128) || num_q_heads / num_kv_heads > 16 ||
      num_q_heads > 65536 || max_query >= (1 << 30) || max_key >= (1 << 30) ||
      num_tokens >= (1 << 30))
    return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

template <typename T, int D>
int launch_prompt(pa::PromptParams &p, const PromptPlan &pl, const CUtensorMap &qmap,
                  const CUtensorMap &kmap, const CUtensorMap &vmap, int dev, cudaStream_t stream) {
  auto kern = pa::prompt_attention_kernel<T, D>;
  constexpr int smem = pa::PromptSmem<D>::BYTES;
  static std::atomic<int> attr_set[kMaxDevices];
  if (!attr_set[dev].load()) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
        cudaSuccess)
      return PA_ERR_CUDA;
    attr_set[dev].store(1);
  }
  if (launch_dependent(kern, dim3((unsigned)(pl.units * pl.pieces)), pa::kPrThreads, smem, stream,
                       qmap, kmap, vmap, p) != cudaSuccess)
    return PA_ERR_CUDA;
  if (pl.pieces > 1 &&
      launch_dependent(pa::prompt_join_kernel<T, D>, dim3((unsigned)pl.units, 32), 256, 0, stream,
                       p) != cudaSuccess)
    return PA_ERR_CUDA;
  return PA_OK;
}

}  // namespace

extern "C" {

int pa_rope_and_cache(void *q_out, const void *q, const void *key, const void *value,
                      void *k_cache, void *v_cache, const int64_t *slot_mapping,
                      const int64_t *positions, const float *cos_sin, const int *sections,
                      int num_axes, int rotary_dim, int max_position, int interleaved,
                      int64_t q_out_stride, int64_t q_stride, int64_t key_stride,
                      int64_t value_stride, int num_tokens, int num_q_heads, int num_kv_heads,
                      int head_dim, int block_size, int num_blocks, pa_dtype dtype,
                      pa_stream_t stream) {
  return rope_and_cache(false, q_out, q, key, value, k_cache, v_cache, nullptr, slot_mapping,
                        positions, cos_sin, sections, num_axes, rotary_dim, max_position,
                        interleaved, q_out_stride, q_stride, key_stride, value_stride, num_tokens,
                        num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, dtype,
                        (cudaStream_t)stream);
}

int pa_rope_and_cache_fp8(void *q_out, const void *q, const void *key, const void *value,
                          void *k_cache, void *v_cache, float *kv_scale,
                          const int64_t *slot_mapping, const int64_t *positions,
                          const float *cos_sin, const int *sections, int num_axes, int rotary_dim,
                          int max_position, int interleaved, int64_t q_out_stride,
                          int64_t q_stride, int64_t key_stride, int64_t value_stride,
                          int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                          int block_size, int num_blocks, pa_dtype dtype, pa_stream_t stream) {
  return rope_and_cache(true, q_out, q, key, value, k_cache, v_cache, kv_scale, slot_mapping,
                        positions, cos_sin, sections, num_axes, rotary_dim, max_position,
                        interleaved, q_out_stride, q_stride, key_stride, value_stride, num_tokens,
                        num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, dtype,
                        (cudaStream_t)stream);
}

int pa_paged_decode_attention_fp8(float *out, const void *q, const void *k_cache,
                                  const void *v_cache, const float *kv_scale,
                                  const int32_t *block_tables, const int32_t *context_lens,
                                  float scale, int num_kv_heads, int num_seqs, int num_q_heads,
                                  int head_dim, int block_size, int max_blocks_per_seq,
                                  int max_context_len, int num_blocks, pa_dtype dtype,
                                  void *workspace, size_t workspace_bytes, pa_stream_t stream) {
  if (num_seqs < 0 || num_kv_heads <= 0 || num_q_heads <= 0 || head_dim <= 0 || block_size <= 0)
    return PA_ERR_ARG;
  if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_ARG;
  if (num_q_heads % num_kv_heads != 0) return PA_ERR_ARG;
  if (!supported_shape(head_dim, block_size) || num_q_heads / num_kv_heads > 16)
    return PA_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PA_OK;
  if (max_blocks_per_seq <= 0 || num_blocks <= 0 || max_context_len < 0 ||
      (long long)max_context_len > (long long)max_blocks_per_seq * block_size)
    return PA_ERR_ARG;
  if ((long long)num_blocks * num_kv_heads * block_size >= (1ll << 31) ||
      (long long)max_blocks_per_seq * block_size >= (1ll << 30))
    return PA_ERR_UNSUPPORTED;
  if (!out || !q || !k_cache || !v_cache || !kv_scale || !block_tables || !context_lens)
    return PA_ERR_ARG;
  if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(kv_scale, 16) || !aligned(block_tables, 4) || !aligned(context_lens, 4))
    return PA_ERR_ARG;
  if (!workspace || !aligned(workspace, 256)) return PA_ERR_WORKSPACE;
  int dev;
  if (current_device(&dev) != PA_OK || dev >= kMaxDevices) return PA_ERR_CUDA;
  const int sms = sm_count(dev);
  if (sms <= 0) return PA_ERR_CUDA;
  CUtensorMap kmap, vmap;
  const long long rows = (long long)num_blocks * num_kv_heads * block_size;
  if (!encode_code_map(&kmap, k_cache, rows, head_dim, block_size) ||
      !encode_code_map(&vmap, v_cache, rows, head_dim, block_size))
    return PA_ERR_CUDA;
  pa::DecodeFp8Params p = {};
  p.out = out;
  p.q = static_cast<const uint8_t *>(q);
  p.kv_scale = kv_scale;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.num_seqs = num_seqs;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.group = num_q_heads / num_kv_heads;
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  p.q_bf16 = dtype == PA_BF16;
  p.wait_ns = g_wait_limit_ns.load();
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  cudaStream_t st = (cudaStream_t)stream;
  return head_dim == 128
             ? dispatch_decode_fp8<128>(p, kmap, vmap, ws, workspace_bytes, max_context_len, dev,
                                        sms, st)
             : dispatch_decode_fp8<64>(p, kmap, vmap, ws, workspace_bytes, max_context_len, dev,
                                        sms, st);
}

int pa_copy_blocks_fp8(void *k_cache, void *v_cache, float *kv_scale, const int64_t *block_mapping,
                       int num_pairs, int num_kv_heads, int head_dim, int block_size,
                       int num_blocks, pa_stream_t stream) {
  if (num_pairs < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks < 0)
    return PA_ERR_ARG;
  if (!supported_shape(head_dim, block_size)) return PA_ERR_UNSUPPORTED;
  if (num_pairs == 0) return PA_OK;
  if (!k_cache || !v_cache || !kv_scale || !block_mapping) return PA_ERR_ARG;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(kv_scale, 16) ||
      !aligned(block_mapping, 8))
    return PA_ERR_ARG;
  const long long code_vec = (long long)num_kv_heads * block_size * head_dim / 16;
  const long long scale_vec = (long long)num_kv_heads * 2 * block_size / 4;
  const long long per_cta = 256ll * pa::kCopy8Unroll;
  const long long chunks = (2 * code_vec + scale_vec + per_cta - 1) / per_cta;
  if (code_vec >= (1ll << 28) || chunks * num_pairs >= (1ll << 31)) return PA_ERR_UNSUPPORTED;
  const cudaError_t e = launch_dependent(
      pa::copy_blocks_fp8_kernel, dim3((unsigned)(chunks * num_pairs)), 256, 0,
      (cudaStream_t)stream, static_cast<uint4 *>(k_cache), static_cast<uint4 *>(v_cache),
      reinterpret_cast<uint4 *>(kv_scale), block_mapping, (int)code_vec, (int)scale_vec,
      (int)chunks, num_blocks);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

int pa_gather_cache_fp8(void *key, void *value, const void *k_cache, const void *v_cache,
                        const float *kv_scale, const int32_t *block_tables,
                        const int32_t *key_start, int num_seqs, int num_tokens, int num_kv_heads,
                        int head_dim, int block_size, int max_blocks_per_seq, int num_blocks,
                        pa_dtype dtype, pa_stream_t stream) {
  if (num_seqs < 0 || num_tokens < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0)
    return PA_ERR_ARG;
  if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_ARG;
  if (!supported_shape(head_dim, block_size)) return PA_ERR_UNSUPPORTED;
  if (num_seqs == 0 || num_tokens == 0) return PA_OK;
  if (max_blocks_per_seq <= 0 || num_blocks <= 0) return PA_ERR_ARG;
  if (num_kv_heads >= (1 << 20) || num_tokens >= (1ll << 31) - pa::kGatherRows)
    return PA_ERR_UNSUPPORTED;
  if (!key || !value || !k_cache || !v_cache || !kv_scale || !block_tables || !key_start)
    return PA_ERR_ARG;
  if (!aligned(key, 16) || !aligned(value, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(kv_scale, 16) || !aligned(block_tables, 4) || !aligned(key_start, 4))
    return PA_ERR_ARG;
  int dev;
  if (current_device(&dev) != PA_OK || dev >= kMaxDevices) return PA_ERR_CUDA;
  const int sms = sm_count(dev);
  if (sms <= 0) return PA_ERR_CUDA;
  pa::GatherParams p;
  p.key = key;
  p.value = value;
  p.k_cache = static_cast<const uint8_t *>(k_cache);
  p.v_cache = static_cast<const uint8_t *>(v_cache);
  p.kv_scale = kv_scale;
  p.block_tables = block_tables;
  p.key_start = key_start;
  p.num_seqs = num_seqs;
  p.num_tokens = num_tokens;
  p.num_kv_heads = num_kv_heads;
  p.block_size = block_size;
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  // Few rows: split the heads over gridDim.y until the grid fills the SMs, a
  // CTA keeping at least one row per lane group.
  const int chunks = (num_tokens + pa::kGatherRows - 1) / pa::kGatherRows;
  const int rows = 2 * num_kv_heads * pa::kGatherRows, groups = 256 / (head_dim / 16);
  const int most = (rows + groups - 1) / groups;
  const int split = std::max(1, std::min(most, 16 * sms / chunks));
  const dim3 grid(chunks, std::min(split, 65535));
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e;
  if (dtype == PA_BF16)
    e = head_dim == 128
            ? launch_dependent(pa::gather_cache_fp8_kernel<__nv_bfloat16, 128>, grid, 256, 0, st, p)
            : launch_dependent(pa::gather_cache_fp8_kernel<__nv_bfloat16, 64>, grid, 256, 0, st, p);
  else
    e = head_dim == 128
            ? launch_dependent(pa::gather_cache_fp8_kernel<__half, 128>, grid, 256, 0, st, p)
            : launch_dependent(pa::gather_cache_fp8_kernel<__half, 64>, grid, 256, 0, st, p);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

size_t pa_prompt_attention_workspace_bytes(int num_seqs, int num_tokens, int num_q_heads,
                                           int num_kv_heads, int head_dim, int max_query_len,
                                           int max_key_len) {
  if (check_prompt(num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim, max_query_len,
                   max_key_len) != PA_OK)
    return 0;
  int dev;
  if (current_device(&dev) != PA_OK) return 0;
  const int sms = sm_count(dev);
  if (sms <= 0) return 0;
  return plan_prompt(num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim, max_query_len,
                     max_key_len, sms)
      .workspace;
}

int pa_prompt_attention(void *out, const void *q, const void *key, const void *value,
                        const int32_t *query_start, const int32_t *key_start, float scale,
                        int num_kv_heads, int num_seqs, int num_tokens, int num_key_tokens,
                        int num_q_heads, int head_dim, int max_query_len, int max_key_len,
                        int64_t q_stride, int64_t key_stride, int64_t value_stride, pa_dtype dtype,
                        void *workspace, size_t workspace_bytes, pa_stream_t stream) {
  if (num_key_tokens < 0 || (dtype != PA_F16 && dtype != PA_BF16)) return PA_ERR_ARG;
  const int bad = check_prompt(num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim,
                               max_query_len, max_key_len);
  if (bad != PA_OK) return bad;
  if (num_seqs == 0 || num_tokens == 0 || (max_query_len == 0 && !query_start)) return PA_OK;
  if (!out || !q || !query_start || !key_start || (num_key_tokens > 0 && (!key || !value)))
    return PA_ERR_ARG;
  if (!aligned(out, 16) || !aligned(q, 16) || !aligned(key, 16) || !aligned(value, 16) ||
      !aligned(query_start, 4) || !aligned(key_start, 4))
    return PA_ERR_ARG;
  if (!aligned_stride(q_stride, head_dim, num_q_heads) ||
      !aligned_stride(key_stride, head_dim, num_kv_heads) ||
      !aligned_stride(value_stride, head_dim, num_kv_heads))
    return PA_ERR_ARG;
  if (q_stride >= (1ll << 38) || key_stride >= (1ll << 38) || value_stride >= (1ll << 38))
    return PA_ERR_UNSUPPORTED;
  int dev;
  if (current_device(&dev) != PA_OK || dev >= kMaxDevices) return PA_ERR_CUDA;
  const int sms = sm_count(dev);
  if (sms <= 0) return PA_ERR_CUDA;
  const PromptPlan pl = plan_prompt(num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim,
                                    max_query_len, max_key_len, sms);
  if (pl.units * pl.pieces >= (1ll << 31)) return PA_ERR_UNSUPPORTED;
  if (pl.workspace > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < pl.workspace))
    return PA_ERR_WORKSPACE;
  const int G = num_q_heads / num_kv_heads;
  // without keys the maps of K and V are never read: they describe q then
  const bool keys = num_key_tokens > 0;
  CUtensorMap qmap, kmap, vmap;
  if (!encode_rows_map(&qmap, q, num_tokens, num_q_heads, head_dim, q_stride, G, pl.tq) ||
      !encode_rows_map(&kmap, keys ? key : q, keys ? num_key_tokens : num_tokens, num_kv_heads,
                       head_dim, keys ? key_stride : q_stride, 1, pa::kPrKeys) ||
      !encode_rows_map(&vmap, keys ? value : q, keys ? num_key_tokens : num_tokens, num_kv_heads,
                       head_dim, keys ? value_stride : q_stride, 1, pa::kPrKeys))
    return PA_ERR_CUDA;
  pa::PromptParams p;
  p.out = out;
  p.query_start = query_start;
  p.key_start = key_start;
  p.part_o = static_cast<float *>(workspace);
  p.part_ml = reinterpret_cast<float2 *>(static_cast<uint8_t *>(workspace) +
                                         (size_t)pl.units * pl.pieces * 256 * head_dim * 4);
  p.part_of = reinterpret_cast<int4 *>(p.part_ml + pl.units * pl.pieces * 256);
  p.scale_log2 = scale * 1.4426950408889634f;
  p.num_seqs = num_seqs;
  p.num_tokens = num_tokens;
  p.num_key_tokens = num_key_tokens;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.group = G;
  p.tq = pl.tq;
  p.max_query = max_query_len;
  p.max_key = max_key_len;
  p.pieces = pl.pieces;
  p.piece_tiles = pl.piece_tiles;
  const unsigned long long limit = std::min(g_wait_limit_ns.load(), 1ull << 60);
  p.wait_cycles = 2 * (long long)limit;
  p.wait_hint = (uint32_t)std::min(limit, 1000000ull);
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == PA_BF16)
    return head_dim == 128
               ? launch_prompt<__nv_bfloat16, 128>(p, pl, qmap, kmap, vmap, dev, st)
               : launch_prompt<__nv_bfloat16, 64>(p, pl, qmap, kmap, vmap, dev, st);
  return head_dim == 128 ? launch_prompt<__half, 128>(p, pl, qmap, kmap, vmap, dev, st)
                         : launch_prompt<__half, 64>(p, pl, qmap, kmap, vmap, dev, st);
}

}  // extern "C"
