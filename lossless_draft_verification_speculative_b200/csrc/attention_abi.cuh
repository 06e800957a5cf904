// C ABI of the cache-side calls (dspark_attention.h): argument checks, the rotary frequencies
// and the launches. Included by dspark_verify.cu, whose launch helpers it uses.
#pragma once

namespace dspark {
namespace {

// A head tensor of the call's rows; written ones must not overlap themselves (extents of one
// have no stride to check).
bool heads_ok(const dspark_heads_t& t, const dspark_rows_t& r, int heads, int D, bool written) {
  if (!t.p || t.token_stride < 0 || t.head_stride < 0 || t.seq_stride < 0) return false;
  if (!written) return true;
  return (heads <= 1 || t.head_stride >= D) && (r.N <= 1 || t.token_stride >= D) &&
         (r.q_start || r.B <= 1 || t.seq_stride >= D);
}

bool heads_vec(const dspark_heads_t& t, const dspark_rows_t& r, int heads) {
  return aligned(t.p, 16) && (heads <= 1 || t.head_stride % 8 == 0) &&
         (r.N <= 1 || t.token_stride % 8 == 0) &&
         (r.q_start || r.B <= 1 || t.seq_stride % 8 == 0);
}

bool cache_vec(const dspark_kv_cache_t& c) {
  return aligned(c.k, 16) && aligned(c.v, 16) &&
         (c.n_pages <= 1 || (c.k_page_stride % 8 == 0 && c.v_page_stride % 8 == 0)) &&
         (c.page_size <= 1 || (c.k_token_stride % 8 == 0 && c.v_token_stride % 8 == 0)) &&
         (c.n_heads <= 1 || (c.k_head_stride % 8 == 0 && c.v_head_stride % 8 == 0));
}

// The checks that both calls share, and the call's number of rows.
dspark_status_t check_cache_call(const dspark_kv_cache_t& c, const dspark_rows_t& r, int Hq,
                                 dspark_dtype_t dtype, int max_dim) {
  if (dtype != DSPARK_BF16 && dtype != DSPARK_F16) return DSPARK_ERR_INVALID_ARG;
  if (r.B < 0 || r.N < 0 || (r.q_start && r.n_new)) return DSPARK_ERR_INVALID_ARG;
  if (Hq < 1 || c.n_heads < 1) return DSPARK_ERR_INVALID_ARG;
  if (c.n_pages < 1 || c.page_size < 1 || c.max_pages < 0 || c.head_dim < 1 ||
      c.ld_table < c.max_pages)
    return DSPARK_ERR_INVALID_ARG;
  if (r.B == 0) return DSPARK_OK;
  if (!c.kv_len || (c.max_pages > 0 && !c.page_table) || !c.k || !c.v)
    return DSPARK_ERR_INVALID_ARG;
  const int64_t D = c.head_dim;  // slots must not overlap
  if ((c.n_pages > 1 && (c.k_page_stride < D || c.v_page_stride < D)) ||
      (c.page_size > 1 && (c.k_token_stride < D || c.v_token_stride < D)) ||
      (c.n_heads > 1 && (c.k_head_stride < D || c.v_head_stride < D)))
    return DSPARK_ERR_INVALID_ARG;
  if (c.head_dim > max_dim || Hq > 4096 || c.n_heads > 4096) return DSPARK_ERR_UNSUPPORTED;
  const long long rows = r.q_start ? r.N : static_cast<long long>(r.B) * r.N;
  if (rows * Hq > INT32_MAX || r.B > 65535 ||
      static_cast<long long>(c.max_pages) * c.page_size > (1 << 30))
    return DSPARK_ERR_UNSUPPORTED;
  if (!aligned(c.k, 2) || !aligned(c.v, 2)) return DSPARK_ERR_UNSUPPORTED;
  return DSPARK_OK;
}

cudaLaunchConfig_t dependent_launch(dim3 grid, int threads, size_t smem, cudaStream_t stream,
                                    cudaLaunchAttribute* attr) {
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

template <typename T>
dspark_status_t rotary_launch(RotaryParams p, bool vec, cudaStream_t stream) {
  const int total = p.rows.q_start ? p.rows.N : p.rows.B * p.rows.N;
  // 2 or 4 tokens a CTA while every SM still has at least 8 CTAs
  p.tokens = 1;
  while (p.tokens < kRotMaxTokens && total >= 8 * kPlanSMs * 2 * p.tokens) p.tokens *= 2;
  int slots = (p.cache.head_dim + 15) / 16;
  p.log_slots = 0;
  while ((1 << p.log_slots) < slots) ++p.log_slots;
  const int ctas = (total + p.tokens - 1) / p.tokens;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg =
      dependent_launch(dim3(static_cast<unsigned>(ctas > 0 ? ctas : 1)), kRotThreads,
                       (static_cast<size_t>(p.tokens) * (p.R / 2) + 8) * sizeof(float2), stream,
                       attr);  // (8: the last slot of interleaved pairs may read past its own)
  const cudaError_t e = vec ? cudaLaunchKernelEx(&cfg, rotary_append_kernel<T, true>, p)
                            : cudaLaunchKernelEx(&cfg, rotary_append_kernel<T, false>, p);
  return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

// Workspace of block_attention: the cut items, then the partial results' (m, l) and O of two
// slots per CTA, for as many rows as an item of the call can have, then the sums of long items of
// two groups per CTA.
struct AttnWs {
  size_t join, ml, o, sums, total;
  int part_rows, sum_rows;
};
AttnWs attention_ws(int N, int Hq, int Hk, int D) {
  const long long rows = static_cast<long long>(N) * (Hq / Hk);
  AttnWs w{};
  w.part_rows = static_cast<int>(rows < kAtItemRows ? rows : kAtItemRows);
  const size_t slots = 2 * static_cast<size_t>(kPlanSMs) * w.part_rows;
  w.ml = align256(sizeof(AttnJoin) * kPlanSMs);
  w.o = w.ml + align256(slots * sizeof(float2));
  w.sums = w.o + align256(slots * (D <= 64 ? 64 : 128) * sizeof(float));
  w.sum_rows = w.part_rows < kAtTile ? w.part_rows : kAtTile;
  w.total = w.sums + 2 * static_cast<size_t>(kPlanSMs) * w.sum_rows *
                         align256((D <= 64 ? 64 : 128) * sizeof(float));
  return w;
}

int log2_of(int pow2) {
  int l = 0;
  while ((1 << l) < pow2) ++l;
  return l;
}

// The tensor map of the pages of a cache tensor: [tensors][pages][heads][slots][head_dim], boxes
// of `box` slots x 64 elements of one head in the 128-byte swizzle; elements past head_dim, and
// boxes of a page index past the last, are filled with zeros. Keys and values of one layout share
// a map (an encoding takes 1.3 us of host time): the two tensors lie `apart` bytes apart from
// the first; 0: one tensor. L2 fetches the 128 bytes of a box's row, no more: with 256 the next
// head's row came along for heads of 64 (186 us instead of 143 for the serving blocks).
bool page_map(CUtensorMap* map, void* base, int64_t apart, int64_t page_stride,
              int64_t token_stride, int64_t head_stride, const dspark_kv_cache_t& c,
              dspark_dtype_t dtype, int box) {
  const EncodeTiledFn enc = tensor_map_encoder();
  if (!enc) return false;
  const int64_t one = c.head_dim;  // any legal stride for an extent of one
  const cuuint64_t dims[5] = {
      static_cast<cuuint64_t>(c.head_dim), static_cast<cuuint64_t>(c.page_size),
      static_cast<cuuint64_t>(c.n_heads), static_cast<cuuint64_t>(c.n_pages), apart ? 2u : 1u};
  const cuuint64_t strides[4] = {2 * static_cast<cuuint64_t>(c.page_size > 1 ? token_stride : one),
                                 2 * static_cast<cuuint64_t>(c.n_heads > 1 ? head_stride : one),
                                 2 * static_cast<cuuint64_t>(c.n_pages > 1 ? page_stride : one),
                                 static_cast<cuuint64_t>(apart ? apart : 2 * one)};
  const cuuint32_t boxes[5] = {64, static_cast<cuuint32_t>(box), 1, 1, 1};
  const cuuint32_t es[5] = {1, 1, 1, 1, 1};
  return enc(map,
             dtype == DSPARK_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                  : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
             5, base, dims, strides, boxes, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The maps of keys and values: one for both where their strides agree and their addresses differ
// by less than a tensor map's largest stride (2^40 bytes), else one each.
bool page_maps(CUtensorMap* kmap, CUtensorMap* vmap, AttnParams* p, dspark_dtype_t dtype) {
  const dspark_kv_cache_t& c = p->cache;
  const uintptr_t k = reinterpret_cast<uintptr_t>(c.k), v = reinterpret_cast<uintptr_t>(c.v);
  const uint64_t apart = v > k ? v - k : k - v;
  if (apart > 0 && apart < (1ull << 40) && c.k_page_stride == c.v_page_stride &&
      c.k_token_stride == c.v_token_stride && c.k_head_stride == c.v_head_stride) {
    p->which_k = v > k ? 0 : 1;
    p->which_v = 1 - p->which_k;
    if (!page_map(kmap, v > k ? c.k : c.v, static_cast<int64_t>(apart), c.k_page_stride,
                  c.k_token_stride, c.k_head_stride, c, dtype, p->box))
      return false;
    *vmap = *kmap;
    return true;
  }
  return page_map(kmap, c.k, 0, c.k_page_stride, c.k_token_stride, c.k_head_stride, c, dtype,
                  p->box) &&
         page_map(vmap, c.v, 0, c.v_page_stride, c.v_token_stride, c.v_head_stride, c, dtype,
                  p->box);
}

template <typename T, int DP>
dspark_status_t attention_launch(AttnParams p, dspark_dtype_t dtype, const AttnWs& ws,
                                 cudaStream_t stream) {
  alignas(64) CUtensorMap kmap, vmap;
  if (!page_maps(&kmap, &vmap, &p, dtype)) return DSPARK_ERR_UNSUPPORTED;
  constexpr size_t smem = AttnSmem<DP>::kTotal;
  cudaError_t e = cudaSuccess;
  const int ctas = resident_ctas(reinterpret_cast<const void*>(&attention_kernel<T, DP>),
                                 kAtThreads, smem, &e);
  if (e != cudaSuccess) return DSPARK_ERR_CUDA;
  if (ctas < 1) return DSPARK_ERR_UNSUPPORTED;
  const unsigned grid = static_cast<unsigned>(ctas < kPlanSMs ? ctas : kPlanSMs);
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = dependent_launch(dim3(grid), kAtThreads, smem, stream, attr);
  if (cudaLaunchKernelEx(&cfg, attention_kernel<T, DP>, kmap, vmap, p) != cudaSuccess)
    return DSPARK_ERR_CUDA;
  // one CTA row per 8 rows of an item, at most 16 (a long item's rows take two turns)
  const int y = (ws.part_rows + kJoinWarps - 1) / kJoinWarps;
  cfg = dependent_launch(dim3(grid, static_cast<unsigned>(y < 1 ? 1 : y > 16 ? 16 : y)),
                         32 * kJoinWarps, 0, stream, attr);
  return cudaLaunchKernelEx(&cfg, attention_join_kernel<T, DP>, p) == cudaSuccess
             ? DSPARK_OK
             : DSPARK_ERR_CUDA;
}

dspark_status_t block_attention_impl(dspark_heads_t q, int n_q_heads, dspark_heads_t out,
                                     dspark_dtype_t dtype, dspark_kv_cache_t cache,
                                     dspark_rows_t rows, float scale, int causal, int window,
                                     float* lse, int32_t* status, void* workspace,
                                     size_t workspace_bytes, void* stream, int withhold) {
  const dspark_status_t st = check_cache_call(cache, rows, n_q_heads, dtype, 128);
  if (st != DSPARK_OK) return st;
  if (!(scale > 0.f) || !std::isfinite(scale) || window < 0 || n_q_heads % cache.n_heads != 0)
    return DSPARK_ERR_INVALID_ARG;
  if (rows.B == 0) return DSPARK_OK;
  const int D = cache.head_dim;
  if (rows.N > 0 &&
      (!heads_ok(q, rows, n_q_heads, D, false) || !heads_ok(out, rows, n_q_heads, D, true)))
    return DSPARK_ERR_INVALID_ARG;
  if (D < 16 || D % 8 != 0 || cache.page_size < 8 || cache.page_size > 1024 ||
      (cache.page_size & (cache.page_size - 1)) != 0)
    return DSPARK_ERR_UNSUPPORTED;
  if (!heads_vec(q, rows, n_q_heads) || !heads_vec(out, rows, n_q_heads) || !cache_vec(cache) ||
      !aligned(lse, 4))
    return DSPARK_ERR_UNSUPPORTED;
  const AttnWs ws = attention_ws(rows.N, n_q_heads, cache.n_heads, D);
  if (!workspace || workspace_bytes < ws.total || !aligned(workspace, 256))
    return DSPARK_ERR_WORKSPACE;
  AttnParams p{};
  p.q = q;
  p.out = out;
  p.cache = cache;
  p.rows = rows;
  p.lse = lse;
  p.status = status;
  p.Hq = n_q_heads;
  p.by_group = fast_div(static_cast<uint32_t>(n_q_heads / cache.n_heads));
  p.causal = causal != 0;
  p.window = window;
  p.scale_log2 = static_cast<float>(scale * 1.4426950408889634);
  if (!std::isfinite(p.scale_log2)) return DSPARK_ERR_INVALID_ARG;
  p.box = cache.page_size < kAtTile ? cache.page_size : kAtTile;
  p.box_log2 = log2_of(p.box);
  p.page_log2 = log2_of(cache.page_size);
  char* w = static_cast<char*>(workspace);
  p.part_rows = ws.part_rows;
  p.withhold = withhold;
  p.join = reinterpret_cast<AttnJoin*>(w + ws.join);
  p.part_ml = reinterpret_cast<float2*>(w + ws.ml);
  p.part_o = reinterpret_cast<float*>(w + ws.o);
  p.sums = reinterpret_cast<float*>(w + ws.sums);
  p.sum_rows = ws.sum_rows;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == DSPARK_BF16)
    return D <= 64 ? attention_launch<__nv_bfloat16, 64>(p, dtype, ws, s)
                   : attention_launch<__nv_bfloat16, 128>(p, dtype, ws, s);
  return D <= 64 ? attention_launch<__half, 64>(p, dtype, ws, s)
                 : attention_launch<__half, 128>(p, dtype, ws, s);
}

}  // namespace
}  // namespace dspark

extern "C" {

dspark_status_t dspark_rotary_frequencies(int R, double theta, dspark_rotary_scaling_t scaling,
                                          double factor, double trained, double low, double high,
                                          float* inv_freq, float* magnitude) {
  if (R < 2 || R > 1024 || R % 2 != 0 || !(theta > 1.0) || !std::isfinite(theta) || !inv_freq ||
      !magnitude)
    return DSPARK_ERR_INVALID_ARG;
  if (scaling < DSPARK_ROTARY_PLAIN || scaling > DSPARK_ROTARY_BANDS) return DSPARK_ERR_INVALID_ARG;
  if (scaling != DSPARK_ROTARY_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
    return DSPARK_ERR_INVALID_ARG;
  const bool ramp = scaling == DSPARK_ROTARY_YARN || scaling == DSPARK_ROTARY_BANDS;
  if (ramp && (!(trained >= 1.0) || !std::isfinite(trained) || !(low > 0.0) || !(high > low) ||
               !std::isfinite(high)))
    return DSPARK_ERR_INVALID_ARG;
  if (scaling == DSPARK_ROTARY_NTK && R == 2) return DSPARK_ERR_INVALID_ARG;  // R / (R - 2)
  const double two_pi = 6.283185307179586477;
  const double base = scaling == DSPARK_ROTARY_NTK
                          ? theta * std::pow(factor, static_cast<double>(R) / (R - 2))
                          : theta;
  double r0 = 0.0, r1 = 0.0;
  if (scaling == DSPARK_ROTARY_YARN) {
    const double k = R / (2.0 * std::log(theta));
    r0 = std::fmax(std::floor(k * std::log(trained / (two_pi * high))), 0.0);
    r1 = std::fmin(std::ceil(k * std::log(trained / (two_pi * low))), R - 1.0);
    if (r1 <= r0) r1 = r0 + 0.001;  // a step instead of a ramp
  }
  for (int i = 0; i < R / 2; ++i) {
    double f = std::pow(base, -2.0 * i / R);
    if (scaling == DSPARK_ROTARY_LINEAR) f /= factor;
    if (scaling == DSPARK_ROTARY_YARN) {
      const double g = std::fmin(std::fmax((i - r0) / (r1 - r0), 0.0), 1.0);
      f = (1.0 - g) * f + g * f / factor;
    }
    if (scaling == DSPARK_ROTARY_BANDS) {
      const double g =
          std::fmin(std::fmax((trained * f / two_pi - low) / (high - low), 0.0), 1.0);
      f = g * f + (1.0 - g) * f / factor;
    }
    inv_freq[i] = static_cast<float>(f);
  }
  *magnitude =
      scaling == DSPARK_ROTARY_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.f;
  return DSPARK_OK;
}

dspark_status_t dspark_rotary_append(dspark_heads_t q, int n_q_heads, dspark_heads_t q_out,
                                     dspark_heads_t k, dspark_heads_t v, dspark_dtype_t dtype,
                                     dspark_kv_cache_t cache, dspark_rows_t rows,
                                     const float* inv_freq, int R, int interleaved,
                                     float magnitude, int32_t* status, void* stream) {
  const dspark_status_t st = check_cache_call(cache, rows, n_q_heads, dtype, 1024);
  if (st != DSPARK_OK || rows.B == 0) return st;
  const int D = cache.head_dim, Hk = cache.n_heads;
  if (R < 0 || R > D || R % 2 != 0 || (R > 0 && !inv_freq) || !std::isfinite(magnitude))
    return DSPARK_ERR_INVALID_ARG;
  if (rows.N > 0 && (!heads_ok(q, rows, n_q_heads, D, false) ||
                     !heads_ok(q_out, rows, n_q_heads, D, true) ||
                     !heads_ok(k, rows, Hk, D, false) || !heads_ok(v, rows, Hk, D, false)))
    return DSPARK_ERR_INVALID_ARG;
  if (!aligned(q.p, 2) || !aligned(q_out.p, 2) || !aligned(k.p, 2) || !aligned(v.p, 2))
    return DSPARK_ERR_UNSUPPORTED;
  const bool vec = D % 8 == 0 && R % (interleaved ? 8 : 16) == 0 && heads_vec(q, rows, n_q_heads) &&
                   heads_vec(q_out, rows, n_q_heads) && heads_vec(k, rows, Hk) &&
                   heads_vec(v, rows, Hk) && cache_vec(cache);
  RotaryParams p{};
  p.q = q;
  p.q_out = q_out;
  p.k = k;
  p.v = v;
  p.cache = cache;
  p.rows = rows;
  p.inv_freq = inv_freq;
  p.status = status;
  p.Hq = n_q_heads;
  p.R = R;
  p.interleaved = interleaved != 0;
  p.magnitude = magnitude;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return dtype == DSPARK_BF16 ? rotary_launch<__nv_bfloat16>(p, vec, s)
                              : rotary_launch<__half>(p, vec, s);
}

size_t dspark_block_attention_workspace_bytes(int N, int n_q_heads, int n_heads, int head_dim) {
  if (N < 0 || n_heads < 1 || n_q_heads < 1 || n_q_heads % n_heads != 0 || head_dim < 16 ||
      head_dim > 128 || head_dim % 8 != 0)
    return 0;
  return attention_ws(N, n_q_heads, n_heads, head_dim).total;
}

dspark_status_t dspark_block_attention(dspark_heads_t q, int n_q_heads, dspark_heads_t out,
                                       dspark_dtype_t dtype, dspark_kv_cache_t cache,
                                       dspark_rows_t rows, float scale, int causal, int window,
                                       float* lse, int32_t* status, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  return block_attention_impl(q, n_q_heads, out, dtype, cache, rows, scale, causal, window, lse,
                              status, workspace, workspace_bytes, stream, 0);
}

dspark_status_t dspark_block_attention_withheld(dspark_heads_t q, int n_q_heads,
                                                dspark_heads_t out, dspark_dtype_t dtype,
                                                dspark_kv_cache_t cache, dspark_rows_t rows,
                                                float scale, int causal, int window, float* lse,
                                                int32_t* status, void* workspace,
                                                size_t workspace_bytes, void* stream) {
  return block_attention_impl(q, n_q_heads, out, dtype, cache, rows, scale, causal, window, lse,
                              status, workspace, workspace_bytes, stream, 1);
}

}  // extern "C"
