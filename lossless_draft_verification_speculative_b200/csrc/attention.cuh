// Attention of a call's new tokens over the paged cache (dspark_block_attention).
#pragma once

#include "rotary.cuh"

namespace dspark {

struct AttnParams {
  dspark_heads_t q, out;
  dspark_kv_cache_t cache;
  dspark_rows_t rows;
  float* lse;
  int32_t* status;
  int Hq, causal, window;
  float scale;
};

// The positions [lo, hi) that new token i (of n, in a cache of L tokens) sees.
__device__ __forceinline__ void seen_range(int L, int n, int i, int causal, int window, int& lo,
                                           int& hi) {
  const int pos = L - n + i;
  hi = causal ? min(L, pos + 1) : L;
  lo = window > 0 && pos >= window ? pos - window + 1 : 0;
  if (hi < lo) hi = lo;
}

// One warp per (new token, query head): 32 positions at a time, a lane scores one, the warp
// keeps the running maximum and sum, and each lane accumulates head_dim / 32 elements.
template <typename T>
__global__ void __launch_bounds__(256) attention_rows_kernel(const AttnParams p) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int lane = threadIdx.x & 31;
  const dspark_kv_cache_t& c = p.cache;
  const int D = c.head_dim, G = p.Hq / c.n_heads;
  const int64_t cap = static_cast<int64_t>(c.max_pages) * c.page_size;
  const int b = blockIdx.y;
  SeqRows s;
  const bool ok = seq_rows(p.rows, c.kv_len, cap, b, s);
  if (p.status && blockIdx.x == 0 && threadIdx.x < 32) {
    bool bad = false;
    if (ok && s.n > 0) {
      int lo, hi, lo1, hi1;
      seen_range(s.L, s.n, 0, p.causal, p.window, lo, hi);
      seen_range(s.L, s.n, s.n - 1, p.causal, p.window, lo1, hi1);
      if (hi1 > lo)
        for (int g = lo / c.page_size + lane; g <= (hi1 - 1) / c.page_size; g += 32) {
          const int page = c.page_table[b * c.ld_table + g];
          bad |= page < 0 || page >= c.n_pages;
        }
    }
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) p.status[b] = !ok ? DSPARK_SEQ_BAD_PARAM : bad ? DSPARK_SEQ_BAD_PAGE : 0;
  }
  const int warps = gridDim.x * 8;
  for (int w = blockIdx.x * 8 + (threadIdx.x >> 5); w < s.n * p.Hq; w += warps) {
    const int i = w / p.Hq, h = w - i * p.Hq, row = s.first + i;
    const T* q = static_cast<const T*>(p.q.p) + row_offset(p.q, p.rows, row) +
                 h * p.q.head_stride;
    const T* kb = static_cast<const T*>(c.k) + (h / G) * c.k_head_stride;
    const T* vb = static_cast<const T*>(c.v) + (h / G) * c.v_head_stride;
    int lo, hi;
    seen_range(s.L, s.n, i, p.causal, p.window, lo, hi);
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int t0 = lo; t0 < hi; t0 += 32) {
      const int t = t0 + lane;
      float z = -INFINITY;
      int page = 0;
      bool bad = false;
      if (t < hi) {
        page = c.page_table[b * c.ld_table + t / c.page_size];
        bad = page < 0 || page >= c.n_pages;
        if (bad) page = 0;
        const T* k = kb + page * c.k_page_stride + (t % c.page_size) * c.k_token_stride;
        z = 0.f;
        for (int d = 0; d < D; ++d) z += Half16<T>::up1(q[d]) * Half16<T>::up1(k[d]);
        z *= p.scale;
        if (bad) z = NAN;
      }
      const float mn = fmaxf(m, warp_max_nan(z));
      const float mu = mn == -INFINITY ? 0.f : mn;
      const float f = __expf(m - mu), e = __expf(z - mu);
      l = l * f + warp_sum(e);
      for (int d = 0; d < 4; ++d) o[d] *= f;
      m = mn;
      for (int j = 0; j < 32 && t0 + j < hi; ++j) {
        const float pj = __shfl_sync(0xffffffffu, e, j);
        const int pg = __shfl_sync(0xffffffffu, page, j);
        const T* v = vb + pg * c.v_page_stride + ((t0 + j) % c.page_size) * c.v_token_stride;
        for (int d = 0; d < 4; ++d)
          if (lane + 32 * d < D) o[d] += pj * Half16<T>::up1(v[lane + 32 * d]);
      }
    }
    T* out = static_cast<T*>(p.out.p) + row_offset(p.out, p.rows, row) + h * p.out.head_stride;
    for (int d = 0; d < 4; ++d)
      if (lane + 32 * d < D) out[lane + 32 * d] = Half16<T>::down1(l == 0.f ? 0.f : o[d] / l);
    if (p.lse && lane == 0)
      p.lse[static_cast<int64_t>(row) * p.Hq + h] = l == 0.f ? -INFINITY : m + __logf(l);
  }
}

}  // namespace dspark
