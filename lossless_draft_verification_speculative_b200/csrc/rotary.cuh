// Rotary embedding of a call's new tokens and their append to the paged cache
// (dspark_rotary_append).
//
// Mathematics: at position p the pair (x1, x2) of frequency f turns by a = p f:
// (x1 cos a - x2 sin a, x2 cos a + x1 sin a), times the magnitude. cos and sin are the same for
// every head of a token, so a CTA takes a few tokens, computes their R/2 pairs once into shared
// memory, and then moves the tokens' heads through registers: one read and one write of q, k
// and v. Far positions: a loses 2^-24 a in float32 (0.06 rad at 10^6), so the angle is reduced
// to a fraction of a turn in float64 (one product and one rounding to the nearest turn per
// pair), and sine and cosine are taken of that fraction in float32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "dspark_attention.h"

namespace dspark {

// ------------------------------------------------------------- rows and cache, on the device

// The rows of sequence b: n new tokens from row `first` of the call's row numbering (block:
// b N + i, packed: q_start[b] + i), in a cache of L tokens. False (and n = 0) when a count, a
// start or the length is out of range.
struct SeqRows {
  int first, n, L;
};
__device__ __forceinline__ bool seq_rows(const dspark_rows_t& r, const int32_t* kv_len,
                                         int64_t capacity, int b, SeqRows& s) {
  s.L = kv_len[b];
  bool ok;
  if (r.q_start) {
    const int s0 = r.q_start[b], s1 = r.q_start[b + 1];
    ok = 0 <= s0 && s0 <= s1 && s1 <= r.N;
    s.first = s0;
    s.n = s1 - s0;
  } else {
    s.n = r.n_new ? r.n_new[b] : r.N;
    s.first = b * r.N;
    ok = 0 <= s.n && s.n <= r.N;
  }
  ok = ok && 0 <= s.L && s.L <= capacity;
  if (!ok) s.n = 0;
  return ok;
}

// Element offset of row `row` (call numbering) of a head tensor.
__device__ __forceinline__ int64_t row_offset(const dspark_heads_t& t, const dspark_rows_t& r,
                                              int row) {
  if (r.q_start) return static_cast<int64_t>(row) * t.token_stride;
  const int b = row / r.N;
  return static_cast<int64_t>(b) * t.seq_stride +
         static_cast<int64_t>(row - b * r.N) * t.token_stride;
}

template <typename T>
struct Half16;  // two 16-bit values of type T in a 32-bit word <-> float2
template <>
struct Half16<__nv_bfloat16> {
  __device__ __forceinline__ static float2 up(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  __device__ __forceinline__ static uint32_t down(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  __device__ __forceinline__ static float up1(__nv_bfloat16 x) { return __bfloat162float(x); }
  __device__ __forceinline__ static __nv_bfloat16 down1(float x) { return __float2bfloat16_rn(x); }
};
template <>
struct Half16<__half> {
  __device__ __forceinline__ static float2 up(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  __device__ __forceinline__ static uint32_t down(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  __device__ __forceinline__ static float up1(__half x) { return __half2float(x); }
  __device__ __forceinline__ static __half down1(float x) { return __float2half_rn(x); }
};

// ---------------------------------------------------------------------------- the kernel

constexpr int kRotThreads = 256;
constexpr int kRotMaxTokens = 4;  // tokens per CTA, at most (a warp finds each)

struct RotaryParams {
  dspark_heads_t q, q_out, k, v;
  dspark_kv_cache_t cache;
  dspark_rows_t rows;
  const float* inv_freq;
  int32_t* status;
  int Hq, R, interleaved, tokens;  // tokens per CTA
  float magnitude;
  int log_slots;  // vector path: slots of a head, rounded up to a power of two
};

struct RotaryToken {
  int row, pos;       // call row; position, or -1: the row belongs to no sequence
  int64_t k_at, v_at;  // the slot's element offset in the cache, or -1
};

// The largest b in [0, B) with q_start[b] <= row, or -1, found by a warp: 32 starts a step, one
// load and ballot per factor of 32 in B. Where the starts decrease somewhere, some index. Rows from
// the last start on, commonly padding, give -1 after the first step.
__device__ __forceinline__ int packed_search(const dspark_rows_t& r, int row, int lane) {
  const int end = r.q_start[r.B];
  int lo = -1, hi = r.B;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + (lane + 1) * step;
    const bool le = at < hi && r.q_start[at] <= row;
    const int cnt = __popc(__ballot_sync(0xffffffffu, le));
    if (row >= end) return -1;
    const int nlo = lo + cnt * step;
    hi = min(hi, nlo + step);
    lo = nlo;
  }
  return lo;
}

// Whether sequence b, by its own bounds, has some of the rows first .. last.
__device__ __forceinline__ bool packed_claims(const dspark_rows_t& r, int b, int first, int last) {
  const int s0 = r.q_start[b], s1 = r.q_start[b + 1];
  return 0 <= s0 && s0 <= last && first < s1 && s0 < s1 && s1 <= r.N;
}

// The first sequence that claims a row, or -1: for rows whose search was misled by starts that
// decrease, and for rows of no sequence (those of a padded batch). A warp over all starts, many
// loads in flight; not inlined, so that they cost the kernel no registers. (4096 rows of which
// 64 sequences have 200: 9.5 us against 9.3 without; 1024 sequences one each: 14.3 against 11.8,
// more by 0.5 us inlined with 4 loads in flight, by 0.9 as a scan that the rows of a CTA share.)
__device__ __noinline__ int packed_scan(const int32_t* q_start, int B, int N, int row, int lane) {
  int b = B;
#pragma unroll 16
  for (int at = lane; at < B; at += 32) {
    const int s0 = q_start[at], s1 = q_start[at + 1];
    if (0 <= s0 && s0 <= row && row < s1 && s1 <= N) b = min(b, at);
  }
  b = __reduce_min_sync(0xffffffffu, b);
  return b < B ? b : -1;
}

// Whether every row of sequence b (packed, well-formed bounds, at least one row) is taken as its
// own: the searches for its first and its last row both end at b (a larger row never ends lower,
// so those between do too), or, where starts decrease, no other sequence claims one of its rows.
__device__ __forceinline__ bool packed_sole(const dspark_rows_t& r, int b, const SeqRows& s,
                                            int lane) {
  const int last = s.first + s.n - 1;
  if (packed_search(r, s.first, lane) == b && packed_search(r, last, lane) == b) return true;
  bool shared = false;
  for (int at = lane; at < r.B; at += 32)
    shared |= at != b && packed_claims(r, at, s.first, last);
  return !__any_sync(0xffffffffu, shared);
}

// Which sequence a row belongs to, its position and its slot, found by one warp: block rows by
// division, packed rows by packed_search. A search that ends at a sequence without the row was
// misled by another sequence's starts, or the row belongs to none: packed_scan tells. Bounds
// out of range are refused by packed_claims and seq_rows, so nothing outside the arrays is read.
__device__ __forceinline__ RotaryToken rotary_token(const RotaryParams& p, int row, int lane) {
  RotaryToken t{row, -1, -1, -1};
  const dspark_kv_cache_t& c = p.cache;
  const int64_t cap = static_cast<int64_t>(c.max_pages) * c.page_size;
  int b = p.rows.q_start ? packed_search(p.rows, row, lane) : row / p.rows.N;
  SeqRows s{};
  // (the length is loaded beside the bounds, before they are looked at)
  bool ok = b >= 0 && seq_rows(p.rows, c.kv_len, cap, b, s);
  if (p.rows.q_start && (b < 0 || !packed_claims(p.rows, b, row, row))) {
    b = packed_scan(p.rows.q_start, p.rows.B, p.rows.N, row, lane);
    ok = b >= 0 && seq_rows(p.rows, c.kv_len, cap, b, s);
  }
  if (!ok || s.L < s.n) return t;
  const int i = row - s.first;
  if (i < 0 || i >= s.n) return t;
  t.pos = s.L - s.n + i;
  const int page = c.page_table[static_cast<int64_t>(b) * c.ld_table + t.pos / c.page_size];
  if (page >= 0 && page < c.n_pages) {
    const int slot = t.pos % c.page_size;
    t.k_at = page * c.k_page_stride + slot * c.k_token_stride;
    t.v_at = page * c.v_page_stride + slot * c.v_token_stride;
  }
  return t;
}

// cos and sin of the tokens' pairs into s_cs[token][pair].
__device__ __forceinline__ void rotary_angles(const RotaryParams& p, const RotaryToken* s_tok,
                                              int nt, float2* s_cs) {
  const int half = p.R / 2;
  for (int j = threadIdx.x; j < nt * half; j += kRotThreads) {
    const int t = j / half, i = j - t * half;
    const int pos = s_tok[t].pos;
    if (pos < 0) continue;
    const double turns = static_cast<double>(pos) * static_cast<double>(__ldg(p.inv_freq + i)) *
                         0.15915494309189533577;  // 1 / (2 pi)
    float sn, cs;
    sincospif(static_cast<float>(2.0 * (turns - rint(turns))), &sn, &cs);
    s_cs[j] = make_float2(p.magnitude * cs, p.magnitude * sn);
  }
}

// status[b] of the sequences, one warp per sequence (the CTAs take them in turn).
__device__ __forceinline__ void rotary_status(const RotaryParams& p) {
  const int lane = threadIdx.x & 31;
  const dspark_kv_cache_t& c = p.cache;
  const int64_t cap = static_cast<int64_t>(c.max_pages) * c.page_size;
  const int warps = gridDim.x * (kRotThreads / 32);
  for (int b = blockIdx.x * (kRotThreads / 32) + (threadIdx.x >> 5); b < p.rows.B; b += warps) {
    SeqRows s;
    int st = 0;
    if (!seq_rows(p.rows, c.kv_len, cap, b, s) || s.L < s.n) {
      st = DSPARK_SEQ_BAD_PARAM;
    } else if (s.n > 0) {
      const int p0 = (s.L - s.n) / c.page_size, p1 = (s.L - 1) / c.page_size;
      bool bad = false;
      for (int g = p0 + lane; g <= p1; g += 32) {
        const int page = c.page_table[static_cast<int64_t>(b) * c.ld_table + g];
        bad |= page < 0 || page >= c.n_pages;
      }
      if (__any_sync(0xffffffffu, bad)) st = DSPARK_SEQ_BAD_PAGE;
      if (p.rows.q_start && !packed_sole(p.rows, b, s, lane)) st |= DSPARK_SEQ_BAD_PARAM;
    }
    if (lane == 0) p.status[b] = st;
  }
}

// One CTA: p.tokens rows, every head. Vector path (kVec): every row start is 16-byte aligned
// and the pairs fall into whole 8-element vectors. A head is cut into slots of two vectors:
// the two halves of eight (i, i + R/2) pairs, or two neighbouring vectors (interleaved pairs,
// the copied rest, v). A thread keeps its slot and takes every (256 / slots)-th (token, head); its
// first one is loaded before the lengths, pages and angles are known, so that both latencies
// overlap. Memory bound: 10205 tokens of 32 + 8 + 8 heads of 128 (251 MB) take 47.6 us, 5.3 TB/s,
// 82% of the measured copy rate. Several loads in flight a thread cost more in registers (resident
// warps) than they bring: where one took 48.5 us, 2, 4 and 6 took 51.2, 54.4 and 70.6; 2 or 8
// tokens a CTA 48.8 and above 50.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kRotThreads) rotary_append_kernel(const RotaryParams p) {
  extern __shared__ __align__(16) float2 s_cs[];
  __shared__ RotaryToken s_tok[kRotMaxTokens];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int total = p.rows.q_start ? p.rows.N : p.rows.B * p.rows.N;
  const int row0 = blockIdx.x * p.tokens;
  const int nt = min(p.tokens, total - row0);
  const int Hk = p.cache.n_heads, H = p.Hq + 2 * Hk, D = p.cache.head_dim, R = p.R;
  const T* q = static_cast<const T*>(p.q.p);
  const T* k = static_cast<const T*>(p.k.p);
  const T* v = static_cast<const T*>(p.v.p);
  T* qo = static_cast<T*>(p.q_out.p);
  T* kp = static_cast<T*>(p.cache.k);
  T* vp = static_cast<T*>(p.cache.v);
  // head h of a token counts q's heads, then k's, then v's
  auto source = [&](int t, int h) {
    if (h < p.Hq) return q + row_offset(p.q, p.rows, row0 + t) + h * p.q.head_stride;
    h -= p.Hq;
    if (h < Hk) return k + row_offset(p.k, p.rows, row0 + t) + h * p.k.head_stride;
    return v + row_offset(p.v, p.rows, row0 + t) + (h - Hk) * p.v.head_stride;
  };
  // null: nothing to write
  auto target = [&](const RotaryToken& tok, int h) -> T* {
    if (tok.pos < 0) return nullptr;
    if (h < p.Hq) return qo + row_offset(p.q_out, p.rows, tok.row) + h * p.q_out.head_stride;
    h -= p.Hq;
    if (h < Hk) return tok.k_at < 0 ? nullptr : kp + tok.k_at + h * p.cache.k_head_stride;
    return tok.v_at < 0 ? nullptr : vp + tok.v_at + (h - Hk) * p.cache.v_head_stride;
  };

  const int slot = tid & ((1 << p.log_slots) - 1), stride = kRotThreads >> p.log_slots;
  const int nvec = D / 8, rvec = R / 8;
  const bool split = !p.interleaved && slot < rvec / 2;  // a pair slot of the half layout
  const bool idle = 2 * slot >= nvec;
  int t = 0, h = tid >> p.log_slots;  // this thread's (token, head)
  while (h >= H) {
    h -= H;
    ++t;
  }
  // the slot's two vectors in head h
  auto vectors = [&](int h, int& a, int& b) {
    const bool pairs = split && h < p.Hq + Hk;
    a = pairs ? slot : 2 * slot;
    b = pairs ? slot + rvec / 2 : 2 * slot + 1;
  };
  uint4 x, y;
  auto load_slot = [&](int t, int h) {
    int a, b;
    vectors(h, a, b);
    const T* src = source(t, h);
    x = *reinterpret_cast<const uint4*>(src + 8 * a);
    if (b < nvec) y = *reinterpret_cast<const uint4*>(src + 8 * b);
  };

  grid_dependency_wait();  // lengths, values and the cache come from the kernels before
  grid_dependents_launch();
  if (kVec && !idle && t < nt) load_slot(t, h);
  if (warp < nt) {
    const RotaryToken tok = rotary_token(p, row0 + warp, lane);
    if (lane == 0) s_tok[warp] = tok;
  }
  __syncthreads();
  rotary_angles(p, s_tok, nt, s_cs);
  if (p.status) rotary_status(p);
  __syncthreads();

  if (kVec) {
    if (idle) return;
    while (t < nt) {
      if (T* dst = target(s_tok[t], h)) {
        int a, b;
        vectors(h, a, b);
        uint32_t* xw = reinterpret_cast<uint32_t*>(&x);
        uint32_t* yw = reinterpret_cast<uint32_t*>(&y);
        const bool turn = h < p.Hq + Hk && (split || (p.interleaved && a < rvec));
        if (turn) {
          float2 w[8];
          const float4* cs = reinterpret_cast<const float4*>(s_cs + t * (R / 2) + 8 * slot);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float4 c = cs[j];
            w[2 * j] = make_float2(c.x, c.y);
            w[2 * j + 1] = make_float2(c.z, c.w);
          }
          if (p.interleaved) {
            // words of x are pairs 0..3 of the slot, words of y pairs 4..7
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 f = Half16<T>::up(xw[j]);
              xw[j] = Half16<T>::down(f.x * w[j].x - f.y * w[j].y, f.y * w[j].x + f.x * w[j].y);
              if (b < rvec) {
                const float2 g = Half16<T>::up(yw[j]), z = w[4 + j];
                yw[j] = Half16<T>::down(g.x * z.x - g.y * z.y, g.y * z.x + g.x * z.y);
              }
            }
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 f = Half16<T>::up(xw[j]), g = Half16<T>::up(yw[j]);
              const float2 c0 = w[2 * j], c1 = w[2 * j + 1];
              xw[j] = Half16<T>::down(f.x * c0.x - g.x * c0.y, f.y * c1.x - g.y * c1.y);
              yw[j] = Half16<T>::down(g.x * c0.x + f.x * c0.y, g.y * c1.x + f.y * c1.y);
            }
          }
        }
        *reinterpret_cast<uint4*>(dst + 8 * a) = x;
        if (b < nvec) *reinterpret_cast<uint4*>(dst + 8 * b) = y;
      }
      h += stride;
      while (h >= H) {
        h -= H;
        ++t;
      }
      if (t < nt) load_slot(t, h);
    }
  } else {
    // element path: a thread per pair, then per copied element
    const int half = R / 2, units = half + (D - R);
    for (int j = tid; j < nt * H * units; j += kRotThreads) {
      const int row = j / units, u = j - row * units, ti = row / H, hi = row - ti * H;
      T* dst = target(s_tok[ti], hi);
      if (!dst) continue;
      const T* src = source(ti, hi);
      if (u >= half) {
        const int d = R + (u - half);
        dst[d] = src[d];
        continue;
      }
      const int d1 = p.interleaved ? 2 * u : u, d2 = p.interleaved ? 2 * u + 1 : u + half;
      const T x1 = src[d1], x2 = src[d2];
      if (hi >= p.Hq + Hk) {
        dst[d1] = x1;
        dst[d2] = x2;
      } else {
        const float f = Half16<T>::up1(x1), g = Half16<T>::up1(x2);
        const float2 w = s_cs[ti * half + u];
        dst[d1] = Half16<T>::down1(f * w.x - g * w.y);
        dst[d2] = Half16<T>::down1(g * w.x + f * w.y);
      }
    }
  }
}

}  // namespace dspark
