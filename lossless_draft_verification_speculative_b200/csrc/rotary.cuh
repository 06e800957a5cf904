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
constexpr int kRotMaxTokens = 4;  // tokens per CTA

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

// Which sequence a row belongs to, its position and its slot, found by one warp: block rows by
// division, packed rows by a 32-way search of the non-decreasing q_start (one load and ballot
// per factor of 32 in B). Ill-formed starts give some sequence or none, and seq_rows refuses
// those out of range, so nothing is read outside the arrays.
__device__ __forceinline__ RotaryToken rotary_token(const RotaryParams& p, int row, int lane) {
  RotaryToken t{row, -1, -1, -1};
  const dspark_kv_cache_t& c = p.cache;
  int b;
  if (p.rows.q_start) {
    // the largest b in [0, B) with q_start[b] <= row, or -1
    int lo = -1, hi = p.rows.B;
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32;
      const int at = lo + (lane + 1) * step;
      const bool le = at < hi && p.rows.q_start[at] <= row;
      const int cnt = __popc(__ballot_sync(0xffffffffu, le));
      const int nlo = lo + cnt * step;
      hi = min(hi, nlo + step);
      lo = nlo;
    }
    b = lo;
  } else {
    b = row / p.rows.N;
  }
  if (b < 0) return t;
  SeqRows s;
  const int64_t cap = static_cast<int64_t>(c.max_pages) * c.page_size;
  if (!seq_rows(p.rows, c.kv_len, cap, b, s) || s.L < s.n) return t;
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
    }
    if (lane == 0) p.status[b] = st;
  }
}

// One CTA: p.tokens rows, every head. Vector path (kVec): every row start is 16-byte aligned
// and the pairs fall into whole 8-element vectors. A head is cut into slots of two vectors:
// the two halves of eight (i, i + R/2) pairs, or two neighbouring vectors (interleaved pairs,
// the copied rest, v); the thread keeps its slot, and its eight cos/sin, over a token's heads.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kRotThreads) rotary_append_kernel(const RotaryParams p) {
  extern __shared__ float2 s_cs[];
  __shared__ RotaryToken s_tok[kRotMaxTokens];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int total = p.rows.q_start ? p.rows.N : p.rows.B * p.rows.N;
  const int row0 = blockIdx.x * p.tokens;
  const int nt = min(p.tokens, total - row0);

  grid_dependency_wait();  // lengths, values and the cache come from the kernels before
  grid_dependents_launch();
  if (warp < nt) {
    const RotaryToken t = rotary_token(p, row0 + warp, lane);
    if (lane == 0) s_tok[warp] = t;
  }
  __syncthreads();
  rotary_angles(p, s_tok, nt, s_cs);
  if (p.status) rotary_status(p);
  __syncthreads();

  const int Hk = p.cache.n_heads, H = p.Hq + 2 * Hk, D = p.cache.head_dim, R = p.R;
  const T* q = static_cast<const T*>(p.q.p);
  const T* k = static_cast<const T*>(p.k.p);
  const T* v = static_cast<const T*>(p.v.p);
  T* qo = static_cast<T*>(p.q_out.p);
  T* kp = static_cast<T*>(p.cache.k);
  T* vp = static_cast<T*>(p.cache.v);
  for (int t = 0; t < nt; ++t) {
    const RotaryToken tok = s_tok[t];
    if (tok.pos < 0) continue;
    const float2* cs = s_cs + t * (R / 2);
    const int64_t q_at = row_offset(p.q, p.rows, tok.row);
    const int64_t o_at = row_offset(p.q_out, p.rows, tok.row);
    const int64_t k_at = row_offset(p.k, p.rows, tok.row);
    const int64_t v_at = row_offset(p.v, p.rows, tok.row);
    // the source and destination of head h (q, then k, then v); false: nothing to write
    auto rows_of = [&](int h, const T*& src, T*& dst) {
      if (h < p.Hq) {
        src = q + q_at + h * p.q.head_stride;
        dst = qo + o_at + h * p.q_out.head_stride;
        return true;
      }
      h -= p.Hq;
      if (h < Hk) {
        src = k + k_at + h * p.k.head_stride;
        dst = kp + tok.k_at + h * p.cache.k_head_stride;
        return tok.k_at >= 0;
      }
      h -= Hk;
      src = v + v_at + h * p.v.head_stride;
      dst = vp + tok.v_at + h * p.cache.v_head_stride;
      return tok.v_at >= 0;
    };
    if (kVec) {
      const int slot = tid & ((1 << p.log_slots) - 1);
      const int nvec = D / 8, rvec = R / 8;
      if (2 * slot >= nvec) continue;
      const bool split = !p.interleaved && slot < rvec / 2;  // a pair slot of the half layout
      const int va = split ? slot : 2 * slot, vb = split ? slot + rvec / 2 : 2 * slot + 1;
      const bool has_b = vb < nvec;
      float2 w[8];
      const int pair0 = 8 * slot;
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = pair0 + i < R / 2 ? cs[pair0 + i] : make_float2(1.f, 0.f);
      const int stride = kRotThreads >> p.log_slots;
#pragma unroll 2
      for (int h = tid >> p.log_slots; h < H; h += stride) {
        const T* src;
        T* dst;
        if (!rows_of(h, src, dst)) continue;
        const bool is_v = h >= p.Hq + Hk;
        const int a0 = is_v ? 2 * slot : va, b0 = is_v ? 2 * slot + 1 : vb;
        const bool hb = is_v ? 2 * slot + 1 < nvec : has_b;
        uint4 x = *reinterpret_cast<const uint4*>(src + 8 * a0);
        uint4 y = hb ? *reinterpret_cast<const uint4*>(src + 8 * b0) : make_uint4(0, 0, 0, 0);
        uint32_t* xw = reinterpret_cast<uint32_t*>(&x);
        uint32_t* yw = reinterpret_cast<uint32_t*>(&y);
        if (!is_v) {
          if (p.interleaved) {
            // words of x are pairs 0..3 of the slot, words of y pairs 4..7
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (a0 < rvec) {
                const float2 f = Half16<T>::up(xw[i]);
                xw[i] = Half16<T>::down(f.x * w[i].x - f.y * w[i].y, f.y * w[i].x + f.x * w[i].y);
              }
              if (b0 < rvec) {
                const float2 f = Half16<T>::up(yw[i]);
                yw[i] = Half16<T>::down(f.x * w[4 + i].x - f.y * w[4 + i].y,
                                        f.y * w[4 + i].x + f.x * w[4 + i].y);
              }
            }
          } else if (split) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 f = Half16<T>::up(xw[i]), g = Half16<T>::up(yw[i]);
              const float2 c0 = w[2 * i], c1 = w[2 * i + 1];
              xw[i] = Half16<T>::down(f.x * c0.x - g.x * c0.y, f.y * c1.x - g.y * c1.y);
              yw[i] = Half16<T>::down(g.x * c0.x + f.x * c0.y, g.y * c1.x + f.y * c1.y);
            }
          }
        }
        *reinterpret_cast<uint4*>(dst + 8 * a0) = x;
        if (hb) *reinterpret_cast<uint4*>(dst + 8 * b0) = y;
      }
    } else {
      // element path: a thread per pair, then per copied element
      const int half = R / 2, units = half + (D - R);
      for (int j = tid; j < H * units; j += kRotThreads) {
        const int h = j / units, u = j - h * units;
        const T* src;
        T* dst;
        if (!rows_of(h, src, dst)) continue;
        if (u >= half) {
          const int d = R + (u - half);
          dst[d] = src[d];
          continue;
        }
        const int d1 = p.interleaved ? 2 * u : u, d2 = p.interleaved ? 2 * u + 1 : u + half;
        const T x1 = src[d1], x2 = src[d2];
        if (h >= p.Hq + Hk) {
          dst[d1] = x1;
          dst[d2] = x2;
        } else {
          const float a = Half16<T>::up1(x1), b = Half16<T>::up1(x2);
          const float2 w = cs[u];
          dst[d1] = Half16<T>::down1(a * w.x - b * w.y);
          dst[d2] = Half16<T>::down1(b * w.x + a * w.y);
        }
      }
    }
  }
}

}  // namespace dspark
