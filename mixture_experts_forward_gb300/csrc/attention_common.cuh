// What the two attention kernels share: where a tile's rows stand, the range
// of keys they see, and the joining of a split tile's parts.
//
// A tile is a run of rows of one (sequence, cache head); row r is new token
// r / group with query head r % group of the head's group, so every head
// layout, from one query head per cache head to all of them, fills tiles alike.
#pragma once

#include "serve_internal.cuh"

namespace moe {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The smaller one; a NaN if one is.
__device__ __forceinline__ float min_nan(float a, float b) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// c * tanh(x / c), by tanh(t) = 1 - 2 / (e^(2t) + 1): absolute error about
// 2^-22 * c (k = 2 log2(e) / c; e^(2t) overflows to inf and underflows to 0 at
// the right ends).
__device__ __forceinline__ float soft_capped(float x, float k, float c) {
  const float e = exp2_approx(x * k);
  return c - 2.0f * c * rcp_approx(e + 1.0f);
}

// One tile's place in its sequence.
struct TileView {
  int b, h, first_row;     // sequence, cache head, first row of the tile
  int rows;                // rows of the tile that exist (0: nothing to do)
  int q0;                  // row of q of the sequence's first new token
  int q_len, kv_len;
  int lo, hi;              // keys that any row of the tile sees (hi <= lo: none)
};

// The keys row r (of the sequence) sees: [row_lo, row_hi).
__device__ __forceinline__ int row_hi(const AttnParams& p, const TileView& t, int tok) {
  return p.causal ? min(t.kv_len, t.kv_len - t.q_len + tok + 1) : t.kv_len;
}
// (compared before the subtraction: a window may be any int, and a sequence may have more new
// tokens than positions)
__device__ __forceinline__ int row_lo(const AttnParams& p, const TileView& t, int tok) {
  const int end = t.kv_len - t.q_len + tok + 1;
  return p.window > 0 && end > p.window ? end - p.window : 0;
}

__device__ __forceinline__ TileView tile_view(const AttnParams& p, int b, int h, int tile,
                                              int tile_rows, bool report) {
  TileView t;
  t.b = b;
  t.h = h;
  t.first_row = tile * tile_rows;
  t.q0 = __ldg(p.cu_q + b);
  t.q_len = __ldg(p.cu_q + b + 1) - t.q0;
  t.kv_len = __ldg(p.kv_lens + b);
  if (t.q0 < 0 || t.q_len < 0 || t.q_len > p.max_q || t.q0 > p.T - t.q_len) {
    if (report) set_error(p.ctrl, MOE_ERR_DEVICE_FAULT, 20);
    t.q_len = 0;
    t.rows = 0;
    t.lo = t.hi = 0;
    return t;
  }
  const int64_t room = static_cast<int64_t>(p.table_stride) << p.c.page_log2;
  if (t.kv_len < 0 || t.kv_len > room) {
    if (report) set_error(p.ctrl, MOE_ERR_DEVICE_FAULT, 21);
    t.kv_len = t.kv_len < 0 ? 0 : static_cast<int>(room);
  }
  t.rows = min(tile_rows, t.q_len * p.group - t.first_row);
  if (t.rows <= 0) {
    t.rows = 0;
    t.lo = t.hi = 0;
    return t;
  }
  t.lo = row_lo(p, t, t.first_row / p.group);
  t.hi = max(0, row_hi(p, t, (t.first_row + t.rows - 1) / p.group));
  return t;
}

// A tile's keys, cut evenly into whole key tiles over at most `parts` CTAs: the range
// of CTA `part`.  count 0: no key is seen (CTA 0 writes the empty rows).
struct Share {
  int k0, k1, n, count;          // keys [k0, k1), in n key tiles; CTAs that have some
};
__device__ __forceinline__ Share share_of(const TileView& t, int parts, int part) {
  constexpr int kTile = kTileKeys;
  Share s;
  const int base = t.lo / kTile * kTile;
  const int all = t.hi > t.lo ? (t.hi - base + kTile - 1) / kTile : 0;
  const int each = max(1, (all + parts - 1) / parts);
  s.count = (all + each - 1) / each;
  s.k0 = base + part * each * kTile;
  s.k1 = all == 0 ? s.k0 : min(t.hi, s.k0 + each * kTile);
  s.n = (s.k1 - s.k0 + kTile - 1) / kTile;
  return s;
}

// Row r's place in out and lse.
__device__ __forceinline__ __nv_bfloat16* out_row(const AttnParams& p, const TileView& t, int r) {
  const int rr = t.first_row + r, tok = rr / p.group;
  return p.out + static_cast<int64_t>(t.q0 + tok) * p.o_st +
         static_cast<int64_t>(t.h * p.group + rr - tok * p.group) * p.o_sh;
}
__device__ __forceinline__ float* lse_at(const AttnParams& p, const TileView& t, int r) {
  const int rr = t.first_row + r, tok = rr / p.group;
  return p.lse + static_cast<int64_t>(t.q0 + tok) * p.q_heads + t.h * p.group + rr -
         tok * p.group;
}

__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.0f ? __int_as_float(0xff800000) : (m + log2f(l)) * kLn2;
}

// A part's result: rows x D sums, then rows maxima, then rows sums of weights
// (the maximum m in log2 units; sums relative to 2^m).
template <int D>
__host__ __device__ __forceinline__ int64_t partial_floats(int rows) {
  return static_cast<int64_t>(rows) * (D + 2);
}

// Called by `threads` threads of the CTA after its part has been written: the last CTA of
// the tile to arrive joins the parts, in their order, and writes out and lse.  `parts`: the
// first of the tile's `count` parts, one after another, part_rows the rows that each has
// room for; `counter` is the tile's own; named barrier `bar` joins the threads; `weights` is
// shared memory for count * part_rows floats.  First a thread per row turns the parts' maxima and sums into
// weights, then all threads stream the parts, kAhead 16-byte loads in flight each.
template <int D>
__device__ __forceinline__ void join_parts(const AttnParams& p, const TileView& t,
                                           const float* parts, unsigned* counter, int part_rows,
                                           int count, int tid, int threads, int bar,
                                           float* weights, int* s_flag) {
  constexpr int kAhead = 8;
  __threadfence();
  named_bar_sync(bar, threads);
  if (tid == 0) {
    const unsigned prev = atomicAdd(counter, 1u);
    const int last = prev == static_cast<unsigned>(count - 1);
    if (last) *counter = 0u;   // every part has arrived
    *s_flag = last;
  }
  named_bar_sync(bar, threads);
  if (!*s_flag) return;
  __threadfence();
  const int64_t stride = partial_floats<D>(part_rows);
  const float* ml = parts + static_cast<int64_t>(part_rows) * D;
  const float ninf = __int_as_float(0xff800000);
  for (int r = tid; r < t.rows; r += threads) {
    float m = ninf, l = 0.0f;
    for (int s0 = 0; s0 < count; s0 += kAhead) {
      float pm[kAhead], pl[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const bool x = s0 + j < count;
        pm[j] = x ? __ldcg(ml + (s0 + j) * stride + r) : ninf;
        pl[j] = x ? __ldcg(ml + (s0 + j) * stride + part_rows + r) : 0.0f;
      }
      float top = m;
#pragma unroll
      for (int j = 0; j < kAhead; ++j) top = fmaxf(top, pm[j]);
      const float ref = top == ninf ? 0.0f : top;
      l *= exp2_approx(m - ref);
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (s0 + j < count) {
          l = fmaf(exp2_approx(pm[j] - ref), pl[j], l);
          weights[(s0 + j) * part_rows + r] = pm[j];
        }
      m = top;
    }
    const float ref = m == ninf ? 0.0f : m;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    for (int s = 0; s < count; ++s)
      weights[s * part_rows + r] = exp2_approx(weights[s * part_rows + r] - ref) * inv;
    if (p.lse != nullptr) *lse_at(p, t, r) = lse_of(m, l);
  }
  named_bar_sync(bar, threads);
  for (int i = tid; i < t.rows * (D / 4); i += threads) {
    const int r = i / (D / 4), d = (i % (D / 4)) * 4;
    const float* src = parts + static_cast<int64_t>(r) * D + d;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < count; s0 += kAhead) {
      float4 x[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (s0 + j < count) x[j] = __ldcg(reinterpret_cast<const float4*>(src + (s0 + j) * stride));
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (s0 + j < count) {
          const float w = weights[(s0 + j) * part_rows + r];
          o.x = fmaf(w, x[j].x, o.x);
          o.y = fmaf(w, x[j].y, o.y);
          o.z = fmaf(w, x[j].z, o.z);
          o.w = fmaf(w, x[j].w, o.w);
        }
    }
    __nv_bfloat162 a = __floats2bfloat162_rn(o.x, o.y);
    __nv_bfloat162 b = __floats2bfloat162_rn(o.z, o.w);
    uint2 u;
    u.x = *reinterpret_cast<uint32_t*>(&a);
    u.y = *reinterpret_cast<uint32_t*>(&b);
    *reinterpret_cast<uint2*>(out_row(p, t, r) + d) = u;
  }
}

// The power of two that brings a row's largest element into [2^8, 2^9), and its
// reciprocal.
__device__ __forceinline__ void row_pow2(float amax, float& mul, float& inv) {
  int ex = static_cast<int>((__float_as_uint(amax) >> 23) & 255u);
  ex = max(ex, 9);
  mul = __uint_as_float(static_cast<uint32_t>(262 - ex) << 23);
  inv = __uint_as_float(static_cast<uint32_t>(ex - 8) << 23);
}

}  // namespace moe
