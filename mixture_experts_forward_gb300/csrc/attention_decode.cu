// Attention of a few rows over the paged cache: single tokens (decode) and
// short drafted runs.
//
// A tile is at most 16 rows (new tokens x query heads of one cache head), so
// every key and value is read once and used 16 times at most: the kernel is
// bound by HBM, and its work is to keep enough loads in flight and stay under
// the bytes' time.  Each warp walks its own groups of keys (32 of 128 codes, 16
// of 128 bf16) through a private ring of cp.async stages, so no barrier
// joins the warps until the end.  Products are mma.sync m16n8k16 (a 128-row
// tensor-core tile would be filled to an eighth): both operands come from shared
// memory as 16-byte pieces of a row, because the contraction's order is free:
// lane (g, t) takes piece t of key g in the first product and piece g of keys
// 2t, 2t+1 in the second, and the query and the output columns are permuted to
// match.  E4M3 codes become binary16 (exact) in registers, the scales
// apply in binary32: per key to the score, and per key inside the weight
// (value_scale).  BF16 caches split the weights in two bf16 terms, so nothing
// but the output is rounded to bf16: the extra product is free under the loads.
//
// The tile's keys are cut into parts over CTAs; the last CTA to finish a
// tile joins the parts in order (join_parts), in the same launch.
#include "attention_common.cuh"

namespace moe {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;

template <int D, bool kFP8>
struct DecodeShape {
  static constexpr int kRowBytes = kFP8 ? D : 2 * D;
  static constexpr int kCpr = kRowBytes / 16;               // 16-byte pieces per row
  static constexpr int kKeys = (!kFP8 && D == 128) ? 16 : 32;  // keys per group
  static constexpr int kKvBytes = kKeys * kRowBytes;
  static constexpr int kScaleBytes = kFP8 ? kKeys * 16 : 0;  // ks, vs, then (log2 vs, 1/vs)
  static constexpr int kStageBytes = 2 * kKvBytes + kScaleBytes;
  static constexpr int kStages = kKvBytes >= 4096 ? 3 : 4;
  static constexpr int kSmem = kWarps * kStages * kStageBytes;
  static_assert(kSmem >= kWarps * kDecodeRows * (D + 2) * 4, "the join fits the ring");
};

// The piece of row `row` that holds its 16 bytes number c, such that the 8
// lanes of each phase of a 16-byte shared load hit different banks in both
// products (keys g, g+1 x pieces t; keys 2t x pieces g, g+1).
template <int kRowBytes>
__device__ __forceinline__ int piece_at(int row, int c) {
  if constexpr (kRowBytes == 64) return c ^ ((row >> 1) & 3);
  return c ^ ((((row >> 1) & 3) << 1) ^ ((row & 1) << 2));
}

__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_async4_or_zero(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 4 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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

template <bool kF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (kF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

template <int D, bool kFP8>
__global__ void __launch_bounds__(kThreads, 2) decode_kernel(const AttnParams p) {
  using S = DecodeShape<D, kFP8>;
  constexpr int kSteps = D / 16;       // k16 steps of the first product
  constexpr int kNt = S::kKeys / 8;    // key tiles of 8
  constexpr int kDt = D / 8;           // output column tiles of 8
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_flag;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  const int64_t tile = blockIdx.x;
  const int rt = static_cast<int>(tile % p.row_tiles);
  const int bh = static_cast<int>(tile / p.row_tiles);
  const int b = bh / p.c.heads, h = bh - b * p.c.heads;
  const int part = blockIdx.y;
  const TileView t = tile_view(p, b, h, rt, kDecodeRows, part == 0 && rt == 0 && tid == 0);
  if (t.rows == 0) return;
  const Parts parts = tile_parts(p, t, 32);
  if (part >= max(1, parts.count)) return;
  const int k0 = parts.base + part * p.chunk;                       // this CTA's keys
  const int k1 = part + 1 >= parts.count ? t.hi : k0 + p.chunk;
  const int keys = parts.count == 0 ? 0 : k1 - k0;
  const int groups = (keys + S::kKeys - 1) / S::kKeys;

  // ---- the query: rows g and g + 8, in the order of the permuted pieces
  uint32_t qa[kSteps][4];
  int hi0 = 0, hi1 = 0, lo0 = 0, lo1 = 0;
  float f0, f1;                        // row factors of the scores
  const float sc = p.softcap > 0.0f ? p.scale : p.scale * kLog2e;
  {
    const int r0 = t.first_row + g, r1 = r0 + 8;
    const int tok0 = r0 / p.group, tok1 = r1 / p.group;
    const bool v0 = g < t.rows, v1 = g + 8 < t.rows;
    if (v0) {
      hi0 = row_hi(p, t, tok0);
      lo0 = row_lo(p, t, tok0);
    }
    if (v1) {
      hi1 = row_hi(p, t, tok1);
      lo1 = row_lo(p, t, tok1);
    }
    const __nv_bfloat16* q0 = p.q + static_cast<int64_t>(t.q0 + tok0) * p.q_st +
                              static_cast<int64_t>(h * p.group + r0 - tok0 * p.group) * p.q_sh;
    const __nv_bfloat16* q1 = p.q + static_cast<int64_t>(t.q0 + tok1) * p.q_st +
                              static_cast<int64_t>(h * p.group + r1 - tok1 * p.group) * p.q_sh;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int d = kFP8 ? (t4 + 4 * (s >> 2)) * 16 + 4 * (s & 3)
                         : (t4 + 4 * (s >> 1)) * 8 + 4 * (s & 1);
      const uint2 z = make_uint2(0u, 0u);
      const uint2 x = v0 ? __ldg(reinterpret_cast<const uint2*>(q0 + d)) : z;
      const uint2 y = v1 ? __ldg(reinterpret_cast<const uint2*>(q1 + d)) : z;
      qa[s][0] = x.x;
      qa[s][1] = y.x;
      qa[s][2] = x.y;
      qa[s][3] = y.y;
    }
    f0 = f1 = sc;
    if constexpr (kFP8) {
      float a0 = 0.0f, a1 = 0.0f;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        a0 = fmaxf(a0, fmaxf(fmaxf(fabsf(bf16_lo(qa[s][0])), fabsf(bf16_hi(qa[s][0]))),
                             fmaxf(fabsf(bf16_lo(qa[s][2])), fabsf(bf16_hi(qa[s][2])))));
        a1 = fmaxf(a1, fmaxf(fmaxf(fabsf(bf16_lo(qa[s][1])), fabsf(bf16_hi(qa[s][1]))),
                             fmaxf(fabsf(bf16_lo(qa[s][3])), fabsf(bf16_hi(qa[s][3])))));
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        a0 = fmaxf(a0, __shfl_xor_sync(0xffffffffu, a0, o));
        a1 = fmaxf(a1, __shfl_xor_sync(0xffffffffu, a1, o));
      }
      float m0, m1, i0, i1;
      row_pow2(a0, m0, i0);
      row_pow2(a1, m1, i1);
      f0 *= i0;
      f1 *= i1;
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float m = (i & 1) ? m1 : m0;
          qa[s][i] = pack_f16(bf16_lo(qa[s][i]) * m, bf16_hi(qa[s][i]) * m);
        }
    }
  }

  // ---- the ring of this warp: groups w, w + kWarps, ...
  const uint32_t ring = smem_u32(smem) + w * (S::kStages * S::kStageBytes);
  const int key_lo = max(k0, t.lo), key_hi = k1;
  const int32_t* table = p.table + static_cast<int64_t>(b) * p.table_stride;
  const int page_mask = (1 << p.c.page_log2) - 1;
  // lanes 0..15 and 16..31 hold the page of a group's first and second 16 keys
  auto fetch_page = [&](int group) -> int {
    const int key = k0 + group * S::kKeys + (lane & 16);
    return (group < groups && key < key_hi) ? __ldg(table + (key >> p.c.page_log2)) : -1;
  };
  auto load_group = [&](int group, int stage, int page) {
    if (group < groups) {
      const int kb = k0 + group * S::kKeys;
      const uint32_t dst = ring + stage * S::kStageBytes;
      if (page >= p.c.num_pages || (page < 0 && kb + (lane & 16) < key_hi)) {
        set_error(p.ctrl, MOE_ERR_DEVICE_FAULT, 22);
        page = -1;
      }
      int64_t base[2];
      bool have[2];
#pragma unroll
      for (int i = 0; i < S::kKeys / 16; ++i) {
        const int pg = __shfl_sync(0xffffffffu, page, 16 * i);
        have[i] = pg >= 0;
        base[i] = ((static_cast<int64_t>(max(pg, 0)) * p.c.heads + h) << p.c.page_log2) +
                  ((kb + 16 * i) & page_mask);
      }
#pragma unroll
      for (int i = 0; i < S::kCpr * S::kKeys / 32; ++i) {
        const int row = (i * 32 + lane) / S::kCpr, c = (i * 32 + lane) % S::kCpr;
        const int half = i * 32 / S::kCpr / 16;
        const bool valid = have[half] && kb + row >= key_lo && kb + row < key_hi;
        const int64_t off = (base[half] + (valid ? row - half * 16 : 0)) * S::kRowBytes + c * 16;
        const uint32_t at = dst + row * S::kRowBytes + piece_at<S::kRowBytes>(row, c) * 16;
        cp_async16_or_zero(at, p.c.k + off, valid);
        cp_async16_or_zero(at + S::kKvBytes, p.c.v + off, valid);
      }
      if constexpr (kFP8) {
        static_assert(!kFP8 || S::kKeys == 32, "a key per lane");
        const bool second = lane >= 16;
        const bool valid = (second ? have[1] : have[0]) && kb + lane >= key_lo && kb + lane < key_hi;
        const int64_t at = (second ? base[1] : base[0]) + (valid ? (lane & 15) : 0);
        const uint32_t sdst = dst + 2 * S::kKvBytes + lane * 4;
        cp_async4_or_zero(sdst, p.c.k_scales + at, valid);
        cp_async4_or_zero(sdst + S::kKeys * 4, p.c.v_scales + at, valid);
      }
    }
    cp_async_commit();
  };

  float o[kDt][4];
#pragma unroll
  for (int i = 0; i < kDt; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) o[i][j] = 0.0f;
  const float ninf = __int_as_float(0xff800000);
  float m0 = ninf, m1 = ninf, l0 = 0.0f, l1 = 0.0f;

  int pages[S::kStages - 1];
#pragma unroll
  for (int i = 0; i < S::kStages - 1; ++i) pages[i] = fetch_page(w + i * kWarps);
  int page_next = fetch_page(w + (S::kStages - 1) * kWarps);
#pragma unroll
  for (int i = 0; i < S::kStages - 1; ++i) load_group(w + i * kWarps, i, pages[i]);

  const float cap = p.softcap, cap_k = cap > 0.0f ? 2.0f * kLog2e / cap : 0.0f;
  const int lo_max = t.lo == 0 && p.window == 0 ? 0
                                                : row_lo(p, t, (t.first_row + t.rows - 1) / p.group);
  const int hi_min = row_hi(p, t, t.first_row / p.group);

  int stage = 0, fill = S::kStages - 1;
  for (int group = w; group < groups; group += kWarps) {
    cp_async_wait<S::kStages - 2>();
    __syncwarp();
    {  // the stage read in the last iteration is free: every lane has passed it
      const int ahead = group + (S::kStages - 1) * kWarps;
      load_group(ahead, fill, page_next);
      page_next = fetch_page(ahead + kWarps);
      fill = fill + 1 == S::kStages ? 0 : fill + 1;
    }
    const int kb = k0 + group * S::kKeys;
    const uint32_t ks_at = ring + stage * S::kStageBytes;
    const uint32_t vs_at = ks_at + S::kKvBytes;
    const uint32_t sc_at = vs_at + S::kKvBytes;
    stage = stage + 1 == S::kStages ? 0 : stage + 1;
    if constexpr (kFP8) {
      // this lane's key: log2 and reciprocal of its value scale
      float vs;
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(vs) : "r"(sc_at + S::kKeys * 4 + lane * 4));
      vs = value_scale(vs);
      asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(sc_at + S::kKeys * 8 + lane * 8),
                   "f"(log2f(vs)), "f"(1.0f / vs)
                   : "memory");
      __syncwarp();
    }
    // ---- scores
    float s[kNt][4];
#pragma unroll
    for (int nb = 0; nb < kNt; ++nb) {
#pragma unroll
      for (int j = 0; j < 4; ++j) s[nb][j] = 0.0f;
      const int row = nb * 8 + g;
#pragma unroll
      for (int i = 0; i < S::kCpr / 4; ++i) {
        const uint4 x = lds128(ks_at + row * S::kRowBytes +
                               piece_at<S::kRowBytes>(row, t4 + 4 * i) * 16);
        if constexpr (kFP8) {
          const uint32_t ww[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma16816<true>(s[nb], qa[4 * i + j], e4m3x2_to_f16x2(static_cast<uint16_t>(ww[j])),
                           e4m3x2_to_f16x2(static_cast<uint16_t>(ww[j] >> 16)));
        } else {
          mma16816<false>(s[nb], qa[2 * i], x.x, x.y);
          mma16816<false>(s[nb], qa[2 * i + 1], x.z, x.w);
        }
      }
    }
    // ---- to log2 units, masked
    const bool whole = kb >= lo_max && kb + S::kKeys <= min(hi_min, key_hi);
    float iv[kNt][2];
    float x0 = ninf, x1 = ninf;
#pragma unroll
    for (int nb = 0; nb < kNt; ++nb) {
      float k0s = 1.0f, k1s = 1.0f, lv0 = 0.0f, lv1 = 0.0f;
      if constexpr (kFP8) {
        const uint2 ks = lds64(sc_at + (nb * 8 + 2 * t4) * 4);
        const uint4 v = lds128(sc_at + S::kKeys * 8 + (nb * 8 + 2 * t4) * 8);
        k0s = __uint_as_float(ks.x);
        k1s = __uint_as_float(ks.y);
        lv0 = __uint_as_float(v.x);
        iv[nb][0] = __uint_as_float(v.y);
        lv1 = __uint_as_float(v.z);
        iv[nb][1] = __uint_as_float(v.w);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float x = s[nb][j] * (j < 2 ? f0 : f1);
        if constexpr (kFP8) x *= (j & 1) ? k1s : k0s;
        if (cap > 0.0f) x = soft_capped(x, cap_k, cap) * kLog2e;
        if constexpr (kFP8) x += (j & 1) ? lv1 : lv0;
        if (!whole) {
          const int key = kb + nb * 8 + 2 * t4 + (j & 1);
          const int a = j < 2 ? max(lo0, key_lo) : max(lo1, key_lo);
          const int z = j < 2 ? min(hi0, key_hi) : min(hi1, key_hi);
          if (key < a || key >= z) x = ninf;
        }
        s[nb][j] = x;
        if (j < 2) x0 = fmaxf(x0, x); else x1 = fmaxf(x1, x);
      }
    }
#pragma unroll
    for (int k = 1; k < 4; k <<= 1) {
      x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, k));
      x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, k));
    }
    // ---- running maximum and sums
    x0 = fmaxf(x0, m0);
    x1 = fmaxf(x1, m1);
    if (__any_sync(0xffffffffu, x0 > m0 || x1 > m1)) {
      const float c0 = m0 == x0 ? 1.0f : exp2_approx(m0 - x0);
      const float c1 = m1 == x1 ? 1.0f : exp2_approx(m1 - x1);
      m0 = x0;
      m1 = x1;
      l0 *= c0;
      l1 *= c1;
#pragma unroll
      for (int i = 0; i < kDt; ++i) {
        o[i][0] *= c0;
        o[i][1] *= c0;
        o[i][2] *= c1;
        o[i][3] *= c1;
      }
    }
    const float ref0 = m0 == ninf ? 0.0f : m0, ref1 = m1 == ninf ? 0.0f : m1;
#pragma unroll
    for (int nb = 0; nb < kNt; ++nb)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float e = exp2_approx(s[nb][j] - (j < 2 ? ref0 : ref1));
        s[nb][j] = e;
        float& l = j < 2 ? l0 : l1;
        if constexpr (kFP8) l = fmaf(e, iv[nb][j & 1], l); else l += e;
      }
    // ---- weights times values
#pragma unroll
    for (int kk = 0; kk < S::kKeys / 16; ++kk) {
      const float(&a)[4] = s[2 * kk];
      const float(&c)[4] = s[2 * kk + 1];
      uint32_t pa[4], pl[4];
      if constexpr (kFP8) {
        pa[0] = pack_f16(a[0], a[1]);
        pa[1] = pack_f16(a[2], a[3]);
        pa[2] = pack_f16(c[0], c[1]);
        pa[3] = pack_f16(c[2], c[3]);
      } else {
        pa[0] = pack_bf16(a[0], a[1]);
        pa[1] = pack_bf16(a[2], a[3]);
        pa[2] = pack_bf16(c[0], c[1]);
        pa[3] = pack_bf16(c[2], c[3]);
        pl[0] = pack_bf16(a[0] - bf16_lo(pa[0]), a[1] - bf16_hi(pa[0]));
        pl[1] = pack_bf16(a[2] - bf16_lo(pa[1]), a[3] - bf16_hi(pa[1]));
        pl[2] = pack_bf16(c[0] - bf16_lo(pa[2]), c[1] - bf16_hi(pa[2]));
        pl[3] = pack_bf16(c[2] - bf16_lo(pa[3]), c[3] - bf16_hi(pa[3]));
      }
      const int r = kk * 16 + 2 * t4;
      auto at = [&](int row, int c16) {
        return vs_at + row * S::kRowBytes + piece_at<S::kRowBytes>(row, c16) * 16;
      };
      if constexpr (kFP8) {
        constexpr int kWords = D / 32;   // 4-code words of this lane's columns in each row
        uint32_t v[4][kWords];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = r + (i & 1) + (i >> 1) * 8;
          if constexpr (D == 128) {
            const uint4 x = lds128(at(row, g));
            v[i][0] = x.x;
            v[i][1] = x.y;
            v[i][2] = x.z;
            v[i][3] = x.w;
          } else {
            const uint2 x = lds64(at(row, g >> 1) + (g & 1) * 8);
            v[i][0] = x.x;
            v[i][1] = x.y;
          }
        }
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
          const uint32_t x0w = __byte_perm(v[0][i], v[1][i], 0x5140);
          const uint32_t x1w = __byte_perm(v[0][i], v[1][i], 0x7362);
          const uint32_t y0w = __byte_perm(v[2][i], v[3][i], 0x5140);
          const uint32_t y1w = __byte_perm(v[2][i], v[3][i], 0x7362);
          mma16816<true>(o[4 * i], pa, e4m3x2_to_f16x2(static_cast<uint16_t>(x0w)),
                         e4m3x2_to_f16x2(static_cast<uint16_t>(y0w)));
          mma16816<true>(o[4 * i + 1], pa, e4m3x2_to_f16x2(static_cast<uint16_t>(x0w >> 16)),
                         e4m3x2_to_f16x2(static_cast<uint16_t>(y0w >> 16)));
          mma16816<true>(o[4 * i + 2], pa, e4m3x2_to_f16x2(static_cast<uint16_t>(x1w)),
                         e4m3x2_to_f16x2(static_cast<uint16_t>(y1w)));
          mma16816<true>(o[4 * i + 3], pa, e4m3x2_to_f16x2(static_cast<uint16_t>(x1w >> 16)),
                         e4m3x2_to_f16x2(static_cast<uint16_t>(y1w >> 16)));
        }
      } else {
#pragma unroll
        for (int half = 0; half < D / 64; ++half) {
          uint32_t v[4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = r + (i & 1) + (i >> 1) * 8;
            const uint4 x = lds128(at(row, g + 8 * half));
            v[i][0] = x.x;
            v[i][1] = x.y;
            v[i][2] = x.z;
            v[i][3] = x.w;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t b00 = __byte_perm(v[0][i], v[1][i], 0x5410);
            const uint32_t b01 = __byte_perm(v[2][i], v[3][i], 0x5410);
            const uint32_t b10 = __byte_perm(v[0][i], v[1][i], 0x7632);
            const uint32_t b11 = __byte_perm(v[2][i], v[3][i], 0x7632);
            mma16816<false>(o[8 * half + 2 * i], pa, b00, b01);
            mma16816<false>(o[8 * half + 2 * i], pl, b00, b01);
            mma16816<false>(o[8 * half + 2 * i + 1], pa, b10, b11);
            mma16816<false>(o[8 * half + 2 * i + 1], pl, b10, b11);
          }
        }
      }
    }
  }

  // ---- join the warps (in the ring's memory), then the parts
#pragma unroll
  for (int k = 1; k < 4; k <<= 1) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, k);
    l1 += __shfl_xor_sync(0xffffffffu, l1, k);
  }
  cp_async_wait<0>();
  __syncthreads();
  float* so = reinterpret_cast<float*>(smem);                 // [warp][16][D]
  float* sm = so + kWarps * kDecodeRows * D;                  // [warp][16] maxima, then sums
  float* sl = sm + kWarps * kDecodeRows;
  {
    float* mine = so + w * kDecodeRows * D;
#pragma unroll
    for (int i = 0; i < kDt; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = 2 * t4 + (j & 1);
        const int d = (!kFP8 && D == 128) ? (i >> 3) * 64 + n * 8 + (i & 7) : n * kDt + i;
        mine[(g + (j >> 1) * 8) * D + d] = o[i][j];
      }
    if (t4 == 0) {
      sm[w * kDecodeRows + g] = m0;
      sm[w * kDecodeRows + g + 8] = m1;
      sl[w * kDecodeRows + g] = l0;
      sl[w * kDecodeRows + g + 8] = l1;
    }
  }
  __syncthreads();
  const bool whole_tile = parts.count <= 1;
  float* dst = p.partial + (tile * p.splits + part) * partial_floats<D>(kDecodeRows);
  for (int i = tid; i < t.rows * (D / 4); i += kThreads) {
    const int r = i / (D / 4), d = (i % (D / 4)) * 4;
    float m = ninf;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) m = fmaxf(m, sm[k * kDecodeRows + r]);
    const float ref = m == ninf ? 0.0f : m;
    float l = 0.0f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      const float e = exp2_approx(sm[k * kDecodeRows + r] - ref);
      const float4 x = *reinterpret_cast<const float4*>(so + (k * kDecodeRows + r) * D + d);
      l = fmaf(e, sl[k * kDecodeRows + r], l);
      acc.x = fmaf(e, x.x, acc.x);
      acc.y = fmaf(e, x.y, acc.y);
      acc.z = fmaf(e, x.z, acc.z);
      acc.w = fmaf(e, x.w, acc.w);
    }
    if (whole_tile) {
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      uint2 u;
      u.x = pack_bf16(acc.x * inv, acc.y * inv);
      u.y = pack_bf16(acc.z * inv, acc.w * inv);
      *reinterpret_cast<uint2*>(out_row(p, t, r) + d) = u;
      if (d == 0 && p.lse != nullptr) *lse_at(p, t, r) = lse_of(m, l);
    } else {
      *reinterpret_cast<float4*>(dst + r * D + d) = acc;
      if (d == 0) {
        dst[kDecodeRows * D + r] = m;
        dst[kDecodeRows * (D + 1) + r] = l;
      }
    }
  }
  if (!whole_tile) join_parts<D>(p, t, tile, kDecodeRows, parts.count, tid, kThreads, 0,
                                     &s_flag);
}

template <int D, bool kFP8>
cudaError_t launch_t(const AttnParams& p, cudaStream_t stream) {
  using S = DecodeShape<D, kFP8>;
  cudaError_t e = cudaFuncSetAttribute(decode_kernel<D, kFP8>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(p.B) * p.c.heads * p.row_tiles, p.splits);
  decode_kernel<D, kFP8><<<grid, kThreads, S::kSmem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention_decode(const AttnParams& p, int head_dim, bool fp8,
                                    cudaStream_t stream) {
  if (head_dim == 128) return fp8 ? launch_t<128, true>(p, stream) : launch_t<128, false>(p, stream);
  return fp8 ? launch_t<64, true>(p, stream) : launch_t<64, false>(p, stream);
}

}  // namespace moe
