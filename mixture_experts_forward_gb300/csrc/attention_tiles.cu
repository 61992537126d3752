// Attention of many rows over the paged cache: chunks of prompts, whole
// prompts and drafted runs.
//
// A CTA takes up to 256 rows (new tokens x query heads of one cache head) as
// two tiles of 128, and walks the keys they see in tiles of 128.  Both products
// run on tcgen05 with their results in tensor memory: S = Q K^T (both operands
// in shared memory) and O += P V with P read from tensor memory, where the
// softmax threads leave it in place of S, and V as it lies in the cache
// (keys x channels, the MN-major form of the B operand).  Per pair of row tiles
// and key tile the tensor core works 4 * 128 * 128 * D * 2 operations, about
// 2 * 1024 cycles at D = 128, and the exponentials take as long (16 per cycle), so
// the two row tiles alternate: while one's softmax runs, the tensor core works for the
// other.  Roles:
//   warps 0-3, 4-7   softmax of row tile 0, 1: a thread owns a row (a lane of
//                    tensor memory), so maxima and sums need no shuffles;
//   warp 8           TMA loads of K and V pages into rings of tiles;
//   warp 9           issues the MMAs;
//   warp 10          (FP8) the tiles' scales;
//   warps 12-15      (FP8) turn V's codes into binary16 tiles.
// E4M3 caches: K's codes go to the tensor core as they are (kind::f8f6f4), against
// the query as the sum of two terms (hi = E4M3(q), lo = E5M2(q - hi), after a
// power of two per row: exact for elements within 2^-13 of the row's largest, to
// 2^-21 of it below), so a score costs what a 16-bit one does and K is never
// rewritten; its scale multiplies the score in binary32.  V's codes become
// code * (vs * 2^-e) in binary16, with 2^(e + 5) the tile's largest value scale (a power
// of two of it), so that the largest codes just fit and smaller values keep the 11 bits
// down to 2^-19 of that scale; 2^e goes into the softmax.  (Splitting the weights in two E4M3 terms instead would spare V's
// conversion, but takes four more conversions per pair of weights, and those run
// at 32 lanes a cycle: 983 cycles per row tile against 230 for V's codes.)
// The softmax takes a maximum only for a row's first keys: later weights are
// taken against that reference, and their sum tells whether one of them came near the end
// of its type (16-bit floats and binary32 sums lose nothing short of that); only
// then do a second pass and a rescale of O follow, which the softmax threads do
// themselves between their S and their P, when no product of theirs is running.
// (With a running maximum in every tile: 2800 cycles per pair of row tiles, 1.48 us.)
// What lies past the last key must not meet a zero weight (0 * NaN): the second
// product runs over the 16-key steps that hold keys, and the rest of a last step is
// zeroed in shared memory before it.
#include <cstring>
#include <type_traits>

#include "attention_tc.cuh"

namespace moe {
namespace {

constexpr int kRows = 128;          // rows per row tile

template <int D, bool kFP8>
struct TileShape {
  static constexpr int kTileBytes = kKeys * D * 2;          // a tile of 16-bit elements
  static constexpr int kCodeBytes = kKeys * D;              // a tile of codes
  // BF16: one ring of K and V tiles.  FP8: a ring of V tiles in binary16, one of K's
  // codes, one of V's codes.
  static constexpr int kSlots = kFP8 ? (D == 128 ? 2 : 3) : (D == 128 ? 5 : 8);
  static constexpr int kKSlots = kFP8 ? (D == 128 ? 3 : 4) : 0;
  static constexpr int kRawSlots = kFP8 ? (D == 128 ? 2 : 4) : 0;
  static constexpr int kScaleSlots = 3;
  static constexpr int kThreads = kFP8 ? 512 : 384;
  // offsets in shared memory.  Q: two row tiles (FP8: each as two tiles of codes)
  static constexpr int oQ = 0;
  static constexpr int oSlots = 2 * kTileBytes;
  static constexpr int oK = oSlots + kSlots * kTileBytes;
  static constexpr int oRaw = oK + kKSlots * kCodeBytes;
  static constexpr int oScale = oRaw + kRawSlots * kCodeBytes;         // [slot][ks f32 | vs * 2^-e f16x2]
  static constexpr int oRowf = oScale + (kFP8 ? kScaleSlots * 1024 : 0);
  static constexpr int kSmem = oRowf + (kFP8 ? 1024 : 0);
  // setmaxnreg shares: softmax, the rest (BF16: 384 x 168 registers at launch, 2 x 128 x 200 +
  // 128 x 96 = 63488 of 64512; FP8: 512 x 128, 2 x 128 x 184 + 2 x 128 x 72 = 65536).  With 80
  // for BF16's rest the MMA warp spills: 681 instead of 666 us for 4096 rows at 16384 keys.
  static constexpr int kRegsSoftmax = kFP8 ? 184 : 200;
  static constexpr int kRegsOther = kFP8 ? 72 : 96;
};

struct Bars {
  uint64_t full[8], empty[8];     // the ring of tiles (FP8: of V)
  uint64_t k_full[4], k_empty[4]; // FP8: K's codes
  uint64_t raw_full[4], raw_empty[4];   // FP8: V's codes
  uint64_t q_full;
  uint64_t s_full[2], p_full[2], o_done[2];
  uint64_t sc_full[3], sc_empty[3];
  uint64_t drain;
  uint32_t tmem;
  int abort;
  int flag;
  int e[3];                       // FP8: exponent of each tile's value scales
};

// kCap: scores are capped (a form of its own: its registers are not the common one's).
template <int D, bool kFP8, bool kCap>
__global__ void __launch_bounds__(TileShape<D, kFP8>::kThreads, 1)
    tiles_kernel(const __grid_constant__ CUtensorMap map_k,
                 const __grid_constant__ CUtensorMap map_v, const AttnParams p) {
  using S = TileShape<D, kFP8>;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ Bars bars;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // ---- what needs no input: barriers, tensor memory
  auto bar = [&](const uint64_t& x) { return smem_u32(&x); };
  if (tid == 0) {
    for (int i = 0; i < S::kSlots; ++i) {
      mbar_init(bar(bars.full[i]), kFP8 ? 4 : 1);
      mbar_init(bar(bars.empty[i]), 1);
    }
    for (int i = 0; i < S::kKSlots; ++i) {
      mbar_init(bar(bars.k_full[i]), 1);
      mbar_init(bar(bars.k_empty[i]), 1);
    }
    for (int i = 0; i < S::kRawSlots; ++i) {
      mbar_init(bar(bars.raw_full[i]), 1);
      mbar_init(bar(bars.raw_empty[i]), 4);
    }
    mbar_init(bar(bars.q_full), 256);
    for (int w = 0; w < 2; ++w) {
      mbar_init(bar(bars.s_full[w]), 1);
      mbar_init(bar(bars.p_full[w]), 4);
      mbar_init(bar(bars.o_done[w]), 1);
    }
    for (int i = 0; i < S::kScaleSlots; ++i) {
      mbar_init(bar(bars.sc_full[i]), 1);
      // the softmax's warps and the converting ones
      mbar_init(bar(bars.sc_empty[i]), 12);
    }
    mbar_init(bar(bars.drain), 1);
    bars.abort = 0;
    mbar_fence_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(&bars.tmem), 512);
    tmem_relinquish();
  }
  if (tid == 256) {
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
  }
  pdl_wait();
  pdl_launch_dependents();

  // ---- what this CTA has to do: first the tiles that are not split, late row tiles (which
  // see most keys) before early ones, then the parts of the last tiles
  const int tiles_bh = p.B * p.c.heads;
  int tile_no = blockIdx.x, part = 0, splits = 1;
  if (tile_no >= p.whole) {
    const int last = tiles_bh * p.row_tiles - p.whole;
    part = (tile_no - p.whole) / last;
    tile_no = p.whole + (tile_no - p.whole) % last;
    splits = p.splits;
  }
  const int rt = p.row_tiles - 1 - tile_no / tiles_bh;
  const int bh = tile_no % tiles_bh;
  const int b = bh / p.c.heads, h = bh - b * p.c.heads;
  const TileView t = tile_view(p, b, h, rt, 2 * kRows, part == 0 && rt == 0 && tid == 0);
  const Share share = share_of(t, splits, part);
  if (t.rows == 0 || part >= max(1, share.count)) {                    // nothing to do here
    if (warp == 9) {
      const uint32_t at = *reinterpret_cast<volatile uint32_t*>(&bars.tmem);
      tmem_dealloc(at, 512);
    }
    return;
  }
  const int k0 = share.k0, k1 = share.k1, n = share.n;           // keys, key tiles
  // key tiles of each group: row tile 0 may end earlier, row tile 1 may not exist
  const int hi0 = min(k1, row_hi(p, t, (t.first_row + min(t.rows, kRows) - 1) / p.group));
  const int n0 = max(0, min(n, (hi0 - k0 + kKeys - 1) / kKeys));
  const int n1 = t.rows > kRows ? n : 0;

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem;
  volatile int* abort_flag = &bars.abort;
  const uint32_t sbase = smem_u32(smem);

  // A bounded wait of a whole warp, whose lanes agree on the result; the first
  // to give up records it and stops the others.
  auto wait = [&](uint32_t at, uint32_t parity) -> bool {
    const bool ok = mbar_wait(at, parity, abort_flag, p.timeout_ns);
    if (!ok && !*abort_flag) {
      *abort_flag = 1;
      set_error(p.ctrl, MOE_ERR_TIMEOUT, 23);
    }
    return __all_sync(0xffffffffu, ok);
  };

  const int32_t* table = p.table + static_cast<int64_t>(b) * p.table_stride;

  if (warp < 8) {
    // =================================================================== softmax
    regs_inc<S::kRegsSoftmax>();
    const int w = warp >> 2;
    const int row = tid & 127;                       // lane of tensor memory
    const int my = w * kRows + row;                  // row of the CTA's rows
    const bool real = my < t.rows;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;   // this warp's lanes (<< 16)
    // ---- the query tiles, in the layout of a K-major operand
    {
      constexpr int kPieces = D / 8;                 // 16-byte pieces of a row
      constexpr int kPerPass = 128 / kPieces;        // rows per pass of the group
      const int c = row % kPieces;
      const uint32_t flip = p.scale < 0.0f ? 0x80008000u : 0u;   // the scores' factor is positive
#pragma unroll 4
      for (int pass = 0; pass < kRows / kPerPass; ++pass) {
        const int tr = row / kPieces + pass * kPerPass;   // row within its tile
        const int cr = w * kRows + tr;                    // row of the CTA's rows
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (cr < t.rows) {
          const int rr = t.first_row + cr, tok = rr / p.group;
          x = __ldg(reinterpret_cast<const uint4*>(
                        p.q + static_cast<int64_t>(t.q0 + tok) * p.q_st +
                        static_cast<int64_t>(h * p.group + rr - tok * p.group) * p.q_sh) + c);
          x.x ^= flip;
          x.y ^= flip;
          x.z ^= flip;
          x.w ^= flip;
        }
        if constexpr (kFP8) {
          uint32_t* xw = reinterpret_cast<uint32_t*>(&x);
          float a = 0.0f;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            a = fmaxf(a, fmaxf(fabsf(__uint_as_float(xw[i] << 16)),
                               fabsf(__uint_as_float(xw[i] & 0xffff0000u))));
#pragma unroll
          for (int o = 1; o < kPieces; o <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
          float mul, inv;
          row_pow2(a, mul, inv);
          mul *= 0.5f;                   // below 2^8: an E4M3 ends at 448
          if (c == 0) reinterpret_cast<float*>(smem + S::oRowf)[cr] = 2.0f * inv;
          uint32_t hi[2], lo[2];
          two_terms({xw[0], xw[1], xw[2], xw[3]}, mul, hi, lo);
          uint8_t* at = smem + S::oQ + w * S::kTileBytes +
                        code_piece<D>(tr, c >> 1) + (c & 1) * 8;
          *reinterpret_cast<uint2*>(at) = make_uint2(hi[0], hi[1]);
          *reinterpret_cast<uint2*>(at + S::kCodeBytes) = make_uint2(lo[0], lo[1]);
        } else {
          uint8_t* at = smem + S::oQ + w * S::kTileBytes + (c >> 3) * kHalfBytes +
                        tr * 128 + (((c & 7) ^ (tr & 7)) << 4);
          *reinterpret_cast<uint4*>(at) = x;
        }
      }
      fence_async_smem();
      mbar_arrive(bar(bars.q_full));
    }
    int r_lo = t.lo, r_hi = t.hi;
    if (real) {
      const int tok = (t.first_row + my) / p.group;
      r_lo = row_lo(p, t, tok);
      r_hi = row_hi(p, t, tok);
    }
    r_lo = max(r_lo, k0);
    r_hi = min(r_hi, k1);
    const bool idle = w * kRows + (warp & 3) * 32 >= t.rows;
    const int my_n = w == 0 ? n0 : n1;
    const float cap = p.softcap;
    float sc = fabsf(p.scale);                       // of the scores
    bool ok = true;
    if constexpr (kFP8) {
      if (my_n > 0) {
        ok = wait(bar(bars.q_full), 0);              // (other threads wrote the factors)
        sc *= reinterpret_cast<const float*>(smem + S::oRowf)[my];
      }
    }
    const float ninf = __int_as_float(0xff800000);
    const float cap_k = kCap ? 2.0f * kLog2e * sc / cap : 0.0f;
    const float f = (kCap ? cap : sc) * kLog2e;   // from s (or tanh) to log2 units
    // (binary16 weights: the first keys' largest is 2^3, so a weight is rounded to 2^-28 of it
    // at worst, or to 2^-25 in a tile whose values' unit is up to 2^3 smaller, and what many small
    // ones add up to beside it is kept)
    constexpr float kFar = kFP8 ? 16384.0f : kFarWeight, kAbove = kFP8 ? 3.0f : 0.0f;
    float ref = 0.0f, l = 0.0f;
    bool started = false;                            // the row has seen a key
    int E = 0, E_top = 0;                            // FP8: O is in units of 2^E
    const uint32_t s_tm = tmem + lanes + w * kKeys, o_tm = tmem + lanes + 256 + w * D;

    // One key tile: the scores of this thread's row, of the keys from kb on, to weights
    // in their place.
    auto tile = [&](int i, int kb, int sslot) {
      constexpr int kCols = kKeys;
      float s[kCols];
#pragma unroll
      for (int j = 0; j < kCols / 32; ++j) tmem_ld32(s_tm + 32 * j, s + 32 * j);
#pragma unroll
      for (int j = 0; j < kCols / 32; ++j) tmem_ld_wait32(s + 32 * j);
      int e = 0;
      if constexpr (kFP8) {
        const float4* ks = reinterpret_cast<const float4*>(smem + S::oScale + sslot * 1024);
#pragma unroll
        for (int j = 0; j < kCols / 4; ++j) {
          const float4 k4 = ks[j];
          mul2(s[4 * j], s[4 * j + 1], s[4 * j], s[4 * j + 1], k4.x, k4.y);
          mul2(s[4 * j + 2], s[4 * j + 3], s[4 * j + 2], s[4 * j + 3], k4.z, k4.w);
        }
        e = bars.e[sslot];
      }
      // the scores of keys that the row does not see become x
      const bool edge = kb + kCols > r_hi || kb < r_lo;
      auto hide = [&](float x) {
        // a bit for each key that the row sees, 32 keys at a time
#pragma unroll
        for (int q = 0; q < kCols / 32; ++q) {
          const int lo = min(max(r_lo - kb - 32 * q, 0), 32), hi = min(max(r_hi - kb - 32 * q, 0), 32);
          const uint32_t below_hi = hi == 32 ? 0xffffffffu : (1u << hi) - 1u;
          const uint32_t seen = lo == 32 ? 0u : below_hi & (0xffffffffu << lo);
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if ((seen >> j & 1u) == 0u) s[32 * q + j] = x;
        }
      };
      if constexpr (kCap) {
        // s becomes tanh(score / cap) = 1 - 2 / (e + 1), e = exp(2 score / cap), with one
        // reciprocal for four scores (e is cut at 2^31, where tanh is 1, so four
        // factors stay finite): 1.25 special functions and 6 other operations per score.
        // (One reciprocal each: 8 cycles of their unit; a polynomial of degree 13: 9
        // operations, and a bound on the scores first.)  A NaN in a
        // score that the row does not see (past the last key anything may lie) must not reach
        // its neighbours: a sum finds it, and the hidden scores become 0.
        if (edge) {
          float x[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int j = 4; j < kCols; j += 4) {
            add2(x[0], x[1], s[j], s[j + 1]);
            add2(x[2], x[3], s[j + 2], s[j + 3]);
          }
          const float all = (x[0] + x[1]) + (x[2] + x[3]);
          if (all != all) hide(0.0f);
        }
#pragma unroll
        for (int j = 0; j < kCols; j += 4) {
          float d[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) d[q] = exp2_approx(min_nan(s[j + q] * cap_k, 31.0f)) + 1.0f;
          const float ab = d[0] * d[1], cd = d[2] * d[3];
          const float r = rcp_approx(ab * cd);
          const float rab = -2.0f * r * cd, rcd = -2.0f * r * ab;
          s[j] = fmaf(rab, d[1], 1.0f);
          s[j + 1] = fmaf(rab, d[0], 1.0f);
          s[j + 2] = fmaf(rcd, d[3], 1.0f);
          s[j + 3] = fmaf(rcd, d[2], 1.0f);
        }
      }
      if (edge) hide(ninf);
      auto row_max = [&]() {
        float x[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int j = 4; j < kCols; ++j) x[j & 3] = fmaxf(x[j & 3], s[j]);
        return fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * f;
      };
      // a row's first keys set its reference (the first of which a score is not -inf: a key may
      // be as low as its type goes)
      const bool first = !started && kb < r_hi && kb + kKeys > r_lo;
      if (__any_sync(0xffffffffu, first)) {
        const float top = row_max();
        if (first && top > ninf) {
          ref = top - kAbove;
          E = e;
          E_top = e;
          started = true;
        }
      }
      // weights, into the place of the scores, and their sum
      auto weigh = [&]() {
        float shift = -ref;
        if constexpr (kFP8) shift += static_cast<float>(e - E);
        float sum0 = 0.0f, sum1 = 0.0f, sum2 = 0.0f, sum3 = 0.0f;
#pragma unroll
        for (int q = 0; q < kCols / 32; ++q) {
          uint32_t r[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float a, bb;
            fma2_bc(a, bb, s[32 * q + 2 * j], s[32 * q + 2 * j + 1], f, shift);
            a = exp2_approx(a);
            bb = exp2_approx(bb);
            if (j & 1) add2(sum2, sum3, a, bb); else add2(sum0, sum1, a, bb);
            if constexpr (kFP8) {
              __half2 hh = __floats2half2_rn(a, bb);
              r[j] = *reinterpret_cast<uint32_t*>(&hh);
            } else {
              __nv_bfloat162 hh = __floats2bfloat162_rn(a, bb);
              r[j] = *reinterpret_cast<uint32_t*>(&hh);
            }
          }
          tmem_st16(s_tm + 16 * q, r);
        }
        return (sum0 + sum1) + (sum2 + sum3);
      };
      float sum = weigh();
      // (FP8: also where the tile's values are far smaller than those that set E, which would
      // leave few bits of the weights; E stays within 40 of the largest, so O stays finite)
      const int to = kFP8 ? max(e, E_top - 40) : 0;
      if (__any_sync(0xffffffffu, sum > kFar || (kFP8 && started && to < E - 3))) {
        // (every row of the warp moves to its largest score so far)
        const float top = row_max();
        const float want = started ? fmaxf(ref, top - kAbove) : ref;
        const float keep = exp2_approx(ref - want);
        const float g = kFP8 ? keep * exp2_approx(static_cast<float>(E - to)) : keep;
        l *= keep;
        ref = want;
        E = to;
        E_top = max(E_top, E);
        if (i > 0) {
          // (these scores are complete, so every earlier product of this group is too)
#pragma unroll 1
          for (int d = 0; d < D; d += 16) {
            float o[16];
            tmem_ld16(o_tm + d, o);
            tmem_ld_wait(o);
            uint32_t r[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) r[j] = __float_as_uint(o[j] * g);
            tmem_st16(o_tm + d, r);
          }
        }
        sum = weigh();
      }
      if constexpr (kFP8) sum *= exp2_approx(static_cast<float>(E - e));
      l += sum;
      tmem_st_wait();
    };

    for (int i = 0; i < my_n && ok; ++i) {
      ok = wait(bar(bars.s_full[w]), i & 1);
      const int sslot = i % S::kScaleSlots;
      if constexpr (kFP8) ok = ok && wait(bar(bars.sc_full[sslot]), (i / S::kScaleSlots) & 1);
      if (!ok) break;
      tc_fence_after();
      if (!idle) tile(i, k0 + i * kKeys, sslot);
      // (one arrival per warp: 32 on one barrier take a hundred cycles)
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(bars.p_full[w]));
        if (kFP8) mbar_arrive(bar(bars.sc_empty[sslot]));
      }
    }
    if constexpr (kFP8) {
      // the key tiles that this group does not see: their scales are done with
      for (int i = my_n; i < n && ok; ++i) {
        const int sslot = i % S::kScaleSlots;
        ok = wait(bar(bars.sc_full[sslot]), (i / S::kScaleSlots) & 1);
        if (lane == 0) mbar_arrive(bar(bars.sc_empty[sslot]));
      }
    }
    if (ok && my_n > 0) ok = wait(bar(bars.o_done[w]), 0);
    tc_fence_after();

    // ---- results
    const bool have = ok && my_n > 0 && !idle;
    if (!have) {
      started = false;
      l = 0.0f;
    }
    if (!started) ref = ninf;
    const bool split = share.count > 1;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const float g = (kFP8 ? exp2_approx(static_cast<float>(E)) : 1.0f) * (split ? 1.0f : inv);
    float* parts = p.partial + static_cast<int64_t>(tile_no - p.whole) * p.splits *
                                   partial_floats<D>(p.part_rows);
    float* dst = parts + part * partial_floats<D>(p.part_rows);
    __nv_bfloat16* orow = real && !split ? out_row(p, t, my) : nullptr;
    if (!idle) {
#pragma unroll 1
      for (int d = 0; d < D; d += 16) {
        float o[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) o[j] = 0.0f;
        if (have) {                       // (the same for all lanes of the warp)
          tmem_ld16(o_tm + d, o);
          tmem_ld_wait(o);
#pragma unroll
          for (int j = 0; j < 16; ++j) o[j] = l == 0.0f ? 0.0f : o[j] * g;   // (0 * NaN)
        }
        if (!real) continue;
        if (split) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            reinterpret_cast<float4*>(dst + static_cast<int64_t>(my) * D + d)[j] =
                make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
        } else {
          uint32_t u[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            __nv_bfloat162 hh = __floats2bfloat162_rn(o[2 * j], o[2 * j + 1]);
            u[j] = *reinterpret_cast<uint32_t*>(&hh);
          }
          reinterpret_cast<uint4*>(orow + d)[0] = make_uint4(u[0], u[1], u[2], u[3]);
          reinterpret_cast<uint4*>(orow + d)[1] = make_uint4(u[4], u[5], u[6], u[7]);
        }
      }
    }
    if (real) {
      if (split) {
        dst[static_cast<int64_t>(p.part_rows) * D + my] = ref;
        dst[static_cast<int64_t>(p.part_rows) * (D + 1) + my] = l;
      } else if (p.lse != nullptr) {
        *lse_at(p, t, my) = lse_of(ref, l);
      }
    }
    if (split)
      join_parts<D>(p, t, parts, p.counters + (tile_no - p.whole), p.part_rows, share.count, tid,
                    256, 1, reinterpret_cast<float*>(smem + S::oSlots), &bars.flag);
  } else if (warp < 12) {
    regs_dec<S::kRegsOther>();
    if (warp == 9 && n > 0) {
      // ================================================================= MMA
      // Everything that an MMA takes is uniform over the warp and says so
      // (shuffles, elect.sync): an issue is then a few instructions, where
      // per-lane registers cost about a hundred cycles each.
      // (formats: E4M3 and binary16 are 0, bf16 is 1)
      const uint32_t idesc_s = make_idesc(kFP8 ? 0u : 1u, kRows, kKeys);
      const uint32_t idesc_o = make_idesc(kFP8 ? 0u : 1u, kRows, D) | (1u << 16);
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const int tiles = __shfl_sync(0xffffffffu, n, 0);
      const int tiles0 = __shfl_sync(0xffffffffu, n0, 0);
      const int tiles1 = __shfl_sync(0xffffffffu, n1, 0);
      const uint32_t q_lo = smem_desc_lo(sbase + S::oQ);
      const uint32_t k_lo = smem_desc_lo(sbase + (kFP8 ? S::oK : S::oSlots));
      const uint32_t v_lo = mn_desc_lo(sbase + S::oSlots);
      const int first_key = max(t.lo, k0);
      const int first_step = max(0, first_key - k0) / 16;     // of the first tile
      const int last_steps = (k1 - (k0 + (n - 1) * kKeys) + 15) / 16;   // of the last tile
      struct Place {           // a tile's slot and the parity of its waits
        int slot;
        uint32_t parity;
      };
      Place at_v = {0, 0}, at_k = {0, 0};
      auto step = [](Place& at, int slots) {
        const Place x = at;
        if (++at.slot == slots) {
          at.slot = 0;
          at.parity ^= 1;
        }
        return x;
      };
      auto next_v = [&]() { return step(at_v, S::kSlots); };
      auto next_k = [&]() { return kFP8 ? step(at_k, S::kKSlots) : step(at_v, S::kSlots); };
      auto wait_v = [&](const Place& x) { return wait(bar(bars.full[0]) + 8 * x.slot, x.parity); };
      auto wait_k = [&](const Place& x) {
        return wait((kFP8 ? bar(bars.k_full[0]) : bar(bars.full[0])) + 8 * x.slot, x.parity);
      };
      auto release_v = [&](const Place& x) {
        if (elect_one()) umma_commit(bar(bars.empty[0]) + 8 * x.slot);
      };
      auto release_k = [&](const Place& x) {
        if (elect_one())
          umma_commit((kFP8 ? bar(bars.k_empty[0]) : bar(bars.empty[0])) + 8 * x.slot);
      };
      // S = Q K^T of group w and the key tile in slot x
      auto scores = [&](int w, const Place& x) {
        const uint32_t q = q_lo + w * (S::kTileBytes >> 4);
        const uint32_t k = k_lo + x.slot * ((kFP8 ? S::kCodeBytes : S::kTileBytes) >> 4);
        tc_fence_after();
        if (elect_one()) {
          if constexpr (kFP8) {
#pragma unroll
            for (int s = 0; s < 2 * (D / 32); ++s) {     // hi, then lo
              const uint32_t off = ((s % (D / 32)) * 32) >> 4;
              umma_codes<D>(tm + w * kKeys, q + (s / (D / 32)) * (S::kCodeBytes >> 4) + off,
                            k + off, s < D / 32 ? idesc_s : idesc_s | kAIsE5M2, s > 0);
            }
          } else {
#pragma unroll
            for (int s = 0; s < D / 16; ++s) {
              const uint32_t off = ((s >> 2) * kHalfBytes + (s & 3) * 32) >> 4;
              umma_lo<false>(tm + w * kKeys, q + off, k + off, idesc_s, s > 0);
            }
          }
          umma_commit(bar(bars.s_full[0]) + 8 * w);
        }
      };
      // O += P V over the 16-key steps of tile i that hold keys
      auto values = [&](int w, int i, const Place& x, bool first) {
        const uint32_t v = v_lo + x.slot * (S::kTileBytes >> 4);
        const uint32_t d = tm + 256 + w * D, pw = tm + w * kKeys;
        tc_fence_after();
        if ((i > 0 || first_step == 0) && (i + 1 < tiles || last_steps == 8)) {
          if (elect_one()) {
#pragma unroll
            for (int s = 0; s < 8; ++s)
              umma_ts(d, pw + s * 8, v + s * (2048u >> 4), idesc_o,
                      s > 0 ? 1u : (first ? 0u : 1u));
          }
        } else if (elect_one()) {
          const int s0 = i == 0 ? first_step : 0, s1 = i + 1 == tiles ? last_steps : 8;
          for (int s = s0; s < s1; ++s)
            umma_ts(d, pw + s * 8, v + s * (2048u >> 4), idesc_o,
                    (first && s == s0) ? 0u : 1u);
        }
      };
      // (BF16) rows of V in those steps that no row sees
      auto clean = [&](int i, const Place& x) {
        if constexpr (!kFP8) {
          if (i > 0 && i + 1 < tiles) return;
          const int kb = k0 + i * kKeys;
          const int lo = max(0, first_key - kb), hi = k1 - kb;
          if ((lo & 15) != 0 || (hi < kKeys && (hi & 15) != 0)) {
            const uint32_t base = sbase + S::oSlots + x.slot * S::kTileBytes;
            auto zero = [&](int r0, int r1) {
              for (int y = lane; y < (r1 - r0) * (D / 8); y += 32) {
                const int r = r0 + y / (D / 8), c = y % (D / 8);
                const uint32_t at = base + (c >> 3) * kHalfBytes + r * 128 + (c & 7) * 16;
                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0)
                             : "memory");
              }
            };
            zero(lo & ~15, lo);
            if (hi < kKeys) zero(hi, (hi + 15) & ~15);
            fence_async_smem();
            __syncwarp();
          }
        }
      };
      bool ok = wait(bar(bars.q_full), 0);
      uint32_t used0 = 0, used1 = 0;       // parity of each row tile's weights
      if (ok) {
        const Place x = next_k();
        ok = wait_k(x);
        if (ok) {
          if (tiles0 > 0) scores(0, x);
          if (tiles1 > 0) scores(1, x);
          release_k(x);
        }
      }
      for (int i = 0; i < tiles && ok; ++i) {
        const Place v = next_v();
        ok = wait_v(v);
        if (!ok) break;
        clean(i, v);
        const bool more = i + 1 < tiles;
        Place k = {0, 0};
        bool have_k = false;
        if (more) k = next_k();
        // a row tile's product, then its next scores
        auto turn = [&](int w, int count, uint32_t& used) -> bool {
          if (i >= count) return true;
          if (!wait(bar(bars.p_full[0]) + 8 * w, used)) return false;
          used ^= 1;
          values(w, i, v, i == 0);
          if (i + 1 < count) {
            if (!have_k && !wait_k(k)) return false;
            have_k = true;
            scores(w, k);
          } else if (elect_one()) {
            umma_commit(bar(bars.o_done[0]) + 8 * w);
          }
          return true;
        };
        ok = turn(0, tiles0, used0) && turn(1, tiles1, used1);
        if (!ok) break;
        release_v(v);
        if (more) release_k(k);
      }
      if (!ok) {                           // products in flight end before the memory goes
        if (elect_one()) umma_commit(bar(bars.drain));
        __syncwarp();
        mbar_wait_drain(bar(bars.drain), 0, p.timeout_ns);
      }
    } else if (warp == 8 && n > 0) {
      // ================================================================= TMA loads
      const int box_log2 = min(p.c.page_log2, 7), box = 1 << box_log2;   // (kKeys = 2^7)
      const int segs = kKeys >> box_log2;
      const int first_key = max(t.lo, k0);           // pages before a window are not read
      const uint64_t policy = p.row_tiles > 1 ? policy_evict_last() : policy_evict_first();
      constexpr int kRowBytes = kFP8 ? D : 2 * D;
      bool ok = p.drop_producer == 0;
      // a ring: its slots, its barriers, how many tiles it was given
      struct Ring {
        uint32_t full, empty, base;
        int slots, bytes, f;
      };
      Ring rv, rk;
      if constexpr (kFP8) {
        rv = {bar(bars.raw_full[0]), bar(bars.raw_empty[0]), sbase + S::oRaw, S::kRawSlots,
              S::kCodeBytes, 0};
        rk = {bar(bars.k_full[0]), bar(bars.k_empty[0]), sbase + S::oK, S::kKSlots,
              S::kCodeBytes, 0};
      } else {
        rv = {bar(bars.full[0]), bar(bars.empty[0]), sbase + S::oSlots, S::kSlots, S::kTileBytes,
              0};
        rk = rv;
      }
      auto load = [&](Ring& r, bool v, int i) {
        const int kb = k0 + i * kKeys;
        const int key = kb + lane * box;
        const bool mine = lane < segs && key < k1 && key + box > first_key;
        int page = mine ? __ldg(table + (key >> p.c.page_log2)) : 0;
        if (page < 0 || page >= p.c.num_pages) {
          set_error(p.ctrl, MOE_ERR_DEVICE_FAULT, 22);
          page = 0;                        // (a place that exists)
        }
        const int slot = r.f % r.slots;
        if (!wait(r.empty + 8 * slot, ((r.f / r.slots) & 1) ^ 1)) return false;
        const uint32_t full = r.full + 8 * slot;
        if (lane == 0) {
          const int loaded = min(segs, (k1 - kb + box - 1) >> box_log2) -
                               max(0, (first_key - kb) >> box_log2);
          mbar_arrive_expect_tx(full, loaded * box * kRowBytes);
        }
        __syncwarp();
        if (mine) {
          const int row = ((page * p.c.heads + h) << p.c.page_log2) +
                          (key & ((1 << p.c.page_log2) - 1));
          const CUtensorMap* map = v ? &map_v : &map_k;
          const uint32_t dst = r.base + slot * r.bytes;
          if constexpr (kFP8) {
            tma_load_2d(dst + lane * box * D, map, full, 0, row, policy);
          } else {
#pragma unroll
            for (int x = 0; x < D / 64; ++x)
              tma_load_2d(dst + x * kHalfBytes + lane * box * 128, map, full, x * 64, row, policy);
          }
        }
        __syncwarp();
        ++r.f;
        return true;
      };
      // in the order that the MMAs take them
      auto keys = [&](int i) { return load(kFP8 ? rk : rv, false, i); };
      ok = ok && keys(0);
      for (int i = 0; i < n && ok; ++i) {
        ok = load(rv, true, i);
        if (ok && i + 1 < n) ok = keys(i + 1);
      }
      if (!ok) {                           // copies in flight land before the memory goes
        for (int g = max(0, rv.f - rv.slots); g < rv.f; ++g)
          mbar_wait_drain(rv.full + 8 * (g % rv.slots), (g / rv.slots) & 1, p.timeout_ns);
        if (kFP8)
          for (int g = max(0, rk.f - rk.slots); g < rk.f; ++g)
            mbar_wait_drain(rk.full + 8 * (g % rk.slots), (g / rk.slots) & 1, p.timeout_ns);
      }
    } else if (kFP8 && warp == 10) {
      // ================================================================= FP8: scales
      // Four keys per lane; pages two tiles ahead, scales one.
      const int page_mask = (1 << p.c.page_log2) - 1;
      auto page_of = [&](int i) {
        const int key = k0 + i * kKeys + 4 * lane;
        return key < k1 ? __ldg(table + (key >> p.c.page_log2)) : -1;
      };
      float ks[4], vs[4];
      auto fetch = [&](int i, int page) {
        const int key = k0 + i * kKeys + 4 * lane;
        const bool have = page >= 0 && page < p.c.num_pages;
        const int64_t at = ((static_cast<int64_t>(have ? page : 0) * p.c.heads + h)
                            << p.c.page_log2) + (key & page_mask);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bool x = have && key + j < k1 && key + j >= t.lo;
          ks[j] = x ? __ldg(p.c.k_scales + at + j) : 0.0f;
          vs[j] = x ? __ldg(p.c.v_scales + at + j) : 0.0f;
        }
      };
      bool ok = p.drop_producer == 0;
      int page_next = page_of(1);
      int ex_top = 0;                  // of the tiles so far
      fetch(0, page_of(0));
      for (int i = 0; i < n && ok; ++i) {
        const int slot = i % S::kScaleSlots;
        ok = wait(bar(bars.sc_empty[slot]), ((i / S::kScaleSlots) & 1) ^ 1);
        if (!ok) break;
        // the tile's largest value scale (scales are not negative: their bits are ordered)
        const uint32_t top = __reduce_max_sync(
            0xffffffffu, __float_as_uint(fmaxf(fmaxf(vs[0], vs[1]), fmaxf(vs[2], vs[3]))));
        // (at least 2^-80 of the largest so far, against which such values count as 0 anyway: a
        // tile of zeros beside large ones must not take the weights, whose unit it is, out of
        // binary32)
        const int ex = max(min(max(static_cast<int>((top >> 23) & 255u), 6), 253), ex_top - 80);
        ex_top = max(ex_top, ex);
        const float mul = __uint_as_float(static_cast<uint32_t>(259 - ex) << 23);   // 2^(5 - e)
        uint32_t g[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          __half2 x = __float2half2_rn(vs[j] * mul);
          g[j] = *reinterpret_cast<uint32_t*>(&x);
        }
        uint8_t* sc = smem + S::oScale + slot * 1024 + lane * 16;
        *reinterpret_cast<float4*>(sc) = make_float4(ks[0], ks[1], ks[2], ks[3]);
        *reinterpret_cast<uint4*>(sc + 512) = make_uint4(g[0], g[1], g[2], g[3]);
        if (lane == 0) bars.e[slot] = ex - 127 - 5;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(bars.sc_full[slot]));
        fetch(i + 1, page_next);
        page_next = page_of(i + 2);
      }
    }
  } else {
    // =================================================================== FP8: V's codes to binary16
    regs_dec<S::kRegsOther>();
    if constexpr (kFP8) {
      const int ct = tid - 384;
      constexpr int kPieces = D / 16;             // 16-code pieces of a row
      constexpr int kPer = kKeys * kPieces / 128; // pieces per thread
      // 8 lanes of a phase take one piece number of 8 rows: different bank groups in the
      // codes' swizzle and in the values'
      const int c = (ct >> 3) % kPieces, r0 = (ct & 7) + 8 * ((ct >> 3) / kPieces);
      const int first_key = max(t.lo, k0);
      const uint32_t half = (c >> 2) * kHalfBytes;
      const int p0 = (2 * c) & 7;
      bool ok = p.drop_producer == 0;
      int rslot = 0, slot = 0, sslot = 0;
      uint32_t rpar = 0, par = 1, spar = 0;
      for (int i = 0; i < n && ok; ++i) {
        ok = wait(bar(bars.sc_full[0]) + 8 * sslot, spar) &&
             wait(bar(bars.raw_full[0]) + 8 * rslot, rpar) &&
             wait(bar(bars.empty[0]) + 8 * slot, par);
        if (!ok) break;
        const int kb = k0 + i * kKeys;
        const uint32_t src = sbase + S::oRaw + rslot * S::kCodeBytes + code_piece<D>(r0, c);
        const uint32_t dst = sbase + S::oSlots + slot * S::kTileBytes + half + r0 * 128;
        const uint32_t a0 = dst + ((p0 ^ (r0 & 7)) << 4), a1 = dst + (((p0 + 1) ^ (r0 & 7)) << 4);
        const __half2* g = reinterpret_cast<const __half2*>(smem + S::oScale + sslot * 1024 + 512);
        const bool edge = kb < first_key || kb + kKeys > k1;
        constexpr int kStep = 128 / kPieces;      // rows between a thread's pieces
        uint4 x[kPer];                            // all of them first: one latency
#pragma unroll
        for (int j = 0; j < kPer; ++j)
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(x[j].x), "=r"(x[j].y), "=r"(x[j].z), "=r"(x[j].w)
                       : "r"(src + j * kStep * D));
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const int r = r0 + j * kStep;
          const __half2 m2 = g[r];
          const uint32_t xw[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
          uint32_t o[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            uint32_t y = e4m3x2_to_f16x2(static_cast<uint16_t>(xw[q >> 1] >> (16 * (q & 1))));
            __half2 z = __hmul2(*reinterpret_cast<__half2*>(&y), m2);
            o[q] = *reinterpret_cast<uint32_t*>(&z);
          }
          if (edge && (kb + r < first_key || kb + r >= k1)) {   // a row that nobody sees
#pragma unroll
            for (int q = 0; q < 8; ++q) o[q] = 0u;
          }
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a0 + j * kStep * 128),
                       "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3])
                       : "memory");
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a1 + j * kStep * 128),
                       "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                       : "memory");
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(bars.full[0]) + 8 * slot);
          mbar_arrive(bar(bars.raw_empty[0]) + 8 * rslot);
          mbar_arrive(bar(bars.sc_empty[0]) + 8 * sslot);
        }
        if (++rslot == S::kRawSlots) { rslot = 0; rpar ^= 1; }
        if (++slot == S::kSlots) { slot = 0; par ^= 1; }
        if (++sslot == S::kScaleSlots) { sslot = 0; spar ^= 1; }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

template <int D, bool kFP8, bool kCap>
cudaError_t launch_t(const AttnParams& p, const CUtensorMap& mk, const CUtensorMap& mv,
                     cudaStream_t stream) {
  using S = TileShape<D, kFP8>;
  cudaError_t e = cudaFuncSetAttribute(tiles_kernel<D, kFP8, kCap>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return e;
  const unsigned tiles = static_cast<unsigned>(p.B) * p.c.heads * p.row_tiles;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = make_cfg(dim3(p.whole + (tiles - p.whole) * p.splits),
                                    dim3(S::kThreads), stream, true, attr);
  cfg.dynamicSmemBytes = S::kSmem;
  return cudaLaunchKernelEx(&cfg, tiles_kernel<D, kFP8, kCap>, mk, mv, p);
}

template <int D, bool kFP8>
cudaError_t launch_c(const AttnParams& p, const CUtensorMap& mk, const CUtensorMap& mv,
                     cudaStream_t stream) {
  return p.softcap > 0.0f ? launch_t<D, kFP8, true>(p, mk, mv, stream)
                          : launch_t<D, kFP8, false>(p, mk, mv, stream);
}

}  // namespace

cudaError_t launch_attention_tiles(const AttnParams& p, int head_dim, bool fp8,
                                   cudaStream_t stream) {
  CUtensorMap mk, mv;
  if (!cache_maps(p, head_dim, fp8, &mk, &mv)) return cudaErrorInvalidValue;
  if (fp8)
    return head_dim == 128 ? launch_c<128, true>(p, mk, mv, stream)
                           : launch_c<64, true>(p, mk, mv, stream);
  return head_dim == 128 ? launch_c<128, false>(p, mk, mv, stream)
                         : launch_c<64, false>(p, mk, mv, stream);
}

}  // namespace moe
