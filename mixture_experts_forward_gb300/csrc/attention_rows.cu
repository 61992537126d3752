// Attention of few rows over the paged cache: single tokens (decode) and
// short drafted runs, up to 64 rows (new tokens x query heads of one cache
// head), 48 over E4M3 codes.  Every cached byte is read once, by TMA, and meets few rows: decode
// is bound by HBM (16 rows, 304 tiles of 8192 keys: 6.5 TB/s from BF16, 6.1 from E4M3), 17 to 48
// rows over E4M3 codes by the softmax warps (conversions of the weights; 3.3 to 4.2 TB/s).
//
// The products are turned round, so that a key is a lane and a row a column:
//   S^T[keys x rows] = K Q^T               (A = the key tile as it lies in the cache)
//   O^T[channels x rows] += V^T P^T   (A = the value tile, MN-major)
// With 128 rows of the tensor core filled by keys and channels, 8 or 40 query rows
// cost no padding to 128; a softmax thread owns a key, so a quantised cache's two
// scales are one register each, and the maxima and sums over keys cross lanes only at
// the first tile and at the end: the reference of a row is the maximum of its first
// keys' scores, and later weights are only checked for the ends of their type (then
// a second pass and a rescale of O follow).
//
// E4M3 caches go to the tensor core as they are, in both products: the query is the
// sum of an E4M3 and an E5M2 term (exact for elements within 2^-13 of the row's largest, to
// 2^-21 of it below), and each weight of two E4M3 terms, hi = E4M3(x), lo = E4M3(16 (x - hi)),
// with sums of their own: 8 to 9 significant bits over 2^-13 .. 448, the first tile's
// largest at 16.  x carries the value scale (relative to 2^E, the first tile's largest), and
// so do the references: a large weight on a small value keeps its bits, and V is never
// rewritten.  BF16 caches split the weights in two bf16 terms.
// Nothing but the output is then rounded to fewer bits than the cache has.
//
// Groups of four warps share the rows of every key tile (a thread per key, 8 or 16 rows
// each); then one warp loads and one issues the MMAs.  Scores are double-buffered in
// tensor memory.  Up to 32 rows two CTAs share an SM (not BF16 heads of 128 above 16 rows, of
// whose 32 KB tiles only two would fit beside a second CTA).
#include <cstring>
#include <type_traits>

#include "attention_tc.cuh"

namespace moe {
namespace {

template <int D, bool kFP8, int N>
struct RowsShape {
  static constexpr int kGroups = N == 16 ? 2 : N / 16;   // of softmax warps
  static constexpr int kSoftmax = kGroups * 128;
  static constexpr int kThreads = kSoftmax + 64;
  static constexpr int kTileBytes = kKeys * D * (kFP8 ? 1 : 2);
  static constexpr int kQTerm = N * D * (kFP8 ? 1 : 2);  // bytes of the query (of each term)
  static constexpr int kChunkRows = kFP8 ? 16 : 8;       // rows in 16 bytes of weights
  static constexpr int kPTerm = N / kChunkRows * kKeys * 16;
  // FP8 is bound by the softmax warps as well as by HBM: two buffers of weights spare them
  // the wait for the product before (BF16: 95 % of the copy bandwidth with one)
  static constexpr int kPBufs = kFP8 ? 2 : 1;
  // offsets in shared memory: weights (hi, lo), query (FP8: hi, lo), the ring
  static constexpr int oP = 0;
  static constexpr int oQ = kPBufs * 2 * kPTerm;
  static constexpr int oSlots = (oQ + (kFP8 ? 2 : 1) * kQTerm + 1023) / 1024 * 1024;
  // two CTAs per SM where each still has three tiles in shared memory
  static constexpr int kHalf = 111 * 1024, kWhole = 222 * 1024;
  static constexpr int kCtas = N <= 32 && (kHalf - oSlots) / kTileBytes >= 3 ? 2 : 1;
  static constexpr int kFit = ((kCtas == 2 ? kHalf : kWhole) - oSlots) / kTileBytes;
  static constexpr int kSlots = kFit > 12 ? 12 : kFit;
  static constexpr int kSmem = oSlots + kSlots * kTileBytes;
  // tensor memory: S twice, O (FP8: hi and lo)
  static constexpr int oO = 2 * N;
  static constexpr int kTmemUsed = oO + 2 * N;
  static constexpr int kTmem = kTmemUsed <= 64 ? 64 : kTmemUsed <= 128 ? 128 : kTmemUsed <= 256 ? 256 : 512;
  static_assert(kSlots >= 3, "two tiles of keys and one of values");
  static_assert(kCtas * kTmem <= 512, "tensor memory");
  static_assert(kSlots * kTileBytes >= kMaxParts * N * 4, "the joining weights fit the ring");
  static_assert(oQ % 1024 == 0, "swizzled tiles start on 1024 bytes");
};

// E4M3 weights end at 2^-13, and many small ones beside a few large ones may add up to
// something.  So a row whose weights in a key tile are all below kSmall moves its reference to
// that tile's maximum (at most kDown below its highest one, in log2 units: sums stay
// finite).  What a tile loses is then at most 128 * 2^-14 = 2^-7 of its largest weight.
// (Drafted runs, 48 rows: 44 us without the check, 46 with it, 51 with kSmall = 4 in every
// fourth tile.  The second pass costs where scores are sharp: queries four times as large, 93 us,
// and decode of 64 sequences to 16384 positions 274 -> 356 us.)
constexpr float kSmall = 1.0f, kDown = 40.0f;

template <int N, int kGroups>
struct RowsBars {
  uint64_t full[12], empty[12];
  uint64_t q_full, s_full[2], p_full[2], o_step, o_last, drain;
  uint32_t tmem;
  int abort, flag;
  int lo[N], hi[N];               // keys that each row sees, in this part
  float top[N];                   // minus the row's highest reference so far
  alignas(16) float factor[N];    // FP8: of the row's scores
  int64_t q[N], out[N];           // the row's place in q and out
  alignas(16) float part[kGroups][4][N / kGroups];   // per group and warp: maxima or sums
  alignas(16) float scale[N];     // of the row's sums at the end
  uint32_t vs[kGroups][4];        // per group and warp: largest value scale (bits)
  // per group and warp: rows that have a large weight (bits).  A buffer for even key tiles and
  // one for odd: with scores and weights double-buffered, nothing but the barrier of the next
  // tile keeps a warp from storing its word while another still reads the tile before's.
  uint32_t large[2][kGroups][4];
};

// D[tmem] (+)= A[smem] * B[smem], any layouts (both descriptors' words given).
template <bool kFP8>
__device__ __forceinline__ void umma_ss(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo,
                                        uint32_t b_hi, uint32_t idesc, uint32_t accumulate) {
  if constexpr (kFP8)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 ad, bd;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "mov.b64 ad, {%1, %2};\n\tmov.b64 bd, {%3, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], ad, bd, %5, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 ad, bd;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "mov.b64 ad, {%1, %2};\n\tmov.b64 bd, {%3, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], ad, bd, %5, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
        : "memory");
}

template <int kCols>
__device__ __forceinline__ void tmem_ld_cols(uint32_t at, float* v) {
  static_assert(kCols == 8 || kCols == 16, "the rows of a group");
  if constexpr (kCols == 16) {
    float(&x)[16] = *reinterpret_cast<float(*)[16]>(v);
    tmem_ld16(at, x);
    tmem_ld_wait(x);
  } else {
    float(&x)[8] = *reinterpret_cast<float(*)[8]>(v);
    tmem_ld8(at, x);
    tmem_ld_wait(x);
  }
}
template <int kCols>
__device__ __forceinline__ void tmem_st_cols(uint32_t at, const uint32_t* r) {
  if constexpr (kCols == 16) {
    tmem_st16(at, r);
  } else {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
                 "r"(r[7])
                 : "memory");
  }
}

// Reduces NH values per lane over the 32 lanes, halving the values with the
// lanes: lane i returns the result of value i / (32 / NH).  x is overwritten.
template <int NH, typename F>
__device__ __forceinline__ float transposed(float (&x)[NH], F op) {
  const int lane = threadIdx.x & 31;
  int o = 16;
#pragma unroll
  for (int n = NH; n > 1; n /= 2, o /= 2) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int k = 0; k < n / 2; ++k) {
      const float give = up ? x[k] : x[k + n / 2], keep = up ? x[k + n / 2] : x[k];
      x[k] = op(keep, __shfl_xor_sync(0xffffffffu, give, o));
    }
  }
#pragma unroll
  for (; o > 0; o /= 2) x[0] = op(x[0], __shfl_xor_sync(0xffffffffu, x[0], o));
  return x[0];
}

// What a CTA has to do: sequence b and cache head h (all their rows are one tile), part
// `part` of `parts`, of which CTA number `first` has part 0.  b < 0: nothing.
struct Job {
  int b, h, part, parts, first;
};

// One CTA per tile.
__device__ __forceinline__ Job whole_job(const AttnParams& p) {
  Job j;
  j.b = blockIdx.x / p.c.heads;
  j.h = blockIdx.x - j.b * p.c.heads;
  j.part = 0;
  j.parts = 1;
  j.first = blockIdx.x;
  return j;
}

// Fewer tiles than the grid has CTAs (one for every place on the SMs): each sequence's
// tiles are cut into as many parts of about `size` key tiles as its length asks for, size the
// smallest, in steps of an eighth, for which the grid holds them all; ragged
// sequences then give CTAs even work in one round.  Every warp finds this out for itself
// from the lengths (at most as many as CTAs).
__device__ __forceinline__ Job shared_job(const AttnParams& p) {
  const int lane = threadIdx.x & 31, places = gridDim.x, unit = p.c.heads;
  // (the first 32 lengths stay in a register)
  auto load_tiles = [&](int b) {
    const int len = b < p.B ? min(max(__ldg(p.kv_lens + b), 0), p.span) : 0;
    return (len + kKeys - 1) / kKeys;
  };
  const int tiles0 = load_tiles(lane);
  auto key_tiles = [&](int b0) { return b0 == 0 ? tiles0 : load_tiles(b0 + lane); };
  auto sum32 = [&](int v) {
    return static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(v)));
  };
  int all = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) all += sum32(key_tiles(b0));
  // (quotients in binary32: every CTA computes the same ones, and any would do)
  float size = fmaxf(2.0f, ceilf(__fdividef(static_cast<float>(all) * unit, static_cast<float>(places))));
  auto parts_of = [&](int b0) {
    const int n = static_cast<int>(ceilf(__fdividef(static_cast<float>(key_tiles(b0)), size) - 1e-4f));
    return b0 + lane < p.B ? max(1, n) : 0;
  };
  for (;;) {
    int parts = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) parts += sum32(parts_of(b0));
    if (static_cast<int64_t>(parts) * unit <= places || size > all) break;
    size = ceilf(size * 1.125f);
  }
  Job j;
  j.b = -1;
  int before = 0;                                  // CTAs of the sequences before
  for (int b0 = 0; b0 < p.B && j.b < 0; b0 += 32) {
    const int parts = parts_of(b0);
    int inc = parts * unit;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    const int c = blockIdx.x;
    const unsigned here = __ballot_sync(0xffffffffu, before + inc > c);
    if (here != 0u) {
      const int l = __ffs(here) - 1;
      const int start = before + __shfl_sync(0xffffffffu, inc - parts * unit, l);
      j.parts = __shfl_sync(0xffffffffu, parts, l);
      j.b = b0 + l;
      j.h = (c - start) / j.parts;
      j.part = (c - start) - j.h * j.parts;
      j.first = c - j.part;
    }
    before += __shfl_sync(0xffffffffu, inc, 31);
  }
  return j;
}

template <int D, bool kFP8, int N>
__global__ void
    __launch_bounds__(RowsShape<D, kFP8, N>::kThreads, RowsShape<D, kFP8, N>::kCtas)
    rows_kernel(const __grid_constant__ CUtensorMap map_k,
                const __grid_constant__ CUtensorMap map_v, const AttnParams p) {
  using S = RowsShape<D, kFP8, N>;
  constexpr int NH = N / S::kGroups;              // rows of a group
  constexpr int kLoadWarp = S::kSoftmax / 32, kMmaWarp = kLoadWarp + 1;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ RowsBars<N, S::kGroups> bars;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // ---- what needs no input: barriers, tensor memory
  auto bar = [&](const uint64_t& x) { return smem_u32(&x); };
  if (tid == 0) {
    for (int i = 0; i < S::kSlots; ++i) {
      mbar_init(bar(bars.full[i]), 1);
      mbar_init(bar(bars.empty[i]), 1);
    }
    mbar_init(bar(bars.q_full), S::kSoftmax);
    mbar_init(bar(bars.s_full[0]), 1);
    mbar_init(bar(bars.s_full[1]), 1);
    mbar_init(bar(bars.p_full[0]), S::kSoftmax / 32);
    mbar_init(bar(bars.p_full[1]), S::kSoftmax / 32);
    mbar_init(bar(bars.o_step), 1);
    mbar_init(bar(bars.o_last), 1);
    mbar_init(bar(bars.drain), 1);
    bars.abort = 0;
    mbar_fence_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&bars.tmem), S::kTmem);
    tmem_relinquish();
  }
  if (tid == kLoadWarp * 32) {
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
  }
  pdl_wait();
  pdl_launch_dependents();

  const Job job = p.splits > 1 ? shared_job(p) : whole_job(p);
  const int b = job.b, h = job.h;
  TileView t;
  Share share;
  if (b >= 0) {
    t = tile_view(p, b, h, 0, N, job.part == 0 && tid == 0);
    share = share_of(t, job.parts, job.part);
  }
  if (b < 0 || t.rows == 0 || job.part >= max(1, share.count)) {   // nothing to do here
    if (warp == kMmaWarp) {
      const uint32_t at = *reinterpret_cast<volatile uint32_t*>(&bars.tmem);
      tmem_dealloc(at, S::kTmem);
    }
    return;
  }
  const int k0 = share.k0, k1 = share.k1, n = share.n;   // keys, key tiles
  if (tid < N) {                                  // the rows' places and keys
    int lo = 0, hi = 0;
    int64_t in = -1, out = 0;
    if (tid < t.rows) {
      const int rr = t.first_row + tid, tok = rr / p.group;
      const int64_t head = h * p.group + rr - tok * p.group;
      lo = max(k0, row_lo(p, t, tok));
      hi = min(k1, row_hi(p, t, tok));
      in = static_cast<int64_t>(t.q0 + tok) * p.q_st + head * p.q_sh;
      out = static_cast<int64_t>(t.q0 + tok) * p.o_st + head * p.o_sh;
    }
    bars.lo[tid] = lo;
    bars.hi[tid] = hi;
    bars.q[tid] = in;
    bars.out[tid] = out;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem;
  volatile int* abort_flag = &bars.abort;
  const uint32_t sbase = smem_u32(smem);
  auto wait = [&](uint32_t at, uint32_t parity) -> bool {
    const bool ok = mbar_wait(at, parity, abort_flag, p.timeout_ns);
    if (!ok && !*abort_flag) {
      *abort_flag = 1;
      set_error(p.ctrl, MOE_ERR_TIMEOUT, 24);
    }
    return __all_sync(0xffffffffu, ok);
  };
  const int32_t* table = p.table + static_cast<int64_t>(b) * p.table_stride;

  if (warp < kLoadWarp) {
    // =================================================================== softmax
    const int w = warp >> 2;
    const int key_lane = (warp & 3) * 32 + lane;         // key of a tile; channel of O
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
    const int page_mask = (1 << p.c.page_log2) - 1;
    // (FP8) this thread's key: its page two tiles ahead, its scales one
    auto page_of = [&](int i) {
      const int key = k0 + i * kKeys + key_lane;
      return kFP8 && key < k1 && key >= t.lo ? __ldg(table + (key >> p.c.page_log2)) : -1;
    };
    float ks_next = 0.0f, vs_next = 0.0f;
    auto fetch = [&](int i, int page) {
      if constexpr (kFP8) {
        ks_next = vs_next = 0.0f;
        if (static_cast<unsigned>(page) < static_cast<unsigned>(p.c.num_pages)) {
          const int at = ((page * p.c.heads + h) << p.c.page_log2) +
                         ((k0 + i * kKeys + key_lane) & page_mask);
          ks_next = __ldg(p.c.k_scales + at);
          vs_next = __ldg(p.c.v_scales + at);
        }
      }
    };
    int page_next = page_of(0);
    // ---- the query, as the B operand of the first product
    {
      constexpr int kPieces = D / 8;                     // 16-byte pieces of a row
      const uint32_t flip = p.scale < 0.0f ? 0x80008000u : 0u;   // the scores' factor is positive
#pragma unroll
      for (int x0 = 0; x0 < N * kPieces; x0 += S::kSoftmax) {
        const int x = x0 + tid;
        if (x0 + (tid & ~31) < N * kPieces) {            // (whole warps)
          const int r = x / kPieces, c = x % kPieces;
          uint4 q = make_uint4(0u, 0u, 0u, 0u);
          if (bars.q[r] >= 0) {
            q = __ldg(reinterpret_cast<const uint4*>(p.q + bars.q[r]) + c);
            q.x ^= flip;
            q.y ^= flip;
            q.z ^= flip;
            q.w ^= flip;
          }
          if constexpr (kFP8) {
            const uint32_t xw[4] = {q.x, q.y, q.z, q.w};
            float a = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              a = fmaxf(a, fmaxf(fabsf(__uint_as_float(xw[i] << 16)),
                                 fabsf(__uint_as_float(xw[i] & 0xffff0000u))));
#pragma unroll
            for (int o = 1; o < kPieces; o <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
            float mul, inv;
            row_pow2(a, mul, inv);
            mul *= 0.5f;                                 // below 2^8: an E4M3 ends at 448
            if (c == 0)
              bars.factor[r] = 2.0f * inv * fabsf(p.scale) * (p.softcap > 0.0f ? 1.0f : kLog2e);
            uint32_t hi[2], lo[2];
            two_terms(xw, mul, hi, lo);
            uint8_t* at = smem + S::oQ + code_piece<D>(r, c >> 1) + (c & 1) * 8;
            *reinterpret_cast<uint2*>(at) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2*>(at + S::kQTerm) = make_uint2(lo[0], lo[1]);
          } else {
            uint8_t* at = smem + S::oQ + (c >> 3) * (N * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
            *reinterpret_cast<uint4*>(at) = q;
          }
        }
      }
      fence_async_smem();
      mbar_arrive(bar(bars.q_full));
    }
    fetch(0, page_next);
    page_next = page_of(1);
    bool ok = wait(bar(bars.q_full), 0);                 // (and the other threads' factors)
    const float ninf = __int_as_float(0xff800000);
    const float cap = p.softcap, cap_k = cap > 0.0f ? 2.0f * kLog2e / cap : 0.0f;
    const float sc = fabsf(p.scale) * (cap > 0.0f ? 1.0f : kLog2e);
    float nref[NH], l[NH];                               // minus the rows' references; sums
    uint32_t pending = 0;                                // rows that have not seen a score above -inf
    int lo_max = k0, hi_min = k1;
#pragma unroll
    for (int r = 0; r < NH; ++r) {
      nref[r] = 0.0f;
      l[r] = 0.0f;
      const int lo = bars.lo[w * NH + r], hi = bars.hi[w * NH + r];
      if (lo < hi) {
        pending |= 1u << r;
        lo_max = max(lo_max, lo);
      }
      if (w * NH + r < t.rows) hi_min = min(hi_min, hi);
    }
    const uint32_t seeing = pending;
    const bool idle = w * NH >= t.rows;
    const int group_bar = 2 + w;
    int E = 0, E_top = 0;                                // FP8: weights carry vs * 2^(4 - E)
    const uint32_t o_tm = tmem + lanes + S::oO + w * NH;
    // Per row over the tile's keys: each thread's x[r] to the maximum over the group.  (A NaN
    // is no maximum: fmaxf passes over it.)
    auto group_max = [&](float (&x)[NH]) {
      const float m = transposed<NH>(x, [](float a, float c) { return fmaxf(a, c); });
      if ((lane & (32 / NH - 1)) == 0) bars.part[w][warp & 3][lane / (32 / NH)] = m;
      named_bar_sync(group_bar, 128);
#pragma unroll
      for (int r = 0; r < NH; ++r)
        x[r] = fmaxf(fmaxf(bars.part[w][0][r], bars.part[w][1][r]),
                     fmaxf(bars.part[w][2][r], bars.part[w][3][r]));
      named_bar_sync(group_bar, 128);
    };
    // the exponent of the tile's largest value scale
    auto group_exponent = [&](float vs) {
      const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(vs));
      if (lane == 0) bars.vs[w][warp & 3] = m;
      named_bar_sync(group_bar, 128);
      const uint32_t top = max(max(bars.vs[w][0], bars.vs[w][1]), max(bars.vs[w][2], bars.vs[w][3]));
      named_bar_sync(group_bar, 128);
      return min(max(static_cast<int>((top >> 23) & 255u), 5), 250) - 127;
    };

    // (A wait that gave up ends the waiting, not the loop: a group's warps still meet at
    // their barriers, and what they compute is dropped.)
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const float ks = ks_next, vs = vs_next;
      fetch(i + 1, page_next);
      page_next = page_of(i + 2);
      if (ok) ok = wait(bar(bars.s_full[i & 1]), (i >> 1) & 1);
      tc_fence_after();
      if (!idle) {
        const int kb = k0 + i * kKeys, key = kb + key_lane;
        const bool edge = kb < lo_max || kb + kKeys > hi_min;
        // x = the scores (in log2 units) + add, masked; they stay in tensor memory
        float x[NH], sum[NH];
        auto scores = [&](auto shifted) {
          float s[NH];
          tmem_ld_cols<NH>(tmem + lanes + (i & 1) * N + w * NH, s);
#pragma unroll
          for (int r = 0; r < NH; r += 4) {
            float4 f = make_float4(sc, sc, sc, sc);
            if constexpr (kFP8) {
              f = *reinterpret_cast<const float4*>(&bars.factor[w * NH + r]);
              mul2(f.x, f.y, f.x, f.y, ks, ks);
              mul2(f.z, f.w, f.z, f.w, ks, ks);
            }
            if (cap > 0.0f) {
              const float g[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
              for (int j = 0; j < 4; ++j)
                x[r + j] = soft_capped(s[r + j] * g[j], cap_k, cap) * kLog2e +
                           (shifted ? nref[r + j] : 0.0f);
            } else if constexpr (shifted) {
              fma2_to(x[r], x[r + 1], s[r], s[r + 1], f.x, f.y, nref[r], nref[r + 1]);
              fma2_to(x[r + 2], x[r + 3], s[r + 2], s[r + 3], f.z, f.w, nref[r + 2], nref[r + 3]);
            } else {
              mul2(x[r], x[r + 1], s[r], s[r + 1], f.x, f.y);
              mul2(x[r + 2], x[r + 3], s[r + 2], s[r + 3], f.z, f.w);
            }
          }
          if (edge) {
#pragma unroll
            for (int r = 0; r < NH; ++r)
              if (key < bars.lo[w * NH + r] || key >= bars.hi[w * NH + r]) x[r] = ninf;
          }
        };
        // rows whose first keys are in this tile
        uint32_t now = 0;
        if (pending != 0u) {
#pragma unroll
          for (int r = 0; r < NH; ++r)
            if (bars.lo[w * NH + r] < kb + kKeys) now |= 1u << r;
          now &= pending;
        }
        // One pass, unless rows start here, or weights are beyond their type or (FP8) too
        // small for it: the group then takes the rows' maxima first.
        auto prepare = [&](bool starts) {
            // (until a row has started, every weight is 0)
            if (kFP8 && starts && pending == seeing) E = E_top = group_exponent(vs);
            const int E2 = !kFP8 ? 0 : starts ? E : max(group_exponent(vs), E_top - static_cast<int>(kDown));
            scores(std::false_type());
            if constexpr (kFP8) {
              // what meets the E4M3 type is the weight times the value scale
              const float lv = fminf(fmaxf(log2f(vs) - static_cast<float>(E2), -kDown), kDown);
#pragma unroll
              for (int r = 0; r < NH; ++r) x[r] += lv;
            }
            group_max(x);
            if (starts) {
#pragma unroll
              for (int r = 0; r < NH; ++r)
                if ((now >> r & 1u) && x[r] > ninf) {    // (all -inf: the next tile's keys)
                  nref[r] = -x[r];
                  if (key_lane == r) bars.top[w * NH + r] = nref[r];
                  pending &= ~(1u << r);
                }
            } else {
              const uint32_t started = seeing & ~pending;
              // to the tile's maximum, but at most kDown below the highest reference so far
#pragma unroll
              for (int r = 0; r < NH; ++r) {
                const bool can = (started >> r & 1u) && x[r] > ninf;
                x[r] = can ? fminf(-x[r], bars.top[w * NH + r] + kDown) : nref[r];
              }
              named_bar_sync(group_bar, 128);
              if (ok && i > 0) ok = wait(bar(bars.o_step), (i - 1) & 1);
              tc_fence_after();
              const float unit = kFP8 ? exp2_approx(static_cast<float>(E - E2)) : 1.0f;
#pragma unroll
              for (int r = 0; r < NH; ++r) {
                const float want = x[r];
                x[r] = exp2_approx(want - nref[r]);
                nref[r] = want;
                l[r] *= x[r];
                if (key_lane == r)
                  bars.top[w * NH + r] = fminf(bars.top[w * NH + r], want);
              }
              E = E2;
              E_top = max(E_top, E);
              if (i > 0) {
#pragma unroll
                for (int term = 0; term < (kFP8 ? 2 : 1); ++term) {
                  float o[NH];
                  tmem_ld_cols<NH>(o_tm + term * N, o);
                  uint32_t u[NH];
#pragma unroll
                  for (int r = 0; r < NH; ++r) u[r] = __float_as_uint(o[r] * x[r] * unit);
                  tmem_st_cols<NH>(o_tm + term * N, u);
                }
                tmem_st_wait();
              }
            }
        };
        auto pass = [&]() -> bool {
          // the weights' two terms, to [buffer][term][chunk of rows][key][16 bytes] (where a
          // pass is done again nobody has read them), and their sums without the value scale
          scores(std::true_type());
#pragma unroll
          for (int r = 0; r < NH; ++r) sum[r] = exp2_approx(x[r]);
          constexpr int kWords = kFP8 ? NH / 4 : NH / 2;   // of this thread's weights, per term
          uint32_t hi[kWords], lo[kWords];
          bool far;
          if constexpr (kFP8) {
            const float vw = vs * exp2_approx(static_cast<float>(4 - E));
            __half2 most = __float2half2_rn(0.0f);
#pragma unroll
            for (int j = 0; j < NH / 4; ++j) {
              uint32_t hw = 0, lw = 0;
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                float a, c;
                mul2(a, c, sum[4 * j + 2 * k], sum[4 * j + 2 * k + 1], vw, vw);
                const uint16_t hc = cvt_e4m3x2(a, c);
                const uint32_t back = e4m3x2_to_f16x2(hc);
                const __half2 full = __floats2half2_rn(a, c);
                most = __hmax2(most, full);
                __half2 d = __hsub2(full, *reinterpret_cast<const __half2*>(&back));
                d = __hmul2(d, __float2half2_rn(16.0f));
                uint16_t lc;
                asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;"
                    : "=h"(lc)
                    : "r"(*reinterpret_cast<uint32_t*>(&d)));
                hw |= static_cast<uint32_t>(hc) << (16 * k);
                lw |= static_cast<uint32_t>(lc) << (16 * k);
              }
              hi[j] = hw;
              lo[j] = lw;
            }
            // (a value scale beyond binary32 in the present unit makes NaN of weights of 0, which
            // the maximum passes over)
            far = fmaxf(__low2float(most), __high2float(most)) > 448.0f || vw > 3.0e38f;
          } else {
            float most = 0.0f;
#pragma unroll
            for (int j = 0; j < NH / 2; ++j) {
              most = fmaxf(most, fmaxf(sum[2 * j], sum[2 * j + 1]));
              __nv_bfloat162 hh = __floats2bfloat162_rn(sum[2 * j], sum[2 * j + 1]);
              const float2 back = __bfloat1622float2(hh);
              __nv_bfloat162 ll =
                  __floats2bfloat162_rn(sum[2 * j] - back.x, sum[2 * j + 1] - back.y);
              hi[j] = *reinterpret_cast<uint32_t*>(&hh);
              lo[j] = *reinterpret_cast<uint32_t*>(&ll);
            }
            far = most > kFarWeight;
          }
          // one buffer of weights: the last product has read those before (that of the tile
          // before it is complete: it came before these scores)
          if (S::kPBufs == 1 && ok && i > 0) ok = wait(bar(bars.o_step), (i - 1) & 1);
          const uint32_t at = sbase + S::oP + (S::kPBufs == 2 ? (i & 1) * 2 * S::kPTerm : 0) +
                              w * NH / S::kChunkRows * (kKeys * 16) + key_lane * 16 +
                              (kWords < 4 ? w * kWords * 4 : 0);
#pragma unroll
          for (int term = 0; term < 2; ++term) {
            const uint32_t* v = term == 0 ? hi : lo;
            if constexpr (kWords < 4) {
              asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at + term * S::kPTerm),
                           "r"(v[0]), "r"(v[1])
                           : "memory");
            } else {
#pragma unroll
              for (int q = 0; q < kWords / 4; ++q)
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                                 at + term * S::kPTerm + q * (kKeys * 16)),
                             "r"(v[4 * q]), "r"(v[4 * q + 1]), "r"(v[4 * q + 2]), "r"(v[4 * q + 3])
                             : "memory");
            }
          }
          return far;
        };
        if (now != 0u) prepare(true);
        const bool far = pass();
        if constexpr (kFP8) {
          // rows of which this tile has a weight of at least kSmall (as E4M3 has it)
          const float least = kSmall * rcp_approx(vs * exp2_approx(static_cast<float>(4 - E)));
          uint32_t large = 0;
#pragma unroll
          for (int r = 0; r < NH; ++r) large |= sum[r] >= least ? 1u << r : 0u;
          large = __reduce_or_sync(0xffffffffu, large);
          if (lane == 0) bars.large[i & 1][w][warp & 3] = large;
        }
        bool again = named_bar_any(group_bar, 128, far);
        if constexpr (kFP8) {
          const uint32_t(&large)[4] = bars.large[i & 1][w];
          again = again ||
                  (seeing & ~pending & ~(large[0] | large[1] | large[2] | large[3])) != 0u;
        }
        if (again) {
          prepare(false);
          pass();
        }
#pragma unroll
        for (int r = 0; r < NH; r += 2) add2(l[r], l[r + 1], sum[r], sum[r + 1]);
        fence_async_smem();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bars.p_full[i & 1]));   // (32 arrivals take a hundred cycles)
    }
    if (ok && n > 0) ok = wait(bar(bars.o_last), 0);
    tc_fence_after();

    // ---- results: the sums over the keys, then a channel per lane
    const bool split = share.count > 1;
    float* parts = p.partial + static_cast<int64_t>(job.first) * partial_floats<D>(p.part_rows);
    float* dst = parts + job.part * partial_floats<D>(p.part_rows);
    if (!idle) {
      float o[NH];
#pragma unroll
      for (int r = 0; r < NH; ++r) o[r] = 0.0f;
      float unit = 1.0f;
      if (n > 0 && ok) {
        tmem_ld_cols<NH>(o_tm, o);
        if constexpr (kFP8) {
          float o2[NH];
          tmem_ld_cols<NH>(o_tm + N, o2);
          unit = exp2_approx(static_cast<float>(E - 4));
#pragma unroll
          for (int r = 0; r < NH; ++r) o[r] = fmaf(o2[r], 0.0625f, o[r]);
        }
      }
      const float sum = transposed<NH>(l, [](float a, float c) { return a + c; });
      if ((lane & (32 / NH - 1)) == 0) bars.part[w][warp & 3][lane / (32 / NH)] = sum;
      float mine = 0.0f;                                 // the reference of row key_lane
#pragma unroll
      for (int r = 0; r < NH; ++r) mine = key_lane == r ? -nref[r] : mine;
      named_bar_sync(group_bar, 128);
      if (key_lane < NH) {
        const int row = w * NH + key_lane;
        const bool saw = ok && (seeing >> key_lane & 1u);
        const float all = saw ? (bars.part[w][0][key_lane] + bars.part[w][1][key_lane]) +
                                    (bars.part[w][2][key_lane] + bars.part[w][3][key_lane])
                              : 0.0f;
        const float rf = all != 0.0f ? mine : ninf;
        bars.scale[row] = !saw ? 0.0f : split ? unit : all == 0.0f ? 0.0f : unit / all;
        if (row < t.rows) {
          if (split) {
            dst[static_cast<int64_t>(p.part_rows) * D + row] = rf;
            dst[static_cast<int64_t>(p.part_rows) * (D + 1) + row] = all;
          } else if (p.lse != nullptr) {
            *lse_at(p, t, row) = lse_of(rf, all);
          }
        }
      }
      named_bar_sync(group_bar, 128);
      if (key_lane < D) {
#pragma unroll
        for (int r = 0; r < NH; ++r) {
          const int row = w * NH + r;
          if (row < t.rows) {
            const float g = bars.scale[row];
            const float y = g == 0.0f ? 0.0f : o[r] * g;
            if (split) dst[static_cast<int64_t>(row) * D + key_lane] = y;
            else p.out[bars.out[row] + key_lane] = __float2bfloat16_rn(y);
          }
        }
      }
    }
    if (split)
      join_parts<D>(p, t, parts, p.counters + job.first, p.part_rows, share.count, tid,
                    S::kSoftmax, 1, reinterpret_cast<float*>(smem + S::oSlots), &bars.flag);
  } else if (warp == kMmaWarp) {
    // =================================================================== MMA
    if (n > 0) {
      // (everything uniform over the warp: see the 256-row kernel)
      constexpr uint32_t kFmt = kFP8 ? 0u : 1u;
      const uint32_t idesc_s = make_idesc(kFmt, 128, N);
      const uint32_t idesc_o = make_idesc(kFmt, 128, N) | (1u << 15) | (1u << 16);
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const int tiles = __shfl_sync(0xffffffffu, n, 0);
      // descriptors.  K and Q are K-major; V is MN-major with its channels in groups of one
      // swizzled row (where D = 64 fills half of the 128, a group stride of 0 repeats them);
      // the weights are MN-major without swizzle, [chunk of rows][8 keys][16 bytes].
      constexpr uint32_t kTileHi = kFP8 ? kCodeDescHi<D> : kDescHi;
      constexpr uint32_t kPHi = ((kKeys * 16) >> 4) | (1u << 14);
      const uint32_t k_lo = smem_desc_lo(sbase + S::oSlots);
      const uint32_t v_lo = ((sbase + S::oSlots) >> 4) |
                            ((D == 128 && !kFP8 ? (kHalfBytes >> 4) : 0u) << 16);
      const uint32_t q_lo = smem_desc_lo(sbase + S::oQ);
      const uint32_t p_lo = ((sbase + S::oP) >> 4) | ((128u >> 4) << 16);
      constexpr int kStepKeys = kFP8 ? 32 : 16;          // keys per MMA of the second product
      constexpr int kSteps = kKeys / kStepKeys;
      constexpr uint32_t kVStep = (kStepKeys * (kFP8 ? D : 128)) >> 4;
      constexpr uint32_t kPStep = (kStepKeys * 16) >> 4;
      const int first_key = max(t.lo, k0);
      const int first_step = max(0, first_key - k0) / kStepKeys;
      const int last_steps = (k1 - (k0 + (n - 1) * kKeys) + kStepKeys - 1) / kStepKeys;
      int slot = 0;
      uint32_t parity = 0;
      auto release = [&]() {
        if (elect_one()) umma_commit(bar(bars.empty[0]) + 8 * slot);
        if (++slot == S::kSlots) {
          slot = 0;
          parity ^= 1;
        }
      };
      auto wait_tile = [&]() { return wait(bar(bars.full[0]) + 8 * slot, parity); };
      auto scores = [&](int buf) {
        const uint32_t a = k_lo + slot * (S::kTileBytes >> 4);
        tc_fence_after();
        if (elect_one()) {
          if constexpr (kFP8) {
#pragma unroll
            for (int s = 0; s < 2 * (D / 32); ++s) {     // the query's hi, then lo
              const uint32_t off = ((s % (D / 32)) * 32) >> 4;
              umma_ss<true>(tm + buf * N, a + off, kTileHi,
                            q_lo + (s / (D / 32)) * (S::kQTerm >> 4) + off, kTileHi,
                            s < D / 32 ? idesc_s : idesc_s | kBIsE5M2, s > 0);
            }
          } else {
#pragma unroll
            for (int s = 0; s < D / 16; ++s) {
              const uint32_t in = ((s & 3) * 32) >> 4;
              umma_ss<false>(tm + buf * N, a + (((s >> 2) * kHalfBytes) >> 4) + in, kTileHi,
                             q_lo + (((s >> 2) * N * 128) >> 4) + in, kTileHi, idesc_s, s > 0);
            }
          }
          umma_commit(bar(bars.s_full[0]) + 8 * buf);
        }
        release();
      };
      auto values = [&](int i) {
        const uint32_t a = v_lo + slot * (S::kTileBytes >> 4);
        const bool first = i == 0;
        const uint32_t pb = p_lo + (S::kPBufs == 2 ? (i & 1) * (2 * S::kPTerm >> 4) : 0);
        const int s0 = first ? first_step : 0, s1 = i + 1 == tiles ? last_steps : kSteps;
        tc_fence_after();
        if (elect_one()) {
          if (s0 == 0 && s1 == kSteps) {
#pragma unroll
            for (int x = 0; x < 2 * kSteps; ++x) {       // the weights' hi, then lo
              const int s = x % kSteps, term = x / kSteps;
              umma_ss<kFP8>(tm + S::oO + (kFP8 ? term * N : 0), a + s * kVStep, kTileHi,
                            pb + term * (S::kPTerm >> 4) + s * kPStep, kPHi, idesc_o,
                            (kFP8 ? s > 0 : x > 0) ? 1u : (first ? 0u : 1u));
            }
          } else {
            for (int term = 0; term < 2; ++term)
              for (int s = s0; s < s1; ++s)
                umma_ss<kFP8>(tm + S::oO + (kFP8 ? term * N : 0), a + s * kVStep, kTileHi,
                              pb + term * (S::kPTerm >> 4) + s * kPStep, kPHi, idesc_o,
                              (s > s0 || (!kFP8 && term > 0)) ? 1u : (first ? 0u : 1u));
          }
        }
        release();
      };
      // rows of V in those steps that no row sees
      auto clean = [&](int i) {
        if (i > 0 && i + 1 < tiles) return;
        const int kb = k0 + i * kKeys;
        const int lo = max(0, first_key - kb), hi = k1 - kb;
        if (lo % kStepKeys != 0 || (hi < kKeys && hi % kStepKeys != 0)) {
          const uint32_t base = sbase + S::oSlots + slot * S::kTileBytes;
          auto zero = [&](int r0, int r1) {
            constexpr int kRowPieces = S::kTileBytes / kKeys / 16;
            for (int y = lane; y < (r1 - r0) * kRowPieces; y += 32) {
              const int r = r0 + y / kRowPieces, c = y % kRowPieces;
              const uint32_t at = base + (kFP8 ? r * D + c * 16
                                               : (c >> 3) * kHalfBytes + r * 128 + (c & 7) * 16);
              asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0) : "memory");
            }
          };
          zero(lo / kStepKeys * kStepKeys, lo);
          if (hi < kKeys) zero(hi, min(kKeys, (hi + kStepKeys - 1) / kStepKeys * kStepKeys));
          fence_async_smem();
          __syncwarp();
        }
      };
      bool ok = wait(bar(bars.q_full), 0);
      for (int i = 0; i < 2 && i < tiles && ok; ++i) {
        ok = wait_tile();
        if (ok) scores(i);
      }
      for (int i = 0; i < tiles && ok; ++i) {
        ok = wait_tile() && wait(bar(bars.p_full[0]) + 8 * (i & 1), (i >> 1) & 1);
        if (!ok) break;
        clean(i);
        values(i);
        // o_step: a phase for every product; o_last: the last one
        if (elect_one()) umma_commit(bar(bars.o_step));
        if (i + 1 == tiles && elect_one()) umma_commit(bar(bars.o_last));
        if (i + 2 < tiles) {
          ok = wait_tile();
          if (ok) scores(i & 1);
        }
      }
      if (!ok) {                           // products in flight end before the memory goes
        if (elect_one()) umma_commit(bar(bars.drain));
        __syncwarp();
        mbar_wait_drain(bar(bars.drain), 0, p.timeout_ns);
      }
    }
  } else {
    // =================================================================== TMA loads
    const int box_log2 = min(p.c.page_log2, 7), box = 1 << box_log2;   // (kKeys = 2^7)
    const int segs = kKeys >> box_log2;
    const int first_key = max(t.lo, k0);                  // pages before a window are not read
    const uint64_t policy = policy_evict_first();         // (read once)
    constexpr int kRowBytes = kFP8 ? D : 2 * D;
    bool ok = p.drop_producer == 0;
    int f = 0;
    auto is_mine = [&](int i) {
      const int key = k0 + i * kKeys + lane * box;
      return lane < segs && key < k1 && key + box > first_key;
    };
    // this lane's page of key tile i; fetched some tiles ahead
    auto page_at = [&](int i) {
      return is_mine(i) ? __ldg(table + ((k0 + i * kKeys + lane * box) >> p.c.page_log2)) : 0;
    };
    int slot = 0;
    uint32_t parity = 1;
    auto load = [&](bool v, int i, int page) -> bool {
      const int kb = k0 + i * kKeys;
      const int key = kb + lane * box;
      const bool mine = is_mine(i);
      if (page < 0 || page >= p.c.num_pages) {
        set_error(p.ctrl, MOE_ERR_DEVICE_FAULT, 22);
        page = 0;                          // (a place that exists)
      }
      if (!wait(bar(bars.empty[0]) + 8 * slot, parity)) return false;
      const uint32_t full = bar(bars.full[0]) + 8 * slot;
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
        const uint32_t dst = sbase + S::oSlots + slot * S::kTileBytes;
        if constexpr (kFP8) {
          tma_load_2d(dst + lane * box * D, map, full, 0, row, policy);
        } else {
#pragma unroll
          for (int x = 0; x < D / 64; ++x)
            tma_load_2d(dst + x * kHalfBytes + lane * box * 128, map, full, x * 64, row, policy);
        }
      }
      __syncwarp();
      ++f;
      if (++slot == S::kSlots) {
        slot = 0;
        parity ^= 1;
      }
      return true;
    };
    // in the order that the MMAs take them: keys of the first two tiles, then each tile's
    // values and the keys of the tile after the next
    int pages[3] = {page_at(0), page_at(1), page_at(2)};
    for (int i = 0; i < 2 && i < n && ok; ++i) ok = load(false, i, pages[i]);
    for (int i = 0; i < n && ok; ++i) {
      const int next = page_at(i + 3);
      ok = load(true, i, pages[0]);
      if (ok && i + 2 < n) ok = load(false, i + 2, pages[2]);
      pages[0] = pages[1];
      pages[1] = pages[2];
      pages[2] = next;
    }
    if (!ok)                               // copies in flight land before the memory goes
      for (int g = max(0, f - S::kSlots); g < f; ++g)
        mbar_wait_drain(bar(bars.full[g % S::kSlots]), (g / S::kSlots) & 1, p.timeout_ns);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, S::kTmem);
}

template <int D, bool kFP8, int N>
cudaError_t launch_n(const AttnParams& p, const CUtensorMap& mk, const CUtensorMap& mv,
                     cudaStream_t stream) {
  using S = RowsShape<D, kFP8, N>;
  cudaError_t e = cudaFuncSetAttribute(rows_kernel<D, kFP8, N>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg =
      make_cfg(dim3(p.whole), dim3(S::kThreads), stream, true, attr);
  cfg.dynamicSmemBytes = S::kSmem;
  return cudaLaunchKernelEx(&cfg, rows_kernel<D, kFP8, N>, mk, mv, p);
}

template <int D, bool kFP8>
cudaError_t launch_d(const AttnParams& p, int tile_rows, const CUtensorMap& mk,
                     const CUtensorMap& mv, cudaStream_t stream) {
  if (tile_rows == 16) return launch_n<D, kFP8, 16>(p, mk, mv, stream);
  if (tile_rows == 32) return launch_n<D, kFP8, 32>(p, mk, mv, stream);
  if (tile_rows == 48) return launch_n<D, kFP8, 48>(p, mk, mv, stream);
  if constexpr (kFP8) return cudaErrorInvalidValue;      // (49 rows and more: 256-row tiles)
  else return launch_n<D, kFP8, 64>(p, mk, mv, stream);
}

}  // namespace

int attention_rows_places(int tile_rows, int head_dim, bool fp8) {
  if (tile_rows > 32) return 1;
  if (tile_rows == 16)
    return head_dim == 128 ? (fp8 ? RowsShape<128, true, 16>::kCtas : RowsShape<128, false, 16>::kCtas)
                           : (fp8 ? RowsShape<64, true, 16>::kCtas : RowsShape<64, false, 16>::kCtas);
  return head_dim == 128 ? (fp8 ? RowsShape<128, true, 32>::kCtas : RowsShape<128, false, 32>::kCtas)
                         : (fp8 ? RowsShape<64, true, 32>::kCtas : RowsShape<64, false, 32>::kCtas);
}

cudaError_t launch_attention_rows(const AttnParams& p, int tile_rows, int head_dim, bool fp8,
                                  cudaStream_t stream) {
  CUtensorMap mk, mv;
  if (!cache_maps(p, head_dim, fp8, &mk, &mv)) return cudaErrorInvalidValue;
  if (fp8)
    return head_dim == 128 ? launch_d<128, true>(p, tile_rows, mk, mv, stream)
                           : launch_d<64, true>(p, tile_rows, mk, mv, stream);
  return head_dim == 128 ? launch_d<128, false>(p, tile_rows, mk, mv, stream)
                         : launch_d<64, false>(p, tile_rows, mk, mv, stream);
}

}  // namespace moe
