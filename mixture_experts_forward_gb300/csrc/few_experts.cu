// The whole gated expert layer for a few tokens (single tokens, drafted runs): two kernels after
// the router.
//
// With T <= 16 tokens nearly every weight is used for one or two of them, so the layer is one
// pass over the active experts' weights and HBM bounds it; everything else has to hide behind
// that stream.  A warp takes 16 weight rows at a time as the A operand of mma.sync and the tokens
// as its 8 columns (twice 8 above 8 tokens), m16n8k16.  The tensor core's legacy path is far from
// its limit at this intensity (an MMA per 256 weights), takes its operands from registers, so E4M3
// codes become binary16 on the way (exact) and no activation has to be quantised, and leaves the
// sums there: no tensor memory to read back for each 128-deep scale block.  (E4M3 operands in
// m16n8k32 took 170 us instead of 96 for 16 tokens through 69 of 256 experts: that form is made of
// conversions too, one for each MMA.)  The order of k inside
// an MMA is free, so a lane loads 16 contiguous bytes of a row and uses them as they lie.  Weights
// come by cp.async into a ring of the warp's own (4 KB a step: 16 rows x 256 bytes).  A lane copies
// one piece of every second row and reads pieces of two rows, mostly other lanes' copies: each wait
// for the ring is followed by a __syncwarp.
//
// Up: a unit is 8 gate rows and the 8 up rows of the same h columns, in one MMA tile, so
// silu(gate) * up is computed where the sums are; several warps share a unit's K where there
// are few units.  Down: a cluster of up to 8 CTAs takes 64 or 128 output rows (as many CTAs as fill the
// SMs once: clusters of 4 for H = 2048, of 2 for 4096), each of its CTAs an equal share of all
// active experts' K; the shares meet over distributed shared memory, in rank order
// (no atomics: repeated calls give the same bits).  The tokens are routed before by moe_route's
// kernel, during which the up kernel stages x; while the up kernel runs, the down kernel fetches
// its first weights as far as it finds room.  (Routing in every CTA of both kernels instead saved a launch but
// took 8 us of each for 16 tokens and 256 experts.)
//
// Measured (HBM's floor for the experts that the tokens reach in brackets), a pass among others: one
// token, 8 FP8 experts of 512 x 2048 15 us (3.8: the chain of three launches); 16 tokens, 69 of them
// 55-59 us (33: 22 + 12 us of stream at 6.4 TB/s, the rest the router and the kernels' beginnings and
// ends); one token, 2 BF16 experts of 1024 x 4096 15-18 us (7.6); 5 tokens, 18 BF16 experts of
// 1408 x 4096 110-127 us (94).  The 128-token path of moe_forward, in a graph each: FP8 experts of
// 512 x 2048 31 us against 16 here for one token, 46 / 37 for 8, 49 / 51 for 12, 55 / 59 for 16; BF16
// of 1408 x 4096 61 / 45, 149 / 152 (8 tokens), 196 / 218 (12), 220 / 263 (16); from 9 tokens on a
// weight tile meets two groups of MMA columns.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ieee_math.cuh"
#include "serve_internal.cuh"

namespace moe {
namespace {

constexpr int kMaxTok = MOE_FEW_TOKENS;
constexpr int kStepBytes = 256;           // of each row and step: two blocks of 128
constexpr int kSlotBytes = 16 * kStepBytes;   // of the ring: a step's rows,
constexpr int kSlot = kSlotBytes + 16;        // and its blocks' scales
constexpr int kCluster = 8;               // CTAs that share output rows, at most

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// c += a x b; codes as binary16, or BF16.
template <bool kFP8>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (kFP8)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The power of two that takes a block's largest element into [2^14, 2^15) of binary16, and its
// inverse (largest below 2^-100: as for 2^-100).
__device__ __forceinline__ void block_scale(float amax, float& up, float& down) {
  const int e = max(static_cast<int>(__float_as_uint(amax) >> 23), 27) - 127;   // <= 128
  up = __uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23);
  down = __uint_as_float(static_cast<uint32_t>(e - 14 + 127) << 23);
}

// Four codes as binary16, two in each half.
__device__ __forceinline__ void codes_to_halves(uint32_t codes, uint32_t& first, uint32_t& second) {
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
      : "=r"(first), "=r"(second)
      : "r"(codes));
}

// Four values, scaled, as binary16.
__device__ __forceinline__ uint2 halves(const float* v, float up) {
  const __half2 a = __floats2half2_rn(v[0] * up, v[1] * up), b = __floats2half2_rn(v[2] * up, v[3] * up);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

struct FewParams {
  const int32_t* ids;          // [T * k] the routes (moe_route)
  const float* weights;        // [T * k]
  const __nv_bfloat16* x;
  const uint8_t* w;
  const float* w_scales;
  const uint8_t* w2;
  const float* w2_scales;
  float* h;                    // [T * k, I], by route
  __nv_bfloat16* out;
  Ctrl* ctrl;
  int T, H, I, E, k;
  int share;                   // warps that share a unit of the up kernel (a power of two)
  int h_rows;                  // rows of h that the down kernel stages at a time
  int tiles;                   // 16-row tiles of output rows that a down CTA takes (4 or 8),
  int cluster;                 // and how many CTAs share them (1, 2, 4 or 8)
};

// What every CTA knows of the routing, in shared memory.
struct Routing {
  int32_t* ids;                // [T * k]
  float* weights;              // [T * k]
  uint32_t* tokens;            // [E] bit t: token t goes there
  int32_t* active;             // [min(E, T * k)] the experts that any token goes to, ascending
  int32_t* before;             // [active + 1] routes to the experts before each of them
  uint32_t* on;                // [32] bit e % 32 of word e / 32: expert e is active
  uint8_t* choice;             // [active][kMaxTok] which of its k choices that is to the token
  __host__ __device__ static int most(int T, int k, int E) { return E < T * k ? E : T * k; }
  __host__ __device__ static int bytes(int T, int k, int E) {
    return (8 * T * k + 4 * E + (8 + kMaxTok) * most(T, k, E) + 4 + 128 + 15) / 16 * 16;
  }
  __device__ Routing(uint8_t* p, int T, int k, int E)
      : ids(reinterpret_cast<int32_t*>(p)),
        weights(reinterpret_cast<float*>(ids + T * k)),
        tokens(reinterpret_cast<uint32_t*>(weights + T * k)),
        active(reinterpret_cast<int32_t*>(tokens + E)),
        before(active + most(T, k, E)),
        on(reinterpret_cast<uint32_t*>(before + most(T, k, E) + 1)),
        choice(reinterpret_cast<uint8_t*>(on + 32)) {}
  __device__ uint32_t tokens_of(int a) const { return tokens[active[a]]; }
};

// Before the routes are there.
__device__ __forceinline__ void route_clear(const FewParams& p, const Routing& r) {
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) r.tokens[e] = 0;
  if (threadIdx.x < 32) r.on[threadIdx.x] = 0;
  __syncthreads();
}

// Reads the routes and finds the active experts, by all threads; returns how many there are.
// kAll: their weights and `before` too (there after the next barrier).
template <bool kAll>
__device__ __forceinline__ int route_join(const FewParams& p, const Routing& r) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int routes = p.T * p.k;
  const uint32_t inverse = 0xffffffffu / p.k + 1;            // i / k = umulhi(i, inverse), k > 1
  auto token_of = [&](int i) { return p.k == 1 ? i : static_cast<int>(__umulhi(i, inverse)); };
  for (int i = threadIdx.x; i < routes; i += blockDim.x) {
    const int e = __ldcg(p.ids + i);
    if constexpr (kAll) r.weights[i] = __ldcg(p.weights + i);
    r.ids[i] = e;
    if (e >= 0 && e < p.E) {
      atomicOr(r.tokens + e, 1u << token_of(i));
      atomicOr(r.on + (e >> 5), 1u << (e & 31));
    } else {
      set_error(p.ctrl, MOE_ERR_DEVICE_FAULT, kFaultFewRoute);   // a NaN logit that no key stands for
    }
  }
  __syncthreads();
  int active = 0;
  for (int w = 0; w < (p.E + 31) / 32; ++w) active += __popc(r.on[w]);
  for (int i = threadIdx.x; i < routes; i += blockDim.x) {
    const int e = r.ids[i], t = token_of(i);
    if (e < 0 || e >= p.E) continue;
    int a = __popc(r.on[e >> 5] & ((1u << (e & 31)) - 1u));
    for (int w = 0; w < (e >> 5); ++w) a += __popc(r.on[w]);
    r.active[a] = e;                        // (its tokens write the same)
    r.choice[a * kMaxTok + t] = static_cast<uint8_t>(i - t * p.k);
  }
  __syncthreads();
  if (kAll && warp == 0) {
    int sum = 0;
    for (int a0 = 0; a0 < active; a0 += 32) {
      const int a = a0 + lane, n = a < active ? __popc(r.tokens[r.active[a]]) : 0;
      int upto = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += u;
      }
      if (a < active) r.before[a] = sum + upto - n;
      sum += __shfl_sync(0xffffffffu, upto, 31);
    }
    if (lane == 0) r.before[active] = sum;
  }
  return active;
}

// One block of 128 bytes of 16 rows, as A operands: the lane's 16 bytes of rows g and g + 8 in
// its two halves.
template <bool kFP8>
struct Block {
  static constexpr int kMmas = kFP8 ? 4 : 2;             // in each half
  uint32_t a[2 * kMmas][4];
  // the lane's piece of row g in the block's two halves (row g + 8 lies 8 rows further)
  __device__ __forceinline__ void load(const uint8_t* first, const uint8_t* second) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint8_t* q = c == 0 ? first : second;
      const uint4 lo = *reinterpret_cast<const uint4*>(q);
      const uint4 hi = *reinterpret_cast<const uint4*>(q + 8 * kStepBytes);
      const uint32_t l[4] = {lo.x, lo.y, lo.z, lo.w}, u[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
      for (int i = 0; i < kMmas; ++i) {
        uint32_t(&m)[4] = a[kMmas * c + i];
        if constexpr (kFP8) {
          codes_to_halves(l[i], m[0], m[2]);
          codes_to_halves(u[i], m[1], m[3]);
        } else {
          m[0] = l[2 * i], m[1] = u[2 * i], m[2] = l[2 * i + 1], m[3] = u[2 * i + 1];
        }
      }
    }
  }
  // times the activations: 128 binary16 or 64 bf16 of the lane's token's row, or zeros
  __device__ __forceinline__ void multiply(float (&c)[4], const uint8_t* row, int t, bool there) const {
#pragma unroll
    for (int i = 0; i < kMmas; ++i) {
      uint4 b = make_uint4(0u, 0u, 0u, 0u);
      const int at = kFP8 ? i / 2 * 128 + t * 32 + i % 2 * 16 : i * 64 + t * 16;
      if (there) b = *reinterpret_cast<const uint4*>(row + at);
      mma<kFP8>(c, a[2 * i], b.x, b.y);
      mma<kFP8>(c, a[2 * i + 1], b.z, b.w);
    }
  }
};

// Copies one step's 16 rows x 256 bytes (128 unless `both`), two rows an instruction: lane l brings
// 16-byte piece l % 16 of row l / 16 of the pair.  src: the lane's piece of the first pair; the
// second eight rows begin `gap` bytes after the first row.  In the slot the pieces of odd rows change places in
// fours, so that the products' loads (four neighbouring pieces of two rows) meet no bank twice.
__device__ __forceinline__ uint32_t piece_at(int row, int piece) {
  return row * kStepBytes + ((piece ^ ((row & 1) << 2)) << 4);
}
__device__ __forceinline__ void copy_step(uint32_t slot, const uint8_t* src, int64_t row_bytes,
                                          int64_t gap, bool both) {
  const int lane = threadIdx.x & 31, piece = lane & 15;
  if (!both && piece >= 8) return;
  const uint32_t d = slot + piece_at(lane >> 4, piece);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    cp_async16(d + 2 * j * kStepBytes, src);
    src += j == 3 ? gap - 6 * row_bytes : 2 * row_bytes;
  }
}

// ----------------------------------------------------------------------------
// Up: h[route, i] = silu(gate_i) * up_i.  x lies in shared memory, FP8 as binary16 scaled by a
// power of two for each 128 elements; tokens' rows are so far apart that a load's eight 16-byte
// pieces (two tokens') fall into different banks.
template <bool kFP8>
__host__ __device__ constexpr int x_pitch(int H) { return 2 * H + (kFP8 ? 16 : 64); }

// Buffers for the sums of warps that share a unit: two in turn need one barrier a unit, but not
// where they would take the room of a ring (32 KB).
__host__ __device__ constexpr int red_buffers(int groups, int warps) { return groups * warps < 32 ? 2 : 1; }

template <bool kFP8, int kGroups, int kWarps, int kDepth>
int up_smem(const FewParams& p) {
  return Routing::bytes(p.T, p.k, p.E) + p.T * x_pitch<kFP8>(p.H) +
         (kFP8 ? p.H / 128 * 8 * kGroups * 4 : 0) + red_buffers(kGroups, kWarps) * kWarps * kGroups * 512 +
         kWarps * kDepth * kSlot;
}

template <bool kFP8, int kGroups, int kWarps, int kDepth>
__global__ void __launch_bounds__(kWarps * 32, kWarps == 8 ? 2 : 1) few_up_kernel(const FewParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  __shared__ int s_ticket[kWarps][8];
  const Routing r(smem, p.T, p.k, p.E);
  const int pitch = x_pitch<kFP8>(p.H);
  uint8_t* s_x = smem + Routing::bytes(p.T, p.k, p.E);
  float* s_xs = reinterpret_cast<float*>(s_x + p.T * pitch);            // FP8: [K/128][tokens]
  float4* s_red = reinterpret_cast<float4*>(s_xs + (kFP8 ? p.H / 128 * 8 * kGroups : 0));
  uint8_t* s_ring = reinterpret_cast<uint8_t*>(s_red + red_buffers(kGroups, kWarps) * kWarps * kGroups * 32) +
                    warp * kDepth * kSlot;
  const uint32_t ring = smem_u32(s_ring);
  // The warps that share units, and the units they take: after the first `ahead`, which are dealt
  // out, tickets from a counter, each drawn `ahead` units before its own, so that no copy waits for
  // one.
  // SMs do not get equal shares of HBM: with equal shares of the units the first of them
  // were done at half the time of the last (five tokens through 18 BF16 experts: 50 and 109 us).
  const int share = p.share, sub = warp & (share - 1);
  const int row_bytes = p.H * (kFP8 ? 1 : 2);
  const int nkb = row_bytes / 128, steps = (nkb + 1) / 2;
  // (unit j's steps copy up to the start of unit j + 1 + kDepth / steps; tickets drawn with unit
  // j - 1 are known then, and fewer than 8 are at any time)
  const int ahead = kDepth / (steps / share) + 2;
  const int groups = gridDim.x * (kWarps / share);
  volatile int* ticket = s_ticket[warp / share];
  if (sub == 0 && lane < ahead) ticket[lane] = lane * groups + blockIdx.x * (kWarps / share) + warp / share;
  // x into shared memory, 8 elements a lane: it was there before the routing kernel began, which
  // is waited for afterwards
  const int blocks = (p.H + 127) / 128;
  {
    const int per_token = p.H / 8, pieces = p.T * per_token;   // (FP8: whole blocks of 16 pieces)
    const uint32_t inverse = 0xffffffffu / per_token + 1;      // (i * per_token < 2^32)
    const uint4* from = reinterpret_cast<const uint4*>(p.x);
    const int first = threadIdx.x, step = kWarps * 32;
    uint4 next = first < pieces ? __ldg(from + first) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
    for (int i = first; i < (pieces + 31) / 32 * 32; i += step) {
      const uint4 raw = next;
      if (i + step < pieces) next = __ldg(from + i + step);
      const int tok = __umulhi(i, inverse), piece = i - tok * per_token;
      uint4* dst = reinterpret_cast<uint4*>(s_x + tok * pitch + piece * 16);
      if constexpr (kFP8) {
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
        float v[8], amax = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[2 * e] = __uint_as_float(w[e] << 16);
          v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
          amax = fmaxf(amax, fmaxf(fabsf(v[2 * e]), fabsf(v[2 * e + 1])));
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        float up, down;
        block_scale(amax, up, down);
        const uint2 a = halves(v, up), b = halves(v + 4, up);
        if (i < pieces) {
          *dst = make_uint4(a.x, a.y, b.x, b.y);
          if (piece % 16 == 0) s_xs[piece / 16 * 8 * kGroups + tok] = down;
        }
      } else if (i < pieces) {
        *dst = raw;
      }
    }
  }
  if (kFP8)      // columns of no token
    for (int i = threadIdx.x; i < blocks * 8 * kGroups; i += kWarps * 32)
      if (i % (8 * kGroups) >= p.T) s_xs[i] = 0.0f;
  route_clear(p, r);
  pdl_wait();
  pdl_launch_dependents();
  const int active = route_join<false>(p, r);

  const int per_expert = p.I / 8;
  const int units = active * per_expert;
  const int64_t to_up = static_cast<int64_t>(p.I) * row_bytes;     // from a gate row to its up row

  // the copies run kDepth steps ahead of the products, over the units' boundaries
  const uint32_t inverse = 0xffffffffu / per_expert + 1;      // (per_expert >= 16)
  auto expert_of = [&](int u) {             // u / per_expert
    const int a = __umulhi(u, inverse);     // (one too many where u * per_expert passes 2^32)
    return a * per_expert > u ? a - 1 : a;
  };
  int lj = 0, lu = ticket[0], ls = sub;     // the unit that is copied, and its next step
  const uint8_t* src = nullptr;             // the lane's piece of the first rows
  const float* scale = nullptr;             // lanes 0, 1: the gate rows' two; 2, 3: the up rows'
  auto aim = [&]() {
    const int a = expert_of(lu);
    const int64_t row = static_cast<int64_t>(r.active[a]) * 2 * p.I + (lu - a * per_expert) * 8;
    src = p.w + (row + (lane >> 4)) * row_bytes + (lane & 15) * 16 + sub * kStepBytes;
    if constexpr (kFP8)
      scale = p.w_scales + (row + (lane & 2 ? p.I : 0)) / 128 * nkb + 2 * sub + (lane & 1);
  };
  if (lu < units) aim();
  auto copy = [&](int slot) {
    if (lu < units) {
      copy_step(ring + slot * kSlot, src, row_bytes, to_up, 2 * ls + 1 < nkb);
      src += share * kStepBytes;
      if constexpr (kFP8) {
        if (lane < 4 && 2 * ls + (lane & 1) < nkb)
          cp_async4(ring + slot * kSlot + kSlotBytes + lane * 4, scale);
        scale += 2 * share;
      }
      ls += share;
      if (ls >= steps) {
        ls = sub;
        lu = ticket[++lj & 7];
        if (lu < units) aim();
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int d = 0; d < kDepth; ++d) copy(d);

  // the columns' tokens (those of no token read token 0's row: their sums are not used)
  const uint8_t* row[kGroups];
#pragma unroll
  for (int n = 0; n < kGroups; ++n) row[n] = s_x + (8 * n + g < p.T ? 8 * n + g : 0) * pitch;
  const float* xs = s_xs + 2 * t;
  const uint32_t half0 = piece_at(g, t), half1 = piece_at(g, 4 + t);
  int slot = 0, parity = 0;
  for (int j = 0, u = ticket[0]; u < units; u = ticket[++j & 7]) {
    int drawn = 0;
    if (sub == 0 && lane == 0) drawn = ahead * groups + atomicAdd(&p.ctrl->queue, 1u);
    const int a = expert_of(u), i0 = (u - a * per_expert) * 8;
    const uint32_t tokens = r.tokens_of(a);
    float acc[kGroups][4];
#pragma unroll
    for (int n = 0; n < kGroups; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
    for (int s = sub; s < steps; s += share) {
      cp_wait<kDepth - 1>();
      __syncwarp();
      const uint8_t* q = s_ring + slot * kSlot;
      const float* sc = reinterpret_cast<const float*>(q + kSlotBytes);
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int kb = 2 * s + b;
        if (b == 1 && kb >= nkb) break;
        Block<kFP8> w;
        w.load(q + half0 + b * 128, q + half1 + b * 128);
#pragma unroll
        for (int n = 0; n < kGroups; ++n) {
          if (kGroups > 1 && ((tokens >> (8 * n)) & 255u) == 0) continue;
          if constexpr (kFP8) {
            float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            w.multiply(c, row[n] + kb * 256, t, true);
            const float2 x2 = *reinterpret_cast<const float2*>(xs + kb * 8 * kGroups + 8 * n);
            acc[n][0] = fmaf(c[0], sc[b] * x2.x, acc[n][0]);
            acc[n][1] = fmaf(c[1], sc[b] * x2.y, acc[n][1]);
            acc[n][2] = fmaf(c[2], sc[2 + b] * x2.x, acc[n][2]);
            acc[n][3] = fmaf(c[3], sc[2 + b] * x2.y, acc[n][3]);
          } else {
            w.multiply(acc[n], row[n] + kb * 128, t, true);
          }
        }
      }
      __syncwarp();                         // the slot has been read by all lanes
      copy(slot);
      slot = slot == kDepth - 1 ? 0 : slot + 1;
    }
    if (sub == 0 && lane == 0) ticket[(j + ahead) & 7] = drawn;
    // the sharing warps' sums meet in the first of them
    if (share == 1) {
      __syncwarp();
    } else {
      constexpr bool kTwo = red_buffers(kGroups, kWarps) == 2;
      float4* red = s_red + parity * kWarps * kGroups * 32;
      if (kTwo) parity ^= 1;
      if (sub > 0)
#pragma unroll
        for (int n = 0; n < kGroups; ++n)
          red[(warp * kGroups + n) * 32 + lane] =
              make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
      asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / share), "r"(share * 32) : "memory");
      if (sub == 0)
        for (int w = 1; w < share; ++w)
#pragma unroll
          for (int n = 0; n < kGroups; ++n) {
            const float4 v = red[((warp + w) * kGroups + n) * 32 + lane];
            acc[n][0] += v.x;
            acc[n][1] += v.y;
            acc[n][2] += v.z;
            acc[n][3] += v.w;
          }
      if (!kTwo) asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / share), "r"(share * 32) : "memory");
    }
    if (sub != 0) continue;
#pragma unroll
    for (int n = 0; n < kGroups; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int tok = 8 * n + 2 * t + i;
        if (((tokens >> tok) & 1u) == 0) continue;
        const int route = tok * p.k + r.choice[a * kMaxTok + tok];
        const float gate = acc[n][i], up = acc[n][2 + i];
        p.h[static_cast<size_t>(route) * p.I + i0 + g] = __fdiv_rn(gate, 1.0f + exp_ieee(-gate)) * up;
      }
  }
}

// ----------------------------------------------------------------------------
// Down: out[t, n] = sum over t's experts of weight * (w2[e, n, :] . h).  A staged row is one
// block of one token's h, times its weight: FP8 as binary16 scaled by a power of two (11 bits),
// BF16 in two terms (16 bits).
template <bool kFP8>
constexpr int h_pitch() {                   // bytes; as x_pitch
  return kFP8 ? 256 + 16 : 2 * 128 + 64;
}

template <bool kFP8, int kGroups, int kWarps, int kDepth>
int down_smem(const FewParams& p) {
  return Routing::bytes(p.T, p.k, p.E) + p.h_rows * (h_pitch<kFP8>() + 4 + 4) +
         kWarps * 16 * 8 * kGroups * 4 + kWarps * kDepth * kSlot;
}

template <bool kFP8, int kGroups, int kWarps, int kDepth>
__global__ void __launch_bounds__(kWarps * 32, kWarps == 8 ? 2 : 1)
    few_down_kernel(const FewParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int kCols = 8 * kGroups;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const Routing r(smem, p.T, p.k, p.E);
  uint8_t* s_h = smem + Routing::bytes(p.T, p.k, p.E);
  float* s_hs = reinterpret_cast<float*>(s_h + p.h_rows * h_pitch<kFP8>());   // FP8: rows' scales
  int* s_what = reinterpret_cast<int*>(s_hs + p.h_rows);        // what a row holds: route, block
  float* s_part = reinterpret_cast<float*>(s_what + p.h_rows);  // [part][row][token]
  uint8_t* s_ring = reinterpret_cast<uint8_t*>(s_part + kWarps * 16 * kCols) + warp * kDepth * kSlot;
  const uint32_t ring = smem_u32(s_ring);
  const int cluster = p.cluster, rank = blockIdx.x % cluster;
  const int tile = warp % p.tiles, part = warp / p.tiles;       // the parts of a tile's warps
  const int parts = kWarps / p.tiles;                           // take its steps in turn
  const int n_cta = blockIdx.x / cluster * p.tiles * 16, n0 = n_cta + tile * 16;
  const bool idle = n0 >= p.H;                                  // (H is a multiple of 16)
  // (the up kernel has begun, so the routing is done)
  route_clear(p, r);
  const int active = route_join<true>(p, r);
  __syncthreads();

  // this CTA's share of the steps (two blocks each, expert by expert)
  const int row_bytes = p.I * (kFP8 ? 1 : 2);
  const int nkb = row_bytes / 128, per = (nkb + 1) / 2;
  const int all = active * per;             // (at most 512 * 256)
  const int s0 = all * rank / cluster, s1 = all * (rank + 1) / cluster;

  int ls = s0 + part, la = ls / per, lp = ls - la * per;
  const int la0 = la, lp0 = lp;
  const uint8_t* src = nullptr;             // the lane's piece of the first rows
  const float* scale = nullptr;             // lanes 0, 1: the step's two
  auto aim = [&]() {
    const int64_t row = static_cast<int64_t>(r.active[la]) * p.H + n0;
    src = p.w2 + (row + (lane >> 4)) * row_bytes + (lane & 15) * 16 + lp * kStepBytes;
    if constexpr (kFP8) scale = p.w2_scales + row / 128 * nkb + 2 * lp + (lane & 1);
  };
  if (!idle && ls < s1) aim();
  auto copy = [&](int slot) {
    if (ls < s1 && !idle) {
      copy_step(ring + slot * kSlot, src, row_bytes, 8 * static_cast<int64_t>(row_bytes), 2 * lp + 1 < nkb);
      src += parts * kStepBytes;
      if constexpr (kFP8) {
        if (lane < 2 && 2 * lp + lane < nkb)
          cp_async4(ring + slot * kSlot + kSlotBytes + lane * 4, scale);
        scale += 2 * parts;
      }
      ls += parts;
      lp += parts;
      if (lp >= per) {
        while (lp >= per) lp -= per, ++la;
        if (ls < s1) aim();
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int d = 0; d < kDepth; ++d) copy(d);
  float acc[kGroups][4];
#pragma unroll
  for (int n = 0; n < kGroups; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
  const uint32_t half0 = piece_at(g, t), half1 = piece_at(g, 4 + t);
  // Row of block kb of expert a's first token, counted over all of them: those of a block are
  // neighbours, then come the expert's next blocks.
  auto row_at = [&](int a, int kb) { return r.before[a] * nkb + (r.before[a + 1] - r.before[a]) * kb; };
  auto row_of_step = [&](int s) {
    const int a = s / per;
    return a >= active ? r.before[active] * nkb : row_at(a, 2 * (s - a * per));
  };
  bool waited = false;                      // for the up kernel: nothing so far depends on it
  int slot = 0;
  int ca = la0, cp = lp0;                   // the warp's next step
  for (int s = s0; s < s1;) {
    // the next steps whose rows of h fit
    const int first = row_of_step(s);
    int end = s1;
    if (row_of_step(end) - first > p.h_rows) {
      int lo = s + 1, hi = s1;              // (one step always fits) the first end that does not
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (row_of_step(mid) - first > p.h_rows) hi = mid; else lo = mid;
      }
      end = lo;
    }
    const int rows = row_of_step(end) - first;
    for (int i = threadIdx.x; i < rows; i += kWarps * 32) {
      const int at = first + i;
      int lo = 0, hi = active;              // its expert
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (r.before[mid] * nkb <= at) lo = mid; else hi = mid;
      }
      const int n = r.before[lo + 1] - r.before[lo];
      const int in = at - r.before[lo] * nkb, kb = in / n;
      uint32_t tokens = r.tokens_of(lo);
      for (int q = in - kb * n; q > 0; --q) tokens &= tokens - 1;
      const int tok = __ffs(tokens) - 1;
      s_what[i] = kb << 16 | (tok * p.k + r.choice[lo * kMaxTok + tok]);
    }
    __syncthreads();
    if (!waited) pdl_wait();
    waited = true;
    // h times its route's weight, in the MMA's types; eight rows' loads in flight
    constexpr int kAtOnce = 8;
    for (int i0 = warp; i0 < rows; i0 += kAtOnce * kWarps) {
      float v[kAtOnce][4];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int i = i0 + j * kWarps;
        if (i >= rows) break;
        const float* src = p.h + static_cast<size_t>(s_what[i] & 0xffff) * p.I;
        const int kb = s_what[i] >> 16;
        if constexpr (kFP8) {
          const float4 f = __ldcg(reinterpret_cast<const float4*>(src + kb * 128) + lane);
          v[j][0] = f.x, v[j][1] = f.y, v[j][2] = f.z, v[j][3] = f.w;
        } else {
          const float2 f = __ldcg(reinterpret_cast<const float2*>(src + kb * 64) + lane);
          v[j][0] = f.x, v[j][1] = f.y;
        }
      }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int i = i0 + j * kWarps;
        if (i >= rows) break;
        const float weight = r.weights[s_what[i] & 0xffff];
        if constexpr (kFP8) {
          float amax = 0.0f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[j][e] *= weight;
            amax = fmaxf(amax, fabsf(v[j][e]));
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          float up, down;
          block_scale(amax, up, down);
          *reinterpret_cast<uint2*>(s_h + i * h_pitch<kFP8>() + lane * 8) = halves(v[j], up);
          if (lane == 0) s_hs[i] = down;
        } else {
          const float x = v[j][0] * weight, y = v[j][1] * weight;
          const __nv_bfloat162 hi = __floats2bfloat162_rn(x, y);
          const float2 back = __bfloat1622float2(hi);
          // (nothing beside an infinity: it would be a NaN)
          const __nv_bfloat162 rest = __floats2bfloat162_rn(isinf(back.x) ? 0.0f : x - back.x,
                                                            isinf(back.y) ? 0.0f : y - back.y);
          uint32_t* dst = reinterpret_cast<uint32_t*>(s_h + i * h_pitch<kFP8>()) + lane;
          dst[0] = *reinterpret_cast<const uint32_t*>(&hi);
          dst[32] = *reinterpret_cast<const uint32_t*>(&rest);
        }
      }
    }
    __syncthreads();
    if (!idle) {
      for (; ca * per + cp < end;) {
        const int a = ca, kb0 = 2 * cp;
        const uint32_t tokens = r.tokens_of(a);
        const bool both = kb0 + 1 < nkb;
        cp += parts;
        while (cp >= per) cp -= per, ++ca;
        cp_wait<kDepth - 1>();
        __syncwarp();
        const uint8_t* q = s_ring + slot * kSlot;
        const float* sc = reinterpret_cast<const float*>(q + kSlotBytes);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          if (b == 1 && !both) break;
          Block<kFP8> w;
          w.load(q + half0 + b * 128, q + half1 + b * 128);
          const int base = row_at(a, kb0 + b) - first;
#pragma unroll
          for (int n = 0; n < kGroups; ++n) {
            if (kGroups > 1 && ((tokens >> (8 * n)) & 255u) == 0) continue;
            auto row_of = [&](int tok) { return base + __popc(tokens & ((1u << tok) - 1u)); };
            const int tok = 8 * n + g;
            const bool there = (tokens >> tok) & 1u;
            const uint8_t* row = s_h + row_of(tok) * h_pitch<kFP8>();
            // A column whose token does not go to the expert keeps its sums: 0 times a weight that
            // is not finite is a NaN.
            const int t0 = 8 * n + 2 * t;
            const bool in0 = (tokens >> t0) & 1u, in1 = (tokens >> (t0 + 1)) & 1u;
            if constexpr (kFP8) {
              float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
              w.multiply(c, row, t, there);
              const float h0 = in0 ? s_hs[row_of(t0)] * sc[b] : 0.0f;
              const float h1 = in1 ? s_hs[row_of(t0 + 1)] * sc[b] : 0.0f;
              acc[n][0] = in0 ? fmaf(c[0], h0, acc[n][0]) : acc[n][0];
              acc[n][1] = in1 ? fmaf(c[1], h1, acc[n][1]) : acc[n][1];
              acc[n][2] = in0 ? fmaf(c[2], h0, acc[n][2]) : acc[n][2];
              acc[n][3] = in1 ? fmaf(c[3], h1, acc[n][3]) : acc[n][3];
            } else {
              float c[4] = {acc[n][0], acc[n][1], acc[n][2], acc[n][3]};
              w.multiply(c, row, t, there);
              w.multiply(c, row + 128, t, there);
              if (in0) acc[n][0] = c[0], acc[n][2] = c[2];
              if (in1) acc[n][1] = c[1], acc[n][3] = c[3];
            }
          }
        }
        __syncwarp();
        copy(slot);
        slot = slot == kDepth - 1 ? 0 : slot + 1;
      }
    }
    s = end;
    __syncthreads();                        // before the next rows overwrite these
  }
  if (!waited) pdl_wait();
  pdl_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) p.ctrl->queue = 0;   // for the next up kernel
  // a tile's parts meet in the first of them, then the shares, in the ranks' order: rank r adds its
  // part of the rows
  auto part_at = [&](int q, int n, int i) -> float& {
    return s_part[((q * p.tiles + tile) * 16 + g + 8 * (i >> 1)) * kCols + 8 * n + 2 * t + (i & 1)];
  };
  if (part > 0)
#pragma unroll
    for (int n = 0; n < kGroups; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) part_at(part, n, i) = acc[n][i];
  __syncthreads();
  if (part == 0) {
    for (int q = 1; q < parts; ++q)
#pragma unroll
      for (int n = 0; n < kGroups; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][i] += part_at(q, n, i);
#pragma unroll
    for (int n = 0; n < kGroups; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) part_at(0, n, i) = acc[n][i];
  }
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  const int rows = p.tiles * 16 / cluster;
  for (int i = threadIdx.x; i < rows * p.T; i += kWarps * 32) {
    const int tok = i / rows, row = rank * rows + i - tok * rows;
    const int n = n_cta + row;
    if (n >= p.H) continue;
    const uint32_t mine = smem_u32(s_part + row * kCols + tok);
    float v[kCluster];
#pragma unroll
    for (int c = 0; c < kCluster; ++c) {
      v[c] = 0.0f;
      if (c >= cluster) continue;
      uint32_t at;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(mine), "r"(c));
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v[c]) : "r"(at));
    }
    float sum = v[0];
#pragma unroll
    for (int c = 1; c < kCluster; ++c) sum += v[c];
    p.out[static_cast<size_t>(tok) * p.H + n] = __float2bfloat16_rn(sum);
  }
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

constexpr int kMaxSmem = 226 * 1024;       // 227 KB a CTA, less the static part

template <bool kFP8, int kGroups, int kWarps, int kDepth>
cudaError_t launch_up(const FewParams& p, int sms, cudaStream_t stream) {
  auto* kernel = few_up_kernel<kFP8, kGroups, kWarps, kDepth>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  if (e == cudaSuccess) e = prefer_max_shared(kernel);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = make_cfg(dim3(sms), dim3(kWarps * 32), stream, true, attr);
  cfg.dynamicSmemBytes = up_smem<kFP8, kGroups, kWarps, kDepth>(p);
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <bool kFP8, int kGroups, int kWarps, int kDepth>
cudaError_t launch_down(const FewParams& p, cudaStream_t stream) {
  auto* kernel = few_down_kernel<kFP8, kGroups, kWarps, kDepth>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  if (e == cudaSuccess) e = prefer_max_shared(kernel);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = make_cfg(dim3((p.H + p.tiles * 16 - 1) / (p.tiles * 16) * p.cluster),
                                    dim3(kWarps * 32), stream, true, attr);
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.numAttrs = 2;
  cfg.dynamicSmemBytes = down_smem<kFP8, kGroups, kWarps, kDepth>(p);
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// Warps that share a unit: the fewest steps of the longest warp if all routes go to experts of their
// own, a step and a half more for a join (one token through 8 FP8 experts: 15, 16 and 18 us with 2,
// 4 and 8; 16 tokens through 69: 66, 66, 69, 77 with 1 to 8; 5 through 18 BF16 experts: 116, 112 and 111
// with 2, 4 and 8).
int unit_share(const FewParams& p, bool fp8, int warps, int sms) {
  const int steps = (p.H * (fp8 ? 1 : 2) / 128 + 1) / 2;
  const int64_t units = static_cast<int64_t>(Routing::most(p.T, p.k, p.E)) * p.I / 8;
  int share = 1;
  double best = 1e30;
  for (int n = 1; n <= warps && n <= steps; n *= 2) {
    const int64_t groups = static_cast<int64_t>(sms) * (warps / n);
    const double cost = static_cast<double>((units + groups - 1) / groups) *
                        ((steps + n - 1) / n + (n > 1 ? 1.5 : 0.0));
    if (cost < best) best = cost, share = n;
  }
  return share;
}

template <bool kFP8, int kGroups>
cudaError_t launch_few(FewParams p, int sms, cudaStream_t stream) {
  // 8 warps an SM leave room for the down kernel's CTAs beside the up kernel's, which pays where the
  // work is small; 16 stream faster.  x takes what room the rings leave.
  const int64_t routed = static_cast<int64_t>(Routing::most(p.T, p.k, p.E)) * 2 * p.I * p.H * (kFP8 ? 1 : 2);
  const bool small = routed <= (32ll << 20);
  // One round over the SMs with as many CTAs as it takes: clusters of 8 find room for 15 on 152
  // SMs with a CTA each, those of 4 for 36.
  p.tiles = (p.H + 63) / 64 <= sms ? 4 : 8;
  const int chunks = (p.H + p.tiles * 16 - 1) / (p.tiles * 16);
  p.cluster = chunks * 8 <= sms * 3 / 4 ? 8 : chunks * 4 <= sms * 15 / 16 ? 4 : chunks * 2 <= sms ? 2 : 1;
  // rows of h at a time: all of a share's if they are spread evenly, as far as there is room
  const int64_t even = static_cast<int64_t>(p.T) * p.k * p.I * (kFP8 ? 1 : 2) / 128 / p.cluster * 5 / 4 + 32;
  p.h_rows = 0;
  const int fixed = small ? down_smem<kFP8, kGroups, 8, 3>(p) : down_smem<kFP8, kGroups, 16, 2>(p);
  const int64_t room = ((small ? kMaxSmem / 2 : kMaxSmem) - fixed) / (h_pitch<kFP8>() + 8);
  p.h_rows = static_cast<int>(even < room ? even : room < 32 ? 32 : room) / 4 * 4;
  cudaError_t e;
  const bool wide = !small && up_smem<kFP8, kGroups, 16, 2>(p) <= kMaxSmem;
  p.share = unit_share(p, kFP8, wide ? 16 : 8, sms);
  if (wide)
    e = launch_up<kFP8, kGroups, 16, 2>(p, sms, stream);
  else if (up_smem<kFP8, kGroups, 8, 3>(p) <= kMaxSmem)
    e = launch_up<kFP8, kGroups, 8, 3>(p, sms, stream);
  else
    e = launch_up<kFP8, kGroups, 8, 2>(p, sms, stream);
  if (e != cudaSuccess) return e;
  return small ? launch_down<kFP8, kGroups, 8, 3>(p, stream)
               : launch_down<kFP8, kGroups, 16, 2>(p, stream);
}

// Whether x of p.T tokens and the routes' tables leave room for the up kernel's smallest rings.
template <bool kFP8>
bool tokens_fit(const FewParams& p) {
  return (p.T <= 8 ? up_smem<kFP8, 1, 8, 2>(p) : up_smem<kFP8, 2, 8, 2>(p)) <= kMaxSmem;
}

}  // namespace

cudaError_t launch_few_experts(const moe_forward_args& f, void* out, uint8_t* ws, int num_sms,
                               cudaStream_t stream) {
  const bool fp8 = f.dtype == MOE_DTYPE_FP8_E4M3;
  // x of one launch fits shared memory beside the rings, and beside the routes' tables: these take up
  // to 20 KB, so with hundreds of experts and 24 or more choices M * K near 65536 needs a pass more
  int most = 65536 / f.K;
  if (most > kMaxTok) most = kMaxTok;
  int passes = (f.M + most - 1) / most;
  for (FewParams p = {};; ++passes) {       // (one token always fits)
    p.T = (f.M + passes - 1) / passes;
    p.H = f.K;
    p.E = f.E;
    p.k = f.top_k;
    if (p.T == 1 || (fp8 ? tokens_fit<true>(p) : tokens_fit<false>(p))) break;
  }
  int32_t* ids = reinterpret_cast<int32_t*>(ws + MOE_CTRL_BYTES);
  float* weights = reinterpret_cast<float*>(ids + kMaxTok * 32);
  cudaError_t e = launch_route(f.logits, f.M, f.E, f.top_k, f.softcap, f.renorm, ids, weights, stream, true);
  if (e != cudaSuccess) return e;
  for (int i = 0; i < passes; ++i) {
    const int t0 = f.M * i / passes, t1 = f.M * (i + 1) / passes;
    FewParams p;
    p.ids = ids + t0 * f.top_k;
    p.weights = weights + t0 * f.top_k;
    p.x = static_cast<const __nv_bfloat16*>(f.x) + static_cast<size_t>(t0) * f.K;
    p.w = static_cast<const uint8_t*>(f.w);
    p.w_scales = f.w_scales;
    p.w2 = static_cast<const uint8_t*>(f.w2);
    p.w2_scales = f.w2_scales;
    p.out = static_cast<__nv_bfloat16*>(out) + static_cast<size_t>(t0) * f.K;
    p.ctrl = reinterpret_cast<Ctrl*>(ws);
    // (every pass has the same place: its kernels wait for those of the pass before)
    p.h = weights + kMaxTok * 32;
    p.T = t1 - t0;
    p.H = f.K;
    p.I = f.N;
    p.E = f.E;
    p.k = f.top_k;
    if (fp8)
      e = p.T <= 8 ? launch_few<true, 1>(p, num_sms, stream) : launch_few<true, 2>(p, num_sms, stream);
    else
      e = p.T <= 8 ? launch_few<false, 1>(p, num_sms, stream) : launch_few<false, 2>(p, num_sms, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace moe
