// The whole gated expert layer for a few tokens (single tokens, drafted runs): two kernels.
//
// With T <= 16 tokens nearly every weight is used for one or two of them, so the layer is one
// pass over the active experts' weights and HBM bounds it; everything else has to hide behind
// that stream.  A warp takes 16 weight rows at a time as the A operand of mma.sync m16n8k16 and
// the tokens as its 8 columns (twice 8 above 8 tokens): the tensor core's legacy path is far
// from its limit at this intensity (one MMA per 256 weights), and it takes the weights from
// registers, so E4M3 codes become binary16 on the way (exact) and no activation has to be
// quantised.  The order of k inside an MMA is free, so a lane loads 16 contiguous bytes of a row
// and uses them as they lie.  Weights come by cp.async into a ring of the warp's own (2 KB a
// step: 16 rows x 128 bytes, kDepth steps ahead); a lane reads back what it copied.
//
// Up: a unit is 8 gate rows and the 8 up rows of the same h columns, in one MMA tile, so
// silu(gate) * up is computed where the sums are; several warps share a unit's K where there
// are few units.  Down: a cluster of 8 CTAs takes 128 output rows, each of its CTAs an equal
// share of all active experts' K; the shares meet over distributed shared memory, in rank order
// (no atomics: repeated calls give the same bits).  Every CTA routes by itself (the same device
// function as moe_route), which costs a microsecond and saves a launch and its wait.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "route_token.cuh"
#include "serve_internal.cuh"

namespace moe {
namespace {

constexpr int kUpThreads = 512, kUpWarps = kUpThreads / 32;
constexpr int kDownThreads = 256, kDownWarps = kDownThreads / 32;
constexpr int kMaxTok = MOE_FEW_TOKENS;
constexpr int kStep = 2048;               // weight bytes of a step: 16 rows x 128
constexpr int kSlot = kStep + 16;         // and the step's block scales
constexpr int kCluster = 8;               // CTAs that share 128 output rows
constexpr int kDownRows = 128;
constexpr int kHRows = 96;                // staged rows of h (128 bytes of weights' k each)

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

template <bool kFP8>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (kFP8)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The power of two that takes a block's largest element into [2^14, 2^15) of binary16, and its
// inverse (largest below 2^-100: as for 2^-100).
__device__ __forceinline__ void block_scale(float amax, float& up, float& down) {
  const int e = max(static_cast<int>(__float_as_uint(amax) >> 23), 27) - 127;   // <= 128
  up = __uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23);
  down = __uint_as_float(static_cast<uint32_t>(e - 14 + 127) << 23);
}

struct FewParams {
  const float* logits;
  const __nv_bfloat16* x;
  const uint8_t* w;
  const float* w_scales;
  const uint8_t* w2;
  const float* w2_scales;
  float* h;                    // [T * k, I], by route
  __nv_bfloat16* out;
  Ctrl* ctrl;
  int T, H, I, E, k;
  float softcap;
  int renorm;
};

__device__ __noinline__ void route_one(const float* row, int E, int k, float softcap, int renorm,
                                       int32_t* ids, float* weights) {
  if (E <= 64) route_token<2>(row, E, k, softcap, renorm, ids, weights);
  else if (E <= 256) route_token<8>(row, E, k, softcap, renorm, ids, weights);
  else route_token<32>(row, E, k, softcap, renorm, ids, weights);
}

// What every CTA knows of the routing, in shared memory.
struct Routing {
  int32_t* ids;                // [T * k]
  float* weights;              // [T * k]
  uint32_t* tokens;            // [E] bit t: token t goes there
  int32_t* active;             // [min(E, T * k)] the experts that any token goes to, ascending
  __host__ __device__ static int bytes(int T, int k, int E) {
    const int routes = T * k;
    return (8 * routes + 4 * E + 4 * (E < routes ? E : routes) + 15) / 16 * 16;
  }
  __device__ Routing(uint8_t* p, int T, int k, int E)
      : ids(reinterpret_cast<int32_t*>(p)),
        weights(reinterpret_cast<float*>(ids + T * k)),
        tokens(reinterpret_cast<uint32_t*>(weights + T * k)),
        active(reinterpret_cast<int32_t*>(tokens + E)) {}
};

// Fills r; returns how many experts are active.  All threads of the CTA.
__device__ __forceinline__ int route_all(const FewParams& p, const Routing& r, int* s_n) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) r.tokens[e] = 0;
  for (int t = warp; t < p.T; t += warps)
    route_one(p.logits + static_cast<size_t>(t) * p.E, p.E, p.k, p.softcap, p.renorm,
              r.ids + t * p.k, r.weights + t * p.k);
  __syncthreads();
  for (int i = threadIdx.x; i < p.T * p.k; i += blockDim.x) {
    const int e = r.ids[i];
    if (e >= 0 && e < p.E)
      atomicOr(r.tokens + e, 1u << (i / p.k));
    else
      set_error(p.ctrl, MOE_ERR_DEVICE_FAULT, 30);   // a NaN logit that no key stands for
  }
  __syncthreads();
  if (warp == 0) {
    int n = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const bool on = e0 + lane < p.E && r.tokens[e0 + lane] != 0;
      const uint32_t m = __ballot_sync(0xffffffffu, on);
      if (on) r.active[n + __popc(m & ((1u << lane) - 1u))] = e0 + lane;
      n += __popc(m);
    }
    if (lane == 0) *s_n = n;
  }
  __syncthreads();
  return *s_n;
}

// The 8 (FP8) or 4 (BF16) MMAs of one step for one group of 8 tokens.  w: the lane's 16 bytes of
// rows g and g + 8 in the two halves of the 128 bytes; b: the lane's token's row at this step.
// FP8: code q of the 16 is k = 16 t + q of its half, and b holds 128 binary16; BF16: 64.
template <bool kFP8>
__device__ __forceinline__ void load_b(uint4 (&b)[4], const uint8_t* row, int t, bool there) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    if constexpr (kFP8) {
      const uint4* q = reinterpret_cast<const uint4*>(row + c * 128 + t * 32);
      b[2 * c] = there ? q[0] : make_uint4(0u, 0u, 0u, 0u);
      b[2 * c + 1] = there ? q[1] : make_uint4(0u, 0u, 0u, 0u);
    } else {
      const uint4* q = reinterpret_cast<const uint4*>(row + c * 64 + t * 16);
      b[c] = there ? q[0] : make_uint4(0u, 0u, 0u, 0u);
    }
  }
}

template <bool kFP8>
struct Weights {
  uint32_t a[kFP8 ? 8 : 4][4];
  // the lane's pieces of a ring slot: row g, row g + 8 of half 0, then of half 1
  __device__ __forceinline__ void load(const uint8_t* slot, int lane) {
    const uint4* q = reinterpret_cast<const uint4*>(slot) + lane;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint4 lo = q[64 * c], hi = q[64 * c + 32];
      const uint32_t l[4] = {lo.x, lo.y, lo.z, lo.w}, u[4] = {hi.x, hi.y, hi.z, hi.w};
      if constexpr (kFP8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[4 * c + i][0] = e4m3x2_to_f16x2(static_cast<uint16_t>(l[i]));
          a[4 * c + i][1] = e4m3x2_to_f16x2(static_cast<uint16_t>(u[i]));
          a[4 * c + i][2] = e4m3x2_to_f16x2(static_cast<uint16_t>(l[i] >> 16));
          a[4 * c + i][3] = e4m3x2_to_f16x2(static_cast<uint16_t>(u[i] >> 16));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          a[2 * c + i][0] = l[2 * i];
          a[2 * c + i][1] = u[2 * i];
          a[2 * c + i][2] = l[2 * i + 1];
          a[2 * c + i][3] = u[2 * i + 1];
        }
      }
    }
  }
  __device__ __forceinline__ void multiply(float (&c)[4], const uint4 (&b)[4]) const {
#pragma unroll
    for (int i = 0; i < (kFP8 ? 4 : 2); ++i) {
      mma16816<kFP8>(c, a[2 * i][0], a[2 * i][1], a[2 * i][2], a[2 * i][3], b[i].x, b[i].y);
      mma16816<kFP8>(c, a[2 * i + 1][0], a[2 * i + 1][1], a[2 * i + 1][2], a[2 * i + 1][3], b[i].z,
                     b[i].w);
    }
  }
};

// Copies one step's 16 rows (two row pointers of the lane, its 16 bytes of both halves).
__device__ __forceinline__ void copy_step(uint32_t slot, const uint8_t* lo, const uint8_t* hi) {
  const uint32_t d = slot + lane_id() * 16;
  cp_async16(d, lo);
  cp_async16(d + 512, hi);
  cp_async16(d + 1024, lo + 64);
  cp_async16(d + 1536, hi + 64);
}

// ----------------------------------------------------------------------------
// Up: h[route, i] = silu(gate_i) * up_i.
template <bool kFP8>
__host__ __device__ constexpr int x_pitch(int H) {   // bytes; tokens 16 or 64 bytes apart in the banks
  return 2 * H + (kFP8 ? 16 : 64);
}

template <bool kFP8, int kGroups, int kDepth>
int up_smem(const FewParams& p) {
  return Routing::bytes(p.T, p.k, p.E) + p.T * x_pitch<kFP8>(p.H) +
         (kFP8 ? p.H / 128 * kMaxTok * 4 : 0) + kUpWarps * kGroups * 512 +
         kUpWarps * kDepth * kSlot;
}

template <bool kFP8, int kGroups, int kDepth>
__global__ void __launch_bounds__(kUpThreads, 1) few_up_kernel(const FewParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int s_n;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const Routing r(smem, p.T, p.k, p.E);
  const int pitch = x_pitch<kFP8>(p.H);
  uint8_t* s_x = smem + Routing::bytes(p.T, p.k, p.E);
  float* s_xs = reinterpret_cast<float*>(s_x + p.T * pitch);            // FP8: [K/128][kMaxTok]
  float4* s_red = reinterpret_cast<float4*>(s_xs + (kFP8 ? p.H / 128 * kMaxTok : 0));
  uint8_t* s_ring = reinterpret_cast<uint8_t*>(s_red + kUpWarps * kGroups * 32) +
                    warp * kDepth * kSlot;
  const uint32_t ring = smem_u32(s_ring);
  pdl_wait();
  pdl_launch_dependents();

  // x into shared memory (a warp per 128 elements of a token)
  const int blocks = (p.H + 127) / 128;
  for (int b = warp; b < p.T * blocks; b += kUpWarps) {
    const int tok = b / blocks, blk = b - tok * blocks;
    const int at = blk * 128 + lane * 4;
    if (!kFP8 && at >= p.H) continue;
    const uint2 raw = __ldg(reinterpret_cast<const uint2*>(p.x + static_cast<size_t>(tok) * p.H + at));
    uint2* dst = reinterpret_cast<uint2*>(s_x + tok * pitch + at * 2);
    if constexpr (kFP8) {
      const float v[4] = {__uint_as_float(raw.x << 16), __uint_as_float(raw.x & 0xffff0000u),
                          __uint_as_float(raw.y << 16), __uint_as_float(raw.y & 0xffff0000u)};
      float amax = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      float up, down;
      block_scale(amax, up, down);
      const __half2 lo = __floats2half2_rn(v[0] * up, v[1] * up);
      const __half2 hi = __floats2half2_rn(v[2] * up, v[3] * up);
      *dst = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
      if (lane == 0) s_xs[blk * kMaxTok + tok] = down;
    } else {
      *dst = raw;
    }
  }
  if (kFP8)      // columns of no token
    for (int i = threadIdx.x; i < blocks * kMaxTok; i += kUpThreads)
      if (i % kMaxTok >= p.T) s_xs[i] = 0.0f;
  const int active = route_all(p, r, &s_n);

  // Warps that share a unit: as many as it takes to give every warp of the grid work.
  const int per_expert = p.I / 8;
  const int units = active * per_expert;
  const int row_bytes = p.H * (kFP8 ? 1 : 2);
  const int nkb = row_bytes / 128;
  int share = 1;
  while (share < 16 && units * share < static_cast<int>(gridDim.x) * kUpWarps && 2 * share <= nkb)
    share *= 2;
  const int sub = warp & (share - 1);
  const int stride = gridDim.x * (kUpWarps / share);
  const int first = blockIdx.x * (kUpWarps / share) + warp / share;

  // the copies run kDepth steps ahead of the products, over the units' boundaries
  int lu = first, lkb = sub;
  const uint8_t* lo = nullptr;
  const float* ls = nullptr;
  auto aim = [&]() {
    if (lu >= units) return;
    const int a = lu / per_expert, i0 = (lu - a * per_expert) * 8;
    const int64_t e = r.active[a];
    lo = p.w + (e * 2 * p.I + i0 + g) * row_bytes + t * 16;
    if constexpr (kFP8) ls = p.w_scales + (e * 2 * p.I + i0) / 128 * nkb;
  };
  aim();
  auto copy = [&](int slot) {
    if (lu < units) {
      const uint32_t d = ring + slot * kSlot;
      const uint8_t* src = lo + lkb * 128;
      copy_step(d, src, src + static_cast<int64_t>(p.I) * row_bytes);
      if (kFP8 && lane < 2) cp_async4(d + kStep + lane * 4, ls + lane * (p.I / 128 * nkb) + lkb);
      lkb += share;
      if (lkb >= nkb) {
        lkb = sub;
        lu += stride;
        aim();
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int d = 0; d < kDepth - 1; ++d) copy(d);

  int slot = 0;
  for (int u = first; u < units; u += stride) {
    const int a = u / per_expert, i0 = (u - a * per_expert) * 8;
    const int e = r.active[a];
    const uint32_t tokens = r.tokens[e];
    float acc[kGroups][4];
#pragma unroll
    for (int n = 0; n < kGroups; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
    for (int kb = sub; kb < nkb; kb += share) {
      __syncwarp();                         // the slot's scales have been read by all lanes
      copy(slot == 0 ? kDepth - 1 : slot - 1);
      cp_wait<kDepth - 1>();
      __syncwarp();
      const uint8_t* s = s_ring + slot * kSlot;
      Weights<kFP8> w;
      w.load(s, lane);
      float gs = 1.0f, us = 1.0f;
      if constexpr (kFP8) {
        gs = *reinterpret_cast<const float*>(s + kStep);
        us = *reinterpret_cast<const float*>(s + kStep + 4);
      }
#pragma unroll
      for (int n = 0; n < kGroups; ++n) {
        if (kGroups > 1 && ((tokens >> (8 * n)) & 255u) == 0) continue;
        const int tok = 8 * n + g;
        uint4 b[4];
        load_b<kFP8>(b, s_x + (tok < p.T ? tok : 0) * pitch + kb * (kFP8 ? 256 : 128), t, true);
        if constexpr (kFP8) {
          float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          w.multiply(c, b);
          const float2 xs = *reinterpret_cast<const float2*>(s_xs + kb * kMaxTok + 8 * n + 2 * t);
          acc[n][0] = fmaf(c[0], gs * xs.x, acc[n][0]);
          acc[n][1] = fmaf(c[1], gs * xs.y, acc[n][1]);
          acc[n][2] = fmaf(c[2], us * xs.x, acc[n][2]);
          acc[n][3] = fmaf(c[3], us * xs.y, acc[n][3]);
        } else {
          w.multiply(acc[n], b);
        }
      }
      slot = slot == kDepth - 1 ? 0 : slot + 1;
    }
    // the sharing warps' sums meet in the first of them
    if (share > 1) {
      const int bar = 1 + warp / share;
      if (sub > 0)
#pragma unroll
        for (int n = 0; n < kGroups; ++n)
          s_red[(warp * kGroups + n) * 32 + lane] =
              make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
      asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(share * 32) : "memory");
      if (sub == 0)
        for (int j = 1; j < share; ++j)
#pragma unroll
          for (int n = 0; n < kGroups; ++n) {
            const float4 v = s_red[((warp + j) * kGroups + n) * 32 + lane];
            acc[n][0] += v.x;
            acc[n][1] += v.y;
            acc[n][2] += v.z;
            acc[n][3] += v.w;
          }
      asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(share * 32) : "memory");
    }
    if (sub != 0) continue;
#pragma unroll
    for (int n = 0; n < kGroups; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int tok = 8 * n + 2 * t + i;
        if (((tokens >> tok) & 1u) == 0) continue;
        int j = 0;
        while (j < p.k - 1 && r.ids[tok * p.k + j] != e) ++j;
        const float gate = acc[n][i], up = acc[n][2 + i];
        p.h[static_cast<size_t>(tok * p.k + j) * p.I + i0 + g] =
            __fdiv_rn(gate, 1.0f + exp_ieee(-gate)) * up;
      }
  }
}

// ----------------------------------------------------------------------------
// Down: out[t, n] = sum over t's experts of weight * (w2[e, n, :] . h).
template <bool kFP8>
constexpr int h_pitch() {                   // bytes; neighbouring rows in other banks
  return kFP8 ? 272 : 320;
}

template <bool kFP8, int kDepth>
int down_smem(const FewParams& p) {
  return Routing::bytes(p.T, p.k, p.E) + kHRows * (h_pitch<kFP8>() + 4 + 8) +
         kDownRows * kMaxTok * 4 + kDownWarps * kDepth * kSlot;
}

template <bool kFP8, int kGroups, int kDepth>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kDownThreads, 2)
    few_down_kernel(const FewParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int s_n;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const Routing r(smem, p.T, p.k, p.E);
  uint8_t* s_h = smem + Routing::bytes(p.T, p.k, p.E);
  float* s_hs = reinterpret_cast<float*>(s_h + kHRows * h_pitch<kFP8>());
  int2* s_step = reinterpret_cast<int2*>(s_hs + kHRows);        // (active expert, first row)
  float* s_part = reinterpret_cast<float*>(s_step + kHRows);    // [row][token]
  uint8_t* s_ring = reinterpret_cast<uint8_t*>(s_part + kDownRows * kMaxTok) + warp * kDepth * kSlot;
  const uint32_t ring = smem_u32(s_ring);
  const int rank = blockIdx.x % kCluster;
  const int n0 = blockIdx.x / kCluster * kDownRows + warp * 16;
  const bool idle = n0 >= p.H;                                  // (H is a multiple of 16)
  const int active = route_all(p, r, &s_n);

  // this CTA's share of the steps (expert by expert, 128 bytes of k each)
  const int row_bytes = p.I * (kFP8 ? 1 : 2);
  const int nkb = row_bytes / 128;
  const int64_t steps = static_cast<int64_t>(active) * nkb;
  const int s0 = static_cast<int>(steps * rank / kCluster);
  const int s1 = static_cast<int>(steps * (rank + 1) / kCluster);

  int ls = s0, la = s0 / nkb, lkb = s0 - la * nkb;
  const uint8_t* lo = nullptr;
  const float* lsc = nullptr;
  auto aim = [&]() {
    if (ls >= s1) return;
    const int64_t e = r.active[la];
    lo = p.w2 + (e * p.H + n0 + g) * row_bytes + t * 16;
    if constexpr (kFP8) lsc = p.w2_scales + (e * (p.H / 128) + n0 / 128) * nkb;
  };
  if (!idle) aim();
  auto copy = [&](int slot) {
    if (ls < s1 && !idle) {
      const uint32_t d = ring + slot * kSlot;
      const uint8_t* src = lo + lkb * 128;
      copy_step(d, src, src + 8 * static_cast<int64_t>(row_bytes));
      if (kFP8 && lane == 0) cp_async4(d + kStep, lsc + lkb);
      ++ls;
      if (++lkb == nkb) {
        lkb = 0;
        ++la;
        aim();
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int d = 0; d < kDepth - 1; ++d) copy(d);
  pdl_wait();                               // the weights above do not depend on the up kernel
  pdl_launch_dependents();

  float acc[kGroups][4];
#pragma unroll
  for (int n = 0; n < kGroups; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
  int slot = 0;
  for (int s = s0; s < s1;) {
    // the next steps whose rows of h (one per token and step) fit
    int count = 0, rows = 0;
    while (s + count < s1) {
      const int a = (s + count) / nkb, kb = (s + count) - a * nkb;
      const int n = __popc(r.tokens[r.active[a]]);
      const int take = min(min(nkb - kb, s1 - s - count), (kHRows - rows) / n);
      if (take == 0) break;
      for (int i = threadIdx.x; i < take; i += kDownThreads) s_step[count + i] = make_int2(a, rows + i * n);
      count += take;
      rows += take * n;
    }
    __syncthreads();
    // h times its route's weight, in the MMA's type
    for (int i = warp; i < count; i += kDownWarps) {
      const int2 at = s_step[i];
      const int e = r.active[at.x], kb = s + i - at.x * nkb;
      uint32_t m = r.tokens[e];
      for (int row = at.y; m != 0; ++row, m &= m - 1) {
        const int tok = __ffs(m) - 1;
        int j = 0;
        while (j < p.k - 1 && r.ids[tok * p.k + j] != e) ++j;
        const int route = tok * p.k + j;
        const float weight = r.weights[route];
        const float* src = p.h + static_cast<size_t>(route) * p.I;
        uint8_t* dst = s_h + row * h_pitch<kFP8>();
        if constexpr (kFP8) {
          float4 v = __ldcg(reinterpret_cast<const float4*>(src + kb * 128) + lane);
          v.x *= weight, v.y *= weight, v.z *= weight, v.w *= weight;
          float amax = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          float up, down;
          block_scale(amax, up, down);
          const __half2 a = __floats2half2_rn(v.x * up, v.y * up);
          const __half2 b = __floats2half2_rn(v.z * up, v.w * up);
          reinterpret_cast<uint2*>(dst)[lane] =
              make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
          if (lane == 0) s_hs[row] = down;
        } else {
          // two bf16 terms: 16 bits of h
          float2 v = __ldcg(reinterpret_cast<const float2*>(src + kb * 64) + lane);
          v.x *= weight, v.y *= weight;
          const __nv_bfloat162 hi = __floats2bfloat162_rn(v.x, v.y);
          const float2 back = __bfloat1622float2(hi);
          const __nv_bfloat162 rest = __floats2bfloat162_rn(v.x - back.x, v.y - back.y);
          reinterpret_cast<uint32_t*>(dst)[lane] = *reinterpret_cast<const uint32_t*>(&hi);
          reinterpret_cast<uint32_t*>(dst + 128)[lane] = *reinterpret_cast<const uint32_t*>(&rest);
        }
      }
    }
    __syncthreads();
    if (!idle) {
      for (int i = 0; i < count; ++i) {
        __syncwarp();
        copy(slot == 0 ? kDepth - 1 : slot - 1);
        cp_wait<kDepth - 1>();
        __syncwarp();
        const uint8_t* sl = s_ring + slot * kSlot;
        Weights<kFP8> w;
        w.load(sl, lane);
        const int2 at = s_step[i];
        const uint32_t tokens = r.tokens[r.active[at.x]];
#pragma unroll
        for (int n = 0; n < kGroups; ++n) {
          if (kGroups > 1 && ((tokens >> (8 * n)) & 255u) == 0) continue;
          auto row_of = [&](int tok) { return at.y + __popc(tokens & ((1u << tok) - 1u)); };
          const int tok = 8 * n + g;
          const bool there = (tokens >> tok) & 1u;
          const uint8_t* row = s_h + (there ? row_of(tok) : at.y) * h_pitch<kFP8>();
          uint4 b[4];
          load_b<kFP8>(b, row, t, there);
          if constexpr (kFP8) {
            const float ws = *reinterpret_cast<const float*>(sl + kStep);
            float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            w.multiply(c, b);
            const int t0 = 8 * n + 2 * t;
            const float h0 = ((tokens >> t0) & 1u) ? s_hs[row_of(t0)] * ws : 0.0f;
            const float h1 = ((tokens >> (t0 + 1)) & 1u) ? s_hs[row_of(t0 + 1)] * ws : 0.0f;
            acc[n][0] = fmaf(c[0], h0, acc[n][0]);
            acc[n][1] = fmaf(c[1], h1, acc[n][1]);
            acc[n][2] = fmaf(c[2], h0, acc[n][2]);
            acc[n][3] = fmaf(c[3], h1, acc[n][3]);
          } else {
            w.multiply(acc[n], b);
            load_b<kFP8>(b, row + 128, t, there);
            w.multiply(acc[n], b);
          }
        }
        slot = slot == kDepth - 1 ? 0 : slot + 1;
      }
    }
    s += count;
    __syncthreads();                        // before the next rows overwrite these
  }
  // the shares meet: rank r adds rows 16 r .. 16 r + 15, in the ranks' order
#pragma unroll
  for (int n = 0; n < kGroups; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      s_part[(warp * 16 + g + 8 * (i >> 1)) * kMaxTok + 8 * n + 2 * t + (i & 1)] = acc[n][i];
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  const int row = threadIdx.x & 15, tok = threadIdx.x >> 4;
  const int n = blockIdx.x / kCluster * kDownRows + rank * 16 + row;
  if (tok < p.T && n < p.H) {
    const uint32_t mine = smem_u32(s_part + (rank * 16 + row) * kMaxTok + tok);
    float part[kCluster];
#pragma unroll
    for (int c = 0; c < kCluster; ++c) {
      uint32_t at;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(mine), "r"(c));
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(part[c]) : "r"(at));
    }
    float sum = part[0];
#pragma unroll
    for (int c = 1; c < kCluster; ++c) sum += part[c];
    p.out[static_cast<size_t>(tok) * p.H + n] = __float2bfloat16_rn(sum);
  }
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

constexpr int kMaxSmem = 226 * 1024;       // 227 KB a CTA, less the static part
constexpr int kDownDepth = 4;

template <bool kFP8, int kGroups, int kDepth>
cudaError_t launch_up(const FewParams& p, int sms, cudaStream_t stream) {
  const int bytes = up_smem<kFP8, kGroups, kDepth>(p);
  cudaError_t e = cudaFuncSetAttribute(few_up_kernel<kFP8, kGroups, kDepth>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = make_cfg(dim3(sms), dim3(kUpThreads), stream, true, attr);
  cfg.dynamicSmemBytes = bytes;
  return cudaLaunchKernelEx(&cfg, few_up_kernel<kFP8, kGroups, kDepth>, p);
}

template <bool kFP8, int kGroups>
cudaError_t launch_few(const FewParams& p, int sms, cudaStream_t stream) {
  // four steps ahead, or two where x takes the room (above 12 tokens of 4096, say)
  cudaError_t e = up_smem<kFP8, kGroups, 4>(p) <= kMaxSmem
                      ? launch_up<kFP8, kGroups, 4>(p, sms, stream)
                      : launch_up<kFP8, kGroups, 2>(p, sms, stream);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(few_down_kernel<kFP8, kGroups, kDownDepth>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = make_cfg(dim3((p.H + kDownRows - 1) / kDownRows * kCluster),
                                    dim3(kDownThreads), stream, true, attr);
  cfg.dynamicSmemBytes = down_smem<kFP8, kDownDepth>(p);
  return cudaLaunchKernelEx(&cfg, few_down_kernel<kFP8, kGroups, kDownDepth>, p);
}

}  // namespace

cudaError_t launch_few_experts(const moe_forward_args& f, void* out, float* h, Ctrl* ctrl,
                               int num_sms, cudaStream_t stream) {
  const bool fp8 = f.dtype == MOE_DTYPE_FP8_E4M3;
  // x of one launch fits shared memory beside the rings
  int most = 65536 / f.K;
  if (most > kMaxTok) most = kMaxTok;
  const int passes = (f.M + most - 1) / most;
  for (int i = 0; i < passes; ++i) {
    const int t0 = f.M * i / passes, t1 = f.M * (i + 1) / passes;
    FewParams p;
    p.logits = f.logits + static_cast<size_t>(t0) * f.E;
    p.x = static_cast<const __nv_bfloat16*>(f.x) + static_cast<size_t>(t0) * f.K;
    p.w = static_cast<const uint8_t*>(f.w);
    p.w_scales = f.w_scales;
    p.w2 = static_cast<const uint8_t*>(f.w2);
    p.w2_scales = f.w2_scales;
    p.h = h + static_cast<size_t>(t0) * f.top_k * f.N;
    p.out = static_cast<__nv_bfloat16*>(out) + static_cast<size_t>(t0) * f.K;
    p.ctrl = ctrl;
    p.T = t1 - t0;
    p.H = f.K;
    p.I = f.N;
    p.E = f.E;
    p.k = f.top_k;
    p.softcap = f.softcap;
    p.renorm = f.renorm;
    cudaError_t e;
    if (fp8)
      e = p.T <= 8 ? launch_few<true, 1>(p, num_sms, stream) : launch_few<true, 2>(p, num_sms, stream);
    else
      e = p.T <= 8 ? launch_few<false, 1>(p, num_sms, stream) : launch_few<false, 2>(p, num_sms, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace moe
