// Rotary positions, alone or on the way into the paged cache.
//
// A CTA takes a few tokens.  Its threads first compute the tokens' cosines and sines into shared
// memory, once for all heads: the angle is position * table mod 2^64, in fractions of a turn, an
// integer product that is exact however far the position is; as binary32 (all 64 bits rounded once)
// it carries a relative error of 2^-24 into sincospif, also for slow pairs at small positions.
// Then each thread takes pieces of 16 elements: two runs of 8 (16-byte loads and stores) that hold
// whole pairs, so a piece needs no other thread's elements: in the half layout runs i .. i+7 and
// i + rotary_dim/2 .., else 16 neighbours.  A row's pieces lie in neighbouring lanes, which share
// its maximum by shuffles where the cache is FP8.
// One pass, bound by HBM; below a few hundred tokens by the launch.  16384 tokens of 32 + 2 x 8
// heads of 128 from a packed projection into an FP8 cache take 70 us (5.3 TB/s, 80 % of a copy's
// rate), 5003 of 24 + 2 x 8 heads of 64 into a BF16 one 12 us in a graph, 32 tokens 4 us.  The next
// pieces loaded a turn ahead gave 69 us for twice the code.
#include "quant_common.cuh"
#include "serve_internal.cuh"

namespace moe {
namespace {

constexpr int kRotThreads = 256;

struct RotaryParams {
  const uint64_t* table;
  const int32_t* positions;
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  __nv_bfloat16* q_out;
  __nv_bfloat16* k_out;
  const int32_t* slots;
  int64_t q_st, q_sh, k_st, k_sh, v_st, v_sh, qo_st, qo_sh, ko_st, ko_sh;
  KvCacheView c;
  Ctrl* ctrl;
  int T, q_heads, kv_heads, head_dim, rotary_dim, tokens;
  float amplitude;
};

__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ uint2 codes8(const float (&v)[8], float inv, uint32_t keep) {
  uint32_t u[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint16_t lo = cvt_e4m3x2(__fmul_rn(v[4 * i], inv), __fmul_rn(v[4 * i + 1], inv));
    const uint16_t hi = cvt_e4m3x2(__fmul_rn(v[4 * i + 2], inv), __fmul_rn(v[4 * i + 3], inv));
    u[i] = (static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16)) & keep;
  }
  return make_uint2(u[0], u[1]);
}

// kD: the head size, or 0 for any (without a cache).  kCache: 0 none, 1 BF16, 2 FP8.
template <int kD, int kCache, bool kInter>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const RotaryParams p) {
  extern __shared__ float s_cos[];          // [tokens][half], then the sines
  __shared__ int s_slot[8];
  pdl_wait();
  pdl_launch_dependents();
  const int D = kD > 0 ? kD : p.head_dim;
  const int half = p.rotary_dim / 2;
  const int t0 = blockIdx.x * p.tokens;
  const int n = min(p.tokens, p.T - t0);
  float* s_sin = s_cos + p.tokens * half;
  for (int i = threadIdx.x; i < n * half; i += kRotThreads) {
    const int tok = i / half;
    const int64_t pos = __ldg(p.positions + t0 + tok);
    const uint64_t turn = static_cast<uint64_t>(pos) * __ldg(p.table + (i - tok * half));
    // half turns in [-1, 1]
    const float x = static_cast<float>(static_cast<int64_t>(turn)) * 0x1p-63f;
    float s, c;
    sincospif(x, &s, &c);
    s_cos[i] = c * p.amplitude;
    s_sin[i] = s * p.amplitude;
  }
  if constexpr (kCache != 0) {
    if (threadIdx.x < n) {
      int slot = __ldg(p.slots + t0 + threadIdx.x);
      if (slot < -1 || (slot >> p.c.page_log2) >= p.c.num_pages) {
        set_error(p.ctrl, MOE_ERR_DEVICE_FAULT, kFaultRotarySlot);
        slot = -1;
      }
      s_slot[threadIdx.x] = slot;
    }
  }
  __syncthreads();

  const int per_row = D / 16;
  const int rows = p.q_heads + p.kv_heads * (kCache != 0 ? 2 : 1);
  const int pieces = rows * per_row;
  // blockIdx.y shares a token's rows where there are few tokens; whole warps, for the shuffles
  for (int i0 = blockIdx.y * kRotThreads; i0 < n * pieces; i0 += gridDim.y * kRotThreads) {
    const int i = i0 + threadIdx.x;
    const bool valid = i < n * pieces;
    const int tok = valid ? i / pieces : 0;
    const int rest = valid ? i - tok * pieces : 0;
    const int row = rest / per_row, piece = rest - row * per_row;
    const int64_t t = t0 + tok;
    const __nv_bfloat16* src;
    int h;
    int kind;                               // 0 q, 1 k, 2 v
    if (row < p.q_heads) {
      kind = 0, h = row, src = p.q + t * p.q_st + h * p.q_sh;
    } else if (kCache == 0 || row < p.q_heads + p.kv_heads) {
      kind = 1, h = row - p.q_heads, src = p.k + t * p.k_st + h * p.k_sh;
    } else {
      kind = 2, h = row - p.q_heads - p.kv_heads, src = p.v + t * p.v_st + h * p.v_sh;
    }
    const bool turned = kind < 2 && piece * 16 < p.rotary_dim;
    // the two runs of 8 elements
    const int e0 = turned && !kInter ? piece * 8 : piece * 16;
    const int e1 = turned && !kInter ? piece * 8 + half : piece * 16 + 8;
    float a[8], b[8];
    {
      uint4 wa = make_uint4(0u, 0u, 0u, 0u), wb = wa;
      if (valid) {
        wa = *reinterpret_cast<const uint4*>(src + e0);
        wb = *reinterpret_cast<const uint4*>(src + e1);
      }
      unpack8(wa, a);
      unpack8(wb, b);
    }
    if (turned) {
      const float4* c4 = reinterpret_cast<const float4*>(s_cos + tok * half + piece * 8);
      const float4* s4 = reinterpret_cast<const float4*>(s_sin + tok * half + piece * 8);
      const float4 c0 = c4[0], c1 = c4[1], n0 = s4[0], n1 = s4[1];
      const float c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
      const float s[8] = {n0.x, n0.y, n0.z, n0.w, n1.x, n1.y, n1.z, n1.w};
      if constexpr (kInter) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x = a[2 * j], y = a[2 * j + 1], u = b[2 * j], w = b[2 * j + 1];
          a[2 * j] = x * c[j] - y * s[j];
          a[2 * j + 1] = x * s[j] + y * c[j];
          b[2 * j] = u * c[4 + j] - w * s[4 + j];
          b[2 * j + 1] = u * s[4 + j] + w * c[4 + j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float x = a[j], y = b[j];
          a[j] = x * c[j] - y * s[j];
          b[j] = x * s[j] + y * c[j];
        }
      }
    }
    if (valid && (kCache == 0 || kind == 0)) {
      __nv_bfloat16* dst = kind == 0 ? p.q_out + t * p.qo_st + h * p.qo_sh
                                     : p.k_out + t * p.ko_st + h * p.ko_sh;
      *reinterpret_cast<uint4*>(dst + e0) = pack8(a);
      *reinterpret_cast<uint4*>(dst + e1) = pack8(b);
    }
    if constexpr (kCache != 0) {
      const int slot = s_slot[tok];
      const int64_t at = ((static_cast<int64_t>(slot >> p.c.page_log2) * p.c.heads + h)
                          << p.c.page_log2) + (slot & ((1 << p.c.page_log2) - 1));
      uint8_t* cache = kind == 1 ? p.c.k : p.c.v;
      const bool store = valid && kind > 0 && slot >= 0;
      if constexpr (kCache == 1) {
        if (!store) continue;
        __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(cache) + at * D;
        *reinterpret_cast<uint4*>(dst + e0) = pack8(a);
        *reinterpret_cast<uint4*>(dst + e1) = pack8(b);
      } else {
        // as moe_kv_write: a = max |x|, s = a/448, code = E4M3(x * (1/s))
        float amax = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fmaxf(fabsf(a[j]), fabsf(b[j])));
#pragma unroll
        for (int o = 1; o < kD / 16; o <<= 1)
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        float scale = 0.0f, inv = 0.0f;
        if (amax >= amax_floor()) {
          scale = __fdiv_rn(amax, 448.0f);
          inv = __fdiv_rn(1.0f, scale);
        }
        if (!store) continue;
        const uint32_t keep = scale == 0.0f ? 0x7f7f7f7fu : 0xffffffffu;
        uint8_t* dst = cache + at * D;
        *reinterpret_cast<uint2*>(dst + e0) = codes8(a, inv, keep);
        *reinterpret_cast<uint2*>(dst + e1) = codes8(b, inv, keep);
        if (piece == 0) (kind == 1 ? p.c.k_scales : p.c.v_scales)[at] = scale;
      }
    }
  }
}

template <int kD, int kCache>
cudaError_t launch(const RotaryParams& p, bool interleaved, dim3 grid, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = make_cfg(grid, dim3(kRotThreads), stream, true, attr);
  cfg.dynamicSmemBytes = p.tokens * p.rotary_dim * 4;
  return interleaved ? cudaLaunchKernelEx(&cfg, rotary_kernel<kD, kCache, true>, p)
                     : cudaLaunchKernelEx(&cfg, rotary_kernel<kD, kCache, false>, p);
}

}  // namespace

cudaError_t launch_rotary(const moe_rotary_args& a, const KvCacheView* cache, Ctrl* ctrl,
                          int num_sms, cudaStream_t stream) {
  RotaryParams p = {};
  p.table = a.table;
  p.positions = a.positions;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.k = static_cast<const __nv_bfloat16*>(a.k);
  p.v = static_cast<const __nv_bfloat16*>(a.v);
  p.q_out = static_cast<__nv_bfloat16*>(a.q_out);
  p.k_out = static_cast<__nv_bfloat16*>(a.k_out);
  p.slots = a.slots;
  p.q_st = a.q_stride_t, p.q_sh = a.q_stride_h;
  p.k_st = a.k_stride_t, p.k_sh = a.k_stride_h;
  p.v_st = a.v_stride_t, p.v_sh = a.v_stride_h;
  p.qo_st = a.q_out_stride_t, p.qo_sh = a.q_out_stride_h;
  p.ko_st = a.k_out_stride_t, p.ko_sh = a.k_out_stride_h;
  if (cache != nullptr) p.c = *cache;
  p.ctrl = ctrl;
  p.T = a.T;
  p.q_heads = a.q_heads;
  p.kv_heads = a.kv_heads;
  p.head_dim = a.head_dim;
  p.rotary_dim = a.rotary_dim;
  p.amplitude = a.amplitude;
  // Four tokens a CTA where that fills the SMs several times over, else one, whose rows then go
  // to several CTAs until every SM has one.
  p.tokens = a.T >= 16 * num_sms ? 4 : 1;
  const int pieces = (a.q_heads + a.kv_heads * (cache != nullptr ? 2 : 1)) * (a.head_dim / 16);
  const int x = (a.T + p.tokens - 1) / p.tokens;
  int y = 1;
  while (x * y < num_sms && y * kRotThreads < pieces) ++y;
  const dim3 grid(x, y);
  if (cache == nullptr) return launch<0, 0>(p, a.interleaved != 0, grid, stream);
  const bool fp8 = a.cache.dtype == MOE_DTYPE_FP8_E4M3;
  if (a.head_dim == 128)
    return fp8 ? launch<128, 2>(p, a.interleaved != 0, grid, stream)
               : launch<128, 1>(p, a.interleaved != 0, grid, stream);
  return fp8 ? launch<64, 2>(p, a.interleaved != 0, grid, stream)
             : launch<64, 1>(p, a.interleaved != 0, grid, stream);
}

}  // namespace moe
