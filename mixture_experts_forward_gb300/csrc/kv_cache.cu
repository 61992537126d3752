// The paged key/value cache: writing new positions (quantised as they are
// written, or copied) and reading positions back.
//
// Write, FP8: per token and head, a = max |x| over the head's row, s = a/448,
// code = E4M3(x * (1/s)): the 1x128 activation rule with the row as its block,
// in IEEE binary32 operations, so codes and scales are exact functions of the
// input.  16 elements per thread (two 16-byte loads of k and two of v in
// flight, one 16-byte store each), 8 or 4 threads per row, the row's maximum
// by shuffles among them.  Read: a CTA takes kReadTokens consecutive output
// rows, finds each one's page once, and its threads walk the rows' pieces of
// 16 elements.  Both are one pass and bound by HBM (or, below a few hundred
// rows, by the launch).
#include "moe_internal.cuh"
#include "quant_common.cuh"
#include "serve_internal.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

// Quantises 16 elements of a row shared by kTpr neighbouring lanes.
template <int kTpr>
__device__ __forceinline__ void quantise_piece(const uint4& raw0, const uint4& raw1, uint4& codes,
                                               float& scale) {
  const uint32_t w[8] = {raw0.x, raw0.y, raw0.z, raw0.w, raw1.x, raw1.y, raw1.z, raw1.w};
  float v[16];
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    amax = fmaxf(amax, fmaxf(fabsf(v[2 * i]), fabsf(v[2 * i + 1])));
  }
#pragma unroll
  for (int o = 1; o < kTpr; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  scale = 0.0f;
  float inv = 0.0f;
  if (amax >= amax_floor()) {
    scale = __fdiv_rn(amax, 448.0f);
    inv = __fdiv_rn(1.0f, scale);
  }
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint16_t c01 = cvt_e4m3x2(__fmul_rn(v[4 * i], inv), __fmul_rn(v[4 * i + 1], inv));
    const uint16_t c23 = cvt_e4m3x2(__fmul_rn(v[4 * i + 2], inv), __fmul_rn(v[4 * i + 3], inv));
    out[i] = static_cast<uint32_t>(c01) | (static_cast<uint32_t>(c23) << 16);
  }
  // a zero (or tiny) row has +0 codes whatever its elements' signs; a NaN, which
  // the maximum skips, keeps its place
  const uint32_t keep = scale == 0.0f ? 0x7f7f7f7fu : 0xffffffffu;
  codes = make_uint4(out[0] & keep, out[1] & keep, out[2] & keep, out[3] & keep);
}

template <int D, bool kFP8>
__global__ void __launch_bounds__(kThreads)
    kv_write_kernel(const __nv_bfloat16* __restrict__ k, const __nv_bfloat16* __restrict__ v,
                    int64_t ks_t, int64_t ks_h, int64_t vs_t, int64_t vs_h,
                    const int32_t* __restrict__ slots, KvCacheView c, int64_t rows, Ctrl* ctrl) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kTpr = D / 16;             // threads per row
  const int64_t idx = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t row = idx / kTpr;
  const int piece = static_cast<int>(idx % kTpr);
  bool valid = row < rows;
  int64_t dst = 0;                         // row of the cache
  uint4 a0 = make_uint4(0u, 0u, 0u, 0u), a1 = a0, b0 = a0, b1 = a0;
  if (valid) {
    const int64_t t = row / c.heads;
    const int h = static_cast<int>(row - t * c.heads);
    const int slot = __ldg(slots + t);
    const uint4* kp = reinterpret_cast<const uint4*>(k + t * ks_t + h * ks_h + piece * 16);
    const uint4* vp = reinterpret_cast<const uint4*>(v + t * vs_t + h * vs_h + piece * 16);
    a0 = __ldg(kp);
    a1 = __ldg(kp + 1);
    b0 = __ldg(vp);
    b1 = __ldg(vp + 1);
    const int page = slot >> c.page_log2;
    if (slot < 0 || page >= c.num_pages) {
      if (slot != -1) set_error(ctrl, MOE_ERR_DEVICE_FAULT, 10);
      valid = false;
    } else {
      dst = ((static_cast<int64_t>(page) * c.heads + h) << c.page_log2) +
            (slot & ((1 << c.page_log2) - 1));
    }
  }
  if constexpr (kFP8) {
    uint4 kq, vq;
    float ks, vs;
    quantise_piece<kTpr>(a0, a1, kq, ks);
    quantise_piece<kTpr>(b0, b1, vq, vs);
    if (!valid) return;
    reinterpret_cast<uint4*>(c.k)[dst * kTpr + piece] = kq;
    reinterpret_cast<uint4*>(c.v)[dst * kTpr + piece] = vq;
    if (piece == 0) {
      c.k_scales[dst] = ks;
      c.v_scales[dst] = vs;
    }
  } else {
    if (!valid) return;
    uint4* kd = reinterpret_cast<uint4*>(c.k) + (dst * kTpr + piece) * 2;
    uint4* vd = reinterpret_cast<uint4*>(c.v) + (dst * kTpr + piece) * 2;
    kd[0] = a0;
    kd[1] = a1;
    vd[0] = b0;
    vd[1] = b1;
  }
}

// bf16(code * scale) of 16 codes
__device__ __forceinline__ void dequantise16(const uint4& q, float s, uint4& o0, uint4& o1) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 f = e4m3x2_to_f32(static_cast<uint16_t>(w[i] >> (16 * j)));
      __nv_bfloat162 b = __floats2bfloat162_rn(__fmul_rn(f.x, s), __fmul_rn(f.y, s));
      o[2 * i + j] = *reinterpret_cast<uint32_t*>(&b);
    }
  }
  o0 = make_uint4(o[0], o[1], o[2], o[3]);
  o1 = make_uint4(o[4], o[5], o[6], o[7]);
}

constexpr int kReadTokens = 16;

template <int D, bool kFP8>
__global__ void __launch_bounds__(kThreads)
    kv_read_kernel(KvCacheView c, const int32_t* __restrict__ table, int table_stride,
                   const int32_t* __restrict__ cu, const int32_t* __restrict__ starts, int B,
                   int rows, uint4* __restrict__ k_out, uint4* __restrict__ v_out, Ctrl* ctrl) {
  constexpr int kTpr = D / 16;
  __shared__ int64_t s_src[kReadTokens];   // row of the cache at head 0, or -1
  pdl_wait();
  pdl_launch_dependents();
  const int r0 = blockIdx.x * kReadTokens;
  if (threadIdx.x < kReadTokens) {
    const int r = r0 + threadIdx.x;
    int64_t src = -1;
    if (r < rows) {
      // the last sequence whose first row is at or below r
      int lo = 0, hi = B;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(cu + mid) <= r) lo = mid; else hi = mid;
      }
      const int64_t pos = static_cast<int64_t>(r) - __ldg(cu + lo) +
                          (starts != nullptr ? __ldg(starts + lo) : 0);
      const int64_t entry = pos >> c.page_log2;
      int page = -1;
      if (pos >= 0 && entry < table_stride && r < __ldg(cu + lo + 1))
        page = __ldg(table + static_cast<int64_t>(lo) * table_stride + entry);
      if (page < 0 || page >= c.num_pages)
        set_error(ctrl, MOE_ERR_DEVICE_FAULT, 11);
      else
        src = ((static_cast<int64_t>(page) * c.heads) << c.page_log2) +
              (pos & ((1 << c.page_log2) - 1));
    }
    s_src[threadIdx.x] = src;
  }
  __syncthreads();
  const int n = min(kReadTokens, rows - r0) * c.heads * kTpr;
  const int per_row = c.heads * kTpr;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int tok = i / per_row;
    const int rest = i - tok * per_row;
    const int h = rest / kTpr, piece = rest % kTpr;
    const int64_t base = s_src[tok];
    const int64_t dst = (static_cast<int64_t>(r0 + tok) * per_row + rest) * 2;
    uint4 k0 = make_uint4(0u, 0u, 0u, 0u), k1 = k0, v0 = k0, v1 = k0;
    if (base >= 0) {
      const int64_t src = base + (static_cast<int64_t>(h) << c.page_log2);
      if constexpr (kFP8) {
        const uint4 kq = __ldg(reinterpret_cast<const uint4*>(c.k) + src * kTpr + piece);
        const uint4 vq = __ldg(reinterpret_cast<const uint4*>(c.v) + src * kTpr + piece);
        const float ks = __ldg(c.k_scales + src), vs = __ldg(c.v_scales + src);
        dequantise16(kq, ks, k0, k1);
        dequantise16(vq, vs, v0, v1);
      } else {
        const uint4* kp = reinterpret_cast<const uint4*>(c.k) + (src * kTpr + piece) * 2;
        const uint4* vp = reinterpret_cast<const uint4*>(c.v) + (src * kTpr + piece) * 2;
        k0 = __ldg(kp);
        k1 = __ldg(kp + 1);
        v0 = __ldg(vp);
        v1 = __ldg(vp + 1);
      }
    }
    k_out[dst] = k0;
    k_out[dst + 1] = k1;
    v_out[dst] = v0;
    v_out[dst + 1] = v1;
  }
}

}  // namespace

cudaError_t launch_kv_write(const KvCacheView& c, int head_dim, bool fp8, const void* k,
                            const void* v, int T, int64_t ks_t, int64_t ks_h, int64_t vs_t,
                            int64_t vs_h, const int32_t* slots, Ctrl* ctrl, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(T) * c.heads;
  const int64_t threads = rows * (head_dim / 16);
  const dim3 grid(static_cast<unsigned>((threads + kThreads - 1) / kThreads));
  const __nv_bfloat16* kb = static_cast<const __nv_bfloat16*>(k);
  const __nv_bfloat16* vb = static_cast<const __nv_bfloat16*>(v);
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = make_cfg(grid, dim3(kThreads), stream, true, attr);
#define MOE_KVW(DD, F)                                                                          \
  return cudaLaunchKernelEx(&cfg, kv_write_kernel<DD, F>, kb, vb, ks_t, ks_h, vs_t, vs_h, slots, \
                            c, rows, ctrl)
  if (head_dim == 128) {
    if (fp8) MOE_KVW(128, true);
    MOE_KVW(128, false);
  }
  if (fp8) MOE_KVW(64, true);
  MOE_KVW(64, false);
#undef MOE_KVW
}

cudaError_t launch_kv_read(const KvCacheView& c, int head_dim, bool fp8, const int32_t* table,
                           int table_stride, const int32_t* cu, const int32_t* starts, int B,
                           int rows, void* k_out, void* v_out, Ctrl* ctrl, cudaStream_t stream) {
  const dim3 grid((rows + kReadTokens - 1) / kReadTokens);
  uint4* ko = static_cast<uint4*>(k_out);
  uint4* vo = static_cast<uint4*>(v_out);
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = make_cfg(grid, dim3(kThreads), stream, true, attr);
#define MOE_KVR(DD, F)                                                                         \
  return cudaLaunchKernelEx(&cfg, kv_read_kernel<DD, F>, c, table, table_stride, cu, starts, B, \
                            rows, ko, vo, ctrl)
  if (head_dim == 128) {
    if (fp8) MOE_KVR(128, true);
    MOE_KVR(128, false);
  }
  if (fp8) MOE_KVR(64, true);
  MOE_KVR(64, false);
#undef MOE_KVR
}

}  // namespace moe
