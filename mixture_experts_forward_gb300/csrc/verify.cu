// Verification of drafted tokens against the target's probabilities from
// given random numbers.
//
// A cluster of up to 8 CTAs takes one sequence.  Every CTA finds the first
// refused draft by itself (one warp, a draft per lane).  The draw then needs
// one pass over a row of p and a row of q: each warp sums its own contiguous
// run of the vocabulary in fixed point (w = trunc(max(p - q, 0) * 2^38), exact
// in any order; a row sums to about 2^38, so 2^24 tokens of full weight still
// fit 64 bits), the CTAs' sums meet over distributed shared memory, and the one
// warp whose run holds the threshold walks that run again, 32 tokens at a time.
// Rows start at any multiple of the element size (odd vocabularies), so loads
// are one element per lane, kUnroll of each row in flight per thread; 128-byte
// requests keep up with HBM.  Bound by HBM for batches, by the latency of the
// dependent steps (drafts, row, sums, run) for single sequences.
#include "serve_internal.cuh"

namespace moe {
namespace {

constexpr int kVThreads = 512;
constexpr int kVWarps = kVThreads / 32;
constexpr int kVUnroll = 8;
constexpr float kFix = 274877906944.0f;  // 2^38

__device__ __forceinline__ float load_prob(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_prob(const __nv_bfloat16* p) {
  return __bfloat162float(__ldg(p));
}

// clamp to [0, 1]; NaN -> 0
__device__ __forceinline__ float unit(float x) { return fminf(fmaxf(x, 0.0f), 1.0f); }

__device__ __forceinline__ uint64_t fixed(float w) { return static_cast<uint64_t>(w * kFix); }

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <typename T>
struct VerifyArgs {
  const T* p;
  const T* q;
  int64_t p_sb, p_si, q_sb, q_si;
  const int32_t* draft;
  const int32_t* draft_lens;
  const float* u_accept;
  const float* u_sample;
  int32_t* accepted;
  int32_t* tokens;
  int n, V;
  Ctrl* ctrl;
};

__device__ __forceinline__ uint64_t ld_cluster_u64(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}

template <typename T>
__global__ void __launch_bounds__(kVThreads) verify_kernel(VerifyArgs<T> a, int ctas) {
  __shared__ uint64_t s_warp[2][kVWarps];  // sums of this CTA's warps: rest, p alone
  __shared__ uint64_t s_cta[2];
  __shared__ int s_r;
  const int b = blockIdx.x / ctas;
  const int rank = blockIdx.x - b * ctas;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int n = a.n, V = a.V;
  int len = n;
  if (a.draft_lens != nullptr) {
    len = __ldg(a.draft_lens + b);
    if (len < 0 || len > n) {
      if (rank == 0 && tid == 0) set_error(a.ctrl, MOE_ERR_DEVICE_FAULT, 30);
      len = min(max(len, 0), n);
    }
  }
  if (w == 0) {
    bool ok = false;
    if (lane < len) {
      const int x = __ldg(a.draft + static_cast<int64_t>(b) * n + lane);
      const float u = __ldg(a.u_accept + static_cast<int64_t>(b) * n + lane);
      if (x >= 0 && x < V) {
        const float px = load_prob(a.p + b * a.p_sb + lane * a.p_si + x);
        const float qx = load_prob(a.q + b * a.q_sb + lane * a.q_si + x);
        ok = __fmul_rn(u, qx) < px;
      } else if (rank == 0) {
        set_error(a.ctrl, MOE_ERR_DEVICE_FAULT, 31);
      }
    }
    const unsigned m = __ballot_sync(0xffffffffu, ok);
    if (lane == 0) s_r = __ffs(~m) - 1 < 0 ? 32 : __ffs(~m) - 1;
  }
  __syncthreads();
  const int r = min(s_r, len);
  const bool has_q = r < len;
  const T* p = a.p + b * a.p_sb + r * a.p_si;
  const T* q = a.q + b * a.q_sb + (has_q ? r : 0) * a.q_si;

  // this warp's run of the vocabulary: a multiple of 32 tokens per warp
  const int warps = ctas * kVWarps;
  const int per = ((V + warps - 1) / warps + 31) & ~31;
  const int64_t first = static_cast<int64_t>(rank * kVWarps + w) * per;
  const int v0 = static_cast<int>(first < V ? first : V);
  const int v1 = min(V, v0 + per);
  uint64_t rest = 0, alone = 0;
  int v = v0 + lane;
  for (; v + 32 * (kVUnroll - 1) < v1; v += 32 * kVUnroll) {
    float x[kVUnroll], y[kVUnroll];
#pragma unroll
    for (int i = 0; i < kVUnroll; ++i) x[i] = unit(load_prob(p + v + 32 * i));
#pragma unroll
    for (int i = 0; i < kVUnroll; ++i) y[i] = has_q ? load_prob(q + v + 32 * i) : 0.0f;
#pragma unroll
    for (int i = 0; i < kVUnroll; ++i) {
      alone += fixed(x[i]);
      rest += fixed(unit(__fsub_rn(x[i], y[i])));
    }
  }
  for (; v < v1; v += 32) {
    const float x = unit(load_prob(p + v));
    alone += fixed(x);
    rest += fixed(unit(__fsub_rn(x, has_q ? load_prob(q + v) : 0.0f)));
  }
  rest = warp_sum(rest);
  alone = warp_sum(alone);
  if (lane == 0) {
    s_warp[0][w] = rest;
    s_warp[1][w] = alone;
  }
  __syncthreads();
  if (w == 0) {
    const uint64_t c0 = warp_sum(lane < kVWarps ? s_warp[0][lane] : 0ull);
    const uint64_t c1 = warp_sum(lane < kVWarps ? s_warp[1][lane] : 0ull);
    if (lane == 0) {
      s_cta[0] = c0;
      s_cta[1] = c1;
    }
  }
  cluster_sync();
  uint64_t total0 = 0, total1 = 0, before0 = 0, before1 = 0;
  for (int c = 0; c < ctas; ++c) {
    const uint32_t at = mapa_shared(smem_u32(s_cta), c);
    const uint64_t x = ld_cluster_u64(at), y = ld_cluster_u64(at + 8);
    total0 += x;
    total1 += y;
    if (c < rank) {
      before0 += x;
      before1 += y;
    }
  }
  cluster_sync();  // every CTA has read the others' sums: they may exit
  const bool from_p = total0 == 0;         // no residual weight: draw from p itself
  const uint64_t total = from_p ? total1 : total0;
  uint64_t u24 = static_cast<uint64_t>(unit(__ldg(a.u_sample + b)) * 16777216.0f);
  if (u24 > 16777215u) u24 = 16777215u;    // 1 is outside [0, 1): the last token
  // floor(u24 * total / 2^24) in 88 bits
  const uint64_t t = (__umul64hi(total, u24) << 40) | ((total * u24) >> 24);
  int32_t* out = a.tokens + static_cast<int64_t>(b) * (n + 1);
  if (rank == 0 && w == 0) {
    for (int i = lane; i <= n; i += 32) {
      if (i < r) out[i] = __ldg(a.draft + static_cast<int64_t>(b) * n + i);
      else if (i > r || total == 0) out[i] = -1;
    }
    if (lane == 0) a.accepted[b] = r;
  }
  const uint64_t* sums = s_warp[from_p ? 1 : 0];
  uint64_t acc = from_p ? before1 : before0;
  for (int i = 0; i < w; ++i) acc += sums[i];
  if (t < acc || t >= acc + sums[w]) return;
  // the threshold lies in this warp's run
  for (int base = v0; base < v1; base += 32) {
    const int j = base + lane;
    uint64_t wt = 0;
    if (j < v1) {
      const float x = unit(load_prob(p + j));
      wt = fixed(from_p ? x : unit(__fsub_rn(x, has_q ? load_prob(q + j) : 0.0f)));
    }
    uint64_t inc = wt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    const unsigned over = __ballot_sync(0xffffffffu, acc + inc > t);
    if (over != 0u) {
      if (lane == 0) out[r] = base + __ffs(over) - 1;
      return;
    }
    acc += __shfl_sync(0xffffffffu, inc, 31);
  }
}

template <typename T>
cudaError_t launch_t(const moe_verify_args& a, Ctrl* ctrl, int num_sms, cudaStream_t stream) {
  VerifyArgs<T> k;
  k.p = static_cast<const T*>(a.p);
  k.q = static_cast<const T*>(a.q);
  k.p_sb = a.p_stride_b;
  k.p_si = a.p_stride_i;
  k.q_sb = a.q_stride_b;
  k.q_si = a.q_stride_i;
  k.draft = a.draft;
  k.draft_lens = a.draft_lens;
  k.u_accept = a.u_accept;
  k.u_sample = a.u_sample;
  k.accepted = a.accepted;
  k.tokens = a.tokens;
  k.n = a.n;
  k.V = a.V;
  k.ctrl = ctrl;
  // CTAs per sequence: enough for two CTAs on every SM, but no warp with
  // fewer than 64 tokens
  int ctas = 1;
  while (ctas < 8 && static_cast<int64_t>(a.B) * ctas < 2 * num_sms &&
         a.V / (2 * ctas * kVWarps) >= 64)
    ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B) * ctas);
  cfg.blockDim = dim3(kVThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, verify_kernel<T>, k, ctas);
}

}  // namespace

cudaError_t launch_verify(const moe_verify_args& a, Ctrl* ctrl, int num_sms, cudaStream_t stream) {
  return a.dtype == MOE_DTYPE_F32 ? launch_t<float>(a, ctrl, num_sms, stream)
                                  : launch_t<__nv_bfloat16>(a, ctrl, num_sms, stream);
}

}  // namespace moe
