// Verification of drafted tokens against the target's probabilities from
// given random numbers.
//
// A cluster of up to 8 CTAs takes one sequence.  Every CTA finds the first
// refused draft by itself (one warp, a draft per lane).  The draw then needs
// one pass over a row of p and a row of q: each warp sums its own contiguous
// run of the vocabulary in fixed point (w = trunc(max(p - q, 0) * 2^38), exact
// in any order; a row sums to about 2^38, so 2^24 tokens of full weight still
// fit 64 bits), and the CTAs' sums meet over distributed shared memory.  The CTA
// whose part holds the threshold splits the one warp's run that holds it over all
// its warps, and one of those walks the last few hundred tokens, 32 at a time.
// Rows start at any multiple of the element size (odd vocabularies), so loads
// are one element per lane, kUnroll of each row in flight per thread; 128-byte
// requests keep up with HBM.  The weights' conversion is shifts of the float's own
// bits: a conversion instruction to 64 bits runs at 2 lanes per cycle and was 60 of 85 us
// for 96 rows of 131071.  Bound by HBM for batches, by the latency of the dependent
// steps (drafts, row, sums, run) for single sequences.
#include "serve_internal.cuh"

namespace moe {
namespace {

constexpr int kVThreads = 512;
constexpr int kVWarps = kVThreads / 32;
constexpr int kVUnroll = 8;

__device__ __forceinline__ float load_prob(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_prob(const __nv_bfloat16* p) {
  return __bfloat162float(__ldg(p));
}

// clamp to [0, 1]; NaN -> 0
__device__ __forceinline__ float unit(float x) { return fminf(fmaxf(x, 0.0f), 1.0f); }

// trunc(w * 2^38) of w in [0, 1]: the 24-bit significand shifted by the exponent
// (2^-23 is one unit of it at exponent 127: 38 - 23 = 15 places left, less 127 - exponent).
__device__ __forceinline__ uint64_t fixed(float w) {
  const uint32_t u = __float_as_uint(w);
  const uint64_t m = static_cast<uint64_t>((u & 0x7fffffu) | 0x800000u) << 15;
  return m >> min(127u - (u >> 23), 63u);      // (zero and subnormals: shifted out)
}

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
  __shared__ uint64_t s_warp[kVWarps];     // sums of this CTA's warps
  __shared__ uint64_t s_cta;
  __shared__ int s_r;
  pdl_wait();
  pdl_launch_dependents();
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

  // a token's weight: what is left of p after q, or (from_p) p itself
  auto weight = [&](int v, bool from_p) -> uint64_t {
    const float x = unit(load_prob(p + v));
    return fixed(from_p || !has_q ? x : unit(__fsub_rn(x, load_prob(q + v))));
  };
  // the sum over this warp's lanes of the weights of [from, to)
  auto run_sum = [&](int from, int to, bool from_p) -> uint64_t {
    const bool both = has_q && !from_p;
    uint64_t sum = 0;
    int v = from + lane;
    for (; v + 32 * (kVUnroll - 1) < to; v += 32 * kVUnroll) {
      float x[kVUnroll], y[kVUnroll];
#pragma unroll
      for (int i = 0; i < kVUnroll; ++i) x[i] = load_prob(p + v + 32 * i);
#pragma unroll
      for (int i = 0; i < kVUnroll; ++i) y[i] = both ? load_prob(q + v + 32 * i) : 0.0f;
#pragma unroll
      for (int i = 0; i < kVUnroll; ++i) {
        const float w = unit(x[i]);
        sum += fixed(both ? unit(__fsub_rn(w, y[i])) : w);
      }
    }
    for (; v < to; v += 32) sum += weight(v, from_p);
    return warp_sum(sum);
  };
  // this warp's run of the vocabulary: a multiple of 32 tokens per warp
  const int warps = ctas * kVWarps;
  const int per = ((V + warps - 1) / warps + 31) & ~31;
  auto run_start = [&](int warp_of_cta) -> int {
    const int64_t first = static_cast<int64_t>(rank * kVWarps + warp_of_cta) * per;
    return static_cast<int>(first < V ? first : V);
  };
  const int v0 = run_start(w), v1 = min(V, v0 + per);
  uint64_t total = 0, before = 0;
  bool from_p = false;
  for (int attempt = 0; attempt < 2; ++attempt) {
    // no residual weight anywhere: draw from p itself
    from_p = attempt == 1;
    const uint64_t mine = run_sum(v0, v1, from_p);
    if (lane == 0) s_warp[w] = mine;
    __syncthreads();
    if (w == 0) {
      const uint64_t c = warp_sum(lane < kVWarps ? s_warp[lane] : 0ull);
      if (lane == 0) s_cta = c;
    }
    cluster_sync();
    total = before = 0;
    for (int c = 0; c < ctas; ++c) {
      const uint64_t x = ld_cluster_u64(mapa_shared(smem_u32(&s_cta), c));
      total += x;
      if (c < rank) before += x;
    }
    cluster_sync();                        // every CTA has read the others' sums
    if (total > 0 || !has_q) break;
  }
  uint64_t u24 = static_cast<uint64_t>(
      __float2uint_rz(unit(__ldg(a.u_sample + b)) * 16777216.0f));
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
  // the warp's run that holds the threshold, if it is this CTA's: the same for all its threads
  int owner = -1;
  uint64_t acc = before;
  for (int i = 0; i < kVWarps; ++i) {
    const uint64_t x = s_warp[i];
    if (owner < 0) {
      if (t >= acc && t < acc + x) owner = i;
      else acc += x;
    }
  }
  if (owner < 0) return;
  __syncthreads();                         // (s_warp is written again)
  const int o0 = run_start(owner), o1 = min(V, o0 + per);
  const int sub = ((o1 - o0 + kVWarps - 1) / kVWarps + 31) & ~31;
  const int q0 = min(o1, o0 + w * sub), q1 = min(o1, q0 + sub);
  const uint64_t mine = run_sum(q0, q1, from_p);
  if (lane == 0) s_warp[w] = mine;
  __syncthreads();
  for (int i = 0; i < w; ++i) acc += s_warp[i];
  if (t < acc || t >= acc + mine) return;
  for (int base = q0; base < q1; base += 32) {
    const int j = base + lane;
    uint64_t inc = j < q1 ? weight(j, from_p) : 0ull;
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
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, verify_kernel<T>, k, ctas);
}

}  // namespace

cudaError_t launch_verify(const moe_verify_args& a, Ctrl* ctrl, int num_sms, cudaStream_t stream) {
  return a.dtype == MOE_DTYPE_F32 ? launch_t<float>(a, ctrl, num_sms, stream)
                                  : launch_t<__nv_bfloat16>(a, ctrl, num_sms, stream);
}

}  // namespace moe
