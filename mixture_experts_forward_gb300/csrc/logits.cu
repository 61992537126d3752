// Penalties, biases and masks on logits, and their probabilities.
//
// A cluster of up to 8 CTAs takes one row at a time, each CTA a contiguous part of the vocabulary
// that its threads hold in registers (kPer values each, one load in flight per value), so the logits are
// read once and the result is written once.  While the first loads are under way the CTA counts the
// history into shared memory, a word for each token of its part (integer atomics: the same in any
// order); further rows of the sequence add one draft each.  Where a CTA takes several rows it also
// lists the tokens named: their values are adjusted by themselves, spread over the threads, and the
// pass over the row finds them in the words' place, in 3 instructions a value instead of a branch
// that most warps take.  The softmax is over each warp's own maximum; the CTA joins its warps' sums
// and the CTAs exchange theirs once over distributed shared memory (max, sum, and the first token of
// the maximum for greedy rows) and join them in rank order, so repeated calls give the same bits.  Without probabilities
// nothing is exchanged and the CTAs stand alone.
// Rows begin at any multiple of the element size (odd vocabularies): one element per lane and
// load.  Bound, for many rows, by a row's chain of steps (the loads, the pass, the maximum, the
// exponentials, the exchange, the stores: 8.5 us with two CTAs an SM, of which HBM explains 5):
// 576 rows of 131071 in 202 us (3.0 TB/s; without penalties, biases and mask 135; from BF16 211), 200
// BF16 rows of 100003 without probabilities in 73 us (1.7 TB/s; without the history 55, without
// anything 37; 68 before rows of a sequence shared their counts, which these do not), one row 8-10 us:
// launch and chain.  Clusters of
// 8 leave a fifth of the SMs empty, those of 4 with 64 values a thread fewer, but one CTA an SM
// overlaps with no other (the rows above 195 us, without the counts 142).  No faster: quads on
// 16-byte boundaries with the next row copied ahead, values kept in shared memory with one exchange
// a row, chunks of tokens dealt to the CTAs in turn, a fixed set of clusters with equal shares of
// all rows, the named tokens of the next row adjusted beside the exchange (208).
#include <algorithm>

#include "serve_internal.cuh"

namespace moe {
namespace {

constexpr int kLThreads = 512;
constexpr int kLWarps = kLThreads / 32;
constexpr int kLMaxCluster = 8;
// A token's word: bit 0 the prompt, then 11 bits the first bias that names it (1 + its place), then how
// often it is among the outputs.
constexpr uint32_t kOnce = 1u << 12;
constexpr int kListShare = 4;             // the list holds a quarter of a CTA's tokens

__device__ __forceinline__ float load_logit(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) {
  return __bfloat162float(__ldg(p));
}

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

template <typename T>
struct LogitsParams {
  const T* logits;
  float* out;
  int64_t l_sb, l_si, o_sb, o_si, m_sb, m_si;
  const int32_t* history;
  const int32_t* history_lens;
  const int32_t* prompt_lens;
  const int32_t* draft;
  const float* repetition;
  const float* presence;
  const float* frequency;
  const float* temperature;
  const int32_t* bias_tokens;
  const float* bias_values;
  const uint32_t* mask;
  Ctrl* ctrl;
  int m, V, history_stride, biases, part, cluster;
  int rows;                                 // rows of a sequence that a cluster takes
};

// A warp's or CTA's share of a row: its maximum, where that is first, and the sum of exponentials.
struct alignas(16) Share {                 // (stored as one vector)
  float max, sum;
  int at, pad;
};

template <typename T, int kPer, bool kProbs>
__global__ void __launch_bounds__(kLThreads, kPer <= 8 ? 3 : kPer <= 32 ? 2 : 1)
    logits_kernel(const LogitsParams<T> p) {
  extern __shared__ __align__(16) uint32_t s_count[];   // [part]: a token's word, later its value's bits, inverted
  __shared__ Share s_share[2][kLMaxCluster];   // every CTA of the cluster writes its own here
  __shared__ Share s_warp[kLWarps];
  __shared__ int s_draft[32], s_named;
  __shared__ float s_number[4];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x % p.cluster;
  const int group = blockIdx.x / p.cluster;           // p.rows rows of a sequence
  const int groups = (p.m + p.rows - 1) / p.rows;     // of a sequence
  const int b = group / groups, i0 = (group - b * groups) * p.rows, i1 = min(p.m, i0 + p.rows);
  const int v0 = rank * p.part, n = min(p.part, p.V - v0);    // n may be <= 0
  constexpr int kWords = (kPer + 31) / 32;
  const bool counts = p.history != nullptr || p.draft != nullptr || p.biases > 0;
  const bool list = p.rows > 1;
  if (counts) {
    for (int at = tid; at < p.part / 4; at += kLThreads)
      reinterpret_cast<uint4*>(s_count)[at] = make_uint4(0u, 0u, 0u, 0u);
    if (tid == 0) s_named = 0;
  }
  pdl_wait();
  pdl_launch_dependents();
  if (kProbs && p.cluster > 1)              // (before any CTA writes to another)
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");

  // the tokens named: a word each, and the list of them (where it has room)
  const int room = p.part / kListShare;
  uint32_t* s_word = s_count + p.part;
  int32_t* s_bias_t = reinterpret_cast<int32_t*>(s_word + room);
  float* s_bias_v = reinterpret_cast<float*>(s_bias_t + p.biases);
  float* s_bias_sum = s_bias_v + p.biases;
  uint16_t* s_token = reinterpret_cast<uint16_t*>(s_bias_sum + p.biases);

  // What the counts and the adjustment need comes before the row, which keeps the load units busy
  // for microseconds.
  float number = 1.0f;                      // the sequence's numbers, one a thread
  if (tid < 4) {
    const float* from = tid == 0 ? p.repetition : tid == 1 ? p.presence : tid == 2 ? p.frequency : p.temperature;
    number = from == nullptr ? (tid == 0 || tid == 3 ? 1.0f : 0.0f) : __ldg(from + b);
  }
  int len = 0, prompt = 0;
  constexpr int kAtOnce = 8;
  int ahead[kAtOnce];                       // the history's next tokens
  const int32_t* history = p.history + static_cast<int64_t>(b) * p.history_stride + tid;
  auto load_history = [&](int at) {
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j)
      ahead[j] = at + tid + j * kLThreads < len ? __ldg(history + at + j * kLThreads) : -1;
  };
  if (p.history != nullptr) {
    len = p.history_lens != nullptr ? __ldg(p.history_lens + b) : p.history_stride;
    if (p.prompt_lens != nullptr) prompt = __ldg(p.prompt_lens + b);
    if (len < 0 || len > p.history_stride || prompt < 0 || prompt > len) {
      if (tid == 0) set_error(p.ctrl, MOE_ERR_DEVICE_FAULT, kFaultHistory);
      len = min(max(len, 0), p.history_stride);
      prompt = min(max(prompt, 0), len);
    }
    load_history(0);
  }
  for (int at = tid; at < p.biases; at += kLThreads) {
    cp_async4(smem_u32(s_bias_t + at), p.bias_tokens + static_cast<int64_t>(b) * p.biases + at);
    cp_async4(smem_u32(s_bias_v + at), p.bias_values + static_cast<int64_t>(b) * p.biases + at);
  }
  if (p.draft != nullptr && tid < p.m - 1) cp_async4(smem_u32(s_draft + tid), p.draft + b * (p.m - 1) + tid);

  float l[kPer];
  uint32_t words[kWords];                   // word j of the mask for this warp's tokens of turn j, by lane j
  auto load_row = [&](int i) {
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
      const int at = (warp + (32 * w + lane) * kLWarps) * 32;
      words[w] = 0xffffffffu;
      if (p.mask != nullptr && 32 * w + lane < kPer && at < n)
        words[w] = __ldg(p.mask + b * p.m_sb + i * p.m_si + (v0 + at) / 32);
    }
    const T* src = p.logits + b * p.l_sb + i * p.l_si + v0 + tid;
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      l[j] = tid + j * kLThreads < n ? load_logit(src + j * kLThreads) : neg_inf();
  };
  load_row(i0);
  if (tid < 4) s_number[tid] = number;

  // The word as it was, of a token of this part (else ~0u): a token's first name enters it in the list.
  auto count = [&](int v, uint32_t what) -> uint32_t {
    if (v < 0 || v >= p.V) {
      if (v != -1) set_error(p.ctrl, MOE_ERR_DEVICE_FAULT, kFaultToken);
      return ~0u;
    }
    v -= v0;
    if (v < 0 || v >= n) return ~0u;
    return what < kOnce ? atomicOr(s_count + v, what) : atomicAdd(s_count + v, what);
  };
  auto enter = [&](int v, int at) {
    if (at < room) s_token[at] = static_cast<uint16_t>(v - v0);
  };
  bool listed = false;
  cp_async_wait_all();
  __syncthreads();
  if (counts) {
    for (int turn = 0; turn < len; turn += kAtOnce * kLThreads) {
      int now[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) now[j] = ahead[j];
      load_history(turn + kAtOnce * kLThreads);
      if (!list) {
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) count(now[j], turn + tid + j * kLThreads < prompt ? 1u : kOnce);
        continue;
      }
      uint32_t entered = 0;
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
        if (count(now[j], turn + tid + j * kLThreads < prompt ? 1u : kOnce) == 0) entered |= 1u << j;
      int at = __popc(entered);             // one draw for a warp's new tokens
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o) at += up;
      }
      int base = 0;
      if (lane == 31 && at > 0) base = atomicAdd(&s_named, at);
      at += __shfl_sync(0xffffffffu, base, 31) - __popc(entered);
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
        if ((entered >> j & 1u) != 0) enter(now[j], at++);
    }
    if (p.draft != nullptr && tid < i0 && count(s_draft[tid], kOnce) == 0 && list)
      enter(s_draft[tid], atomicAdd(&s_named, 1));
    // the first bias of a token gets all of them, added up in their order; a warp for each
    for (int at = warp; at < p.biases; at += kLWarps) {
      const int t = s_bias_t[at];
      if ((t < -1 || t >= p.V) && lane == 0) set_error(p.ctrl, MOE_ERR_DEVICE_FAULT, kFaultToken);
      if (t < v0 || t >= v0 + n || t < 0 || t >= p.V) continue;
      int first = -1;
      float sum = 0.0f;
      for (int q = 0; q < p.biases; q += 32) {
        uint32_t same = __ballot_sync(0xffffffffu, q + lane < p.biases && s_bias_t[min(q + lane, p.biases - 1)] == t);
        if (first < 0 && same != 0) first = q + __ffs(same) - 1;
        if (first >= 0 && first != at) break;
        for (; same != 0; same &= same - 1) sum += s_bias_v[q + __ffs(same) - 1];
      }
      if (first != at || lane != 0) continue;
      s_bias_sum[at] = sum;
      if (count(t, static_cast<uint32_t>(at + 1) << 1) == 0 && list) enter(t, atomicAdd(&s_named, 1));
    }
    __syncthreads();
    if (list && p.draft != nullptr) {       // drafts of the rows to come get places, with nothing counted
      if (tid >= i0 && tid < i1 - 1) {
        const int t = s_draft[tid], v = t - v0;
        if (t < -1 || t >= p.V) set_error(p.ctrl, MOE_ERR_DEVICE_FAULT, kFaultToken);
        bool is_new = t >= 0 && t < p.V && v >= 0 && v < n && s_count[v] == 0;
        for (int d = i0; d < tid; ++d) is_new = is_new && s_draft[d] != t;
        if (is_new) enter(t, atomicAdd(&s_named, 1));
      }
      __syncthreads();
    }
    listed = list && s_named <= room;
  }
  float rep = s_number[0], temp = s_number[3];
  const float presence = s_number[1], frequency = s_number[2];
  if (!(rep > 0.0f) || !(temp >= 0.0f)) {
    if (tid == 0) set_error(p.ctrl, MOE_ERR_DEVICE_FAULT, kFaultNumber);
    if (!(rep > 0.0f)) rep = 1.0f;
    if (!(temp >= 0.0f)) temp = 1.0f;
  }
  const float inverse = __fdiv_rn(1.0f, rep);

  auto adjusted = [&](float x, uint32_t c) {
    const uint32_t bias = (c >> 1) & (kOnce / 2 - 1);
    if ((c & 1u) != 0 || c >= kOnce) x *= x > 0.0f ? inverse : rep;
    if (c >= kOnce) x = x - frequency * static_cast<float>(c / kOnce) - presence;
    if (bias != 0 && x > neg_inf()) x += s_bias_sum[bias - 1];
    return x;
  };

  for (int i = i0; i < i1; ++i) {
    if (i > i0) {
      load_row(i);
      if (!kProbs) __syncthreads();         // (with probabilities the exchange has ordered the readers before)
    }
    if (listed) {
      // The listed tokens' values by themselves; each is put where the pass finds it, inverted, so
      // that it is never 0 (that would be a NaN, which counts as -inf).
      const T* row = p.logits + b * p.l_sb + i * p.l_si + v0;
      const int draft = i > i0 && p.draft != nullptr ? s_draft[i - 1] - v0 : -1;   // one more is counted
      for (int at = tid; at < s_named; at += 2 * kLThreads) {
        const bool two = at + kLThreads < s_named;
        const int v[2] = {s_token[at], two ? s_token[at + kLThreads] : -1};
        const float x[2] = {load_logit(row + v[0]), two ? load_logit(row + v[1]) : 0.0f};
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (v[q] < 0) break;
          uint32_t c = i == i0 ? s_count[v[q]] : s_word[at + q * kLThreads];
          if (v[q] == draft) c += kOnce;
          s_word[at + q * kLThreads] = c;
          s_count[v[q]] = ~__float_as_uint(fmaxf(adjusted(x[q], c), neg_inf()));
        }
      }
      __syncthreads();
    } else if (i > i0 && p.draft != nullptr) {
      if (tid == 0) count(s_draft[i - 1], kOnce);
      __syncthreads();
    }
    if (i + 1 < i1) {                       // the next row comes to L2 meanwhile, 128 bytes a thread
      const char* next = reinterpret_cast<const char*>(p.logits + b * p.l_sb + (i + 1) * p.l_si + v0);
      for (int at = tid * 128; at < n * static_cast<int>(sizeof(T)); at += kLThreads * 128)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(next + at));
    }
    // the mask's bits turned round: bit j for this lane's value of turn j
#pragma unroll
    for (int w = 0; w < kWords; ++w)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const uint32_t low = 0xffffffffu / ((1u << o) + 1u);      // the bits whose place has no o
        const uint32_t other = __shfl_xor_sync(0xffffffffu, words[w], o);
        words[w] = (lane & o) == 0 ? (words[w] & low) | ((other & low) << o)
                                   : (words[w] & ~low) | ((other & ~low) >> o);
      }
    if (listed) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const uint32_t c = s_count[tid + j * kLThreads];
        if (c != 0) l[j] = __uint_as_float(~c);
      }
    } else if (counts) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const uint32_t c = s_count[tid + j * kLThreads];
        if (c != 0) l[j] = adjusted(l[j], c);
      }
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      l[j] = fmaxf(l[j], neg_inf());        // (a NaN counts as -inf)
      if ((words[j / 32] >> (j % 32) & 1u) == 0) l[j] = neg_inf();
    }
    float* out = p.out + b * p.o_sb + i * p.o_si + v0 + tid;
    if constexpr (!kProbs) {
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (tid + j * kLThreads < n) out[j * kLThreads] = l[j];
    } else {
      // the warp's maximum, then (greedy) its first place or the sum
      float top = neg_inf();
#pragma unroll
      for (int j = 0; j < kPer; ++j) top = fmaxf(top, l[j]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const bool greedy = temp == 0.0f;
      int first = 0x7fffffff;
      float sum = 0.0f;
      // exp((l - top) / temp) as a power of two; the rate stays between the ends of the type, so
      // that a difference of 0 gives 1 and one of -inf gives 0
      const float rate = fminf(fmaxf(__fdiv_rn(1.4426950408889634f, temp), 1.2e-38f), 3.0e38f);
      if (greedy) {
#pragma unroll
        for (int j = kPer - 1; j >= 0; --j)
          if (l[j] == top && top > neg_inf()) first = v0 + tid + j * kLThreads;
        first = __reduce_min_sync(0xffffffffu, first);
      } else {
        if (top == -neg_inf()) {
#pragma unroll
          for (int j = 0; j < kPer; ++j) {
            l[j] = l[j] == top ? 1.0f : 0.0f;
            sum += l[j];
          }
        } else {
          const float base = top == neg_inf() ? 0.0f : top;
#pragma unroll
          for (int j = 0; j < kPer; ++j) {
            asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(l[j]) : "f"((l[j] - base) * rate));
            sum += l[j];
          }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      }
      if (lane == 0) s_warp[warp] = {top, sum, first, 0};
      __syncthreads();
      // a share's sum, taken to another maximum
      auto taken_to = [&](const Share& s, float max) {
        float f;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(f) : "f"((s.max - max) * rate));
        return s.max == max ? s.sum : s.max == neg_inf() ? 0.0f : s.sum * f;
      };
      // the CTAs' shares (two buffers in turn: no CTA is two rows ahead of another)
      Share* share = s_share[(i - i0) & 1];
      if (p.cluster > 1 && i == i0) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
      if (warp == 0) {
        Share mine = s_warp[lane % kLWarps];
        float max = mine.max;
#pragma unroll
        for (int o = kLWarps / 2; o > 0; o >>= 1) max = fmaxf(max, __shfl_xor_sync(0xffffffffu, max, o));
        float part = taken_to(mine, max);
#pragma unroll
        for (int o = kLWarps / 2; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
        const int at = __reduce_min_sync(0xffffffffu, mine.max == max ? mine.at : 0x7fffffff);
        if (lane < p.cluster) {
          uint32_t to;
          asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                       : "=r"(to)
                       : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(share + rank))), "r"(lane));
          asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to),
                       "r"(__float_as_uint(max)), "r"(__float_as_uint(part)), "r"(at), "r"(0)
                       : "memory");
        }
      }
      if (p.cluster > 1) {
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
      } else {
        __syncthreads();
      }
      float all = neg_inf(), total = 0.0f;
      int choice = 0x7fffffff;
      for (int c = 0; c < p.cluster; ++c) all = fmaxf(all, share[c].max);
      for (int c = 0; c < p.cluster; ++c) {
        const Share s = share[c];
        if (s.max == all) choice = min(choice, s.at);
        total += taken_to(s, all);
      }
      if (greedy) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) l[j] = v0 + tid + j * kLThreads == choice ? 1.0f : 0.0f;
      }
      const float scale = greedy ? 1.0f : all == neg_inf() ? 0.0f : __fdiv_rn(taken_to({top, 1.0f, 0, 0}, all), total);
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (tid + j * kLThreads < n) out[j * kLThreads] = l[j] * scale;
    }
  }
}

template <typename T, int kPer, bool kProbs>
cudaError_t launch(LogitsParams<T> p, int B, int cluster, int num_sms, cudaStream_t stream) {
  p.part = kPer * kLThreads;
  if (!kProbs) cluster = (p.V + p.part - 1) / p.part;   // (CTAs of their own: no more than have tokens)
  p.cluster = cluster;
  // Rows of a sequence that share their counts: what takes the fewest rounds of the clusters that
  // find room (of 152 SMs clusters of 8 use 120, of 4 144); counting costs about half a row.  (2, 3
  // and 6 rows of 96 sequences' 6 a cluster: 219, 204 and 204 us.)
  const int sms = !kProbs || cluster <= 2 ? num_sms : cluster == 4 ? num_sms * 18 / 19 : num_sms * 15 / 19;
  const int room = std::max(1, sms * (kPer <= 8 ? 3 : kPer <= 32 ? 2 : 1) / cluster);
  double best = 1e30;
  for (int rows = 1; rows <= p.m; ++rows) {
    const int64_t clusters = static_cast<int64_t>(B) * ((p.m + rows - 1) / rows);
    const double cost = static_cast<double>((clusters + room - 1) / room) * (rows + 0.5);
    if (cost < best) best = cost, p.rows = rows;
  }
  const int bytes = p.part * 4 + p.part / kListShare * 6 + p.biases * 12;
  // (also below 48 KB: a kernel's limit by default is that less its static part)
  const cudaError_t e = cudaFuncSetAttribute(logits_kernel<T, kPer, kProbs>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kPer * kLThreads * 4 + kPer * kLThreads / kListShare * 6 +
                                                 1024 * 12);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  const unsigned groups = static_cast<unsigned>(B) * ((p.m + p.rows - 1) / p.rows);
  cudaLaunchConfig_t cfg = make_cfg(dim3(groups * cluster), dim3(kLThreads), stream, true, attr);
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kProbs ? cluster : 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.numAttrs = 2;
  cfg.dynamicSmemBytes = bytes;
  return cudaLaunchKernelEx(&cfg, logits_kernel<T, kPer, kProbs>, p);
}

template <typename T, bool kProbs>
cudaError_t launch_rows(const LogitsParams<T>& p, int B, int num_sms, cudaStream_t stream) {
  // As many CTAs of 4096 tokens as the row has, up to 8; longer rows give each CTA more.
  const int parts = (p.V + 4095) / 4096;
  const int cluster = parts >= 5 ? 8 : parts >= 3 ? 4 : parts;
  const int per = (p.V + cluster * kLThreads - 1) / (cluster * kLThreads);
  if (per <= 8) return launch<T, 8, kProbs>(p, B, cluster, num_sms, stream);
  if (per <= 16) return launch<T, 16, kProbs>(p, B, cluster, num_sms, stream);
  if (per <= 32) return launch<T, 32, kProbs>(p, B, cluster, num_sms, stream);
  return launch<T, 64, kProbs>(p, B, cluster, num_sms, stream);
}

template <typename T>
cudaError_t launch_typed(const moe_logits_args& a, Ctrl* ctrl, int num_sms, cudaStream_t stream) {
  LogitsParams<T> p = {};
  p.logits = static_cast<const T*>(a.logits);
  p.out = a.out;
  p.l_sb = a.logits_stride_b, p.l_si = a.logits_stride_i;
  p.o_sb = a.out_stride_b, p.o_si = a.out_stride_i;
  p.m_sb = a.mask_stride_b, p.m_si = a.mask_stride_i;
  p.history = a.history_stride > 0 ? a.history : nullptr;
  p.history_lens = a.history_lens;
  p.prompt_lens = a.prompt_lens;
  p.draft = a.m > 1 ? a.draft : nullptr;
  p.repetition = a.repetition;
  p.presence = a.presence;
  p.frequency = a.frequency;
  p.temperature = a.temperature;
  p.bias_tokens = a.bias_tokens;
  p.bias_values = a.bias_values;
  p.mask = a.mask;
  p.ctrl = ctrl;
  p.m = a.m;
  p.V = a.V;
  p.history_stride = a.history_stride;
  p.biases = a.biases;
  return a.probabilities ? launch_rows<T, true>(p, a.B, num_sms, stream)
                         : launch_rows<T, false>(p, a.B, num_sms, stream);
}

}  // namespace

cudaError_t launch_adjust_logits(const moe_logits_args& a, Ctrl* ctrl, int num_sms,
                                 cudaStream_t stream) {
  return a.dtype == MOE_DTYPE_F32 ? launch_typed<float>(a, ctrl, num_sms, stream)
                                  : launch_typed<__nv_bfloat16>(a, ctrl, num_sms, stream);
}

}  // namespace moe
