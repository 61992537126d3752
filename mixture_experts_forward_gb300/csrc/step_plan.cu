// The plan of one step: pages for the sequences that grow, slots and positions for their new
// tokens; and the release of pages.
//
// Every CTA scans the whole batch by itself (block-wide, 1024 sequences a round) and keeps the
// prefix sums of the rows and of the pages needed in shared memory, so one launch does: a row
// finds its sequence by a binary search there, and a page's place on the stack follows from the
// prefix.  Nothing that a CTA reads is written before all have read it: the table entries written
// lie past held[], and held[] and free_count[] are updated by the last CTA to finish (a counter in
// the control block).  A few bytes per row: bound by the launch and the chain of dependent loads
// (lengths, scan, table entry, slot).  Plan and release together take 9 us for 8 sequences and
// 12 us for 1024 with 18432 new tokens (in a graph; the plan alone 7, the release 5), where the
// bytes would take 0.03; the Python calls take 30 and 38.
#include "serve_internal.cuh"

namespace moe {
namespace {

constexpr int kPlanThreads = 1024;

// Inclusive block-wide sums of two numbers; total: the block's.  s: 2 x 33 words.
__device__ __forceinline__ void block_scan(long long& a, int& b, long long* s_a, int* s_b,
                                           long long& total_a, int& total_b) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long ua = __shfl_up_sync(0xffffffffu, a, o);
    const int ub = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) a += ua, b += ub;
  }
  if (lane == 31) s_a[warp] = a, s_b[warp] = b;
  __syncthreads();
  if (warp == 0) {
    long long wa = s_a[lane];
    int wb = s_b[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long ua = __shfl_up_sync(0xffffffffu, wa, o);
      const int ub = __shfl_up_sync(0xffffffffu, wb, o);
      if (lane >= o) wa += ua, wb += ub;
    }
    s_a[lane] = wa, s_b[lane] = wb;
  }
  __syncthreads();
  if (warp > 0) a += s_a[warp - 1], b += s_b[warp - 1];
  total_a = s_a[31];
  total_b = s_b[31];
  __syncthreads();
}

// Whether this CTA is the last to come here; its earlier reads are done, and in the last one
// everybody's are.
__device__ __forceinline__ bool last_to_finish(Ctrl* ctrl) {
  __shared__ int s_last;
  __syncthreads();
  if (threadIdx.x == 0) {
    unsigned prev;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;"
                 : "=r"(prev) : "l"(&ctrl->done) : "memory");
    s_last = prev == gridDim.x - 1;
    if (s_last) ctrl->done = 0;
  }
  __syncthreads();
  return s_last != 0;
}

__global__ void __launch_bounds__(kPlanThreads)
    plan_kernel(const moe_page_state p, int page_log2, int num_pages,
                const int32_t* __restrict__ lens, const int32_t* __restrict__ news, int rows,
                int32_t* __restrict__ slots, int32_t* __restrict__ positions,
                int32_t* __restrict__ cu_q, int32_t* __restrict__ kv_lens, Ctrl* ctrl) {
  extern __shared__ int s_cu[];             // [B+1] first rows
  int* s_pages = s_cu + p.B + 1;            // [B+1] pages needed before each sequence
  uint32_t* s_bad = reinterpret_cast<uint32_t*>(s_pages + p.B + 1);   // bit b: not to be served
  __shared__ long long s_a[32];
  __shared__ int s_b[32];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int page = 1 << page_log2;
  const int said = *p.free_count;
  const int count = min(max(said, 0), p.free_capacity);
  if (said != count && tid == 0) set_error(ctrl, MOE_ERR_DEVICE_FAULT, kFaultPlanCount);

  long long row0 = 0;
  int page0 = 0;
  for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int len = 0, n = 0, held = 0;
    bool bad = false;
    if (b < p.B) {
      len = __ldg(lens + b);
      n = __ldg(news + b);
      held = p.held[b];
      const long long room = static_cast<long long>(p.table_stride) << page_log2;
      bad = len < 0 || n < 0 || held < 0 || held > p.table_stride ||
            static_cast<long long>(len) + n > room ||
            (static_cast<long long>(held) << page_log2) < len;
      n = max(n, 0);
    }
    // (len + n <= room < 2^31 unless bad)
    int need = bad ? 0 : max(0, ((len + n - 1) >> page_log2) + 1 - held);
    long long end = n;
    int upto = need, pages;
    long long total;
    block_scan(end, upto, s_a, s_b, total, pages);
    if (row0 + end > rows && n > 0) {
      bad = true;
    }
    // a sequence past the last row takes no pages: those after it are past it too, so no later
    // prefix counts what it would have taken
    if (b < p.B) {
      s_cu[b + 1] = static_cast<int>(min(row0 + end, static_cast<long long>(rows)));
      s_pages[b + 1] = page0 + upto;
    }
    const uint32_t m = __ballot_sync(0xffffffffu, bad);
    if (lane == 0 && b < p.B) s_bad[b >> 5] = m;
    if (bad && blockIdx.x == 0) set_error(ctrl, MOE_ERR_DEVICE_FAULT, kFaultPlanSequence);
    row0 += total;
    page0 += pages;
  }
  if (tid == 0) s_cu[0] = 0, s_pages[0] = 0;
  __syncthreads();

  auto is_bad = [&](int b) { return (s_bad[b >> 5] >> (b & 31)) & 1u; };
  auto need_of = [&](int b) { return s_pages[b + 1] - s_pages[b]; };
  auto served = [&](int b) {
    return !is_bad(b) && (need_of(b) == 0 || s_pages[b + 1] <= count);
  };

  // rows
  for (int r = blockIdx.x * kPlanThreads + tid; r < rows; r += gridDim.x * kPlanThreads) {
    int slot = -1, pos = 0;
    if (r < s_cu[p.B]) {
      int lo = 0, hi = p.B;                 // the last sequence whose first row is at or below r
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_cu[mid] <= r) lo = mid; else hi = mid;
      }
      const int len = __ldg(lens + lo);
      const long long at = static_cast<long long>(len) + (r - s_cu[lo]);
      if (len >= 0 && at <= 0x7fffffffll) pos = static_cast<int>(at);
      if (served(lo)) {
        const int entry = pos >> page_log2, held = p.held[lo];
        const int id = entry < held
                           ? p.block_table[static_cast<int64_t>(lo) * p.table_stride + entry]
                           : p.free_pages[count - 1 - (s_pages[lo] + entry - held)];
        if (id >= 0 && id < num_pages)
          slot = (id << page_log2) + (pos & (page - 1));
        else
          set_error(ctrl, MOE_ERR_DEVICE_FAULT, kFaultPlanPage);
      }
    }
    slots[r] = slot;
    positions[r] = pos;
  }
  // the new pages enter the tables, a warp per sequence
  const int warps = gridDim.x * (kPlanThreads / 32);
  for (int b = blockIdx.x * (kPlanThreads / 32) + warp; b < p.B; b += warps) {
    const int need = need_of(b);
    if (need == 0 || !served(b)) continue;
    int32_t* row = p.block_table + static_cast<int64_t>(b) * p.table_stride + p.held[b];
    for (int j = lane; j < need; j += 32) row[j] = p.free_pages[count - 1 - (s_pages[b] + j)];
  }
  for (int b = blockIdx.x * kPlanThreads + tid; b <= p.B; b += gridDim.x * kPlanThreads) {
    cu_q[b] = s_cu[b];
    if (b < p.B) kv_lens[b] = served(b) ? __ldg(lens + b) + __ldg(news + b) : 0;
  }
  if (!last_to_finish(ctrl)) return;
  int taken = 0;
  for (int b = tid; b < p.B; b += kPlanThreads)
    if (need_of(b) > 0 && served(b)) {
      p.held[b] += need_of(b);
      taken += need_of(b);
    }
  taken = __reduce_add_sync(0xffffffffu, taken);
  if (lane == 0) s_b[warp] = taken;
  __syncthreads();
  if (warp == 0) {
    taken = __reduce_add_sync(0xffffffffu, s_b[lane]);
    if (lane == 0) *p.free_count = count - taken;
  }
}

__global__ void __launch_bounds__(kPlanThreads)
    release_kernel(const moe_page_state p, int page_log2, const int32_t* __restrict__ keep,
                   Ctrl* ctrl) {
  extern __shared__ int s_give[];           // [B+1] pages given back before each sequence
  __shared__ long long s_a[32];
  __shared__ int s_b[32];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int said = *p.free_count;
  const int count = min(max(said, 0), p.free_capacity);
  if (said != count && tid == 0) set_error(ctrl, MOE_ERR_DEVICE_FAULT, kFaultReleaseCount);
  int before = 0;
  for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int give = 0;
    if (b < p.B) {
      const int held = p.held[b], kept = __ldg(keep + b);
      if (held < 0 || held > p.table_stride)
        set_error(ctrl, MOE_ERR_DEVICE_FAULT, kFaultReleaseHeld);
      else if (kept >= 0)
        give = max(0, held - (kept == 0 ? 0 : ((kept - 1) >> page_log2) + 1));
    }
    long long none = 0, total;
    int pages;
    block_scan(none, give, s_a, s_b, total, pages);
    if (b < p.B) s_give[b + 1] = before + give;
    before += pages;
  }
  if (tid == 0) s_give[0] = 0;
  __syncthreads();
  const bool fits = before <= p.free_capacity - count;
  if (!fits && tid == 0) set_error(ctrl, MOE_ERR_DEVICE_FAULT, kFaultReleaseRoom);
  if (fits) {
    const int warps = gridDim.x * (kPlanThreads / 32);
    for (int b = blockIdx.x * (kPlanThreads / 32) + warp; b < p.B; b += warps) {
      const int first = s_give[b], give = s_give[b + 1] - first;
      if (give == 0) continue;
      int32_t* row = p.block_table + static_cast<int64_t>(b) * p.table_stride + p.held[b] - give;
      for (int j = lane; j < give; j += 32) {
        p.free_pages[count + before - 1 - (first + j)] = row[j];
        row[j] = -1;
      }
    }
  }
  if (!last_to_finish(ctrl) || !fits) return;
  for (int b = tid; b < p.B; b += kPlanThreads) p.held[b] -= s_give[b + 1] - s_give[b];
  if (tid == 0) *p.free_count = count + before;
}

int page_bits(int page_size) {
  int n = 0;
  while ((1 << n) < page_size) ++n;
  return n;
}

}  // namespace

cudaError_t launch_plan_step(const moe_page_state& p, const int32_t* lens, const int32_t* news,
                             int rows, int num_pages, int32_t* slots, int32_t* positions,
                             int32_t* cu_q, int32_t* kv_lens, Ctrl* ctrl, int num_sms,
                             cudaStream_t stream) {
  const int most = rows > 32 * p.B ? rows : 32 * p.B;      // a warp per sequence
  int grid = (most + kPlanThreads - 1) / kPlanThreads;
  grid = grid < 1 ? 1 : grid > num_sms ? num_sms : grid;
  const int bytes = (2 * (p.B + 1) + (p.B + 31) / 32) * 4;
  cudaError_t e = cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (2 * (kMaxPlanned + 1) + kMaxPlanned / 32) * 4);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = make_cfg(dim3(grid), dim3(kPlanThreads), stream, true, attr);
  cfg.dynamicSmemBytes = bytes;
  return cudaLaunchKernelEx(&cfg, plan_kernel, p, page_bits(p.page_size), num_pages, lens, news,
                            rows, slots, positions, cu_q, kv_lens, ctrl);
}

cudaError_t launch_release_pages(const moe_page_state& p, const int32_t* keep, Ctrl* ctrl,
                                 int num_sms, cudaStream_t stream) {
  int grid = (p.B + 31) / 32;
  grid = grid < 1 ? 1 : grid > num_sms ? num_sms : grid;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = make_cfg(dim3(grid), dim3(kPlanThreads), stream, true, attr);
  cfg.dynamicSmemBytes = (p.B + 1) * 4;
  return cudaLaunchKernelEx(&cfg, release_kernel, p, page_bits(p.page_size), keep, ctrl);
}

}  // namespace moe
