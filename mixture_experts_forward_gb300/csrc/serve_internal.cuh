// Declarations shared by the serving operators: the paged cache, attention
// over it, and the verification of drafted tokens.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "moe_internal.cuh"

namespace moe {

// moe_kv_cache as the kernels take it.  A cache row is one position of one
// head: row ((page * heads + head) << page_log2) + position % page_size.
struct KvCacheView {
  uint8_t* k;
  uint8_t* v;
  float* k_scales;
  float* v_scales;
  int num_pages, heads, page_log2;
};

// Two E4M3 codes (low byte first) as binary16 (exact), and as binary32.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(codes));
  return h;
}
__device__ __forceinline__ float2 e4m3x2_to_f32(uint16_t codes) {
  uint32_t h = e4m3x2_to_f16x2(codes);
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

// Attention: what the kernels need of moe_attention_args.
struct AttnParams {
  KvCacheView c;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  float* lse;
  int64_t q_st, q_sh, o_st, o_sh;
  const int32_t* cu_q;
  const int32_t* kv_lens;
  const int32_t* table;
  int table_stride;
  int B, T, q_heads, group, max_q;
  float scale, softcap;
  int window, causal;
  int row_tiles;                 // row tiles per (sequence, head)
  int splits;                    // parts of a tile's keys at most
  int whole;                     // many rows: tiles before the ones that are split; few: CTAs
  int span;                      // keys that a tile sees at most (few rows)
  int part_rows;                 // rows that a part's result has room for
  unsigned* counters;            // one per (sequence, head, row tile); zero between calls
  float* partial;                // per (tile, part): rows x (head_dim sums, maximum, sum)
  Ctrl* ctrl;
  unsigned long long timeout_ns;
  int drop_producer;
};

cudaError_t launch_kv_write(const KvCacheView& c, int head_dim, bool fp8, const void* k,
                            const void* v, int T, int64_t ks_t, int64_t ks_h, int64_t vs_t,
                            int64_t vs_h, const int32_t* slots, Ctrl* ctrl, cudaStream_t stream);
cudaError_t launch_kv_read(const KvCacheView& c, int head_dim, bool fp8, const int32_t* table,
                           int table_stride, const int32_t* cu, const int32_t* starts, int B,
                           int rows, void* k_out, void* v_out, Ctrl* ctrl, cudaStream_t stream);
// Parts of a tile (and CTAs that share tiles) at most.
constexpr int kMaxParts = 320;
// Up to 16, 32, 48 or (BF16) 64 rows per tile (tile_rows), tcgen05 with keys and channels as the
// rows.
int attention_rows_places(int tile_rows, int head_dim, bool fp8);   // CTAs per SM
cudaError_t launch_attention_rows(const AttnParams& p, int tile_rows, int head_dim, bool fp8,
                                  cudaStream_t stream);
// Up to 256 rows per tile, tcgen05.
constexpr int kTileRows = 256;
constexpr int kTileKeys = 128;
cudaError_t launch_attention_tiles(const AttnParams& p, int head_dim, bool fp8,
                                   cudaStream_t stream);
// moe_kv_cache checked, and as the kernels take it (serve_api.cu).
moe_status_t check_cache(const moe_kv_cache* c, KvCacheView* view);

// Where a fault of these operators was first seen (Ctrl::err_info): they may share a control block
// with the forward (1 .. 6), the cache (10, 11), attention (20 .. 24) and the verification (30, 31).
enum FaultPlace {
  kFaultToken = 40,            // logits: a token id,
  kFaultHistory = 41,          //   a length of the history or the prompt,
  kFaultNumber = 42,           //   a repetition or a temperature
  kFaultPlanCount = 50,        // plan: free_count,
  kFaultPlanSequence = 51,     //   a sequence's lengths, held or rows,
  kFaultPlanPage = 52,         //   a page id
  kFaultReleaseCount = 53,     // release: free_count,
  kFaultReleaseHeld = 54,      //   held,
  kFaultReleaseRoom = 55,      //   no room on the stack
  kFaultRotarySlot = 60,
  kFaultFewRoute = 70,         // few tokens: a route to no expert
};

// Sequences of one plan at most: their prefix sums stay in shared memory.
constexpr int kMaxPlanned = 8192;
cudaError_t launch_plan_step(const moe_page_state& p, const int32_t* lens, const int32_t* news,
                             int rows, int num_pages, int32_t* slots, int32_t* positions,
                             int32_t* cu_q, int32_t* kv_lens, Ctrl* ctrl, int num_sms,
                             cudaStream_t stream);
cudaError_t launch_release_pages(const moe_page_state& p, const int32_t* keep, Ctrl* ctrl,
                                 int num_sms, cudaStream_t stream);
cudaError_t launch_rotary(const moe_rotary_args& a, const KvCacheView* cache, Ctrl* ctrl,
                          int num_sms, cudaStream_t stream);
// ws: kFewWsBytes (the control block and the routes), then h in binary32, [M * top_k, N]
constexpr size_t kFewWsBytes = MOE_CTRL_BYTES + MOE_FEW_TOKENS * 32 * 8;
cudaError_t launch_few_experts(const moe_forward_args& f, void* out, uint8_t* ws, int num_sms,
                               cudaStream_t stream);
cudaError_t launch_adjust_logits(const moe_logits_args& a, Ctrl* ctrl, int num_sms,
                                 cudaStream_t stream);
cudaError_t launch_verify(const moe_verify_args& a, Ctrl* ctrl, int num_sms, cudaStream_t stream);

}  // namespace moe
